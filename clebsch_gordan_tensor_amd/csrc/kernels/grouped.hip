// Channel mixing within each irrep (e3j A.3 Eq.5) with weights per group, and
// its gradients: for the rows r of group g (chemical element, expert)
//   y[r][o, m][k]  = sum over sources i of sum_k' x[r][i, m][k'] W[g][io][k'][k]
//   dx: the same product over dy with W transposed
//   dW[g][io]      = sum over the group's r and m of x[r][i, m]^T dy[r][o, m].
// Rows stand in any order; the index of e3_group_index lists them by group,
// and the kernels gather and scatter through it.  The rows of the products are
// the (r, m) of an output block, cut into tiles that belong to one group.
//
// All products run on the bf16 matrix cores (v_mfma_f32_16x16x32_bf16, fp32
// accumulation).  A float32 operand is split into three bf16 parts, a = a1 +
// a2 + a3 with each part the rest rounded to nearest: 24 bits and the range of
// float32, down to 2^-110 (bf16's least value is 2^-133: of a smaller operand
// what lies below 2^-134 is lost).  Of the nine products of two split operands
// the six largest are kept; what is left out is below 2^-26 of a product.  Six
// bf16 products cost 6/16 of a float32 one's matrix-core time.
//
// Layout of the operands (A[i][k]: lane i + 16 (k / 8) holds 8 consecutive k;
// B[k][j] likewise; D[i][j]: register r of lane j + 16 h is i = 4 h + r): W is
// taken as A and the rows of x as B, so that a lane ends with consecutive
// columns of one row of y and stores 16 bytes at once.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.h"
#include "group_tiles.h"
#include "registry.h"
#include "row_halves.h"
#include "tile128.h"

namespace e3k {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;   // 4 wavefronts, 64 x 64 of the tile each
constexpr int kTile = 128;      // rows and columns of a workgroup's tile

template <class T>
constexpr int kParts = sizeof(T) == 4 ? 3 : 1;  // bf16 parts of an operand

// Where 16 bytes (8 values) `piece` of row r of K values lie in LDS, in values:
// the pieces of 8 consecutive rows (K = 32: of 8 rows, two a 128-byte line) are
// exchanged so that reads of one piece of 16 rows meet every bank alike.
// (Padded rows left half of the LDS cycles to conflicts.)
template <int K>
__device__ __forceinline__ int lds_at(int r, int piece) {
  return r * K + ((piece ^ (K >= 64 ? r & 7 : (r >> 1) & 3)) << 3);
}

// Parts of 4 consecutive values.
__device__ __forceinline__ void split3(const f32x4 v, bf16x4 (&p)[3]) {
  p[0] = __builtin_convertvector(v, bf16x4);
  f32x4 r = v - __builtin_convertvector(p[0], f32x4);
  p[1] = __builtin_convertvector(r, bf16x4);
  r -= __builtin_convertvector(p[1], f32x4);
  p[2] = __builtin_convertvector(r, bf16x4);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// c[i][j] += a[i] b[j] of split operands, smallest products first; one product
// of every pair in turn, so that none waits for the one before.
template <int PARTS, int M, int N>
__device__ __forceinline__ void products(const bf16x8 (&a)[M][PARTS], const bf16x8 (&b)[N][PARTS],
                                         f32x4 (&c)[M][N]) {
  constexpr int kA[6] = {2, 0, 1, 1, 0, 0}, kB[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
  for (int t = PARTS == 3 ? 0 : 5; t < 6; ++t)
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) c[i][j] = mfma(a[i][kA[t]], b[j][kB[t]], c[i][j]);
}

// ------------------------------------------------------------ the mixing

// float32: chunks of 32 k pass through registers, where they are split, to LDS;
// the next chunk is on its way meanwhile.
template <bool WT>
__global__ void __launch_bounds__(kThreads) k_mix(const MixArgs a, const MixList l) {
  constexpr int BK = 32;
  constexpr int TPR = BK / 4;             // threads of a row of a chunk, 4 values each
  constexpr int PASS = kThreads / TPR;    // rows of a pass: 32
  constexpr int CT = kTile / 4;           // threads of a row of W
  __shared__ __attribute__((aligned(16))) __bf16 s_x[3][kTile * BK], s_w[3][kTile * BK];
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups);
  const unsigned wg = a.wg0 + blockIdx.x;
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(wg)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  int col_tile;
  if (!find_tile_xcd(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, kTile,
                     wg - unsigned(blk.wg0), unsigned((a.cout + kTile - 1) / kTile), tile,
                     col_tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.x);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave & 1, wn = wave >> 1, q = lane & 15, h = lane >> 4;
  const int col0 = col_tile * kTile;
  const int n_rows = int(min(int64_t(kTile), tile.rows - tile.at));
  const TileRows rows(tile.at, blk.deg);

  f32x4 acc[4][4];  // [columns][rows] of 16
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};

  // the rows this thread stages, and its 4 values of them; the rows this lane
  // ends with
  const int piece = tid % TPR, r0 = tid / TPR;
  const float* xrow[4];
  int load_row[4], load_m[4], row[4], comp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    load_row[j] = order(rows.place(min(r0 + j * PASS, n_rows - 1), load_m[j]));
    row[j] = order(rows.place(min(wm * 64 + j * 16 + q, n_rows - 1), comp[j]));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    xrow[j] = static_cast<const float*>(a.x) +
              (int64_t(load_row[j]) * a.din + load_m[j]) * a.cin + piece * 4;
  const int n_src = tile.group < a.n_groups ? blk.n_src : 0;
  const int chunks = (a.cin + BK - 1) / BK;
  const float* W0 = static_cast<const float*>(a.W) + int64_t(tile.group) * a.pairs * a.cin * a.cout;

  f32x4 xv[4], wv[4];
  const auto fetch = [&](int step) {
    const int src = step / chunks, k0 = (step - src * chunks) * BK;
    const MixSource sc = l.src[blk.src0 + src];
    const float* W = W0 + int64_t(sc.pair) * a.cin * a.cout;
    const bool in = k0 + piece * 4 < a.cin;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xv[j] = in ? *reinterpret_cast<const f32x4*>(xrow[j] + int64_t(sc.in_off) * a.cin + k0)
                 : f32x4{};
    if constexpr (WT) {  // rows of W are columns here, k along them
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = col0 + r0 + j * PASS;
        wv[j] = n < a.cout && in
                    ? *reinterpret_cast<const f32x4*>(W + int64_t(n) * a.cin + k0 + piece * 4)
                    : f32x4{};
      }
    } else {  // 4 columns of 4 consecutive k
      const int n = col0 + tid % CT * 4, k = k0 + tid / CT * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        wv[j] = n < a.cout && k + j < a.cin
                    ? *reinterpret_cast<const f32x4*>(W + int64_t(k + j) * a.cout + n)
                    : f32x4{};
    }
  };
  // parts of 4 values along k into row r of an operand in LDS
  const auto put = [&](__bf16 (&s)[3][kTile * BK], int r, int k, f32x4 v) {
    bf16x4 p[3];
    split3(v, p);
#pragma unroll
    for (int t = 0; t < 3; ++t)
      *reinterpret_cast<bf16x4*>(&s[t][lds_at<BK>(r, k / 8) + k % 8]) = p[t];
  };
  const auto stage = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) put(s_x, r0 + j * PASS, piece * 4, xv[j]);
    if constexpr (WT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) put(s_w, r0 + j * PASS, piece * 4, wv[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        put(s_w, tid % CT * 4 + e, tid / CT * 4, f32x4{wv[0][e], wv[1][e], wv[2][e], wv[3][e]});
    }
  };

  const int steps = n_src * chunks;
  if (steps > 0) fetch(0);
  for (int step = 0; step < steps; ++step) {
    __syncthreads();  // the last chunk's reads are done
    stage();
    __syncthreads();
    if (step + 1 < steps) fetch(step + 1);
    bf16x8 xf[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 3; ++t)
        xf[j][t] = *reinterpret_cast<const bf16x8*>(
            &s_x[t][lds_at<BK>(wm * 64 + j * 16 + q, h)]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x8 wf[1][3];
#pragma unroll
      for (int t = 0; t < 3; ++t)
        wf[0][t] = *reinterpret_cast<const bf16x8*>(
            &s_w[t][lds_at<BK>(wn * 64 + i * 16 + q, h)]);
      products<3, 1, 4>(wf, xf, reinterpret_cast<f32x4(&)[1][4]>(acc[i]));
    }
  }

#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (wm * 64 + j * 16 + q >= n_rows) continue;
    float* y = static_cast<float*>(a.y) +
               (int64_t(row[j]) * a.dout + blk.out_off + comp[j]) * a.cout;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = col0 + wn * 64 + i * 16 + h * 4;
      if (n < a.cout) *reinterpret_cast<f32x4*>(y + n) = acc[i][j];
    }
  }
}

// bf16: chunks of 64 k go straight to LDS, one is multiplied while the next is
// on its way; two workgroups on a compute unit.  W lies along k when it is
// transposed, and along its columns when not: then it is read across.
// 16,384 rows in 16 groups, 1024 to 2048 channels: 98 us (700 TFLOP/s), its dx
// 95-110; 40-44% of the cycles are products, no LDS read meets another's bank, and the
// rest are waits for chunks: 1.1 GB pass from the caches to LDS.
template <bool WT>
__global__ void __launch_bounds__(kThreads, 2) k_mix_along(const MixArgs a, const MixList l) {
  // a name for every stage: reads of one are then known not to wait for loads
  // into the other
  __shared__ __attribute__((aligned(128))) uint8_t s_x0[TileLoad::kBytes], s_w0[TileLoad::kBytes];
  __shared__ __attribute__((aligned(128))) uint8_t s_x1[TileLoad::kBytes], s_w1[TileLoad::kBytes];
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups);
  const unsigned wg = a.wg0 + blockIdx.x;
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(wg)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  int col_tile;
  if (!find_tile_xcd(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, kTile,
                     wg - unsigned(blk.wg0), unsigned((a.cout + kTile - 1) / kTile), tile,
                     col_tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.x);
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const TileLoad load;
  const AcrossLoad<4> across;
  const int wm = load.wave & 1, wn = load.wave >> 1, col0 = col_tile * kTile;
  const int n_rows = int(min(int64_t(kTile), tile.rows - tile.at));
  const TileRows rows(tile.at, blk.deg);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  // the rows this lane loads, and those it ends with; rows past the end are
  // the last one again, and so are columns
  int load_row[4], load_m[4], row[4], comp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    load_row[j] = order(rows.place(min(load.row + j * 32, n_rows - 1), load_m[j]));
    row[j] = order(rows.place(min(wm * 64 + j * 16 + q, n_rows - 1), comp[j]));
  }
  const uint8_t *xrow[4], *wrow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xrow[j] = static_cast<const uint8_t*>(a.x) +
              ((int64_t(load_row[j]) * a.din + load_m[j]) * a.cin + load.piece * 8) * 2;
    // slot s of the columns holds column 8 (s >> 2 & 3) + 4 (s >> 4 & 1) + (s & 3) of its 32
    const int s = load.row + j * 32;
    const int n = min(col0 + ((s & ~31) | ((s >> 2) & 3) << 3 | ((s >> 4) & 1) << 2 | (s & 3)),
                      a.cout - 1);
    const int64_t W0 = int64_t(tile.group) * a.pairs * a.cin * a.cout;
    wrow[j] = static_cast<const uint8_t*>(a.W) +
              (W0 + (WT ? int64_t(n) * a.cin + load.piece * 8
                        : int64_t(across.row + j * 16) * a.cout + col0 + across.piece * 8)) * 2;
  }
  const bool in_col = col0 + across.piece * 8 < a.cout;
  const int chunks = (a.cin + 63) / 64;
  const int steps = tile.group < a.n_groups ? blk.n_src * chunks : 0;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kTileZeros);
  int64_t xo = 0, wo = 0;  // bytes to the chunk asked for next
  int src = -1, b = chunks - 1;
  const auto fetch = [&](uint8_t* x, uint8_t* w) {
    if (b + 1 < chunks) {  // past the last chunk it is asked for again
      ++b;
      xo += 128;
      wo += WT ? 128 : int64_t(a.cout) * 128;
    } else if (src + 1 < blk.n_src) {
      const MixSource sc = l.src[blk.src0 + ++src];
      b = 0;
      xo = int64_t(sc.in_off) * a.cin * 2;
      wo = int64_t(sc.pair) * a.cout * a.cin * 2;
    }
    const bool in = b * 64 + load.piece * 8 < a.cin;
#pragma unroll
    for (int j = 0; j < 4; ++j) load.ask(in ? xrow[j] + xo : zeros, x, j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool have = WT ? in : in_col && b * 64 + across.row + j * 16 < a.cin;
      load.ask(have ? wrow[j] + wo : zeros, w, j);
    }
  };
  const auto turn = [&](const uint8_t* x, const uint8_t* w, uint8_t* x_free, uint8_t* w_free,
                        int step) {
    tile_wait();
    fetch(x_free, w_free);
    if (step >= steps) return;
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      bf16x8 xf[4][1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        xf[j][0] = *reinterpret_cast<const bf16x8*>(tile_at(x, wm * 64 + j * 16 + q, kk * 4 + h));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x8 wf[1][1];
        if constexpr (WT)
          wf[0][0] = *reinterpret_cast<const bf16x8*>(tile_at(w, wn * 64 + i * 16 + q, kk * 4 + h));
        else wf[0][0] = across.read(w, kk, wn * 8 + (i >> 1) * 4 + (lane & 3), i & 1);
        products<1, 1, 4>(wf, xf, reinterpret_cast<f32x4(&)[1][4]>(acc[i]));
      }
    }
  };
  if (steps > 0) fetch(s_x0, s_w0);
  for (int step = 0; step < steps; step += 2) {
    turn(s_x0, s_w0, s_x1, s_w1, step);
    turn(s_x1, s_w1, s_x0, s_w0, step + 1);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load writes to LDS after the end
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (wm * 64 + j * 16 + q >= n_rows) continue;
    bf16_t* y = static_cast<bf16_t*>(a.y) +
                (int64_t(row[j]) * a.dout + blk.out_off + comp[j]) * a.cout;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const int n = col0 + wn * 64 + i * 16 + h * 8;
      bf16x8 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __bf16(acc[i][j][e]);
        v[4 + e] = __bf16(acc[i + 1][j][e]);
      }
      if (n < a.cout) *reinterpret_cast<bf16x8*>(y + n) = v;
    }
  }
}

// The mixing where every block has one source and its rows of W are short (K =
// 32 NK channels at most): a wavefront holds 32 columns of W in registers, in
// parts, and a workgroup walks over its group's rows, 64 at a time.  Their x
// passes through LDS once, split there; the next 64 rows are under way in
// registers meanwhile, and where they lie is known two tiles ahead.  CW
// wavefronts share out the output channels, 4 / CW the tile's rows.  64,000 x 16
// rows of 128 channels, float32: 245-275 us, 4.0 TB/s; 41% of the cycles are
// products, the rest loads and stores that wait for memory.
//
// Nothing in the walk is conditional: a wait for loads counts what was issued
// after them, and with stores that may or may not have been issued it waits
// for these as well.  Rows past the end of the walk are rows of the group all
// the same, the last atom's; their results are written twice.
constexpr int kStreamRows = 64;

template <class T, bool WT, int NK, int CW, bool FULL>
__global__ void __launch_bounds__(kThreads, 2) k_mix_stream(const MixArgs a, const MixList l,
                                                            int chunk) {
  constexpr int PARTS = kParts<T>, K = 32 * NK;
  constexpr int VEC = 16 / sizeof(T), TPR = K / VEC, PASS = kThreads / TPR;
  constexpr int NP = kStreamRows / PASS, RT = CW;  // row tiles of a wavefront
  static_assert(NP >= 1);
  __shared__ __attribute__((aligned(16))) __bf16 s_x[PARTS][kStreamRows * K];
  __shared__ int2 s_row[3][kStreamRows];  // row and component
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups);
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(blockIdx.x)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  if (!find_tile(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, chunk,
                 int64_t(blockIdx.x) - blk.wg0, tile) || !valid)
    return;
  const int* order = a.index ? a.index + a.order + tile.first : nullptr;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int q = lane & 15, h = lane >> 4, wn = wave % CW, wm = wave / CW;
  const int col0 = int(blockIdx.y) * (32 * CW) + wn * 32;
  const int n = int(min(int64_t(chunk), tile.rows - tile.at));
  const int deg = blk.deg;

  // where the rows are: thread r of the first wavefront keeps to row r of the
  // tiles, and has the next one's place in `place`
  // (places count on past the last one, and that may be 2^31 - 2: unsigned)
  const unsigned last = unsigned((tile.at + n - 1) / deg), step_at = unsigned(kStreamRows / deg);
  const int step_m = kStreamRows % deg;
  const int64_t from = tile.at / deg;
  const unsigned u = unsigned(tile.at - from * deg) + unsigned(lane);
  unsigned at = unsigned(from) + u / unsigned(deg);
  int m = int(u % unsigned(deg));
  const int* source = order ? order : static_cast<const int*>(a.x);  // (read in any case)
  const auto look = [&]() {
    const unsigned t = min(at, last);
    const int row = source[order ? t : 0u];
    return order ? row : int(t);
  };
  const auto put = [&](int buf, int place) {
    if (wave == 0) s_row[buf][lane] = {place, m};
    at += step_at;
    m += step_m;
    if (m >= deg) {
      m -= deg;
      ++at;
    }
  };
  int place = look();
  if (tile.group >= a.n_groups || blk.n_src == 0) {  // zeros
    for (int t0 = 0; t0 < n; t0 += kStreamRows) {
      put(0, place);
      place = look();
      __syncthreads();
      for (int e = tid; e < min(kStreamRows, n - t0) * 32 * CW; e += kThreads) {
        const int2 to = s_row[0][e / (32 * CW)];
        const int c = int(blockIdx.y) * (32 * CW) + e % (32 * CW);
        if (c < a.cout)
          static_cast<T*>(a.y)[(int64_t(to.x) * a.dout + blk.out_off + to.y) * a.cout + c] = T{};
      }
      __syncthreads();
    }
    return;
  }
  put(0, place);
  place = look();
  put(1, place);
  place = look();
  __syncthreads();

  const RowHalves halves;
  const MixSource sc = l.src[blk.src0];
  const int piece = tid % TPR, r0 = tid / TPR;
  const bool in = piece * VEC < a.cin;
  const T* x0 = static_cast<const T*>(a.x) + int64_t(sc.in_off) * a.cin + (in ? piece * VEC : 0);
  u32x4 xv[NP];
  const auto fetch = [&](int buf) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int2 r = s_row[buf][r0 + j * PASS];
      xv[j] = *reinterpret_cast<const u32x4*>(x0 + (int64_t(r.x) * a.din + r.y) * a.cin);
    }
  };
  fetch(0);

  // this wavefront's columns of W: product i's row q of A.  All of them are
  // asked for before the first is split (piece by piece the loads' delays add up).
  bf16x8 wf[NK][2][PARTS];
  {
    const T* W = static_cast<const T*>(a.W) +
                 (int64_t(tile.group) * a.pairs + sc.pair) * a.cin * a.cout;
    T v[NK][2][8];
#pragma unroll
    for (int s = 0; s < NK; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = std::is_same_v<T, float> ? i * 16 + q : 8 * (q >> 2) + 4 * i + (q & 3);
        const int col = min(col0 + c, a.cout - 1);  // (columns past the end are not stored)
        const int k = s * 32 + h * 8 < a.cin ? s * 32 + h * 8 : 0;
        if constexpr (WT) {
          const T* w = W + int64_t(col) * a.cin + k;
#pragma unroll
          for (int e = 0; e < 8; e += VEC)
            *reinterpret_cast<u32x4*>(&v[s][i][e]) = *reinterpret_cast<const u32x4*>(w + e);
        } else {
          const T* w = W + int64_t(k) * a.cout + col;
#pragma unroll
          for (int e = 0; e < 8; ++e) v[s][i][e] = w[int64_t(e) * a.cout];
        }
      }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < NK; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool have = s * 32 + h * 8 < a.cin;
        if constexpr (PARTS == 3) {
          const T* w = v[s][i];
          bf16x4 lo[3], hi[3];
          split3(have ? f32x4{w[0], w[1], w[2], w[3]} : f32x4{}, lo);
          split3(have ? f32x4{w[4], w[5], w[6], w[7]} : f32x4{}, hi);
#pragma unroll
          for (int t = 0; t < 3; ++t)
            wf[s][i][t] = __builtin_shufflevector(lo[t], hi[t], 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            wf[s][i][0][e] = have ? __builtin_bit_cast(__bf16, v[s][i][e]) : __bf16(0.0f);
        }
      }
  }

  // everything asked for so far is here: at the walk's top only a turn's own
  // loads and stores are left to count
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  for (int t0 = 0, buf = 0; t0 < n; t0 += kStreamRows, buf = buf == 2 ? 0 : buf + 1) {
    constexpr int JB = RT < 2 ? RT : 2;  // row tiles whose products alternate
    f32x4 acc[RT / JB][2][JB];
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[j / JB][i][j % JB] = f32x4{};
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int r = r0 + j * PASS;
      const u32x4 v = in ? xv[j] : u32x4{};
      const int to = lds_at<K>(r, piece * VEC / 8) + piece * VEC % 8;
      if constexpr (PARTS == 3) {
        bf16x4 p[3];
        split3(__builtin_bit_cast(f32x4, v), p);
#pragma unroll
        for (int t = 0; t < 3; ++t) *reinterpret_cast<bf16x4*>(&s_x[t][to]) = p[t];
      } else {
        *reinterpret_cast<u32x4*>(&s_x[0][to]) = v;
      }
    }
    const int next = buf == 2 ? 0 : buf + 1, after = next == 2 ? 0 : next + 1;
    put(after, place);
    __syncthreads();
    place = look();
    fetch(next);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the products
#pragma unroll
    for (int s = 0; s < NK; ++s)
#pragma unroll
      for (int j = 0; j < RT / JB; ++j) {
        bf16x8 xf[JB][PARTS];
#pragma unroll
        for (int b = 0; b < JB; ++b)
#pragma unroll
          for (int t = 0; t < PARTS; ++t)
            xf[b][t] = *reinterpret_cast<const bf16x8*>(
                &s_x[t][lds_at<K>((wm * RT + j * JB + b) * 16 + q, s * 4 + h)]);
        products<PARTS, 2, JB>(wf[s], xf, acc[j]);
      }
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if constexpr (PARTS == 3) {  // 32 columns are a line
        f32x4 v0 = acc[j / JB][0][j % JB], v1 = acc[j / JB][1][j % JB];
        halves.trade(v0, v1);
        const int c = col0 + halves.column / 4, r = (wm * RT + j) * 16 + (q & 7);
        const int2 r0 = s_row[buf][r], r1 = s_row[buf][r + 8];
        T* y = static_cast<T*>(a.y) + int64_t(blk.out_off) * a.cout + c;
        if (FULL || c < a.cout) {
          __builtin_nontemporal_store(
              v0, reinterpret_cast<f32x4*>(y + (int64_t(r0.x) * a.dout + r0.y) * a.cout));
          __builtin_nontemporal_store(
              v1, reinterpret_cast<f32x4*>(y + (int64_t(r1.x) * a.dout + r1.y) * a.cout));
        }
      } else {
        const int2 to = s_row[buf][(wm * RT + j) * 16 + q];
        T* y = static_cast<T*>(a.y) + (int64_t(to.x) * a.dout + blk.out_off + to.y) * a.cout;
        bf16x8 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = __bf16(acc[j / JB][0][j % JB][e]);
          v[4 + e] = __bf16(acc[j / JB][1][j % JB][e]);
        }
        if (FULL || col0 + h * 8 < a.cout) *reinterpret_cast<bf16x8*>(y + col0 + h * 8) = v;
      }
    }
    __syncthreads();  // s_x and the rows' oldest buffer are written next
  }
}

// Rows of a workgroup's walk: a few workgroups for every one that is resident
// (two on a compute unit).
int stream_chunk(int64_t rows) {
  const int64_t n = (rows / 2048 + kStreamRows - 1) / kStreamRows * kStreamRows;
  return int(std::min<int64_t>(1024, std::max<int64_t>(kStreamRows, n)));
}

template <class T, bool WT, int NK>
hipError_t launch_stream(const MixArgs& a, MixList l, hipStream_t s) {
  int64_t wgs = 0, comps = 0;
  for (int i = 0; i < l.n_blocks; ++i) comps += l.blk[i].deg;
  const int chunk = stream_chunk(a.n_rows * comps);
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, chunk, a.index != nullptr);
  }
  const auto go = [&](auto cw) {
    constexpr int CW = decltype(cw)::value;
    const dim3 grid(unsigned(wgs), unsigned((a.cout + 32 * CW - 1) / (32 * CW)));
    if (a.cout % (32 * CW) == 0)
      hipLaunchKernelGGL((k_mix_stream<T, WT, NK, CW, true>), grid, dim3(kThreads), 0, s, a, l,
                         chunk);
    else
      hipLaunchKernelGGL((k_mix_stream<T, WT, NK, CW, false>), grid, dim3(kThreads), 0, s, a, l,
                         chunk);
    return hipGetLastError();
  };
  if (a.cout > 64) return go(std::integral_constant<int, 4>{});
  if (a.cout > 32) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

template <class T, bool WT>
hipError_t launch_stream_k(const MixArgs& a, const MixList& l, hipStream_t s) {
  if (a.cin <= 32) return launch_stream<T, WT, 1>(a, l, s);
  if (a.cin <= 64) return launch_stream<T, WT, 2>(a, l, s);
  return launch_stream<T, WT, 4>(a, l, s);
}

// Whether W's columns fit into registers.  (20,000 x 4 rows in 10 groups, bf16,
// 256 to 256 channels: 43 us so, 28 through tiles; 20,000 x 16 rows of 128: 32
// and 39; of 64: 17 and 31.)
bool streams(const MixArgs& a, const MixList& l) {
  for (int i = 0; i < l.n_blocks; ++i)
    if (l.blk[i].n_src > 1) return false;
  return a.cin <= 128;
}

// Few rows of a group: what counts is that the weights are asked for at once.
// A wavefront takes 16 rows and 16 columns, straight from memory into the
// products' operands, and asks for 4 (bf16: 8) times 32 k before it multiplies
// the first; the products are added in the other kernels' order, so that a
// row's result stays the same.
template <class T, bool WT>
__global__ void __launch_bounds__(64) k_mix_few(const MixArgs a, const MixList l) {
  constexpr int PARTS = kParts<T>, VEC = 16 / sizeof(T), N = PARTS == 3 ? 4 : 8;
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups);
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(blockIdx.x)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  if (!find_tile(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, 16,
                 int64_t(blockIdx.x) - blk.wg0, tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.x);
  const int lane = threadIdx.x, q = lane & 15, h = lane >> 4;
  const int n_rows = int(min(int64_t(16), tile.rows - tile.at)), col0 = int(blockIdx.y) * 16;
  const TileRows rows(tile.at, blk.deg);
  int m;
  const int row = order(rows.place(min(q, n_rows - 1), m));
  const int chunks = (a.cin + 31) / 32;
  const int steps = tile.group < a.n_groups ? blk.n_src * chunks : 0;
  const T* x = static_cast<const T*>(a.x) + (int64_t(row) * a.din + m) * a.cin;
  const int col = min(col0 + q, a.cout - 1);  // (columns past the end are not stored)
  const T* W = static_cast<const T*>(a.W) + int64_t(tile.group) * a.pairs * a.cin * a.cout +
               (WT ? int64_t(col) * a.cin : col);
  f32x4 acc[1][1] = {};
  for (int s0 = 0; s0 < steps; s0 += N) {
    T xv[N][8], wv[N][8];
    bool have[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {  // past the last step it is asked for again
      const int s = min(s0 + i, steps - 1), of = s / chunks;
      int k = (s - of * chunks) * 32 + h * 8;
      have[i] = k < a.cin;
      k = have[i] ? k : 0;
      const MixSource sc = l.src[blk.src0 + of];
      const T* xp = x + int64_t(sc.in_off) * a.cin + k;
      const T* w = W + int64_t(sc.pair) * a.cin * a.cout + (WT ? k : int64_t(k) * a.cout);
#pragma unroll
      for (int e = 0; e < 8; e += VEC)
        *reinterpret_cast<u32x4*>(&xv[i][e]) = *reinterpret_cast<const u32x4*>(xp + e);
      if constexpr (WT) {
#pragma unroll
        for (int e = 0; e < 8; e += VEC)
          *reinterpret_cast<u32x4*>(&wv[i][e]) = *reinterpret_cast<const u32x4*>(w + e);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) wv[i][e] = w[int64_t(e) * a.cout];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    const auto operand = [&](const T (&v)[8], bool have, bf16x8 (&out)[PARTS]) {
      if constexpr (PARTS == 3) {
        bf16x4 lo[3], hi[3];
        split3(have ? f32x4{v[0], v[1], v[2], v[3]} : f32x4{}, lo);
        split3(have ? f32x4{v[4], v[5], v[6], v[7]} : f32x4{}, hi);
#pragma unroll
        for (int t = 0; t < 3; ++t)
          out[t] = __builtin_shufflevector(lo[t], hi[t], 0, 1, 2, 3, 4, 5, 6, 7);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          out[0][e] = have ? __builtin_bit_cast(__bf16, v[e]) : __bf16(0.0f);
      }
    };
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (s0 + i < steps) {
        bf16x8 xf[1][PARTS], wf[1][PARTS];
        operand(xv[i], have[i], xf[0]);
        operand(wv[i], have[i], wf[0]);
        products<PARTS, 1, 1>(wf, xf, acc);
      }
  }
  if (q >= n_rows || col0 + h * 4 >= a.cout) return;
  T* y = static_cast<T*>(a.y) + (int64_t(row) * a.dout + blk.out_off + m) * a.cout + col0 + h * 4;
  if constexpr (PARTS == 3) *reinterpret_cast<f32x4*>(y) = acc[0][0];
  else *reinterpret_cast<bf16x4*>(y) = __builtin_convertvector(acc[0][0], bf16x4);
}

template <class T>
hipError_t launch_few(const MixArgs& a, MixList l, hipStream_t s) {
  int64_t wgs = 0;
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, 16, a.index != nullptr);
  }
  const dim3 grid(unsigned(wgs), unsigned((a.cout + 15) / 16));
  if (a.w_trans) hipLaunchKernelGGL((k_mix_few<T, true>), grid, dim3(64), 0, s, a, l);
  else hipLaunchKernelGGL((k_mix_few<T, false>), grid, dim3(64), 0, s, a, l);
  return hipGetLastError();
}

template <class T>
hipError_t launch_mix_t(const MixArgs& a, MixList l, hipStream_t s) {
  const bool stream = streams(a, l);
  if (stream ? few_rows(a.n_rows, a.n_groups, l)
             : small_tiles(a.n_rows, a.n_groups, l, a.cout) <= (sizeof(T) == 4 ? 6000 : 1200))
    return launch_few<T>(a, l, s);
  if (stream)
    return a.w_trans ? launch_stream_k<T, true>(a, l, s) : launch_stream_k<T, false>(a, l, s);
  int64_t wgs = 0;
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += xcd_workgroups(most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, kTile,
                                     a.index != nullptr), (a.cout + kTile - 1) / kTile);
    if (wgs > (int64_t(1) << 30)) return hipErrorInvalidValue;
  }
  return launch_tiles(wgs, kThreads, [&](unsigned n, unsigned first) {
    MixArgs part = a;
    part.wg0 = first;
    const dim3 grid{n};
    if constexpr (sizeof(T) == 2) {
      if (a.w_trans) hipLaunchKernelGGL((k_mix_along<true>), grid, dim3(kThreads), 0, s, part, l);
      else hipLaunchKernelGGL((k_mix_along<false>), grid, dim3(kThreads), 0, s, part, l);
    } else {
      if (a.w_trans) hipLaunchKernelGGL((k_mix<true>), grid, dim3(kThreads), 0, s, part, l);
      else hipLaunchKernelGGL((k_mix<false>), grid, dim3(kThreads), 0, s, part, l);
    }
  });
}

// ------------------------------------------------------- weight gradients

struct MixDwList {
  int n_pairs;
  MixPair p[kMixSources];
};

// Rows of a workgroup's part of a group's sum.  Parts of a group that has
// several are written to the workspace and added afterwards; the only part of a
// group goes straight to dW.  Parts are short enough to fill the chip, in bf16
// about once (with dx, 384 parts and 512 of all tiles: 20,000 x 16 rows of 128
// channels 94 us and 104, 100,000 x 9 rows of 64 138 and 125, 16,411 rows of
// 1024 x 2048 243 both), in float32, whose rows take
// longest, twice; but not so short that a part's beginning and end outweigh its
// rows, or that all of them are more than half of what x and dy are (3,051 rows
// in 9 groups, 744 x 256 channels in float32 with dx: 57 us, 89 with parts of an
// eighth).  Where one group's tiles fill the chip there are no parts.
int64_t dw_rows(int64_t n_rows, int cin, int cout, const MixPair* p, int n_pairs, int esize) {
  const int64_t tiles = int64_t((cin + kTile - 1) / kTile) * ((cout + kTile - 1) / kTile);
  if (tiles >= 256) return int64_t(1) << 40;
  int64_t comps = 0;
  for (int i = 0; i < n_pairs; ++i) comps += p[i].deg;
  const int64_t least = std::max(int64_t(8) * cin * cout / (int64_t(cin + cout) * esize),
                                 int64_t(esize == 4 ? 128 : 512));
  const int64_t rows = std::max(n_rows * comps * tiles / (esize == 4 ? 1024 : 384), least);
  return (rows + 63) / 64 * 64;
}
// Most parts that groups with several can have together: each holds half of
// `rows` at least on average.
__host__ __device__ inline int64_t dw_parts(int64_t n_rows, int deg, int64_t rows) {
  const int64_t n = n_rows * deg;
  return n > rows ? 2 * n / rows : 0;
}
// Parts of the groups before group g that have several.
__device__ __forceinline__ int parts_before(const int* offsets, int g, int deg, int64_t rows) {
  int total = 0;
  for (int g0 = 0; g0 < g; g0 += 64) {
    const int i = g0 + int(threadIdx.x & 63);
    int n = 0;
    if (i < g) n = int((int64_t(offsets[i + 1] - offsets[i]) * deg + rows - 1) / rows);
    n = n > 1 ? n : 0;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    total += n;
  }
  return total;
}

// What a workgroup adds up: rows of a group for 128 x 128 elements of a pair.
struct DwTile {
  GroupTile tile;
  int pair, a0, b0;  // first channels
  int64_t n;         // rows
  int last;          // last of the group's rows that has one
  const int* order;
  __device__ __forceinline__ bool find(const MixDwArgs& a, const MixDwList& l, int64_t part_rows) {
    const bool valid = index_matches(a.index, a.n_rows, a.n_groups);
    const int* offsets = a.index ? a.index + a.offsets : nullptr;
    pair = int(blockIdx.y);
    const int deg = l.p[pair].deg;
    // neighbouring workgroups are on different XCDs, each of which takes
    // neighbouring tiles, whose rows of x and dy meet in its L2
    const int row_tiles = (a.cin + kTile - 1) / kTile;
    const int tiles = row_tiles * ((a.cout + kTile - 1) / kTile);
    int of = int(blockIdx.x) % tiles;
    if (tiles % 8 == 0) of = of % 8 * (tiles / 8) + of / 8;
    a0 = of % row_tiles * kTile;
    b0 = of / row_tiles * kTile;
    if (!find_tile(offsets, a.n_groups, a.n_rows, deg, part_rows, int(blockIdx.x) / tiles, tile,
                   1) || tile.group >= a.n_groups || !valid)
      return false;
    n = min(part_rows, tile.rows - tile.at);
    order = a.index ? a.index + a.order + tile.first : nullptr;
    last = int((tile.at + n - 1) / deg);
    return true;
  }
  // Where the sums go.
  __device__ __forceinline__ float* out(const MixDwArgs& a, const MixDwList& l,
                                        int64_t part_rows) const {
    const int64_t size = int64_t(a.cin) * a.cout;
    if (tile.rows <= part_rows) return a.dW + (int64_t(tile.group) * a.pairs + pair) * size;
    int64_t at = tile.at / part_rows;
    for (int i = 0; i < pair; ++i) at += dw_parts(a.n_rows, l.p[i].deg, part_rows);
    if (a.index)
      at += parts_before(a.index + a.offsets, tile.group, l.p[pair].deg, part_rows);
    return a.part + at * size;
  }
};

// NR rows that a lane loads, k, k + STRIDE and so on of a chunk of BK, in memory
// (row, component).  A chunk's rows are asked for a chunk ahead of their channels;
// past the end they are the last row again (places count on, and the last one
// may be 2^31 - 2: unsigned).
template <int STRIDE, int BK, int NR>
struct DwRows {
  unsigned at[NR], last, step_at;
  int m[NR], row[NR], deg, step_m;
  const int* order;
  __device__ __forceinline__ DwRows(const DwTile& d, int deg_, int k)
      : last(unsigned(d.last)), step_at(unsigned(BK / deg_)), deg(deg_), step_m(BK % deg_),
        order(d.order) {
    const int64_t from = d.tile.at / deg;
    const unsigned m0 = unsigned(d.tile.at - from * deg);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const unsigned u = m0 + unsigned(k + j * STRIDE), e = u / unsigned(deg);
      at[j] = unsigned(from) + e;
      m[j] = int(u - e * unsigned(deg));
    }
  }
  __device__ __forceinline__ void find() {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const unsigned t = min(at[j], last);
      row[j] = order ? order[t] : int(t);
    }
  }
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      at[j] += step_at;
      m[j] += step_m;
      if (m[j] >= deg) {
        m[j] -= deg;
        ++at[j];
      }
    }
  }
};

// float32: rows pass through registers, where they are split and turned, to
// LDS (64,000 x 16 rows of 128 channels: 275 us, 41% of the cycles products).
// Channel 4 c + e of a tile lies in LDS row 32 e + c, so that neighbouring
// threads write neighbouring rows.
__global__ void __launch_bounds__(kThreads, 2)
    k_mix_dw(const MixDwArgs a, const MixDwList l, int64_t part_rows) {
  constexpr int BK = 32, CT = kTile / 4;
  static_assert(kThreads / CT * 4 == BK);
  __shared__ __attribute__((aligned(16))) __bf16 s_x[3][kTile * BK], s_y[3][kTile * BK];
  DwTile d;
  if (!d.find(a, l, part_rows)) return;
  const MixPair p = l.p[d.pair];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave & 1, wn = wave >> 1, q = lane & 15, h = lane >> 4;

  f32x4 acc[4][4];  // [input channels][output channels]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};

  // this thread's 4 channels of 4 consecutive rows of a chunk.  Channels and
  // rows past the end are read at the last ones' place and then cleared.
  const int c = tid % CT, k = tid / CT * 4;
  const bool in_x = d.a0 + c * 4 < a.cin, in_y = d.b0 + c * 4 < a.cout;
  const float* x0 = static_cast<const float*>(a.x) + int64_t(p.in_off) * a.cin +
                    (in_x ? d.a0 + c * 4 : 0);
  const float* y0 = static_cast<const float*>(a.dy) + int64_t(p.out_off) * a.cout +
                    (in_y ? d.b0 + c * 4 : 0);
  DwRows<1, BK, 4> rows(d, p.deg, k);
  f32x4 xv[4], yv[4];
  const auto fetch = [&]() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = rows.row[j];
      xv[j] = *reinterpret_cast<const f32x4*>(x0 + (r * a.din + rows.m[j]) * a.cin);
      yv[j] = *reinterpret_cast<const f32x4*>(y0 + (r * a.dout + rows.m[j]) * a.cout);
    }
    rows.next();
  };
  const bool whole = d.a0 + kTile <= a.cin && d.b0 + kTile <= a.cout;
  const auto stage = [&](__bf16 (&s)[3][kTile * BK], f32x4 (&v)[4], bool in, int64_t left) {
    if (!whole || left < BK) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!in || k + j >= left) v[j] = f32x4{};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bf16x4 part[3];
      split3(f32x4{v[0][e], v[1][e], v[2][e], v[3][e]}, part);
#pragma unroll
      for (int u = 0; u < 3; ++u)
        *reinterpret_cast<bf16x4*>(&s[u][lds_at<BK>(e * CT + c, k / 8) + k % 8]) = part[u];
    }
  };

  if (d.n > 0) {
    rows.find();
    fetch();
    rows.find();
  }
  for (int64_t k0 = 0; k0 < d.n; k0 += BK) {
    __syncthreads();
    stage(s_x, xv, in_x, d.n - k0);
    stage(s_y, yv, in_y, d.n - k0);
    __syncthreads();
    fetch();  // (past the end: the last rows again)
    rows.find();
    bf16x8 yf[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int t = 0; t < 3; ++t)
        yf[j][t] = *reinterpret_cast<const bf16x8*>(&s_y[t][lds_at<BK>(j * CT + wn * 16 + q, h)]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x8 xf[1][3];
#pragma unroll
      for (int t = 0; t < 3; ++t)
        xf[0][t] = *reinterpret_cast<const bf16x8*>(&s_x[t][lds_at<BK>(i * CT + wm * 16 + q, h)]);
      products<3, 1, 4>(xf, yf, reinterpret_cast<f32x4(&)[1][4]>(acc[i]));
    }
  }

  float* out = d.out(a, l, part_rows);
  const int col = d.b0 + (wn * 16 + q) * 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = d.a0 + (wm * 16 + 4 * h + r) * 4 + i;
      f32x4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = acc[i][j][r];
      if (row < a.cin && col < a.cout)
        *reinterpret_cast<f32x4*>(out + int64_t(row) * a.cout + col) = v;
    }
  }
}

// The same in bf16: rows of x and dy go straight to LDS as they lie in memory
// and are read across them; one chunk of 32 rows is multiplied while the next is
// on its way, three workgroups on a compute unit (16,411 rows in 16 groups, 1024
// x 2048 channels with dx: 245 us, chunks of 64 and two workgroups 252, where
// runs of either lie between 245 and 270).  Rows past the end are zeros.
// (Turned in registers on their way to LDS instead: 13,742 rows in 6 groups,
// 1264 x 312 channels, 92 us, 65 so.)
__global__ void __launch_bounds__(kThreads, 3)
    k_mix_dw_across(const MixDwArgs a, const MixDwList l, int64_t part_rows) {
  constexpr int BK = 32, BYTES = BK * kTile * 2;
  __shared__ __attribute__((aligned(128))) uint8_t s_x0[BYTES], s_y0[BYTES];
  __shared__ __attribute__((aligned(128))) uint8_t s_x1[BYTES], s_y1[BYTES];
  DwTile d;
  if (!d.find(a, l, part_rows)) return;
  const MixPair p = l.p[d.pair];
  const TileLoad load;
  const AcrossLoad<2> across;
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const int wm = load.wave & 1, wn = load.wave >> 1;
  f32x4 acc[4][4];  // [input channels][output channels]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  const int ca = d.a0 + across.piece * 8, cb = d.b0 + across.piece * 8;
  const bool in_x = ca < a.cin, in_y = cb < a.cout;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.x) + (int64_t(p.in_off) * a.cin + ca) * 2;
  const uint8_t* y0 = static_cast<const uint8_t*>(a.dy) + (int64_t(p.out_off) * a.cout + cb) * 2;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kTileZeros);
  DwRows<16, BK, 2> rows(d, p.deg, across.row);
  int64_t left = d.n - across.row;
  const auto fetch = [&](uint8_t* x, uint8_t* y) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bool in = j * 16 < left;
      const int64_t xo = (int64_t(rows.row[j]) * a.din + rows.m[j]) * a.cin * 2;
      const int64_t yo = (int64_t(rows.row[j]) * a.dout + rows.m[j]) * a.cout * 2;
      load.ask(in && in_x ? x0 + xo : zeros, x, j);
      load.ask(in && in_y ? y0 + yo : zeros, y, j);
    }
    left -= BK;
    rows.next();
    rows.find();
  };
  const int64_t steps = (d.n + BK - 1) / BK;
  const auto turn = [&](const uint8_t* x, const uint8_t* y, uint8_t* x_free, uint8_t* y_free,
                        int64_t step) {
    tile_wait();
    fetch(x_free, y_free);
    if (step >= steps) return;
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 yf[4][1];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      yf[j][0] = across.read(y, 0, wn * 8 + j * 2 + ((lane & 3) >> 1), lane & 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x8 xf[1][1] = {
          {across.read(x, 0, wm * 8 + i * 2 + ((lane & 3) >> 1), lane & 1)}};
      // rows of the products: output channels
      products<1, 4, 1>(yf, xf, reinterpret_cast<f32x4(&)[4][1]>(acc[i]));
    }
  };
  if (steps > 0) {
    rows.find();
    fetch(s_x0, s_y0);
  }
  for (int64_t step = 0; step < steps; step += 2) {
    turn(s_x0, s_y0, s_x1, s_y1, step);
    turn(s_x1, s_y1, s_x0, s_y0, step + 1);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load writes to LDS after the end
  // dW past the caches, which x and dy need (16,384 rows in 16 groups, 1024 x
  // 2048, in chunks of 64 rows, with dx: 199 us, 226 without, where they are in
  // the caches from a call before; 253 and 257 where not, no more than runs
  // differ; in float32, whose products take longer, no difference either); parts
  // are read again soon
  float* out = d.out(a, l, part_rows);
  const bool part = d.tile.rows > part_rows;
  const RowHalves halves;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ch = d.a0 + wm * 64 + i * 16 + (q & 7);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {  // 32 columns are a line
      halves.trade(acc[i][j], acc[i][j + 1]);
      const int col = d.b0 + wn * 64 + j * 16 + halves.column / 4;
      f32x4* to0 = reinterpret_cast<f32x4*>(out + int64_t(ch) * a.cout + col);
      f32x4* to1 = reinterpret_cast<f32x4*>(out + int64_t(ch + 8) * a.cout + col);
      const bool in0 = col < a.cout && ch < a.cin, in1 = col < a.cout && ch + 8 < a.cin;
      if (part) {
        if (in0) *to0 = acc[i][j];
        if (in1) *to1 = acc[i][j + 1];
      } else {
        if (in0) __builtin_nontemporal_store(acc[i][j], to0);
        if (in1) __builtin_nontemporal_store(acc[i][j + 1], to1);
      }
    }
  }
}

// dW of the groups with several parts, added in their order, 1024 elements of a
// (group, pair) at a time; most groups may have nothing here, so that the
// launch is of kSumTarget workgroups rather than of one for every 1024 elements
// (16 groups of 1024 x 2048 without parts: 18 us and 4.6).
constexpr int kSumTarget = 1024;
__global__ void __launch_bounds__(256) k_mix_dw_sum(const MixDwArgs a, const MixDwList l,
                                                    int64_t part_rows) {
  if (!index_matches(a.index, a.n_rows, a.n_groups)) return;
  const int g = int(blockIdx.y), pi = int(blockIdx.z), deg = l.p[pi].deg;
  const int64_t size = int64_t(a.cin) * a.cout;
  const int* offsets = a.index ? a.index + a.offsets : nullptr;
  const int64_t rows = (offsets ? offsets[g + 1] - offsets[g] : a.n_rows) * deg;
  const int n = int((rows + part_rows - 1) / part_rows);
  if (n < 2) return;
  int64_t at = offsets ? parts_before(offsets, g, deg, part_rows) : 0;
  for (int i = 0; i < pi; ++i) at += dw_parts(a.n_rows, l.p[i].deg, part_rows);
  const float* part = a.part + at * size;
  float* dW = a.dW + (int64_t(g) * a.pairs + pi) * size;
  const int64_t step = int64_t(gridDim.x) * 1024;
  for (int64_t e = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; e < size; e += step) {
    f32x4 s{};
#pragma unroll 4
    for (int i = 0; i < n; ++i) s += *reinterpret_cast<const f32x4*>(part + i * size + e);
    *reinterpret_cast<f32x4*>(dW + e) = s;
  }
}

template <class T>
hipError_t launch_mix_dw_t(const MixDwArgs& a, const MixPair* p, hipStream_t s) {
  MixDwList l;
  l.n_pairs = a.pairs;
  int deg = 1;
  for (int i = 0; i < a.pairs; ++i) {
    l.p[i] = p[i];
    deg = std::max(deg, p[i].deg);
  }
  const int64_t rows = dw_rows(a.n_rows, a.cin, a.cout, p, a.pairs, sizeof(T));
  const int64_t slots = most_tiles(a.n_rows, a.n_groups, deg, rows, true) + 1;
  const int64_t tiles = int64_t((a.cin + kTile - 1) / kTile) * ((a.cout + kTile - 1) / kTile);
  const dim3 grid(unsigned(slots * tiles), unsigned(a.pairs));
  if constexpr (sizeof(T) == 2)
    hipLaunchKernelGGL(k_mix_dw_across, grid, dim3(kThreads), 0, s, a, l, rows);
  else hipLaunchKernelGGL(k_mix_dw, grid, dim3(kThreads), 0, s, a, l, rows);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n_rows * deg <= rows) return e;
  const int64_t runs = std::min((int64_t(a.cin) * a.cout + 1023) / 1024,
                                kSumTarget / (int64_t(a.n_groups) * a.pairs) + 1);
  hipLaunchKernelGGL(k_mix_dw_sum,
                     dim3(unsigned(runs), unsigned(a.n_groups), unsigned(a.pairs)), dim3(256), 0, s,
                     a, l, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mix(const MixArgs& a, const MixList& l, int bf16, hipStream_t s) {
  return bf16 ? launch_mix_t<bf16_t>(a, l, s) : launch_mix_t<float>(a, l, s);
}

size_t mix_dw_part_floats(int64_t n_rows, int cin, int cout, const MixPair* p, int n_pairs) {
  int64_t most = 0;  // for either storage type
  for (int esize : {2, 4}) {
    const int64_t rows = dw_rows(n_rows, cin, cout, p, n_pairs, esize);
    int64_t parts = 0;
    for (int i = 0; i < n_pairs; ++i) parts += dw_parts(n_rows, p[i].deg, rows);
    most = std::max(most, parts);
  }
  return size_t(most) * cin * cout;
}

hipError_t launch_mix_dw(const MixDwArgs& a, const MixPair* p, int bf16, hipStream_t s) {
  return bf16 ? launch_mix_dw_t<bf16_t>(a, p, s) : launch_mix_dw_t<float>(a, p, s);
}

}  // namespace e3k
