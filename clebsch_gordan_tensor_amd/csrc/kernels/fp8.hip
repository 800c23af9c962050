// Channel mixing of 8-bit features with 8-bit weights (e4m3), next to the
// quantisation of both: with s_x a scale for 128 channels of a component row
// of x and s_W one for 128 x 128 weights,
//   y[r][n] = sum over blocks b of 128 channels of
//             s_x[r][b] s_W[b][n / 128] sum_{k in b} x8[r][k] W8[k][n].
// The inner sum of a block enters the float32 result by one multiply-add with
// the product of the two scales, which the columns of a block and a lane's row
// share.  It is formed
//   for bf16 y by one instruction, v_mfma_f32_16x16x128_f8f6f4.  Within 8
//     consecutive products that drops what lies below 2^-13 of the largest one
//     (measured, and so does v_mfma_f32_16x16x32_fp8_fp8); the eights are added
//     in float32.  On normal values the sums are off by 1.5e-5 (root mean
//     square, relative), a hundredth of the rounding to bf16 that follows; of
//     a small difference of large terms they are off by as much of the terms;
//   for float32 y from the codes' values in bf16, which are exact, by four
//     v_mfma_f32_16x16x32_bf16 (2e-8 off on the same values).
//
// Operands: a lane q + 16 h holds 32 bytes of row (or column) q, the bytes
// 16 h .. 16 h + 15 of either half of the block; which k these are does not
// matter as long as both operands agree.  W is taken as A: register r of lane
// q + 16 h is column 4 h + r of row q.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.h"
#include "fp8.h"
#include "group_tiles.h"
#include "registry.h"
#include "row_halves.h"
#include "tile128.h"

namespace e3k {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;

// ------------------------------------------------------------ quantisation

// A run of 128 channels of a row: L lanes of 4 channels (float32) or 8 (bf16),
// fewer than a run's 128 channels need where rows are shorter (972,000 rows of
// 32 float32 channels: 87 us with 32 lanes each, 26 with 8).
template <class T, int L>
__global__ void __launch_bounds__(kThreads)
    k_fp8_quantize(int64_t n_runs, int runs, int C, const T* __restrict__ x,
                   uint8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x % L;
  for (int64_t t = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / L; t < n_runs;
       t += int64_t(gridDim.x) * (kThreads / L)) {
    const int64_t row = L * V < kFp8Run      ? t
                        : n_runs < (1 << 30) ? unsigned(t) / unsigned(runs)
                                             : t / runs;
    const int k = int(t - row * runs) * kFp8Run + lane * V;
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.0f;
    if (k < C) load_ch<T, V>(x + row * C + k, v);
    float top = fp8_top(v);
#pragma unroll
    for (int o = 1; o < L; o <<= 1) top = fp8_max(top, __shfl_xor(top, o));
    const Fp8Scale s(top);
    if (k < C) fp8_store<V, false>(q + row * C + k, v, s);
    if (lane == 0) scale[t] = s.scale;
  }
}

// Whether the weights are packed for this call; without pairs there are none,
// nor a header.
__device__ __forceinline__ bool weights_match(const Fp8MixArgs& a) {
  if (a.pairs == 0) return true;
  const int* header = static_cast<const int*>(a.packed);
  return (header[0] == kFp8Magic) & (header[1] == a.cin) & (header[2] == a.cout) &
         (header[3] == a.pairs) & (header[4] == a.n_groups);
}

// A block of 128 x 128 weights a workgroup: thread (c, k) takes 4 columns of
// 16 consecutive k, whose codes it stores side by side.  16 x 2048 x 1024: 27 us
// (6.2 TB/s, in part from the caches).
__global__ void __launch_bounds__(kThreads)
    k_fp8_pack(int pairs, int groups, int cin, int cout, Fp8Layout l, const float* __restrict__ W,
               uint8_t* __restrict__ packed) {
  __shared__ float s_top[kThreads / 64];
  const int64_t mat = blockIdx.x / l.in_blocks;
  const int kb = int(blockIdx.x % l.in_blocks), nb = int(blockIdx.y), tid = threadIdx.x;
  if (kb == 0 && nb == 0 && mat == 0 && tid == 0) {
    int* header = reinterpret_cast<int*>(packed);
    header[0] = kFp8Magic;
    header[1] = cin;
    header[2] = cout;
    header[3] = pairs;
    header[4] = groups;
  }
  const int n = nb * 128 + tid % 32 * 4, k0 = kb * 128 + tid / 32 * 16;
  const float* w = W + mat * cin * cout;
  f32x4 v[16];
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    v[j] = k0 + j < cin && n < cout
               ? *reinterpret_cast<const f32x4*>(w + int64_t(k0 + j) * cout + n)
               : f32x4{};
    const float t[4] = {v[j][0], v[j][1], v[j][2], v[j][3]};
    top = fp8_max(top, fp8_top(t));
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) top = fp8_max(top, __shfl_xor(top, o));
  if ((tid & 63) == 0) s_top[tid >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kThreads / 64; ++j) top = fp8_max(top, s_top[j]);
  const Fp8Scale s(top);
  if (tid == 0)
    reinterpret_cast<float*>(packed + l.scales)[(mat * l.out_blocks + nb) * l.in_blocks + kb] =
        s.scale;
  if (n >= cout) return;
  uint8_t* out = packed + l.codes + (mat * cout + n) * (int64_t(l.in_blocks) * 128) + k0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    u32x4 c;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = fp8_codes(v[4 * j][e], v[4 * j + 1][e], v[4 * j + 2][e], v[4 * j + 3][e], s);
    *reinterpret_cast<u32x4*>(out + int64_t(e) * l.in_blocks * 128) = c;
  }
}

// --------------------------------------------------------------- the mixing

// A block's operand of one row or column: the codes, or their values.
struct Values {
  bf16x8 v[4];
};
template <class T>
struct Operand {
  using type = i32x8;
  __device__ __forceinline__ static i32x8 of(i32x8 c) { return c; }
};
template <>
struct Operand<float> {
  using type = Values;
  __device__ __forceinline__ static Values of(i32x8 c) {
    Values r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true);
      r.v[i / 2][i % 2 * 4] = lo[0];
      r.v[i / 2][i % 2 * 4 + 1] = lo[1];
      r.v[i / 2][i % 2 * 4 + 2] = hi[0];
      r.v[i / 2][i % 2 * 4 + 3] = hi[1];
    }
    return r;
  }
};
__device__ __forceinline__ f32x4 product(const i32x8& a, const i32x8& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 product(const Values& a, const Values& b) {
  f32x4 c{};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

// Column of a tile in slot s: as the results are stored 16 bytes at once, for
// bf16 two products' columns alternate by fours.
template <class T>
__device__ __forceinline__ int column_in(int s) {
  if constexpr (std::is_same_v<T, float>) return s;
  else return (s & ~31) | ((s >> 2) & 3) << 3 | ((s >> 4) & 1) << 2 | (s & 3);
}

// Steps whose scales of the rows are in LDS at once.  Asked for step by step
// they cost more of the L1 than the tiles (a line of memory for every row):
// 16 experts of 2048 x 1024 channels took 96 us, 69 without any.
constexpr int kScaleSteps = 16;

// Tiles of 128 rows by 128 columns, one chunk of 128 k multiplied while the
// next is on its way; two workgroups on a compute unit.  16,411 rows of 16
// experts, 2048 to 1024 channels: 73 us (940 TFLOP/s), to float32 107 (its bf16
// products and twice the results); 256 columns a
// workgroup, alone on its compute unit with two chunks on their way, 85 us,
// three rounds of workgroups where 2.3 would do.
template <class T>
__global__ void __launch_bounds__(kThreads, 2) k_fp8_mix(const Fp8MixArgs a, const MixList l,
                                                      const Fp8Layout at) {
  // a name for every stage: reads of one are then known not to wait for loads
  // into the other
  __shared__ __attribute__((aligned(128))) uint8_t s_x0[TileLoad::kBytes], s_w0[TileLoad::kBytes];
  __shared__ __attribute__((aligned(128))) uint8_t s_x1[TileLoad::kBytes], s_w1[TileLoad::kBytes];
  __shared__ float s_scale[kTileRows][kScaleSteps + 1];
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups) && weights_match(a);
  const unsigned wg = a.wg0 + blockIdx.x;
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(wg)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  int col_tile;
  if (!find_tile_xcd(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg,
                     kTileRows, wg - unsigned(blk.wg0),
                     unsigned((a.cout + 127) / 128), tile, col_tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.q);
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const TileLoad load;
  const int wm = load.wave & 1, wn = load.wave >> 1;
  const int col0 = col_tile * 128;
  const int n_rows = int(min(int64_t(kTileRows), tile.rows - tile.at));
  const TileRows rows(tile.at, blk.deg);
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};

  // the rows this lane loads, and those it ends with; rows past the end are
  // the last one again, and so are columns
  const int runs = at.in_blocks;
  const int64_t kpad = int64_t(runs) * 128;
  const uint8_t* packed = static_cast<const uint8_t*>(a.packed);
  int load_row[4], load_m[4], row[4], comp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    load_row[j] = order(rows.place(min(load.row + j * 32, n_rows - 1), load_m[j]));
    row[j] = order(rows.place(min(wm * 64 + j * 16 + q, n_rows - 1), comp[j]));
  }
  int scale_m;  // two threads share a row's scales
  const int scale_of = order(rows.place(min(int(threadIdx.x) / 2, n_rows - 1), scale_m));
  const float* scale_row = a.scale + (int64_t(scale_of) * a.din + scale_m) * runs;
  const uint8_t *xrow[4], *wrow[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    xrow[j] = static_cast<const uint8_t*>(a.q) +
              (int64_t(load_row[j]) * a.din + load_m[j]) * a.cin + load.piece * 16;
    const int n = min(col0 + column_in<T>(load.row + j * 32), a.cout - 1);
    wrow[j] = packed + at.codes + (int64_t(tile.group) * a.pairs * a.cout + n) * kpad +
              load.piece * 16;
  }

  // step s is run s % runs of source s / runs
  const int steps = tile.group < a.n_groups ? blk.n_src * runs : 0;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kTileZeros);
  int64_t xo = 0, wo = 0;  // of the chunk asked for next
  int src = -1, b = runs - 1;
  const auto advance = [&]() {  // past the last chunk it is asked for again
    if (b + 1 < runs) {
      ++b;
      xo += 128;
      wo += 128;
    } else if (src + 1 < blk.n_src) {
      const MixSource sc = l.src[blk.src0 + ++src];
      b = 0;
      xo = int64_t(sc.in_off) * a.cin;
      wo = int64_t(sc.pair) * a.cout * kpad;
    }
  };
  const auto fetch = [&](uint8_t* x, uint8_t* w) {
    advance();
    const bool in = b * 128 + load.piece * 16 < a.cin;
#pragma unroll
    for (int j = 0; j < 4; ++j) load.ask(in ? xrow[j] + xo : zeros, x, j);
#pragma unroll
    for (int j = 0; j < 4; ++j) load.ask(wrow[j] + wo, w, j);
  };
  // scales of the next kScaleSteps steps: the rows' into LDS, this wavefront's
  // columns' into its lanes
  float sw_lane = 0.0f;
  constexpr int SS = kScaleSteps;
  const auto scales = [&](int step0) {
    float v[SS / 2];
#pragma unroll
    for (int i = 0; i < SS / 2; ++i) {
      const int s = min(step0 + int(threadIdx.x) % 2 + i * 2, steps - 1), of = s / runs;
      v[i] = scale_row[l.src[blk.src0 + of].in_off * runs + s - of * runs];
    }
#pragma unroll
    for (int i = 0; i < SS / 2; ++i) s_scale[threadIdx.x / 2][threadIdx.x % 2 + i * 2] = v[i];
    const int s = min(step0 + lane % SS, steps - 1), of = s / runs;
    const int64_t mat = int64_t(tile.group) * a.pairs + l.src[blk.src0 + of].pair;
    sw_lane = reinterpret_cast<const float*>(packed + at.scales)[
        (mat * at.out_blocks + col_tile) * runs + s - of * runs];
    asm volatile("" ::"v"(sw_lane));  // here, and not where it is used: the walk waits for no loads
  };
  const auto turn = [&](const uint8_t* x, const uint8_t* w, uint8_t* x_free, uint8_t* w_free,
                        int step) {
    tile_wait();
    fetch(x_free, w_free);
    if (step >= steps) return;
    const int at_step = step % SS;
    const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sw_lane), at_step));
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = s_scale[wm * 64 + j * 16 + q][at_step] * sw;
    const auto operand = [&](const uint8_t* s, int r) {
      const u32x4 lo = *reinterpret_cast<const u32x4*>(tile_at(s, r, h));
      const u32x4 hi = *reinterpret_cast<const u32x4*>(tile_at(s, r, 4 + h));
      return Operand<T>::of(i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                                  int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])});
    };
    typename Operand<T>::type xf[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xf[j] = operand(x, wm * 64 + j * 16 + q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto wf = operand(w, wn * 64 + i * 16 + q);
      f32x4 t[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) t[j] = product(wf, xf[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(t[j][r], f[j], acc[i][j][r]);
    }
  };
  if (steps > 0) fetch(s_x0, s_w0);
  for (int step = 0; step < steps; step += 2) {
    if (step % SS == 0) {
      __syncthreads();
      scales(step);
      __syncthreads();
    }
    turn(s_x0, s_w0, s_x1, s_w1, step);
    turn(s_x1, s_w1, s_x0, s_w0, step + 1);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no load writes to LDS after the end
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (wm * 64 + j * 16 + q >= n_rows) continue;
    T* y = static_cast<T*>(a.y) + (int64_t(row[j]) * a.dout + blk.out_off + comp[j]) * a.cout;
    if constexpr (std::is_same_v<T, float>) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = col0 + wn * 64 + i * 16 + h * 4;
        if (n < a.cout) *reinterpret_cast<f32x4*>(y + n) = acc[i][j];
      }
    } else {
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
}

// Where every block has one source of at most 128 channels, that is one step:
// a wavefront holds 128 columns of W in registers and walks over its group's
// rows, 16 at a time, whose x goes from memory into the products' operand
// without passing through LDS; no wavefront waits for another.  The next 16
// rows' x and scales are under way meanwhile, and where the 16 after them lie.
// Nothing in the walk is conditional (a wait for loads would have to wait for
// stores that may not have been issued): rows past the end are the last atom's
// again, written with the same values.
constexpr int kStreamRows = 64;  // of a workgroup's wavefronts together

template <class T, bool FULL>
__global__ void __launch_bounds__(kThreads, 2) k_fp8_stream(const Fp8MixArgs a, const MixList l,
                                                            const Fp8Layout lay, int chunk) {
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups) && weights_match(a);
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(blockIdx.x)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  if (!find_tile(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, chunk,
                 int64_t(blockIdx.x) - blk.wg0, tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.q);
  const int lane = threadIdx.x & 63, q = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int col0 = int(blockIdx.y) * 128, deg = blk.deg;
  const int n = int(min(int64_t(chunk), tile.rows - tile.at));
  // (places count on past the last one, and that may be 2^31 - 2: unsigned)
  const unsigned last = unsigned((tile.at + n - 1) / deg), step_at = unsigned(kStreamRows / deg);
  const TileRows rows(tile.at, deg);
  const int step_m = kStreamRows % deg;
  int m;
  unsigned at = unsigned(rows.place(wave * 16 + q, m));  // of the next row to look up
  struct Row {
    int row, m;
  };
  const auto look = [&]() {
    const Row r{order(int(min(at, last))), m};
    at += step_at;
    m += step_m;
    if (m >= deg) {
      m -= deg;
      ++at;
    }
    return r;
  };
  if (tile.group >= a.n_groups || blk.n_src == 0) {  // zeros
    for (int t0 = wave * 16; t0 < n; t0 += kStreamRows) {
      const Row r = look();
      T* y = static_cast<T*>(a.y) + (int64_t(r.row) * a.dout + blk.out_off + r.m) * a.cout;
      for (int c = col0 + h; c < min(col0 + 128, a.cout); c += 4) y[c] = T{};
    }
    return;
  }
  const MixSource sc = l.src[blk.src0];
  const RowHalves halves;
  const uint8_t* x0 = static_cast<const uint8_t*>(a.q) + int64_t(sc.in_off) * a.cin;
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kTileZeros);
  const bool in_lo = h * 16 < a.cin, in_hi = 64 + h * 16 < a.cin;
  struct X {
    u32x4 lo, hi;
    float s;
  };
  const auto fetch = [&](const Row& r) {
    const int64_t at_row = int64_t(r.row) * a.din + r.m;
    const uint8_t* p = x0 + at_row * a.cin + h * 16;
    return X{*reinterpret_cast<const u32x4*>(in_lo ? p : zeros),
             *reinterpret_cast<const u32x4*>(in_hi ? p + 64 : zeros),
             a.scale[at_row + sc.in_off]};
  };
  Row now = look(), next = look();
  X x = fetch(now);

  const int64_t mat = int64_t(tile.group) * a.pairs + sc.pair;
  const uint8_t* packed = static_cast<const uint8_t*>(a.packed);
  const float sw =
      reinterpret_cast<const float*>(packed + lay.scales)[mat * lay.out_blocks + blockIdx.y];
  const auto operand = [&](u32x4 lo, u32x4 hi) {
    return Operand<T>::of(i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                                int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])});
  };
  typename Operand<T>::type wf[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = min(col0 + column_in<T>(i * 16 + q), a.cout - 1);
    const uint8_t* w = packed + lay.codes + (mat * a.cout + c) * 128 + h * 16;
    wf[i] = operand(*reinterpret_cast<const u32x4*>(w), *reinterpret_cast<const u32x4*>(w + 64));
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the walk counts its own loads alone
  for (int t0 = wave * 16; t0 < n; t0 += kStreamRows) {
    const X cur = x;
    x = fetch(next);
    const Row after = look();
    __builtin_amdgcn_sched_barrier(0);
    const auto xf = operand(cur.lo, cur.hi);
    const float f = cur.s * sw;
    Row r0, r1;
    halves.rows(now.row, r0.row, r1.row);
    halves.rows(now.m, r0.m, r1.m);
    const auto start = [&](const Row& r) {
      return reinterpret_cast<uint8_t*>(static_cast<T*>(a.y) +
                                        (int64_t(r.row) * a.dout + blk.out_off + r.m) * a.cout +
                                        col0) + halves.column;
    };
    uint8_t *y0 = start(r0), *y1 = start(r1);
    constexpr int LINE = 128 / sizeof(T), PER = LINE / 16;  // columns, products of a line
#pragma unroll
    for (int c = 0; c < 128 / LINE; ++c) {
      f32x4 u[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const f32x4 t = product(wf[c * PER + i], xf);
#pragma unroll
        for (int r = 0; r < 4; ++r) u[i][r] = t[r] * f;
      }
      u32x4 v[2];
      if constexpr (std::is_same_v<T, float>) {
        v[0] = __builtin_bit_cast(u32x4, u[0]);
        v[1] = __builtin_bit_cast(u32x4, u[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bf16x8 b;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            b[r] = __bf16(u[2 * i][r]);
            b[4 + r] = __bf16(u[2 * i + 1][r]);
          }
          v[i] = __builtin_bit_cast(u32x4, b);
        }
      }
      halves.trade(v[0], v[1]);
      if (FULL || col0 + c * LINE + halves.column / int(sizeof(T)) < a.cout) {
        __builtin_nontemporal_store(v[0], reinterpret_cast<u32x4*>(y0 + c * 128));
        __builtin_nontemporal_store(v[1], reinterpret_cast<u32x4*>(y1 + c * 128));
      }
    }
    now = next;
    next = after;
  }
}

// Rows of a workgroup's walk: some workgroups for every one that is resident.
int stream_chunk(int64_t rows) {
  const int64_t n = (rows / 1024 + kStreamRows - 1) / kStreamRows * kStreamRows;
  return int(std::min<int64_t>(4096, std::max<int64_t>(kStreamRows, n)));
}

template <class T>
hipError_t launch_fp8_stream(const Fp8MixArgs& a, MixList l, hipStream_t s) {
  int64_t wgs = 0, comps = 0;
  for (int i = 0; i < l.n_blocks; ++i) comps += l.blk[i].deg;
  const int chunk = stream_chunk(a.n_rows * comps);
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, chunk, a.index != nullptr);
  }
  const Fp8Layout at = fp8_layout(a.n_groups, a.pairs, a.cin, a.cout);
  const dim3 grid(unsigned(wgs), unsigned((a.cout + 127) / 128));
  if (a.cout % 128 == 0)
    hipLaunchKernelGGL((k_fp8_stream<T, true>), grid, dim3(kThreads), 0, s, a, l, at, chunk);
  else
    hipLaunchKernelGGL((k_fp8_stream<T, false>), grid, dim3(kThreads), 0, s, a, l, at, chunk);
  return hipGetLastError();
}

// Few rows of a group: what counts is that the weights are asked for at once.
// A wavefront takes 16 rows and 16 columns and asks for 8 steps (float32: 4)
// before it multiplies the first; the steps' sums are added in the other
// kernels' order, so that a row's result stays the same.
template <class T>
__global__ void __launch_bounds__(64) k_fp8_few(const Fp8MixArgs a, const MixList l,
                                                const Fp8Layout lay) {
  constexpr int N = std::is_same_v<T, float> ? 4 : 8;
  const bool valid = index_matches(a.index, a.n_rows, a.n_groups) && weights_match(a);
  int bi = 0;
  while (bi + 1 < l.n_blocks && l.blk[bi + 1].wg0 <= int(blockIdx.x)) ++bi;
  const MixBlock blk = l.blk[bi];
  GroupTile tile;
  if (!find_tile(a.index ? a.index + a.offsets : nullptr, a.n_groups, a.n_rows, blk.deg, 16,
                 int64_t(blockIdx.x) - blk.wg0, tile) || !valid)
    return;
  const RowOrder order(a.index, a.order, tile, a.q);
  const int lane = threadIdx.x, q = lane & 15, h = lane >> 4;
  const int n_rows = int(min(int64_t(16), tile.rows - tile.at)), col0 = int(blockIdx.y) * 16;
  const TileRows rows(tile.at, blk.deg);
  int m;
  const int row = order(rows.place(min(q, n_rows - 1), m));
  const int64_t at_row = int64_t(row) * a.din + m;
  const int runs = lay.in_blocks;
  const int steps = tile.group < a.n_groups ? blk.n_src * runs : 0;
  const uint8_t* x = static_cast<const uint8_t*>(a.q) + at_row * a.cin + h * 16;
  const float* sx = a.scale + at_row * runs;
  const uint8_t* packed = static_cast<const uint8_t*>(a.packed);
  const float* sw = reinterpret_cast<const float*>(packed + lay.scales);
  const uint8_t* zeros = reinterpret_cast<const uint8_t*>(kTileZeros);
  const auto operand = [&](u32x4 lo, u32x4 hi) {
    return Operand<T>::of(i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                                int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])});
  };
  f32x4 acc{};
  for (int s0 = 0; s0 < steps; s0 += N) {
    u32x4 xv[N][2], wv[N][2];
    float fx[N], fw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {  // past the last step it is asked for again
      const int s = min(s0 + i, steps - 1), of = s / runs, b = s - of * runs;
      const MixSource sc = l.src[blk.src0 + of];
      const int64_t mat = int64_t(tile.group) * a.pairs + sc.pair;
      const uint8_t* xp = x + int64_t(sc.in_off) * a.cin + b * 128;
      const uint8_t* wp = packed + lay.codes + ((mat * a.cout + col0 + q) * runs + b) * 128 + h * 16;
      xv[i][0] = *reinterpret_cast<const u32x4*>(b * 128 + h * 16 < a.cin ? xp : zeros);
      xv[i][1] = *reinterpret_cast<const u32x4*>(b * 128 + 64 + h * 16 < a.cin ? xp + 64 : zeros);
      wv[i][0] = *reinterpret_cast<const u32x4*>(wp);
      wv[i][1] = *reinterpret_cast<const u32x4*>(wp + 64);
      fx[i] = sx[sc.in_off * runs + b];
      fw[i] = sw[(mat * lay.out_blocks + col0 / 128) * runs + b];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (s0 + i < steps) {
        const f32x4 t = product(operand(wv[i][0], wv[i][1]), operand(xv[i][0], xv[i][1]));
        const float f = fx[i] * fw[i];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(t[r], f, acc[r]);
      }
  }
  if (q >= n_rows) return;
  T* y = static_cast<T*>(a.y) + (int64_t(row) * a.dout + blk.out_off + m) * a.cout + col0 + h * 4;
  if constexpr (std::is_same_v<T, float>)
    *reinterpret_cast<f32x4*>(y) = acc;
  else
    *reinterpret_cast<bf16x4*>(y) = __builtin_convertvector(acc, bf16x4);
}

template <class T>
hipError_t launch_fp8_few(const Fp8MixArgs& a, MixList l, hipStream_t s) {
  int64_t wgs = 0;
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, 16, a.index != nullptr);
  }
  hipLaunchKernelGGL((k_fp8_few<T>), dim3(unsigned(wgs), unsigned(a.cout / 16)), dim3(64), 0, s,
                     a, l, fp8_layout(a.n_groups, a.pairs, a.cin, a.cout));
  return hipGetLastError();
}

template <class T>
hipError_t launch_fp8_mix_t(const Fp8MixArgs& a, MixList l, hipStream_t s) {
  bool one = a.cin <= 128;
  for (int i = 0; i < l.n_blocks; ++i) one &= l.blk[i].n_src <= 1;
  // us by small tiles and by large, 1024 to 1024 channels: float32, one group,
  // 512 rows 12.5 and 17.5, 1024 21.7 and 17.6; 16 groups, 512 17.1 and 19.1;
  // bf16, one group, 256 rows 10.3 and 11.7, 512 12.2 and 11.7; 16 groups of
  // 2048 to 512, 512 rows 17.0 and 19.3, 1024 26.2 and 21.1
  if (one ? few_rows(a.n_rows, a.n_groups, l)
          : small_tiles(a.n_rows, a.n_groups, l, a.cout) <= (sizeof(T) == 4 ? 3000 : 1600))
    return launch_fp8_few<T>(a, l, s);
  if (one) return launch_fp8_stream<T>(a, l, s);
  int64_t wgs = 0;
  for (int i = 0; i < l.n_blocks; ++i) {
    l.blk[i].wg0 = int(wgs);
    wgs += xcd_workgroups(most_tiles(a.n_rows, a.n_groups, l.blk[i].deg, kTileRows,
                                     a.index != nullptr), (a.cout + 127) / 128);
    if (wgs > (int64_t(1) << 30)) return hipErrorInvalidValue;
  }
  const Fp8Layout at = fp8_layout(a.n_groups, a.pairs, a.cin, a.cout);
  return launch_tiles(wgs, kThreads, [&](unsigned n, unsigned first) {
    Fp8MixArgs part = a;
    part.wg0 = first;
    hipLaunchKernelGGL((k_fp8_mix<T>), dim3(n), dim3(kThreads), 0, s, part, l, at);
  });
}

}  // namespace

Fp8Layout fp8_layout(int n_groups, int pairs, int cin, int cout) {
  Fp8Layout l;
  l.in_blocks = fp8_runs(cin);
  l.out_blocks = fp8_runs(cout);
  const int64_t mats = int64_t(n_groups) * pairs;
  l.scales = 64;
  l.codes = l.scales + (mats * l.in_blocks * l.out_blocks * 4 + 63) / 64 * 64;
  l.bytes = l.codes + mats * cout * l.in_blocks * 128;
  return l;
}

hipError_t launch_fp8_pack(int n_groups, int pairs, int cin, int cout, const float* W, void* packed,
                           hipStream_t s) {
  const Fp8Layout l = fp8_layout(n_groups, pairs, cin, cout);
  hipLaunchKernelGGL(k_fp8_pack,
                     dim3(unsigned(l.in_blocks) * n_groups * pairs, unsigned(l.out_blocks)),
                     dim3(kThreads), 0, s, pairs, n_groups, cin, cout, l, W,
                     static_cast<uint8_t*>(packed));
  return hipGetLastError();
}

hipError_t launch_fp8_quantize(int64_t n_rows, int C, const void* x, int bf16, void* q,
                               float* scale, hipStream_t s) {
  const int runs = fp8_runs(C);
  const int64_t n = n_rows * runs;
  const auto go = [&](auto t, auto lanes) {
    using T = decltype(t);
    constexpr int L = decltype(lanes)::value, per = kThreads / L;  // runs of a workgroup
    const int64_t wgs = std::min<int64_t>((n + per - 1) / per, 1 << 20);
    hipLaunchKernelGGL((k_fp8_quantize<T, L>), dim3(unsigned(wgs)), dim3(kThreads), 0, s, n, runs,
                       C, static_cast<const T*>(x), static_cast<uint8_t*>(q), scale);
    return hipGetLastError();
  };
  const auto by_width = [&](auto t) {
    constexpr int L = kFp8Run * int(sizeof(t)) / 16;  // lanes of a whole run
    if (C <= kFp8Run / 8) return go(t, std::integral_constant<int, L / 8>{});
    if (C <= kFp8Run / 4) return go(t, std::integral_constant<int, L / 4>{});
    if (C <= kFp8Run / 2) return go(t, std::integral_constant<int, L / 2>{});
    return go(t, std::integral_constant<int, L>{});
  };
  return bf16 ? by_width(bf16_t{}) : by_width(float{});
}

hipError_t launch_fp8_mix(const Fp8MixArgs& a, const MixList& l, int bf16, hipStream_t s) {
  return bf16 ? launch_fp8_mix_t<bf16_t>(a, l, s) : launch_fp8_mix_t<float>(a, l, s);
}

}  // namespace e3k
