// Normalisation of irreps features and its gradients.  A segment is one
// (row, irrep block): nc = 2l+1 component rows of C channels, contiguous in
// the [rows][components][channels] layout, K = nc C values.
//   xc   = x - mean(x)            (centred blocks: scalars), else x
//   rstd = 1 / sqrt(sum xc^2 / K + eps)
//   y    = xc rstd w[k] + b[k]
//   dx   = rstd (g - [mean g] - xc rstd^2 mean(g xc)),  g = dy w[k]
//   dw[k] = sum over rows and components of dy xc rstd,  db[k] = sum of dy
// Each is one pass over its operands: a team of lanes holds a segment in
// registers (a lane owns the same V channels of every component row), so the
// statistics cost no second read; the backward forms them again from x, which
// it reads anyway, and nothing is kept from the forward.
//
// A workgroup stays with one block, so a lane's dw and db accumulate in V
// registers each over all its rows; per-workgroup partials are then added in
// a fixed order (reproducible).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.h"
#include "registry.h"

namespace e3k {
namespace {

// V consecutive channels from an address aligned to the element only (any C).
typedef float nf4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 nb4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float rf4 __attribute__((ext_vector_type(4)));

template <class T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (std::is_same_v<T, float>) v[0] = *p;
    else v[0] = float(*reinterpret_cast<const __bf16*>(p));
  } else {
    static_assert(V == 4);
    rf4 t;
    if constexpr (std::is_same_v<T, float>) t = *reinterpret_cast<const nf4*>(p);
    else t = __builtin_convertvector(*reinterpret_cast<const nb4*>(p), rf4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t[i];
  }
}

template <class T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (std::is_same_v<T, float>) *p = v[0];
    else *reinterpret_cast<__bf16*>(p) = __bf16(v[0]);
  } else {
    const rf4 t = {v[0], v[1], v[2], v[3]};
    if constexpr (std::is_same_v<T, float>) *reinterpret_cast<nf4*>(p) = t;
    else *reinterpret_cast<nb4*>(p) = __builtin_convertvector(t, nb4);
  }
}

// Sums of N values over a team; every lane of the team gets them.  Teams of
// at most 64 lanes (TEAM == 64: g of them, a power of two) lie in one
// wavefront; larger ones are the workgroup and join through LDS, in one of
// two buffers in turn, so one barrier separates a buffer's use from its next.
template <int N>
__device__ __forceinline__ void wave_team_sum(float (&v)[N], int g) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (g > 1) v[i] += dpp<0xB1>(v[i]);   // lane ^ 1
    if (g > 2) v[i] += dpp<0x4E>(v[i]);   // lane ^ 2
    if (g > 4) v[i] += dpp<0x141>(v[i]);  // half-row mirror
    if (g > 8) v[i] += dpp<0x140>(v[i]);  // row mirror
    if (g > 16) {
      float t = v[i];
      swap16(v[i], t);
      v[i] += t;
    }
    if (g > 32) {
      float t = v[i];
      swap32(v[i], t);
      v[i] += t;
    }
  }
}

template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int g, float* lds, int& phase) {
  if constexpr (TEAM == 64) {
    wave_team_sum(v, g);
  } else {
    constexpr int W = TEAM / 64;
    wave_team_sum(v, 64);
    float* buf = lds + phase * (W * 4);
    phase ^= 1;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[w * 4 + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
      for (int j = 0; j < W; ++j) s += buf[j * 4 + i];
      v[i] = s;
    }
  }
}

// What a lane owns: V channels from k0, of which the first `skip` belong to
// its neighbour (the last vector is moved back inside the row when C is no
// multiple of V) and count as zero.
struct Lane {
  int k0, skip;
};
template <int V>
__device__ __forceinline__ Lane lane_of(int q, int C) {
  const int k = q * V;
  const int skip = max(0, k - (C - V));
  return {k - skip, skip};
}

template <class T, int V, int NC>
__device__ __forceinline__ void load_segment(const T* p, int C, int skip, bool valid,
                                             float (&x)[NC][V]) {
#pragma unroll
  for (int c = 0; c < NC; ++c) load_vec<T, V>(p + c * C, x[c]);
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int v = 0; v < V; ++v) x[c][v] = valid && v >= skip ? x[c][v] : 0.0f;
}

// x becomes xc; the sum over the segment's centred values' squares comes from
// the caller's second reduction.
template <int TEAM, int V>
__device__ __forceinline__ void center(float (&x)[1][V], int C, int skip, int g, float* lds,
                                       int& phase) {
  float s[1] = {0.0f};
#pragma unroll
  for (int v = 0; v < V; ++v) s[0] += x[0][v];
  team_sum<TEAM>(s, g, lds, phase);
  const float mu = s[0] / float(C);
#pragma unroll
  for (int v = 0; v < V; ++v) x[0][v] = v >= skip ? x[0][v] - mu : 0.0f;
}

template <int TEAM>
struct Team {
  static constexpr int kThreads = TEAM == 64 ? 256 : TEAM;
};

template <class T, int V, int TEAM, int NC>
__device__ __forceinline__ void fwd_rows(const NormArgs& a, const NormBlock& b, int wg, float* lds) {
  const int g = TEAM == 64 ? a.group : TEAM;
  const int teams = Team<TEAM>::kThreads / g;
  const int team = int(threadIdx.x) / g;
  const Lane ln = lane_of<V>(int(threadIdx.x) % g, a.C);
  float w[V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) w[v] = 1.0f, bias[v] = 0.0f;
  if (a.w) load_vec<float, V>(a.w + int64_t(b.index) * a.C + ln.k0, w);
  if (a.b && b.bias >= 0) load_vec<float, V>(a.b + int64_t(b.bias) * a.C + ln.k0, bias);
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.y);
  int phase = 0;
  for (int64_t r0 = int64_t(wg) * teams; r0 < a.n_rows; r0 += int64_t(b.n_wg) * teams) {
    const bool valid = r0 + team < a.n_rows;
    const int64_t row = valid ? r0 + team : r0;
    const int64_t at = (row * a.dim + b.comp0) * a.C + ln.k0;
    float xs[NC][V];
    load_segment<T, V, NC>(x + at, a.C, ln.skip, valid, xs);
    if constexpr (NC == 1)
      if (b.centered) center<TEAM, V>(xs, a.C, ln.skip, g, lds, phase);
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int v = 0; v < V; ++v) s[0] += xs[c][v] * xs[c][v];
    team_sum<TEAM>(s, g, lds, phase);
    const float rstd = 1.0f / sqrtf(s[0] / float(NC * a.C) + a.eps);
    if (valid && ln.skip < V) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = fmaf(xs[c][v] * rstd, w[v], bias[v]);
        if (ln.skip == 0) {
          store_vec<T, V>(y + at + c * a.C, o);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v >= ln.skip) {
              const float one[1] = {o[v]};
              store_vec<T, 1>(y + at + c * a.C + v, one);
            }
        }
      }
    }
  }
}

template <class T, int V, int TEAM, int NC>
__device__ __forceinline__ void bwd_rows(const NormArgs& a, const NormBlock& b, int wg, float* lds,
                                         float (&aw)[V], float (&ab)[V]) {
  const int g = TEAM == 64 ? a.group : TEAM;
  const int teams = Team<TEAM>::kThreads / g;
  const int team = int(threadIdx.x) / g;
  const Lane ln = lane_of<V>(int(threadIdx.x) % g, a.C);
  float w[V];
#pragma unroll
  for (int v = 0; v < V; ++v) w[v] = 1.0f;
  if (a.w) load_vec<float, V>(a.w + int64_t(b.index) * a.C + ln.k0, w);
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  T* dx = static_cast<T*>(a.y);
  const float inv = 1.0f / float(NC * a.C);
  int phase = 0;
  for (int64_t r0 = int64_t(wg) * teams; r0 < a.n_rows; r0 += int64_t(b.n_wg) * teams) {
    const bool valid = r0 + team < a.n_rows;
    const int64_t row = valid ? r0 + team : r0;
    const int64_t at = (row * a.dim + b.comp0) * a.C + ln.k0;
    float xs[NC][V], d[NC][V];
    load_segment<T, V, NC>(x + at, a.C, ln.skip, valid, xs);
    load_segment<T, V, NC>(dy + at, a.C, ln.skip, valid, d);
    if constexpr (NC == 1)
      if (b.centered) center<TEAM, V>(xs, a.C, ln.skip, g, lds, phase);
    float s[3] = {0.0f, 0.0f, 0.0f};  // of xc^2, g xc, g
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float gv = d[c][v] * w[v];
        s[0] += xs[c][v] * xs[c][v];
        s[1] += gv * xs[c][v];
        if (NC == 1) s[2] += gv;
      }
    team_sum<TEAM>(s, g, lds, phase);
    const float rstd = 1.0f / sqrtf(s[0] * inv + a.eps);
    const float along = s[1] * inv * rstd;
    const float mg = NC == 1 && b.centered ? s[2] * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float xh = xs[c][v] * rstd;
        aw[v] = fmaf(d[c][v], xh, aw[v]);
        if (NC == 1) ab[v] += d[c][v];
        o[v] = rstd * (d[c][v] * w[v] - mg - xh * along);
      }
      if (valid && ln.skip < V) {
        if (ln.skip == 0) {
          store_vec<T, V>(dx + at + c * a.C, o);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v)
            if (v >= ln.skip) {
              const float one[1] = {o[v]};
              store_vec<T, 1>(dx + at + c * a.C + v, one);
            }
        }
      }
    }
  }
}

// The block this workgroup belongs to: a lane per block compares, one load deep.
__device__ __forceinline__ int block_of(const NormArgs& a) {
  static_assert(kNormMaxBlocks <= 64);
  const int lane = threadIdx.x & 63;
  const bool below = lane < a.n_blocks && a.blk[lane].wg0 <= int(blockIdx.x);
  return __popcll(__ballot(below)) - 1;
}

// Calls f(integral_constant<NC>) for the block's component count.
template <int NCMAX, class F>
__device__ __forceinline__ void with_components(int nc, F&& f) {
  if constexpr (NCMAX == 7) {
    switch (nc) {
      case 1: f(std::integral_constant<int, 1>{}); break;
      case 3: f(std::integral_constant<int, 3>{}); break;
      case 5: f(std::integral_constant<int, 5>{}); break;
      default: f(std::integral_constant<int, 7>{}); break;
    }
  } else {
    switch (nc) {
      case 9: f(std::integral_constant<int, 9>{}); break;
      case 11: f(std::integral_constant<int, 11>{}); break;
      case 13: f(std::integral_constant<int, 13>{}); break;
      case 15: f(std::integral_constant<int, 15>{}); break;
      default: f(std::integral_constant<int, 17>{}); break;
    }
  }
}

template <class T, int V, int TEAM, int NCMAX>
__global__ void __launch_bounds__(Team<TEAM>::kThreads) k_norm_fwd(const NormArgs a) {
  __shared__ float lds[TEAM == 64 ? 1 : 2 * (TEAM / 64) * 4];
  const int i = block_of(a);
  const NormBlock b = a.blk[i];
  const int wg = int(blockIdx.x) - b.wg0;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    fwd_rows<T, V, TEAM, decltype(nc)::value>(a, b, wg, lds);
  });
}

// dw and db of this workgroup's rows to its partials (or, where it is the
// block's only one, to the results).
template <class T, int V, int TEAM, int NCMAX>
__global__ void __launch_bounds__(Team<TEAM>::kThreads) k_norm_bwd(const NormArgs a) {
  __shared__ float lds[TEAM == 64 ? 4 * 64 * V * 2 : 2 * (TEAM / 64) * 4];
  const int i = block_of(a);
  const NormBlock b = a.blk[i];
  const int wg = int(blockIdx.x) - b.wg0;
  float aw[V], ab[V];
#pragma unroll
  for (int v = 0; v < V; ++v) aw[v] = ab[v] = 0.0f;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    bwd_rows<T, V, TEAM, decltype(nc)::value>(a, b, wg, lds, aw, ab);
  });
  const bool only = b.n_wg == 1;
  float* ow = only ? (a.dw ? a.dw + int64_t(b.index) * a.C : nullptr)
                   : a.part + int64_t(blockIdx.x) * 2 * a.C;
  float* ob = b.bias < 0 ? nullptr
              : only     ? (a.db ? a.db + int64_t(b.bias) * a.C : nullptr)
                         : a.part + (int64_t(blockIdx.x) * 2 + 1) * a.C;
  if constexpr (TEAM == 64) {
    // the groups of a wavefront, then the wavefronts in order
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    for (int o = a.group; o < 64; o <<= 1)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        aw[v] += __shfl_xor(aw[v], o);
        ab[v] += __shfl_xor(ab[v], o);
      }
    const Lane ln = lane_of<V>(lane, a.C);
    if (lane < a.group) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v >= ln.skip) {
          lds[wv * 64 * V + ln.k0 + v] = aw[v];
          lds[(4 + wv) * 64 * V + ln.k0 + v] = ab[v];
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.C; k += 256) {
      float sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sw += lds[j * 64 * V + k];
        sb += lds[(4 + j) * 64 * V + k];
      }
      if (ow) ow[k] = sw;
      if (ob) ob[k] = sb;
    }
  } else {
    const Lane ln = lane_of<V>(threadIdx.x, a.C);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v >= ln.skip) {
        if (ow) ow[ln.k0 + v] = aw[v];
        if (ob) ob[ln.k0 + v] = ab[v];
      }
  }
}

// dw and db from the partials: a workgroup per 16 channels of one block, its
// 64 groups of 16 lanes taking every 64th partial, their sums added in order
// (64 channels and every 16th partial, on a quarter of the workgroups, took
// 24 us against 8 at 1001 channels and 1024 partials).
__global__ void __launch_bounds__(1024) k_norm_sum(const NormArgs a) {
  __shared__ float s_sum[2][64][17];
  const NormBlock b = a.blk[blockIdx.y];
  if (b.n_wg == 1) return;
  const int c = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int k = blockIdx.x * 16 + c;
  float sw = 0.0f, sb = 0.0f;
  if (k < a.C) {
    const float* p = a.part + int64_t(b.wg0) * 2 * a.C + k;
#pragma unroll 4
    for (int j = part; j < b.n_wg; j += 64) {
      sw += p[int64_t(j) * 2 * a.C];
      if (b.bias >= 0) sb += p[(int64_t(j) * 2 + 1) * a.C];
    }
  }
  s_sum[0][part][c] = sw;
  s_sum[1][part][c] = sb;
  __syncthreads();
  // wavefront 0: lane (half of the partials' sums, w or b, channel), halves added in order
  if (threadIdx.x >= 64) return;
  const int which = part & 1, half = part >> 1;
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) s += s_sum[which][half * 32 + j][c];
  s += __shfl(s, (int(threadIdx.x) + 32) & 63);
  if (half != 0 || k >= a.C) return;
  if (which == 0 && a.dw) a.dw[int64_t(b.index) * a.C + k] = s;
  if (which == 1 && a.db && b.bias >= 0) a.db[int64_t(b.bias) * a.C + k] = s;
}

// Lanes of a team and channels per lane.  A lane owns 4 channels, or 1 when
// the row has fewer than 4; teams of up to 64 lanes share a wavefront.
struct Shape {
  int v, team, group;
};
Shape shape_of(int C) {
  if (C < 4) return {1, 64, C <= 1 ? 1 : C <= 2 ? 2 : 4};
  int g = 1;
  while (g * 4 < C && g < 64) g *= 2;
  if (C <= 256) return {4, 64, g};
  if (C <= 1024) return {4, 256, 256};
  return {4, 1024, 1024};
}

// Workgroups of every block of [first, last), in proportion to its components.
int plan(NormArgs& a, const NormBlock* blocks, int n_blocks, int budget) {
  const Shape sh = shape_of(a.C);
  const int teams = (sh.team == 64 ? 256 : sh.team) / sh.group;
  a.group = sh.group;
  a.n_blocks = n_blocks;
  int dim = 0, wg = 0;
  for (int i = 0; i < n_blocks; ++i) dim += blocks[i].nc;
  const int64_t steps = (a.n_rows + teams - 1) / teams;
  for (int i = 0; i < n_blocks; ++i) {
    a.blk[i] = blocks[i];
    const int64_t share = std::max<int64_t>(1, int64_t(budget) * blocks[i].nc / dim);
    a.blk[i].wg0 = wg;
    a.blk[i].n_wg = int(std::max<int64_t>(1, std::min(share, (steps + 3) / 4)));
    wg += a.blk[i].n_wg;
  }
  return wg;
}

constexpr int kFwdBudget = 4096, kBwdBudget = 1024;

template <class T, int NCMAX>
hipError_t launch(bool bwd, const NormArgs& a, int wgs, hipStream_t s) {
  const Shape sh = shape_of(a.C);
  const dim3 grid{unsigned(wgs)}, wg{unsigned(sh.team == 64 ? 256 : sh.team)};
#define E3_NORM_LAUNCH(V, TEAM)                                                             \
  if (bwd) hipLaunchKernelGGL((k_norm_bwd<T, V, TEAM, NCMAX>), grid, wg, 0, s, a);          \
  else hipLaunchKernelGGL((k_norm_fwd<T, V, TEAM, NCMAX>), grid, wg, 0, s, a)
  if (sh.v == 1) { E3_NORM_LAUNCH(1, 64); }
  else if (sh.team == 64) { E3_NORM_LAUNCH(4, 64); }
  else if (sh.team == 256) { E3_NORM_LAUNCH(4, 256); }
  else if constexpr (NCMAX == 7) { E3_NORM_LAUNCH(4, 1024); }
  else return hipErrorInvalidValue;
#undef E3_NORM_LAUNCH
  return hipGetLastError();
}

// Calls f(blocks, count) for runs of at most kNormMaxBlocks blocks, the
// degrees up to 3 and those above apart (their kernels differ in registers).
template <class F>
hipError_t for_runs(const NormBlock* blocks, int n, F&& f) {
  for (int high = 0; high < 2; ++high) {
    NormBlock run[kNormMaxBlocks];
    int m = 0;
    for (int i = 0; i <= n; ++i) {
      if (i < n && (blocks[i].nc > 7) == bool(high)) run[m++] = blocks[i];
      if (m > 0 && (i == n || m == kNormMaxBlocks)) {
        const hipError_t e = f(run, m, bool(high));
        if (e != hipSuccess) return e;
        m = 0;
      }
    }
  }
  return hipSuccess;
}

}  // namespace

size_t norm_part_floats(int64_t n_rows, int C, const NormBlock* blocks, int n_blocks) {
  size_t most = 0;
  (void)for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, bool) {
    NormArgs a{};
    a.n_rows = n_rows;
    a.C = C;
    most = std::max(most, size_t(plan(a, run, m, kBwdBudget)) * 2 * C);
    return hipSuccess;
  });
  return most;
}

hipError_t launch_norm(bool bwd, const NormArgs& args, const NormBlock* blocks, int n_blocks,
                       int bf16, hipStream_t s) {
  return for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, bool high) {
    NormArgs a = args;
    const int wgs = plan(a, run, m, bwd ? kBwdBudget : kFwdBudget);
    hipError_t e = high ? (bf16 ? launch<bf16_t, 17>(bwd, a, wgs, s) : launch<float, 17>(bwd, a, wgs, s))
                        : (bf16 ? launch<bf16_t, 7>(bwd, a, wgs, s) : launch<float, 7>(bwd, a, wgs, s));
    bool sum = false;
    for (int i = 0; i < m; ++i) sum |= a.blk[i].n_wg > 1;
    if (e != hipSuccess || !bwd || !sum) return e;
    hipLaunchKernelGGL(k_norm_sum, dim3(unsigned((a.C + 15) / 16), unsigned(m)), dim3(1024), 0, s,
                       a);
    return hipGetLastError();
  });
}

}  // namespace e3k
