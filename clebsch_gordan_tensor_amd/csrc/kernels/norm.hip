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
    if constexpr (std::is_same_v<T, float>) t = __builtin_nontemporal_load(reinterpret_cast<const nf4*>(p));
    else t = __builtin_convertvector(__builtin_nontemporal_load(reinterpret_cast<const nb4*>(p)), rf4);
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
    if constexpr (std::is_same_v<T, float>)
      __builtin_nontemporal_store(nf4(t), reinterpret_cast<nf4*>(p));
    else
      __builtin_nontemporal_store(__builtin_convertvector(t, nb4), reinterpret_cast<nb4*>(p));
  }
}

constexpr int kNormThreads = 256;

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

constexpr int kTeamSums = 6;  // sums at once, at most
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], int g, float* lds, int& phase) {
  if constexpr (TEAM == 64) {
    wave_team_sum(v, g);
  } else {
    constexpr int W = TEAM / 64;
    wave_team_sum(v, 64);
    static_assert(N <= kTeamSums);
    float* buf = lds + phase * (W * kTeamSums);
    phase ^= 1;
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[w * kTeamSums + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
      for (int j = 0; j < W; ++j) s += buf[j * kTeamSums + i];
      v[i] = s;
    }
  }
}

// What a lane owns of a component row: K vectors of V channels, vector i from
// channel k0[i]; the first skip[i] of them belong to a neighbour (the row's
// last vector is moved back inside the row when C is no multiple of V, and
// vectors past it altogether) and count as zero.
template <int V, int K>
struct Lane {
  int k0[K], skip[K];
  __device__ __forceinline__ Lane(int q, int g, int C) {
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const int k = (q + i * g) * V;
      skip[i] = max(0, k - (C - V));
      k0[i] = k - skip[i];
    }
  }
};

template <class T, int V, int K, int NC>
__device__ __forceinline__ void load_segment(const T* p, int C, const Lane<V, K>& ln,
                                             float (&x)[NC][K][V]) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < K; ++i) load_vec<T, V>(p + c * C + ln.k0[i], x[c][i]);
}
template <int V, int K, int NC>
__device__ __forceinline__ void clear_others(float (&x)[NC][K][V], const Lane<V, K>& ln,
                                             bool valid) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) x[c][i][v] = valid && v >= ln.skip[i] ? x[c][i][v] : 0.0f;
}
template <class T, int V, int K, int NC>
__device__ __forceinline__ void store_segment(T* p, int C, const Lane<V, K>& ln,
                                              const float (&o)[NC][K][V]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    if (ln.skip[i] >= V) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      T* at = p + c * C + ln.k0[i];
      if (ln.skip[i] == 0) {
        store_vec<T, V>(at, o[c][i]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v >= ln.skip[i]) {
            const float one[1] = {o[c][i][v]};
            store_vec<T, 1>(at + v, one);
          }
      }
    }
  }
}
// A row of per-channel float32 weights; `other` where there are none.
template <int V, int K>
__device__ __forceinline__ void load_weights(const float* p, const Lane<V, K>& ln, float other,
                                             float (&w)[K][V]) {
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) w[i][v] = p ? p[ln.k0[i] + v] : other;
}

// Rows a team takes at once: of scalars two, so that their loads are under way
// together and their sums share the joining steps.
constexpr int rows_at_once(int nc, int k) { return nc == 1 && k == 1 ? 2 : 1; }

// x becomes xc (one component row a segment).
template <int TEAM, int V, int K, int U>
__device__ __forceinline__ void center(float (&x)[U][1][K][V], float inv, const Lane<V, K>& ln,
                                       int g, float* lds, int& phase) {
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s[u] += x[u][0][i][v];
  }
  team_sum<TEAM>(s, g, lds, phase);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float mu = s[u] * inv;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) x[u][0][i][v] = v >= ln.skip[i] ? x[u][0][i][v] - mu : 0.0f;
  }
}

// The rows a team takes at once; those past the end repeat the last one, not
// valid.  (Asking for the next rows before these are reduced changed nothing
// beyond 3% either way, forward or backward.)
template <int U>
struct Rows {
  int64_t at[U];
  bool valid[U];
  __device__ __forceinline__ Rows(int64_t r0, int teams, int team, int64_t n) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      at[u] = r0 + u * teams + team;
      valid[u] = at[u] < n;
      at[u] = valid[u] ? at[u] : n - 1;
    }
  }
};
// Calls f(rows) over the rows of this workgroup.
template <int U, class F>
__device__ __forceinline__ void for_rows(const NormArgs& a, const NormBlock& b, int wg, int teams,
                                         int team, F&& f) {
  const int64_t step = int64_t(teams) * U;
  for (int64_t r0 = wg * step; r0 < a.n_rows; r0 += b.n_wg * step)
    f(Rows<U>(r0, teams, team, a.n_rows));
}

template <class T, int V, int K, int TEAM, int NC>
__device__ __forceinline__ void fwd_rows(const NormArgs& a, const NormBlock& b, int wg, float* lds) {
  constexpr int U = rows_at_once(NC, K);
  const int g = TEAM == 64 ? a.group : TEAM;
  const int teams = kNormThreads / g;
  const Lane<V, K> ln(int(threadIdx.x) % g, g, a.C);
  float w[K][V], bias[K][V];
  load_weights(a.w ? a.w + int64_t(b.index) * a.C : nullptr, ln, 1.0f, w);
  load_weights(a.b && b.bias >= 0 ? a.b + int64_t(b.bias) * a.C : nullptr, ln, 0.0f, bias);
  const T* x = static_cast<const T*>(a.x) + int64_t(b.comp0) * a.C;
  T* y = static_cast<T*>(a.y) + int64_t(b.comp0) * a.C;
  const int64_t ld = int64_t(a.dim) * a.C;
  const float inv = 1.0f / float(NC * a.C);
  int phase = 0;
  for_rows<U>(a, b, wg, teams, int(threadIdx.x) / g, [&](const Rows<U>& r) {
    float xs[U][NC][K][V], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load_segment<T>(x + r.at[u] * ld, a.C, ln, xs[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) clear_others(xs[u], ln, true);
    if constexpr (NC == 1)
      if (b.centered) center<TEAM>(xs, inv, ln, g, lds, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) s[u] += xs[u][c][i][v] * xs[u][c][i][v];
    }
    team_sum<TEAM>(s, g, lds, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float rstd = 1.0f / sqrtf(s[u] * inv + a.eps);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v)
            xs[u][c][i][v] = fmaf(xs[u][c][i][v] * rstd, w[i][v], bias[i][v]);
      if (r.valid[u]) store_segment<T>(y + r.at[u] * ld, a.C, ln, xs[u]);
    }
  });
}

template <class T, int V, int K, int TEAM, int NC>
__device__ __forceinline__ void bwd_rows(const NormArgs& a, const NormBlock& b, int wg, float* lds,
                                         float (&aw)[K][V], float (&ab)[K][V]) {
  constexpr int U = rows_at_once(NC, K);
  const int g = TEAM == 64 ? a.group : TEAM;
  const int teams = kNormThreads / g;
  const Lane<V, K> ln(int(threadIdx.x) % g, g, a.C);
  float w[K][V];
  load_weights(a.w ? a.w + int64_t(b.index) * a.C : nullptr, ln, 1.0f, w);
  const T* x = static_cast<const T*>(a.x) + int64_t(b.comp0) * a.C;
  const T* dy = static_cast<const T*>(a.dy) + int64_t(b.comp0) * a.C;
  T* dx = static_cast<T*>(a.y) + int64_t(b.comp0) * a.C;
  const int64_t ld = int64_t(a.dim) * a.C;
  const float inv = 1.0f / float(NC * a.C);
  int phase = 0;
  for_rows<U>(a, b, wg, teams, int(threadIdx.x) / g, [&](const Rows<U>& r) {
    float xs[U][NC][K][V], d[U][NC][K][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load_segment<T>(x + r.at[u] * ld, a.C, ln, xs[u]);
      load_segment<T>(dy + r.at[u] * ld, a.C, ln, d[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      clear_others(xs[u], ln, r.valid[u]);
      clear_others(d[u], ln, r.valid[u]);
    }
    if constexpr (NC == 1)
      if (b.centered) center<TEAM>(xs, inv, ln, g, lds, phase);
    constexpr int S = NC == 1 ? 3 : 2;  // sums of xc^2, g xc and, for scalars, g
    float s[U * S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float* q = s + u * S;
#pragma unroll
      for (int i = 0; i < S; ++i) q[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float gv = d[u][c][i][v] * w[i][v];
            q[0] += xs[u][c][i][v] * xs[u][c][i][v];
            q[1] += gv * xs[u][c][i][v];
            if constexpr (NC == 1) q[2] += gv;
          }
    }
    team_sum<TEAM>(s, g, lds, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float* q = s + u * S;
      const float rstd = 1.0f / sqrtf(q[0] * inv + a.eps);
      const float along = q[1] * inv * rstd;
      float mg = 0.0f;
      if constexpr (NC == 1) mg = b.centered ? q[2] * inv : 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const float xh = xs[u][c][i][v] * rstd, dv = d[u][c][i][v];
            aw[i][v] = fmaf(dv, xh, aw[i][v]);
            if constexpr (NC == 1) ab[i][v] += dv;
            xs[u][c][i][v] = rstd * (dv * w[i][v] - mg - xh * along);
          }
      if (r.valid[u]) store_segment<T>(dx + r.at[u] * ld, a.C, ln, xs[u]);
    }
  });
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
  if constexpr (NCMAX == 1) {
    f(std::integral_constant<int, 1>{});
  } else if constexpr (NCMAX == 7) {
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

template <class T, int V, int K, int TEAM, int NCMAX>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(const NormArgs a) {
  __shared__ float lds[TEAM == 64 ? 1 : 2 * (TEAM / 64) * kTeamSums];
  const int i = block_of(a);
  const NormBlock b = a.blk[i];
  const int wg = int(blockIdx.x) - b.wg0;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    fwd_rows<T, V, K, TEAM, decltype(nc)::value>(a, b, wg, lds);
  });
}

// dw and db of this workgroup's rows to its partials (or, where it is the
// block's only one, to the results).
template <class T, int V, int K, int TEAM, int NCMAX>
__global__ void __launch_bounds__(kNormThreads) k_norm_bwd(const NormArgs a) {
  constexpr int kRow = 64 * V * K;  // most channels of a team within a wavefront
  __shared__ float lds[TEAM == 64 ? 2 * 4 * kRow : 2 * (TEAM / 64) * kTeamSums];
  const int bi = block_of(a);
  const NormBlock b = a.blk[bi];
  const int wg = int(blockIdx.x) - b.wg0;
  float aw[K][V], ab[K][V];
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) aw[i][v] = ab[i][v] = 0.0f;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    bwd_rows<T, V, K, TEAM, decltype(nc)::value>(a, b, wg, lds, aw, ab);
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
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          aw[i][v] += __shfl_xor(aw[i][v], o);
          ab[i][v] += __shfl_xor(ab[i][v], o);
        }
    if (lane < a.group) {
      const Lane<V, K> ln(lane, a.group, a.C);
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v >= ln.skip[i]) {
            lds[wv * kRow + ln.k0[i] + v] = aw[i][v];
            lds[(4 + wv) * kRow + ln.k0[i] + v] = ab[i][v];
          }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.C; k += kNormThreads) {
      float sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sw += lds[j * kRow + k];
        sb += lds[(4 + j) * kRow + k];
      }
      if (ow) ow[k] = sw;
      if (ob) ob[k] = sb;
    }
  } else {
    const Lane<V, K> ln(threadIdx.x, TEAM, a.C);
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v >= ln.skip[i]) {
          if (ow) ow[ln.k0[i] + v] = aw[i][v];
          if (ob) ob[ln.k0[i] + v] = ab[i][v];
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

// Team and lanes for C channels.  A lane owns vectors of 4 channels, or single
// channels when the row has fewer than 4; teams of up to 64 lanes share a
// wavefront.  Longer rows of scalars stay in one wavefront to 1024 channels (2
// or 4 vectors a lane: no barrier, the loads of a row under way together);
// those of other degrees, and all beyond 1024, take the workgroup.
struct Shape {
  int v, k, team, group;
};
Shape shape_of(int C, int top) {
  if (C < 4) return {1, 1, 64, C <= 1 ? 1 : C <= 2 ? 2 : 4};
  int g = 1;
  while (g * 4 < C && g < 64) g *= 2;
  if (C <= 256) return {4, 1, 64, g};
  if (top == 1 && C <= 1024) return {4, C <= 512 ? 2 : 4, 64, 64};
  return {4, C <= 1024 ? 1 : 4, 256, 256};
}

// Workgroups of every block, in proportion to its components: 6 on a compute
// unit, what the forward's registers let be resident (64,000 rows of
// 128x(0e+1o+2e+3o), us: forward 1536 workgroups 197, 2048 209, 4096 203;
// backward 1024 301, 1536 296, 2048 314).  The backward's
// each leave 8 C bytes of partials to write and read again: past 256 of them a
// workgroup has at least 128 bytes of every channel to read, and a single
// block's are as many on each of the 256 compute units (1001 scalar channels,
// 20,011 rows: 512 workgroups 52 us, 556 62, 768 56, 1024 59).
constexpr int kBudget = 1536;

int plan(NormArgs& a, const NormBlock* blocks, int n_blocks, int top, bool bwd, int esize) {
  const Shape sh = shape_of(a.C, top);
  const int teams = kNormThreads / sh.group;
  a.group = sh.group;
  a.n_blocks = n_blocks;
  int dim = 0, wg = 0;
  for (int i = 0; i < n_blocks; ++i) dim += blocks[i].nc;
  const int64_t steps = (a.n_rows + teams - 1) / teams;
  for (int i = 0; i < n_blocks; ++i) {
    a.blk[i] = blocks[i];
    const int64_t nc = blocks[i].nc;
    int64_t n = std::min<int64_t>(int64_t(kBudget) * nc / dim, steps);
    if (bwd) n = std::min(n, std::max<int64_t>(256, a.n_rows * nc * esize / 128));
    if (bwd && n_blocks == 1 && n > 256) n -= n % 256;
    a.blk[i].wg0 = wg;
    n = std::max<int64_t>(1, n);
    const int64_t turns = std::max<int64_t>(1, (steps + n - 1) / n);
    a.blk[i].n_wg = int(std::max<int64_t>(1, (steps + turns - 1) / turns));  // alike in length
    wg += a.blk[i].n_wg;
  }
  return wg;
}

template <class T, int NCMAX>
hipError_t launch_top(bool bwd, const NormArgs& a, int wgs, hipStream_t s) {
  const Shape sh = shape_of(a.C, NCMAX);
  const dim3 grid{unsigned(wgs)}, wg{unsigned(kNormThreads)};
  const auto go = [&](auto v, auto k, auto team) {
    constexpr int V = decltype(v)::value, K = decltype(k)::value, TEAM = decltype(team)::value;
    if (bwd) hipLaunchKernelGGL((k_norm_bwd<T, V, K, TEAM, NCMAX>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<T, V, K, TEAM, NCMAX>), grid, wg, 0, s, a);
    return hipGetLastError();
  };
  constexpr std::integral_constant<int, 1> one{};
  constexpr std::integral_constant<int, 4> four{};
  constexpr std::integral_constant<int, 64> wave{};
  constexpr std::integral_constant<int, 256> group{};
  if (sh.v == 1) return go(one, one, wave);
  if (sh.team == 64) {
    if (sh.k == 1) return go(four, one, wave);
    if constexpr (NCMAX == 1)
      return sh.k == 2 ? go(four, std::integral_constant<int, 2>{}, wave) : go(four, four, wave);
  } else {
    if constexpr (NCMAX > 1)
      if (sh.k == 1) return go(four, one, group);
    if constexpr (NCMAX <= 7)
      if (sh.k == 4) return go(four, four, group);
  }
  return hipErrorInvalidValue;
}

template <class T>
hipError_t launch(int top, bool bwd, const NormArgs& a, int wgs, hipStream_t s) {
  return top == 1   ? launch_top<T, 1>(bwd, a, wgs, s)
         : top == 7 ? launch_top<T, 7>(bwd, a, wgs, s)
                    : launch_top<T, 17>(bwd, a, wgs, s);
}

// Calls f(blocks, count, most components) for runs of at most kNormMaxBlocks
// blocks, the degrees up to 3 and those above apart, and lists of scalars by
// themselves: their kernels differ in registers.
template <class F>
hipError_t for_runs(const NormBlock* blocks, int n, F&& f) {
  int top = 1;
  for (int i = 0; i < n; ++i) top = std::max(top, blocks[i].nc);
  for (int high = 0; high < 2; ++high) {
    NormBlock run[kNormMaxBlocks];
    int m = 0;
    for (int i = 0; i <= n; ++i) {
      if (i < n && (blocks[i].nc > 7) == bool(high)) run[m++] = blocks[i];
      if (m > 0 && (i == n || m == kNormMaxBlocks)) {
        const hipError_t e = f(run, m, high ? 17 : top == 1 ? 1 : 7);
        if (e != hipSuccess) return e;
        m = 0;
      }
    }
  }
  return hipSuccess;
}

}  // namespace

size_t norm_part_floats(int64_t n_rows, int C, const NormBlock* blocks, int n_blocks, int esize) {
  size_t most = 0;
  (void)for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, int top) {
    NormArgs a{};
    a.n_rows = n_rows;
    a.C = C;
    most = std::max(most, size_t(plan(a, run, m, top, true, esize)) * 2 * C);
    return hipSuccess;
  });
  return most;
}

hipError_t launch_norm(bool bwd, const NormArgs& args, const NormBlock* blocks, int n_blocks,
                       int bf16, hipStream_t s) {
  return for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, int top) {
    NormArgs a = args;
    const int wgs = plan(a, run, m, top, bwd, bf16 ? 2 : 4);
    const hipError_t e = bf16 ? launch<bf16_t>(top, bwd, a, wgs, s) : launch<float>(top, bwd, a, wgs, s);
    bool sum = false;
    for (int i = 0; i < m; ++i) sum |= a.blk[i].n_wg > 1;
    if (e != hipSuccess || !bwd || !sum) return e;
    hipLaunchKernelGGL(k_norm_sum, dim3(unsigned((a.C + 15) / 16), unsigned(m)), dim3(1024), 0, s,
                       a);
    return hipGetLastError();
  });
}

}  // namespace e3k
