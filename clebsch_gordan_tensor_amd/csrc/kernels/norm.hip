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
// Bound by memory.  Three ways to walk it, by the length of a component row:
//   k_norm_fwd, k_norm_bwd  a workgroup stays with one block, so a lane's dw
//     and db accumulate in V registers each over all its rows;
//   k_norm_whole  a workgroup takes its rows' blocks one after another, where
//     blocks share lines of memory;
//   k_norm_rows  whole rows through LDS, where a row of channels is shorter
//     than a vector.
// dw and db go to per-workgroup partials, which are then added in a fixed
// order (reproducible).  At 64,000 rows of 128x(0e+1o+2e+3o) in float32 the
// forward takes 197 us (5.3 TB/s), the backward 299 us (5.3 TB/s); a copy of
// the size reaches 4.5 to 4.8 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.h"
#include "registry.h"

// A row's results must not hang on where it stands: rows at the end take the
// masked form of the same steps, and both have to round alike.  Products and
// sums are fused only where fmaf says so.
#pragma clang fp contract(off)

namespace e3k {
namespace {

// V consecutive channels from an address aligned to the element only (any C).
// STREAM: whole lines of memory, read or written once.
template <class T, int V>
struct Vec;
template <int V>
struct Vec<float, V> {
  typedef float mem __attribute__((ext_vector_type(V), aligned(4)));
};
template <int V>
struct Vec<bf16_t, V> {
  typedef __bf16 mem __attribute__((ext_vector_type(V), aligned(2)));
};

template <bool STREAM, class T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (std::is_same_v<T, float>) v[0] = *p;
    else v[0] = float(*reinterpret_cast<const __bf16*>(p));
  } else {
    typedef float reg __attribute__((ext_vector_type(V)));
    const auto* q = reinterpret_cast<const typename Vec<T, V>::mem*>(p);
    const reg t = __builtin_convertvector(STREAM ? __builtin_nontemporal_load(q) : *q, reg);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = t[i];
  }
}

template <bool STREAM, class T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (std::is_same_v<T, float>) *p = v[0];
    else *reinterpret_cast<__bf16*>(p) = __bf16(v[0]);
  } else {
    typedef float reg __attribute__((ext_vector_type(V)));
    reg t;
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = v[i];
    typedef typename Vec<T, V>::mem mem;
    mem* q = reinterpret_cast<mem*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(__builtin_convertvector(t, mem), q);
    else *q = __builtin_convertvector(t, mem);
  }
}

constexpr int kNormThreads = 256;

// Sums of N values over a team; every lane of the team gets them.  Teams of
// at most 64 lanes (TEAM == 64: g of them, a power of two) lie in one
// wavefront; larger ones are 2 or 4 wavefronts and join through LDS, in one of
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
    float* buf = lds + phase * (kNormThreads / 64 * kTeamSums);
    phase ^= 1;
    const int w = threadIdx.x >> 6, w0 = w / W * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) buf[w * kTeamSums + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = 0.0f;
      for (int j = 0; j < W; ++j) s += buf[(w0 + j) * kTeamSums + i];
      v[i] = s;
    }
  }
}

// What a lane owns of a component row: K vectors of V channels, vector i from
// channel k0[i].  The row's last vector is moved back inside the row when C is
// no multiple of V, and vectors past it altogether: their first skip[i]
// channels are a neighbour's, whose results they repeat but to whose sums
// they add nothing.
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

template <class T, bool STREAM, int V, int K, int NC>
__device__ __forceinline__ void load_segment(const T* p, int C, const Lane<V, K>& ln,
                                             float (&x)[NC][K][V]) {
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < K; ++i) load_vec<STREAM>(p + c * C + ln.k0[i], x[c][i]);
}
template <class T, bool STREAM, bool MASK, int V, int K, int NC>
__device__ __forceinline__ void store_segment(T* p, int C, const Lane<V, K>& ln,
                                              const float (&o)[NC][K][V]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    if (MASK && ln.skip[i] >= V) continue;
#pragma unroll
    for (int c = 0; c < NC; ++c) store_vec<STREAM>(p + c * C + ln.k0[i], o[c][i]);
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

// 1 / sqrt(t), t a mean square + eps; NaN (infinity x 0) where t is not finite:
// an infinity, or squares past float32's range.  The root alone would answer
// these with 0, and every finite value of the segment with it.
__device__ __forceinline__ float inv_root(float t) {
  return fmaf(t, 0.0f, __builtin_amdgcn_rsqf(t));
}

// Rows a team takes at once: of scalars two, so that their loads are under way
// together and their sums share the joining steps.
constexpr int rows_at_once(int nc, int k) { return nc == 1 && k == 1 ? 2 : 1; }

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

// x becomes xc (one component row a segment).
template <int TEAM, bool MASK, int V, int K, int U>
__device__ __forceinline__ void center(float (&x)[U][1][K][V], float inv, const Lane<V, K>& ln,
                                       int g, float* lds, int& phase) {
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = 0.0f;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) s[u] += !MASK || v >= ln.skip[i] ? x[u][0][i][v] : 0.0f;
  }
  team_sum<TEAM>(s, g, lds, phase);
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) x[u][0][i][v] = fmaf(-s[u], inv, x[u][0][i][v]);
}

// What a workgroup's lanes need of a block: the team's share of its memory.
template <class T, int V, int K>
struct Block {
  const T* x;
  const T* dy;
  T* y;
  int64_t ld;  // of a row
  int C, group;
  bool centered;
  float eps;
  __device__ __forceinline__ Block(const NormArgs& a, const NormBlock& b, int g)
      : x(static_cast<const T*>(a.x) + int64_t(b.comp0) * a.C),
        dy(static_cast<const T*>(a.dy) + int64_t(b.comp0) * a.C),
        y(static_cast<T*>(a.y) + int64_t(b.comp0) * a.C),
        ld(int64_t(a.dim) * a.C), C(a.C), group(g), centered(b.centered), eps(a.eps) {}
};

template <int NC, int TEAM, bool STREAM, bool MASK, class T, int V, int K, int U>
__device__ __forceinline__ void fwd_step(const Block<T, V, K>& b, const Rows<U>& r,
                                         const Lane<V, K>& ln, const float (&w)[K][V],
                                         const float (&bias)[K][V], float* lds, int& phase) {
  const float inv = 1.0f / float(NC * b.C);
  float xs[U][NC][K][V], s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load_segment<T, STREAM>(b.x + r.at[u] * b.ld, b.C, ln, xs[u]);
  if constexpr (NC == 1)
    if (b.centered) center<TEAM, MASK>(xs, inv, ln, b.group, lds, phase);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float xm = !MASK || v >= ln.skip[i] ? xs[u][c][i][v] : 0.0f;
          s[u] = fmaf(xm, xm, s[u]);
        }
  }
  team_sum<TEAM>(s, b.group, lds, phase);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float rstd = inv_root(fmaf(s[u], inv, b.eps));
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          xs[u][c][i][v] = fmaf(xs[u][c][i][v] * rstd, w[i][v], bias[i][v]);
    if (!MASK || r.valid[u])
      store_segment<T, STREAM, MASK>(b.y + r.at[u] * b.ld, b.C, ln, xs[u]);
  }
}

// dx of the rows; adds to the lane's dw (aw) and, for scalars, db (ab).  What
// a repeated channel adds is never read.
template <int NC, int TEAM, bool STREAM, bool MASK, class T, int V, int K, int U>
__device__ __forceinline__ void bwd_step(const Block<T, V, K>& b, const Rows<U>& r,
                                         const Lane<V, K>& ln, const float (&w)[K][V],
                                         float (&aw)[K][V], float (&ab)[K][V], float* lds,
                                         int& phase) {
  const float inv = 1.0f / float(NC * b.C);
  float xs[U][NC][K][V], d[U][NC][K][V];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    load_segment<T, STREAM>(b.x + r.at[u] * b.ld, b.C, ln, xs[u]);
    load_segment<T, STREAM>(b.dy + r.at[u] * b.ld, b.C, ln, d[u]);
  }
  if constexpr (NC == 1)
    if (b.centered) center<TEAM, MASK>(xs, inv, ln, b.group, lds, phase);
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
          if (MASK && !r.valid[u]) d[u][c][i][v] = 0.0f;
          const bool mine = !MASK || v >= ln.skip[i];
          const float xm = mine ? xs[u][c][i][v] : 0.0f;
          const float gv = mine ? d[u][c][i][v] * w[i][v] : 0.0f;
          q[0] = fmaf(xm, xm, q[0]);
          q[1] = fmaf(gv, xm, q[1]);
          if constexpr (NC == 1) q[2] += gv;
        }
  }
  team_sum<TEAM>(s, b.group, lds, phase);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float* q = s + u * S;
    const float rstd = inv_root(fmaf(q[0], inv, b.eps));
    const float along = q[1] * inv * rstd;
    float mg = 0.0f;
    if constexpr (NC == 1) mg = b.centered ? q[2] * inv : 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          // an invalid row adds nothing, even where its x is not finite
          const float xh = MASK && !r.valid[u] ? 0.0f : xs[u][c][i][v] * rstd;
          const float dv = d[u][c][i][v];
          aw[i][v] = fmaf(dv, xh, aw[i][v]);
          if constexpr (NC == 1) ab[i][v] += dv;
          // g as it was summed: a single channel's dx is exactly 0
          xs[u][c][i][v] = rstd * fmaf(-xh, along, dv * w[i][v] - mg);
        }
    if (!MASK || r.valid[u])
      store_segment<T, STREAM, MASK>(b.y + r.at[u] * b.ld, b.C, ln, xs[u]);
  }
}

// Calls f(rows, masked) over the rows of this workgroup; nothing is to be
// masked where the lanes' vectors are the row's (C = group x V) and all rows
// are there.
template <int U, class F>
__device__ __forceinline__ void for_rows(const NormArgs& a, const NormBlock& b, int wg, int teams,
                                         int team, F&& f) {
  const int64_t step = int64_t(teams) * U;
  for (int64_t r0 = wg * step; r0 < a.n_rows; r0 += b.n_wg * step) {
    const Rows<U> rows(r0, teams, team, a.n_rows);
    if (a.whole && r0 + step <= a.n_rows) f(rows, std::false_type{});
    else f(rows, std::true_type{});
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
    if constexpr (NCMAX == 18) {  // all of them
      switch (nc) {
        case 1: f(std::integral_constant<int, 1>{}); return;
        case 3: f(std::integral_constant<int, 3>{}); return;
        case 5: f(std::integral_constant<int, 5>{}); return;
        case 7: f(std::integral_constant<int, 7>{}); return;
        default: break;
      }
    }
    switch (nc) {
      case 9: f(std::integral_constant<int, 9>{}); break;
      case 11: f(std::integral_constant<int, 11>{}); break;
      case 13: f(std::integral_constant<int, 13>{}); break;
      case 15: f(std::integral_constant<int, 15>{}); break;
      default: f(std::integral_constant<int, 17>{}); break;
    }
  }
}

__device__ __forceinline__ const float* row_of(const float* p, int row, int C) {
  return p && row >= 0 ? p + int64_t(row) * C : nullptr;
}

template <class T, int V, int K, int TEAM, int NCMAX>
__global__ void __launch_bounds__(kNormThreads) k_norm_fwd(const NormArgs a) {
  __shared__ float lds[TEAM == 64 ? 1 : 2 * (kNormThreads / 64) * kTeamSums];
  const NormBlock b = a.blk[block_of(a)];
  const int g = TEAM == 64 ? a.group : TEAM, team = int(threadIdx.x) / g;
  const Lane<V, K> ln(int(threadIdx.x) % g, g, a.C);
  const Block<T, V, K> blk(a, b, g);
  float w[K][V], bias[K][V];
  load_weights(row_of(a.w, b.index, a.C), ln, 1.0f, w);
  load_weights(row_of(a.b, b.bias, a.C), ln, 0.0f, bias);
  int phase = 0;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    constexpr int NC = decltype(nc)::value, U = rows_at_once(NC, K);
    for_rows<U>(a, b, int(blockIdx.x) - b.wg0, kNormThreads / g, team,
                [&](const Rows<U>& r, auto mask) {
                  fwd_step<NC, TEAM, true, decltype(mask)::value>(blk, r, ln, w, bias, lds, phase);
                });
  });
}

// Wavefronts on a SIMD of the backward for scalars, by registers held to it;
// as many of its workgroups are resident on a compute unit.  At k = 1 (and k =
// 2, v = 4) 2 to 11 registers spill under these caps, and one wavefront less,
// without spills, is faster (us, caps as here and one less): float32, 128
// channels of 150,000 rows 52 and 50, 512 of 40,000 53 and 52; bf16 35 and 29.5,
// 38 and 32.  Without spills there is nothing in it (1000 channels of 20,000
// rows 50.5 and 50.7, in bf16 38 and 38).
constexpr int scalar_waves(int v, int k) {
  return v == 8 ? (k == 1 ? 4 : k == 2 ? 3 : 2) : k == 1 ? 6 : k == 2 ? 5 : 2;
}

// dw and db of this workgroup's rows to its partials (or, where it is the
// block's only one, to the results).
template <class T, int V, int K, int TEAM, int NCMAX>
__global__ void __attribute__((amdgpu_waves_per_eu(NCMAX == 1 ? scalar_waves(V, K) : 1)))
__launch_bounds__(kNormThreads) k_norm_bwd(const NormArgs a) {
  // the sums of the wavefronts (teams within one) or of the teams meet in LDS
  constexpr int kParts = kNormThreads / TEAM, kRow = TEAM * V * K;
  constexpr int kJoin = kParts > 1 ? 2 * kParts * kRow : 0;
  constexpr int kSums = TEAM == 64 ? 0 : 2 * (kNormThreads / 64) * kTeamSums;
  __shared__ float lds[kSums + kJoin];
  const NormBlock b = a.blk[block_of(a)];
  const int g = TEAM == 64 ? a.group : TEAM, team = int(threadIdx.x) / g;
  const Lane<V, K> ln(int(threadIdx.x) % g, g, a.C);
  const Block<T, V, K> blk(a, b, g);
  float w[K][V], aw[K][V], ab[K][V];
  load_weights(row_of(a.w, b.index, a.C), ln, 1.0f, w);
#pragma unroll
  for (int i = 0; i < K; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v) aw[i][v] = ab[i][v] = 0.0f;
  int phase = 0;
  with_components<NCMAX>(b.nc, [&](auto nc) {
    constexpr int NC = decltype(nc)::value, U = rows_at_once(NC, K);
    for_rows<U>(a, b, int(blockIdx.x) - b.wg0, kNormThreads / g, team,
                [&](const Rows<U>& r, auto mask) {
                  bwd_step<NC, TEAM, true, decltype(mask)::value>(blk, r, ln, w, aw, ab, lds, phase);
                });
  });
  const bool only = b.n_wg == 1;
  float* ow = only ? (a.dw ? a.dw + int64_t(b.index) * a.C : nullptr)
                   : a.part + int64_t(blockIdx.x) * 2 * a.C;
  float* ob = b.bias < 0 ? nullptr
              : only     ? (a.db ? a.db + int64_t(b.bias) * a.C : nullptr)
                         : a.part + (int64_t(blockIdx.x) * 2 + 1) * a.C;
  const int lane = threadIdx.x % TEAM, part = threadIdx.x / TEAM;
  if constexpr (TEAM == 64)  // the groups of a wavefront
    for (int o = a.group; o < 64; o <<= 1)
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          aw[i][v] += __shfl_xor(aw[i][v], o);
          ab[i][v] += __shfl_xor(ab[i][v], o);
        }
  if constexpr (kParts > 1) {
    float* join = lds + kSums;
    if (TEAM > 64 || lane < a.group) {
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v >= ln.skip[i]) {
            join[part * kRow + ln.k0[i] + v] = aw[i][v];
            join[(kParts + part) * kRow + ln.k0[i] + v] = ab[i][v];
          }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.C; k += kNormThreads) {
      float sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < kParts; ++j) {
        sw += join[j * kRow + k];
        sb += join[(kParts + j) * kRow + k];
      }
      if (ow) ow[k] = sw;
      if (ob) ob[k] = sb;
    }
  } else {
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

// ------------------------------------------------------------- staged rows
//
// Rows of several blocks with fewer channels than a vector: a workgroup takes
// as many rows as fit a few KB of LDS, copied in and out as one contiguous
// piece in 16-byte vectors; teams of lanes form the statistics of every
// (row, block) from LDS, then every thread keeps to one position of the row,
// so that its weight stays in a register and dw and db add up over the rows.
// 3 channels of 0e+1o+2e+3o, forward and backward, TB/s: 2.3 and 2.8, a block
// a workgroup 1.5 and 1.6.  From 8 channels on k_norm_whole is faster (3.3
// and 3.0 against 2.3 and 2.8): this form works on single elements.

typedef uint32_t raw16 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t reg16 __attribute__((ext_vector_type(4)));

// n elements between memory (aligned to the element) and LDS.
template <class T>
__device__ __forceinline__ void copy_in(const T* src, T* dst, int n) {
  constexpr int V = 16 / sizeof(T);
  const int nv = n / V;
  for (int v0 = threadIdx.x; v0 < nv; v0 += 4 * kNormThreads) {
    reg16 t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + j * kNormThreads;
      if (v < nv) t[j] = __builtin_nontemporal_load(reinterpret_cast<const raw16*>(src + int64_t(v) * V));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = v0 + j * kNormThreads;
      if (v < nv) *reinterpret_cast<reg16*>(dst + v * V) = t[j];
    }
  }
  for (int e = nv * V + threadIdx.x; e < n; e += kNormThreads) dst[e] = src[e];
}
template <class T>
__device__ __forceinline__ void copy_out(T* dst, const T* src, int n) {
  constexpr int V = 16 / sizeof(T);
  const int nv = n / V;
  for (int v = threadIdx.x; v < nv; v += kNormThreads)
    __builtin_nontemporal_store(raw16(*reinterpret_cast<const reg16*>(src + v * V)),
                                reinterpret_cast<raw16*>(dst + int64_t(v) * V));
  for (int e = nv * V + threadIdx.x; e < n; e += kNormThreads) dst[e] = src[e];
}
template <class T>
__device__ __forceinline__ float value_of(const T* p) {
  if constexpr (std::is_same_v<T, float>) return *p;
  else return float(*reinterpret_cast<const __bf16*>(p));
}
template <class T>
__device__ __forceinline__ void put(T* p, float v) {
  if constexpr (std::is_same_v<T, float>) *p = v;
  else *reinterpret_cast<__bf16*>(p) = __bf16(v);
}

struct RowStats {
  float mu, rstd, along, mg;
};

// LDS of a workgroup, in bytes from its start (each part 16-byte aligned).
struct StagedLayout {
  int x, dy, weight, of, stats, sums, bytes;
};
__host__ __device__ inline int up16(int n) { return (n + 15) / 16 * 16; }
__host__ __device__ inline StagedLayout staged_layout(int esize, int row, int rows, int blocks,
                                                      bool bwd) {
  StagedLayout l;
  l.x = 0;
  l.dy = up16(rows * row * esize);
  l.weight = l.dy + (bwd ? up16(rows * row * esize) : 0);
  l.of = l.weight + up16(4 * row);
  l.stats = l.of + up16(row);
  l.sums = l.stats + rows * blocks * int(sizeof(RowStats));
  l.bytes = l.sums + (bwd ? 2 * 4 * (row > kNormThreads ? row : kNormThreads) : 0);
  return l;
}

template <class T, bool BWD>
__global__ void __launch_bounds__(kNormThreads) k_norm_rows(const NormArgs a, int n_rows_at_once) {
  extern __shared__ reg16 s_raw[];
  unsigned char* lds = reinterpret_cast<unsigned char*>(s_raw);
  const int row = a.dim * a.C, R = n_rows_at_once, nb = a.n_blocks;
  const StagedLayout at = staged_layout(sizeof(T), row, R, nb, BWD);
  T* xs = reinterpret_cast<T*>(lds + at.x);
  T* ds = reinterpret_cast<T*>(lds + at.dy);
  float* weight = reinterpret_cast<float*>(lds + at.weight);
  uint8_t* of = lds + at.of;
  RowStats* stats = reinterpret_cast<RowStats*>(lds + at.stats);
  float* sum_w = reinterpret_cast<float*>(lds + at.sums);
  float* sum_b = sum_w + max(row, kNormThreads);
  const int tid = threadIdx.x;
  for (int i = 0; i < nb; ++i) {  // weight and block of every position of a row
    const NormBlock b = a.blk[i];
    for (int j = tid; j < b.nc * a.C; j += kNormThreads) {
      weight[b.comp0 * a.C + j] = a.w ? a.w[int64_t(b.index) * a.C + j % a.C] : 1.0f;
      of[b.comp0 * a.C + j] = uint8_t(i);
    }
  }
  // threads share out the positions of a row; short rows several at a time
  const int groups = max(1, kNormThreads / row), group = tid / row;
  if constexpr (BWD)
    for (int j = tid; j < max(row, kNormThreads); j += kNormThreads) sum_w[j] = sum_b[j] = 0.0f;

  const int64_t pieces = (a.n_rows + R - 1) / R;
  for (int64_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
    const int64_t r0 = piece * R;
    const int rows = int(min(int64_t(R), a.n_rows - r0));
    copy_in(static_cast<const T*>(a.x) + r0 * row, xs, rows * row);
    if constexpr (BWD) copy_in(static_cast<const T*>(a.dy) + r0 * row, ds, rows * row);
    __syncthreads();
    for (int i = 0; i < nb; ++i) {
      const NormBlock b = a.blk[i];
      const int len = b.nc * a.C, from = b.comp0 * a.C;
      const float inv = 1.0f / float(len);
      int g = 1;  // lanes of a segment: about 4 values each
      while (4 * g < len && g < 64) g *= 2;
      const int lane = tid & (g - 1), teams = kNormThreads / g;
      for (int q = 0; q < rows; q += teams) {
        const int r = min(q + tid / g, rows - 1);
        const T* xr = xs + r * row + from;
        float mu = 0.0f;
        if (b.centered) {
          float s[1] = {0.0f};
          for (int e = lane; e < len; e += g) s[0] += value_of(xr + e);
          wave_team_sum(s, g);
          mu = s[0] * inv;
        }
        float s[3] = {0.0f, 0.0f, 0.0f};
        const T* dr = ds + r * row + from;
        for (int e = lane; e < len; e += g) {
          const float xc = value_of(xr + e) - mu;
          s[0] = fmaf(xc, xc, s[0]);
          if constexpr (BWD) {
            const float gv = value_of(dr + e) * weight[from + e];
            s[1] = fmaf(gv, xc, s[1]);
            s[2] += gv;
          }
        }
        wave_team_sum(s, g);
        const float rstd = inv_root(s[0] * inv + a.eps);
        if (lane == 0 && q + tid / g < rows)
          stats[r * nb + i] = {mu, rstd, s[1] * inv * rstd, b.centered ? s[2] * inv : 0.0f};
      }
    }
    __syncthreads();
    if (group < groups)
      for (int j = tid - group * row; j < row; j += kNormThreads) {
        const int i = of[j];
        const float w = weight[j];
        if constexpr (BWD) {
          float aw = 0.0f, ab = 0.0f;
          for (int r = group; r < rows; r += groups) {
            const RowStats st = stats[r * nb + i];
            const float xh = (value_of(xs + r * row + j) - st.mu) * st.rstd;
            const float d = value_of(ds + r * row + j);
            aw = fmaf(d, xh, aw);
            ab += d;
            put(xs + r * row + j, st.rstd * fmaf(-xh, st.along, d * w - st.mg));
          }
          sum_w[group * row + j] += aw;
          sum_b[group * row + j] += ab;
        } else {
          const int bias_row = a.blk[i].bias;
          const float bias = a.b && bias_row >= 0
                                 ? a.b[int64_t(bias_row) * a.C + j - a.blk[i].comp0 * a.C] : 0.0f;
          for (int r = group; r < rows; r += groups) {
            const RowStats st = stats[r * nb + i];
            put(xs + r * row + j, fmaf((value_of(xs + r * row + j) - st.mu) * st.rstd, w, bias));
          }
        }
      }
    __syncthreads();
    copy_out(static_cast<T*>(a.y) + r0 * row, xs, rows * row);
    __syncthreads();  // the next piece lands where this one was read
  }
  if constexpr (BWD) {
    __syncthreads();  // there may have been no piece
    // a wavefront for each (block, channel) in turn
    const int lane = tid & 63;
    for (int p = tid >> 6; p < nb * a.C; p += kNormThreads / 64) {
      const NormBlock b = a.blk[p / a.C];
      const int k = p % a.C;
      float s[2] = {0.0f, 0.0f};
      for (int e = lane; e < groups * b.nc; e += 64) {
        const int at = e / b.nc * row + (b.comp0 + e % b.nc) * a.C + k;
        s[0] += sum_w[at];
        s[1] += sum_b[at];
      }
      wave_team_sum(s, 64);
      const bool only = b.n_wg == 1;
      float* at = a.part + (int64_t(blockIdx.x) * a.part_step + b.wg0) * 2 * a.C;
      float* ow = only ? (a.dw ? a.dw + int64_t(b.index) * a.C : nullptr) : at;
      float* ob = b.bias < 0 ? nullptr
                  : only     ? (a.db ? a.db + int64_t(b.bias) * a.C : nullptr)
                             : at + a.C;
      if (lane == 0 && ow) ow[k] = s[0];
      if (lane == 0 && ob) ob[k] = s[1];
    }
  }
}

// -------------------------------------------------------------- whole rows
//
// Where a component row is not whole 128-byte lines of memory, workgroups that
// each keep to one block write parts of lines, and lines travel more than
// once.  Here a workgroup takes its rows' blocks one after another, so that
// the lines that blocks share meet in its L2; the blocks' weights lie in LDS,
// and so do the sums of dw and db, each lane's own.  0e+1o+2e+3o in float32,
// forward and backward, TB/s, against a block a workgroup: 8 channels 3.3 and
// 3.0 (1.4 and 1.8), 24 channels 4.5 and 4.0 (3.1 and 3.5), 50 channels 4.6
// and 4.0 (3.5 and 4.1), 100 channels 4.8 and 4.2 (4.2 and 4.7).
__host__ __device__ constexpr int lane_row(int v) { return kNormThreads * v; }

template <class T, int V, int NCMAX, bool BWD>
__global__ void __launch_bounds__(kNormThreads) k_norm_whole(const NormArgs a) {
  extern __shared__ float4 s_weights[];
  float* weight = reinterpret_cast<float*>(s_weights);  // [blocks][group][V], then biases or sums
  const int g = a.group, nb = a.n_blocks, per = g * V, tid = threadIdx.x;
  float* bias = weight + nb * per;  // [scalars][group][V]
  float* sums = weight + nb * per;  // [blocks + scalars][threads][V]
  const int q = tid % g, team = tid / g;
  const Lane<V, 1> ln(q, g, a.C);
  for (int i = team; i < nb; i += kNormThreads / g) {
    float w[1][V];
    load_weights(row_of(a.w, a.blk[i].index, a.C), ln, 1.0f, w);
#pragma unroll
    for (int v = 0; v < V; ++v) weight[i * per + q * V + v] = w[0][v];
    if constexpr (!BWD)
      if (a.blk[i].slot >= 0) {
        load_weights(row_of(a.b, a.blk[i].bias, a.C), ln, 0.0f, w);
#pragma unroll
        for (int v = 0; v < V; ++v) bias[a.blk[i].slot * per + q * V + v] = w[0][v];
      }
  }
  if constexpr (BWD)
    for (int i = 0; i < nb + a.n_scalars; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v) sums[i * lane_row(V) + tid * V + v] = 0.0f;
  __syncthreads();
  const int teams = kNormThreads / g;
  int phase = 0;
  for (int64_t r0 = int64_t(blockIdx.x) * teams; r0 < a.n_rows; r0 += int64_t(gridDim.x) * teams) {
    const Rows<1> r(r0, teams, team, a.n_rows);
    for (int i = 0; i < nb; ++i) {
      const NormBlock b = a.blk[i];
      const Block<T, V, 1> blk(a, b, g);
      float w[1][V];
#pragma unroll
      for (int v = 0; v < V; ++v) w[0][v] = weight[i * per + q * V + v];
      with_components<NCMAX>(b.nc, [&](auto nc) {
        constexpr int NC = decltype(nc)::value;
        float ab[1][V];
#pragma unroll
        for (int v = 0; v < V; ++v) ab[0][v] = 0.0f;
        if constexpr (BWD) {
          float aw[1][V];
#pragma unroll
          for (int v = 0; v < V; ++v) aw[0][v] = 0.0f;
          bwd_step<NC, 64, false, true>(blk, r, ln, w, aw, ab, nullptr, phase);
          float* sw = sums + i * lane_row(V) + tid * V;
#pragma unroll
          for (int v = 0; v < V; ++v) sw[v] += aw[0][v];
          if (NC == 1 && b.slot >= 0) {
            float* sb = sums + (nb + b.slot) * lane_row(V) + tid * V;
#pragma unroll
            for (int v = 0; v < V; ++v) sb[v] += ab[0][v];
          }
        } else {
          if (NC == 1 && b.slot >= 0)
#pragma unroll
            for (int v = 0; v < V; ++v) ab[0][v] = bias[b.slot * per + q * V + v];
          fwd_step<NC, 64, false, true>(blk, r, ln, w, ab, nullptr, phase);
        }
      });
    }
  }
  if constexpr (BWD) {
    // the lanes that hold an element: 4 teams' in every thread, the threads of
    // a wavefront by permutes, the rest (4 at most) in order
    const int e = tid % per, stride = kNormThreads / per, wave = tid >> 6;
    const int part = per < 64 ? wave : tid / per, parts = per < 64 ? kNormThreads / 64 : stride;
    const int all = nb + a.n_scalars;
    __syncthreads();
    for (int i = 0; i < all; ++i) {
      float* of = sums + i * lane_row(V);
      float s = 0.0f;
      for (int j = tid / per; j < teams; j += stride) s += of[j * per + e];
      for (int o = per; o < 64; o <<= 1) s += __shfl_xor(s, o);
      __syncthreads();
      of[part * per + e] = s;
    }
    __syncthreads();
    for (int idx = tid; idx < all * per; idx += kNormThreads) {
      const int i = idx / per, el = idx - i * per;
      // block i's dw, or the db of the scalar in slot i - nb
      int of = i;
      if (i >= nb)
        for (of = 0; a.blk[of].slot != i - nb;) ++of;
      const NormBlock b = a.blk[of];
      const bool only = b.n_wg == 1;
      float* at = a.part + (int64_t(blockIdx.x) * a.part_step + b.wg0) * 2 * a.C;
      float* out = i < nb ? (only ? a.dw ? a.dw + int64_t(b.index) * a.C : nullptr : at)
                          : (only ? a.db ? a.db + int64_t(b.bias) * a.C : nullptr : at + a.C);
      const Lane<V, 1> own(el / V, g, a.C);
      float s = 0.0f;
      for (int j = 0; j < parts; ++j) s += sums[i * lane_row(V) + j * per + el];
      if (out && el % V >= own.skip[0]) out[own.k0[0] + el % V] = s;
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
    const int64_t step = int64_t(a.part_step) * 2 * a.C;
#pragma unroll 4
    for (int j = part; j < b.n_wg; j += 64) {
      sw += p[j * step];
      if (b.bias >= 0) sb += p[j * step + a.C];
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

// Team and lanes for C channels: k vectors of v channels a lane, 16 bytes each
// (8 for degrees above 3, whose kernels hold most; single channels when the
// row has fewer than a vector).  Teams of up to 64 lanes share a wavefront, others take
// 2 or 4.  Longer rows of scalars stay in one wavefront to 256 vectors (2 or
// 4 a lane: no barrier, a row's loads under way together).
struct Shape {
  int v, k, team, group;
};
Shape shape_of(int C, int top, int esize) {
  const int v = C < 4 ? 1 : esize == 2 && C >= 8 && top == 1 ? 8 : 4;
  const int n = (C + v - 1) / v;  // vectors of a row
  int g = 1;
  while (g < n && g < 64) g *= 2;
  if (n <= 64) return {v, 1, 64, g};
  if (top == 1 && n <= (v == 8 ? 128 : 256)) return {v, n <= 128 ? 2 : 4, 64, 64};
  if (top > 1 && n <= 128) return {v, 1, 128, 128};
  if (n <= 256) return {v, 1, 256, 256};
  return {v, n <= 512 ? 2 : 4, 256, 256};
}

// Workgroups of every block, in proportion to its components: a few for every
// one that is resident, so that blocks of different lengths even out (64,000
// rows of 128x(0e+1o+2e+3o), us: forward 1536 workgroups 202, 1792 202, 2048
// 195.5, 2560 196.3, 4096 203; other shapes take 2048 and 2560 alike to 5%
// either way: 3,000 rows 12.0 and 12.7, 10,000 rows of 300 channels in bf16
// 45.6 and 44.4; backward 768 340, 1536 299, 1792 303, 2304 313), but a single
// block's exactly as many as are resident.  Each of the backward's leaves 8 C
// bytes of partials to write and read again: past 256 each of its teams has at
// least 8 rows (4 turns where a team takes two at once), or 128 bytes of every
// channel (1001 scalar channels, 20,011 rows: 512 workgroups 52 us, 556 62,
// 768 56, 1024 59).
int plan(NormArgs& a, const NormBlock* blocks, int n_blocks, int top, bool bwd, int esize) {
  const Shape sh = shape_of(a.C, top, esize);
  const int teams = kNormThreads / sh.group;
  a.group = sh.group;
  a.whole = a.C == sh.v * sh.k * sh.group;
  a.n_blocks = n_blocks;
  a.part_step = 1;
  int dim = 0, wg = 0;
  for (int i = 0; i < n_blocks; ++i) dim += blocks[i].nc;
  const int64_t steps = (a.n_rows + teams - 1) / teams;
  const int64_t budget = bwd && top == 1 ? 256 * scalar_waves(sh.v, sh.k)
                         : bwd || top == 1 ? 1536 : 2560;
  for (int i = 0; i < n_blocks; ++i) {
    a.blk[i] = blocks[i];
    const int64_t nc = blocks[i].nc;
    int64_t n = std::min<int64_t>(budget * nc / dim, steps);
    if (bwd)
      n = std::min(n, std::max<int64_t>(256, n_blocks == 1 ? steps / 8
                                                           : a.n_rows * nc * esize / 128));
    if (bwd && n_blocks == 1 && n > 256) n -= n % 256;
    a.blk[i].wg0 = wg;
    a.blk[i].n_wg = int(std::max<int64_t>(1, n));
    wg += a.blk[i].n_wg;
  }
  return wg;
}

constexpr int kStagedRow = 2048;       // most elements of a staged row
constexpr int kStagedBytes = 8192;     // of one operand's rows in LDS
constexpr int kStagedSegments = 1024;  // (row, block) pairs at once, at most
constexpr int kStagedBudget = 1024;    // workgroups

bool staged(int C, int dim, int n_blocks) {
  return C < 4 && n_blocks > 1 && n_blocks <= kNormMaxBlocks && dim * C <= kStagedRow;
}

int staged_rows(int row, int n_blocks, int esize) {
  int r = std::max(1, std::min(kStagedBytes / (row * esize), kStagedSegments / n_blocks));
  // whole 128-byte lines a piece, where so many rows fit
  int line = 128, bytes = row * esize;
  while (line > 1 && bytes % 2 == 0) line /= 2, bytes /= 2;
  return r >= line ? r - r % line : r;
}

// Every block's partials lie side by side, a workgroup after the other.
int plan_staged(NormArgs& a, const NormBlock* blocks, int n_blocks, int esize) {
  const int64_t rows = staged_rows(a.dim * a.C, n_blocks, esize);
  const int64_t wgs = std::max<int64_t>(1, std::min<int64_t>((a.n_rows + rows - 1) / rows,
                                                             kStagedBudget));
  a.n_blocks = n_blocks;
  a.part_step = n_blocks;
  for (int i = 0; i < n_blocks; ++i) {
    a.blk[i] = blocks[i];
    a.blk[i].wg0 = i;
    a.blk[i].n_wg = int(wgs);
  }
  return int(wgs);
}

template <class T>
hipError_t launch_staged(bool bwd, const NormArgs& a, int wgs, hipStream_t s) {
  const int row = a.dim * a.C, rows = staged_rows(row, a.n_blocks, sizeof(T));
  const size_t lds = size_t(staged_layout(sizeof(T), row, rows, a.n_blocks, bwd).bytes);
  const dim3 grid{unsigned(wgs)}, wg{unsigned(kNormThreads)};
  if (bwd) hipLaunchKernelGGL((k_norm_rows<T, true>), grid, wg, lds, s, a, rows);
  else hipLaunchKernelGGL((k_norm_rows<T, false>), grid, wg, lds, s, a, rows);
  return hipGetLastError();
}

constexpr int kWholeBudget = 2048;      // workgroups
constexpr size_t kWholeLds = 65536;

size_t whole_lds(int C, int n_blocks, int n_scalars, bool bwd) {
  const Shape sh = shape_of(C, 17, 4);
  return sizeof(float) * (size_t(n_blocks) * sh.group * sh.v +
                          (bwd ? size_t(n_blocks + n_scalars) * lane_row(sh.v)
                               : size_t(n_scalars) * sh.group * sh.v));
}
// Parts of lines, in the forward to degree 3 at any such width, otherwise where
// a component row is shorter than two lines.
bool whole_rows(int C, int n_blocks, int n_scalars, int top, bool bwd, int esize) {
  if (C < 4 || C > 256 || n_blocks < 2 || n_blocks > kNormMaxBlocks) return false;
  if (C * esize % 128 == 0 || whole_lds(C, n_blocks, n_scalars, true) > kWholeLds) return false;
  return C * esize < 256 || (!bwd && top <= 7);
}
// Every block's partials lie side by side, a workgroup after the other.
int plan_whole(NormArgs& a, const NormBlock* blocks, int n_blocks, bool bwd) {
  const Shape sh = shape_of(a.C, 17, 4);
  const int64_t teams = kNormThreads / sh.group, steps = (a.n_rows + teams - 1) / teams;
  const int wgs = int(std::max<int64_t>(1, std::min<int64_t>(steps, kWholeBudget)));
  a.group = sh.group;
  a.n_blocks = a.part_step = n_blocks;
  a.n_scalars = 0;
  for (int i = 0; i < n_blocks; ++i) {
    a.blk[i] = blocks[i];
    a.blk[i].wg0 = i;
    a.blk[i].n_wg = wgs;
    a.blk[i].slot = blocks[i].bias >= 0 ? a.n_scalars++ : -1;
  }
  return wgs;
}
template <class T>
hipError_t launch_whole(bool bwd, const NormArgs& a, int top, int wgs, hipStream_t s) {
  const dim3 grid{unsigned(wgs)}, wg{unsigned(kNormThreads)};
  const size_t lds = whole_lds(a.C, a.n_blocks, a.n_scalars, bwd);
  const auto go = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    if (bwd) hipLaunchKernelGGL((k_norm_whole<T, 4, NC, true>), grid, wg, lds, s, a);
    else hipLaunchKernelGGL((k_norm_whole<T, 4, NC, false>), grid, wg, lds, s, a);
    return hipGetLastError();
  };
  return top > 7 ? go(std::integral_constant<int, 18>{}) : go(std::integral_constant<int, 7>{});
}

template <int N>
using Int = std::integral_constant<int, N>;

template <class T, int NCMAX>
hipError_t launch_top(bool bwd, const NormArgs& a, int wgs, hipStream_t s) {
  constexpr bool kHalf = sizeof(T) == 2;
  constexpr int kV = kHalf && NCMAX == 1 ? 8 : 4;
  const Shape sh = shape_of(a.C, NCMAX, sizeof(T));
  const dim3 grid{unsigned(wgs)}, wg{unsigned(kNormThreads)};
  const auto go = [&](auto v, auto k, auto team) {
    constexpr int V = decltype(v)::value, K = decltype(k)::value, TEAM = decltype(team)::value;
    if (bwd) hipLaunchKernelGGL((k_norm_bwd<T, V, K, TEAM, NCMAX>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((k_norm_fwd<T, V, K, TEAM, NCMAX>), grid, wg, 0, s, a);
    return hipGetLastError();
  };
  if (sh.v == 1) return go(Int<1>{}, Int<1>{}, Int<64>{});
  if constexpr (kV == 8)
    if (sh.v == 4) return go(Int<4>{}, Int<1>{}, Int<64>{});
  if (sh.team == 64 && sh.k == 1) return go(Int<kV>{}, Int<1>{}, Int<64>{});
  if constexpr (NCMAX == 1) {
    if (sh.team == 64 && sh.k == 2) return go(Int<kV>{}, Int<2>{}, Int<64>{});
    if constexpr (kV == 4)
      if (sh.team == 64) return go(Int<kV>{}, Int<4>{}, Int<64>{});
  } else {
    if (sh.team == 128) return go(Int<kV>{}, Int<1>{}, Int<128>{});
  }
  if constexpr (NCMAX > 1 || kV == 8)
    if (sh.k == 1) return go(Int<kV>{}, Int<1>{}, Int<256>{});
  if constexpr (NCMAX <= 7) {
    if (sh.k == 2) return go(Int<kV>{}, Int<2>{}, Int<256>{});
    if constexpr (kV == 4) return go(Int<kV>{}, Int<4>{}, Int<256>{});
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

struct ScalarsAndTop {
  int scalars, top;  // 0e blocks, most components of a block
};
ScalarsAndTop scalars_and_top(const NormBlock* blocks, int n) {
  ScalarsAndTop r{0, 1};
  for (int i = 0; i < n; ++i) {
    r.scalars += blocks[i].bias >= 0;
    r.top = std::max(r.top, blocks[i].nc);
  }
  return r;
}

}  // namespace

size_t norm_part_floats(int64_t n_rows, int dim, int C, const NormBlock* blocks, int n_blocks,
                        int esize) {
  NormArgs a{};
  a.n_rows = n_rows;
  a.dim = dim;
  a.C = C;
  const auto [scalars, top] = scalars_and_top(blocks, n_blocks);
  if (whole_rows(C, n_blocks, scalars, top, true, esize))
    return size_t(plan_whole(a, blocks, n_blocks, true)) * n_blocks * 2 * C;
  if (staged(C, dim, n_blocks))
    return size_t(plan_staged(a, blocks, n_blocks, esize)) * n_blocks * 2 * C;
  size_t most = 0;
  (void)for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, int top) {
    most = std::max(most, size_t(plan(a, run, m, top, true, esize)) * 2 * C);
    return hipSuccess;
  });
  return most;
}

hipError_t launch_norm(bool bwd, const NormArgs& args, const NormBlock* blocks, int n_blocks,
                       int bf16, hipStream_t s) {
  const int esize = bf16 ? 2 : 4;
  NormArgs a = args;
  const auto sums = [&](int m) {
    bool any = false;
    for (int i = 0; i < m; ++i) any |= a.blk[i].n_wg > 1;
    if (!any) return hipSuccess;
    hipLaunchKernelGGL(k_norm_sum, dim3(unsigned((a.C + 15) / 16), unsigned(m)), dim3(1024), 0, s,
                       a);
    return hipGetLastError();
  };
  const auto [scalars, top] = scalars_and_top(blocks, n_blocks);
  if (whole_rows(a.C, n_blocks, scalars, top, bwd, esize)) {
    const int wgs = plan_whole(a, blocks, n_blocks, bwd);
    const hipError_t e = bf16 ? launch_whole<bf16_t>(bwd, a, top, wgs, s)
                              : launch_whole<float>(bwd, a, top, wgs, s);
    return e != hipSuccess || !bwd ? e : sums(n_blocks);
  }
  if (staged(a.C, a.dim, n_blocks)) {
    const int wgs = plan_staged(a, blocks, n_blocks, esize);
    const hipError_t e = bf16 ? launch_staged<bf16_t>(bwd, a, wgs, s)
                              : launch_staged<float>(bwd, a, wgs, s);
    return e != hipSuccess || !bwd ? e : sums(n_blocks);
  }
  return for_runs(blocks, n_blocks, [&](const NormBlock* run, int m, int top) {
    const int wgs = plan(a, run, m, top, bwd, esize);
    const hipError_t e = bf16 ? launch<bf16_t>(top, bwd, a, wgs, s) : launch<float>(top, bwd, a, wgs, s);
    return e != hipSuccess || !bwd ? e : sums(m);
  });
}

}  // namespace e3k
