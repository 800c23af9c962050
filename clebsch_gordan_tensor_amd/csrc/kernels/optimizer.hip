// The update of a network's weights: the 2-norm of all gradients with its
// clip factor, and the AdamW step, each over a list of tensors whose pointers
// travel in the kernel arguments (no table in device memory, nothing copied
// to the device, so the calls can be captured into a graph).
//
//   g = s grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
//   p = p - lr wd p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// Moments in 8 bits: every 256 consecutive elements of a tensor share a
// float32 scale per moment,
//   m = s c |c|,  c in [-127, 127],  s = max|m| / 127^2
//   v = (s c^2)^2, c in [0, 255],    s = sqrt(max v) / 255^2
// so the step between codes shrinks towards zero: relative steps of 2/c over
// a range of 1.6e4 (m) and 6.5e4 (sqrt v).  A code is the number of borders
// s (k + 1/2)^2, or (s (k + 1/2)^2)^2, below the value; a v that is not zero
// takes at least code 1, so no element is divided by eps alone because its v
// was rounded away.  Codes are those of the moments in 64 bits, where both
// products above are exact or rounded once: they do not hang on how a 32-bit
// evaluation would round.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "common.h"
#include "registry.h"

namespace e3k {
namespace {

typedef float of4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 ob4 __attribute__((ext_vector_type(4), aligned(2)));
typedef float tf4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32u __attribute__((aligned(1)));

constexpr int kParamThreads = 256;
constexpr int kQBlock = 256;  // elements per scale
constexpr int kPass = 4 * kParamThreads;  // elements a workgroup takes at once
constexpr int64_t kMaxWorkgroups = (int64_t(1) << 32) / kParamThreads - 1;  // 2^32 threads a launch
static_assert(sizeof(ParamList) + sizeof(AdamArgs) <= 4096, "kernel arguments");
static_assert(sizeof(GradList) + sizeof(double*) <= 4096, "kernel arguments");
static_assert(kMaxParamElements / kPass < kMaxWorkgroups);

// Four consecutive elements, those at n and beyond 0.  The step streams (61M
// packed elements 365 -> 351 us, 101M with 8-bit moments 478 -> 460); the
// gradients' norm does not (130M in bf16 59 us, streaming 65).
template <bool kStream>
__device__ __forceinline__ void load4(const float* p, int64_t i, int64_t n, float (&v)[4]) {
  if (i + 4 <= n) {
    const of4* q = reinterpret_cast<const of4*>(p + i);
    const tf4 t = kStream ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? p[i + e] : 0.0f;
  }
}
template <bool kStream>
__device__ __forceinline__ void load4(const __bf16* p, int64_t i, int64_t n, float (&v)[4]) {
  if (i + 4 <= n) {
    const ob4* q = reinterpret_cast<const ob4*>(p + i);
    const tf4 t = __builtin_convertvector(kStream ? __builtin_nontemporal_load(q) : *q, tf4);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < n ? float(p[i + e]) : 0.0f;
  }
}
__device__ __forceinline__ void load4_grad(const ParamTensor& t, int64_t i, float (&v)[4]) {
  if (t.grad_bf16) load4<true>(static_cast<const __bf16*>(t.grad), i, t.n, v);
  else load4<true>(static_cast<const float*>(t.grad), i, t.n, v);
}
__device__ __forceinline__ void store4(float* p, int64_t i, int64_t n, const float (&v)[4]) {
  if (i + 4 <= n) {
    const tf4 t = {v[0], v[1], v[2], v[3]};
    __builtin_nontemporal_store(of4(t), reinterpret_cast<of4*>(p + i));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) p[i + e] = v[e];
  }
}
__device__ __forceinline__ void store4(__bf16* p, int64_t i, int64_t n, const float (&v)[4]) {
  if (i + 4 <= n) {
    const tf4 t = {v[0], v[1], v[2], v[3]};
    __builtin_nontemporal_store(__builtin_convertvector(t, ob4), reinterpret_cast<ob4*>(p + i));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) p[i + e] = __bf16(v[e]);
  }
}
// Four codes as the bytes of a word.
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t i, int64_t n) {
  if (i + 4 <= n) return __builtin_nontemporal_load(reinterpret_cast<const u32u*>(p + i));
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) w |= uint32_t(p[i + e]) << (8 * e);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t i, int64_t n, uint32_t w) {
  if (i + 4 <= n) {
    __builtin_nontemporal_store(w, reinterpret_cast<u32u*>(p + i));
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (i + e < n) p[i + e] = uint8_t(w >> (8 * e));
}

// The tensor this workgroup belongs to: a lane per tensor compares, one load
// deep (walking the list took 0.1 us a tensor).
template <int N>
__device__ __forceinline__ int tensor_of(const int (&wg0)[N], int n) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll
  for (int i = 0; i < N; i += 64) {
    const bool below = i + lane < n && wg0[min(i + lane, N - 1)] <= int(blockIdx.x);
    before += __popcll(__ballot(below));
  }
  return before - 1;
}

// ------------------------------------------------------- the gradients' norm

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A thread's part of the squares of elements [base, end): four vectors of 16
// bytes at a time, all asked for before the first is added.
template <class T>
__device__ __forceinline__ double sum_squares(const T* p, int64_t base, int64_t end) {
  constexpr int V = 16 / sizeof(T);
  double s[2] = {0.0, 0.0};
  for (int64_t i0 = base + int(threadIdx.x) * V; i0 < end; i0 += 4 * V * kParamThreads) {
    float g[4][V];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = i0 + j * V * kParamThreads;
#pragma unroll
      for (int h = 0; h < V; h += 4) {
        float q[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (i + h < end) load4<false>(p, i + h, end, q);
#pragma unroll
        for (int e = 0; e < 4; ++e) g[j][h + e] = q[e];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) s[e & 1] = fma(double(g[j][e]), double(g[j][e]), s[e & 1]);
  }
  return s[0] + s[1];
}

// One partial per workgroup; squares and sums in 64 bits, so no gradient of
// float32's range overflows and the order of summation does not show.
__global__ void __launch_bounds__(kParamThreads) k_grad_norm(const GradList l, double* part) {
  __shared__ double s_sum[kParamThreads / 64];
  const int ti = tensor_of(l.wg0, l.n);
  const int64_t size = l.size[ti], n = size < 0 ? ~size : size;
  const int64_t base = int64_t(int(blockIdx.x) - l.wg0[ti]) * l.chunk;
  const int64_t end = min(n, base + l.chunk);
  double s = size < 0 ? sum_squares(static_cast<const __bf16*>(l.grad[ti]), base, end)
                      : sum_squares(static_cast<const float*>(l.grad[ti]), base, end);
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int j = 1; j < kParamThreads / 64; ++j) s += s_sum[j];
    part[blockIdx.x] = s;
  }
}

// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN where the
// norm (as float32) is not finite.
__global__ void __launch_bounds__(1024)
    k_grad_norm_total(int64_t n, const double* part, double max_norm, float* out) {
  __shared__ double s_sum[16];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 1024) s += part[i];
  s = wave_sum64(s);
  if ((threadIdx.x & 63) == 0) s_sum[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int j = 1; j < 16; ++j) s += s_sum[j];
  const double norm = sqrt(s), f = max_norm / (norm + 1e-6);
  out[0] = float(norm);
  out[1] = isfinite(float(norm)) ? float(f < 1.0 ? f : 1.0) : __builtin_nanf("");
}

// ------------------------------------------------------------------ the step

struct Step {
  float lr, size, root, eps;  // size = lr / (1 - b1^t), root = 1 / sqrt(1 - b2^t)
  float scale;                  // of the gradients
  bool skip;
};

__device__ __forceinline__ double pow_int(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1, b *= b)
    if (t & 1) r *= b;
  return r;
}

__device__ __forceinline__ Step step_of(const AdamArgs& a) {
  Step s{a.lr_f, a.size, a.root, a.eps, 1.0f, false};
  if (a.step_dev || a.lr_dev) {
    const double lr = a.lr_dev ? double(*a.lr_dev) : a.lr;
    const int64_t t = a.step_dev ? max(int64_t(1), *a.step_dev) : a.step;
    s.lr = float(lr);
    s.size = float(lr / (1.0 - pow_int(a.beta1, t)));
    s.root = float(1.0 / sqrt(1.0 - pow_int(a.beta2, t)));
  }
  if (a.grad_scale) {
    s.scale = *a.grad_scale;
    s.skip = a.skip_nonfinite && !isfinite(s.scale);
  }
  return s;
}

// p after the step, from sqrt(v).  Decay and update are added first and taken
// off together: one rounding of p, and lr wd is not lost in 1 - lr wd.  Root
// and reciprocal are the hardware's, off by a step at most.
__device__ __forceinline__ float stepped(float p, float m, float root_v, float lr_wd,
                                         const Step& s) {
  const float d = fmaf(root_v, s.root, s.eps);
  return p - fmaf(s.size * m, __builtin_amdgcn_rcpf(d), lr_wd * p);
}

// Float32 moments: a workgroup per 1024 elements, which it takes at once (four
// times as many in a loop: 351 us against 326 at 61M packed elements).
__global__ void __launch_bounds__(kParamThreads) k_adamw(const ParamList l, const AdamArgs a) {
  const Step st = step_of(a);
  if (st.skip) return;
  const int ti = tensor_of(l.wg0, l.n);
  const ParamTensor t = l.t[ti];
  const int64_t i = int64_t(int(blockIdx.x) - l.wg0[ti]) * kPass + int(threadIdx.x) * 4;
  if (i >= t.n) return;
  const float lr_wd = st.lr * t.weight_decay;
  const float b1 = float(a.beta1), c1 = float(1.0 - a.beta1);
  const float b2 = float(a.beta2), c2 = float(1.0 - a.beta2);
  float* m = static_cast<float*>(t.m);
  float* v = static_cast<float*>(t.v);
  float p4[4], g4[4], m4[4], v4[4];
  load4<true>(t.p, i, t.n, p4);
  load4_grad(t, i, g4);
  load4<true>(m, i, t.n, m4);
  load4<true>(v, i, t.n, v4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float g = g4[e] * st.scale;
    m4[e] = fmaf(b1, m4[e], c1 * g);
    v4[e] = fmaf(b2, v4[e], c2 * g * g);
    p4[e] = stepped(p4[e], m4[e], __builtin_amdgcn_sqrtf(v4[e]), lr_wd, st);
  }
  store4(t.p, i, t.n, p4);
  store4(m, i, t.n, m4);
  store4(v, i, t.n, v4);
  if (t.copy) store4(static_cast<__bf16*>(t.copy), i, t.n, p4);
}

// ------------------------------------------------------------ 8-bit moments

// Largest of two bit patterns over the wavefront, in every lane.
__device__ __forceinline__ void wave_max2(uint32_t& a, uint32_t& b) {
  const auto step = [&](auto ctrl) {
    constexpr int C = decltype(ctrl)::value;
    a = max(a, uint32_t(__builtin_amdgcn_mov_dpp(int(a), C, 0xF, 0xF, false)));
    b = max(b, uint32_t(__builtin_amdgcn_mov_dpp(int(b), C, 0xF, 0xF, false)));
  };
  step(std::integral_constant<int, 0xB1>{});   // lane ^ 1
  step(std::integral_constant<int, 0x4E>{});   // lane ^ 2
  step(std::integral_constant<int, 0x141>{});  // half-row mirror
  step(std::integral_constant<int, 0x140>{});  // row mirror
  auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  a = max(uint32_t(r[0]), uint32_t(r[1]));
  r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  b = max(uint32_t(r[0]), uint32_t(r[1]));
  r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
  a = max(uint32_t(r[0]), uint32_t(r[1]));
  r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  b = max(uint32_t(r[0]), uint32_t(r[1]));
}

constexpr uint32_t kFlip = 0x80808080u;  // int8 codes as bytes c + 128

// Byte e of a word as a float.
template <int E>
__device__ __forceinline__ float byte_of(uint32_t w) {
  return float((w >> (8 * E)) & 255u);
}

// c |c| and c^2 of the codes: at most 16 bits, exact.
template <int E>
__device__ __forceinline__ float square_m(uint32_t flipped) {
  const float c = byte_of<E>(flipped) - 128.0f;
  return c * fabsf(c);
}
template <int E>
__device__ __forceinline__ float square_v(uint32_t w) {
  const float c = byte_of<E>(w);
  return c * c;
}

// A code from its 32-bit root t, off by 3e-5 (m: values to 127) or 7e-5 (v: to
// 255) at most: nearer to a border than `kNear` 64 bits decide, as they do all
// over when the scale is so small that 32-bit roots lose the value (`tiny`).
constexpr float kNear = 1e-4f;
constexpr float kTinyM = 1e-36f, kTinyV = 1e-18f;

__device__ __forceinline__ bool near_border(float t, float c) {
  return fabsf(t - c) > 0.5f - kNear;
}
// P = 1: borders s (k + 1/2)^2; P = 2: their squares.
template <int P>
__device__ float code_exact(float t, double value, double s, bool tiny) {
  if (tiny) {
    const double q = P == 1 ? value / s : sqrt(value) / s;
    t = float(sqrt(q));
  }
  const float f = floorf(t), r = t - f - 0.5f;
  if (fabsf(r) > 2.0f * kNear) return f + (r > 0.0f ? 1.0f : 0.0f);
  const double h = double(f) + 0.5, b = s * (h * h);
  return f + ((P == 1 ? b : b * b) < value ? 1.0f : 0.0f);
}

// A wavefront per block of 256 elements, four consecutive ones a lane.  The
// maxima are taken over the bit patterns of |m| and v (so a NaN wins): a
// block that holds a value that is not finite reads back as NaN.
__global__ void __launch_bounds__(kParamThreads) k_adamw8(const ParamList l, const AdamArgs a) {
  const Step st = step_of(a);
  if (st.skip) return;
  const int ti = tensor_of(l.wg0, l.n);
  const ParamTensor t = l.t[ti];
  const int64_t base = int64_t(int(blockIdx.x) - l.wg0[ti]) * l.chunk;
  const int64_t end = min(t.n, base + l.chunk);
  const float lr_wd = st.lr * t.weight_decay;
  const double scale = double(st.scale);
  const double c1 = (1.0 - a.beta1) * scale, c2 = (1.0 - a.beta2) * scale * scale;
  uint8_t* mc = static_cast<uint8_t*>(t.m);
  uint8_t* vc = static_cast<uint8_t*>(t.v);
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (int64_t b0 = base + wv * kQBlock; b0 < end; b0 += kParamThreads / 64 * kQBlock) {
    const int64_t i = b0 + lane * 4, blk = b0 / kQBlock;
    float p4[4], g4[4];
    load4<true>(t.p, i, t.n, p4);
    load4_grad(t, i, g4);
    const uint32_t mw = load_codes(mc, i, t.n) ^ kFlip;
    const uint32_t vw = load_codes(vc, i, t.n);
    const double sm = a.beta1 * double(t.m_scale[blk]), sv = double(t.v_scale[blk]);
    const double sv2 = a.beta2 * (sv * sv);
    const float qm[4] = {square_m<0>(mw), square_m<1>(mw), square_m<2>(mw), square_m<3>(mw)};
    const float qv[4] = {square_v<0>(vw), square_v<1>(vw), square_v<2>(vw), square_v<3>(vw)};
    double m4[4], v4[4];
    float mf[4], root[4];
    uint32_t am = 0, av = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double g = double(g4[e]), q = double(qv[e]);
      m4[e] = fma(sm, double(qm[e]), c1 * g);
      v4[e] = fma(sv2, q * q, c2 * (g * g));
      mf[e] = float(m4[e]);
      const float vf = float(v4[e]);
      am = max(am, __float_as_uint(fabsf(mf[e])));
      av = max(av, __float_as_uint(vf) & 0x7FFFFFFFu);
      root[e] = __builtin_amdgcn_sqrtf(vf);
      p4[e] = stepped(p4[e], mf[e], root[e], lr_wd, st);
    }
    store4(t.p, i, t.n, p4);
    if (t.copy) store4(static_cast<__bf16*>(t.copy), i, t.n, p4);
    wave_max2(am, av);
    float nm = float(double(__uint_as_float(am)) * (1.0 / 16129.0));
    float nv = float(sqrt(double(__uint_as_float(av))) * (1.0 / 65025.0));
    nm = isfinite(nm) ? nm : __builtin_nanf("");
    nv = isfinite(nv) ? nv : __builtin_nanf("");
    const bool tiny_m = nm < kTinyM && nm > 0.0f, tiny_v = nv < kTinyV && nv > 0.0f;
    const float im = nm > 0.0f ? __builtin_amdgcn_rcpf(nm) : 0.0f;
    const float iv = nv > 0.0f ? __builtin_amdgcn_rcpf(nv) : 0.0f;
    float tm[4], tv[4], cm[4], cv[4];
    bool near = tiny_m || tiny_v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      tm[e] = __builtin_amdgcn_sqrtf(fabsf(mf[e]) * im);
      tv[e] = __builtin_amdgcn_sqrtf(root[e] * iv);
      cm[e] = rintf(tm[e]);
      cv[e] = rintf(tv[e]);
      near = near || near_border(tm[e], cm[e]) || near_border(tv[e], cv[e]);
    }
    if (near) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cm[e] = nm > 0.0f ? code_exact<1>(tm[e], fabs(m4[e]), double(nm), tiny_m) : 0.0f;
        cv[e] = nv > 0.0f ? code_exact<2>(tv[e], v4[e], double(nv), tiny_v) : 0.0f;
      }
    }
    uint32_t mo = 0, vo = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float c = copysignf(fminf(cm[e], 127.0f), mf[e]) + 128.0f;
      mo = __builtin_amdgcn_cvt_pk_u8_f32(c, e, mo);
      vo = __builtin_amdgcn_cvt_pk_u8_f32(v4[e] > 0.0 ? fmaxf(cv[e], 1.0f) : 0.0f, e, vo);
    }
    store_codes(mc, i, t.n, mo ^ kFlip);
    store_codes(vc, i, t.n, vo);
    if (lane == 0) {
      t.m_scale[blk] = nm;
      t.v_scale[blk] = nv;
    }
  }
}

// The moments as float32: p and grad hold the destinations of m and v.
__global__ void __launch_bounds__(kParamThreads) k_moments8(const ParamList l) {
  const int ti = tensor_of(l.wg0, l.n);
  const ParamTensor t = l.t[ti];
  const int64_t base = int64_t(int(blockIdx.x) - l.wg0[ti]) * l.chunk;
  const int64_t end = min(t.n, base + l.chunk);
  float* mo = t.p;
  float* vo = static_cast<float*>(const_cast<void*>(t.grad));
  for (int64_t i = base + int(threadIdx.x) * 4; i < end; i += 4 * kParamThreads) {
    const uint32_t mw = load_codes(static_cast<const uint8_t*>(t.m), i, t.n) ^ kFlip;
    const uint32_t vw = load_codes(static_cast<const uint8_t*>(t.v), i, t.n);
    const double sm = double(t.m_scale[i / kQBlock]), sv = double(t.v_scale[i / kQBlock]);
    const float qm[4] = {square_m<0>(mw), square_m<1>(mw), square_m<2>(mw), square_m<3>(mw)};
    const float qv[4] = {square_v<0>(vw), square_v<1>(vw), square_v<2>(vw), square_v<3>(vw)};
    float m4[4], v4[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const double r = sv * double(qv[e]);
      m4[e] = float(sm * double(qm[e]));
      v4[e] = float(r * r);
    }
    store4(mo, i, t.n, m4);
    store4(vo, i, t.n, v4);
  }
}

// Elements of a workgroup: one pass of its threads while that does not fill the
// card (2048 workgroups), up to `most` for long lists.  Measured, us, at 130M
// bf16 gradients: norm 16384 59, 65536 57; at 101M elements with 8-bit moments:
// step 1024 +42, 4096 0, 8192 +4; reading them back 1024 +6, 2048 -10, 4096 0.
int64_t chunk_of(const ParamTensor* t, int n, int64_t pass, int64_t most) {
  int64_t total = 0;
  for (int i = 0; i < n; ++i) total += t[i].n;
  const int64_t even = (total + 2048 * pass - 1) / (2048 * pass) * pass;
  return std::clamp(even, pass, most);
}

// Calls f(list, workgroups) for runs of at most kParamsPerLaunch of the
// tensors that `take` picks, empty ones left out.
template <class P, class F>
hipError_t for_lists(const ParamTensor* t, int n, int64_t chunk, P&& take, F&& f) {
  ParamList l;
  l.n = 0;
  l.chunk = int(chunk);
  int64_t wgs = 0;
  const auto flush = [&]() -> hipError_t {
    if (l.n == 0) return hipSuccess;
    const hipError_t e = f(static_cast<const ParamList&>(l), unsigned(wgs));
    l.n = 0;
    wgs = 0;
    return e;
  };
  for (int i = 0; i < n; ++i) {
    if (t[i].n == 0 || !take(t[i])) continue;
    const int64_t w = (t[i].n + chunk - 1) / chunk;
    if (l.n == kParamsPerLaunch || wgs + w > kMaxWorkgroups) {
      const hipError_t e = flush();
      if (e != hipSuccess) return e;
    }
    l.t[l.n] = t[i];
    l.wg0[l.n++] = int(wgs);
    wgs += w;
  }
  return flush();
}

}  // namespace

size_t grad_norm_partials(const ParamTensor* t, int n) {
  const int64_t chunk = chunk_of(t, n, kPass, kNormChunk);
  size_t w = 0;
  for (int i = 0; i < n; ++i) w += size_t((t[i].n + chunk - 1) / chunk);
  return w;
}

hipError_t launch_grad_norm(const ParamTensor* t, int n, double max_norm, double* part, float* out,
                            hipStream_t s) {
  GradList l;
  l.n = 0;
  l.chunk = int(chunk_of(t, n, kPass, kNormChunk));
  int64_t done = 0, wgs = 0;
  for (int i = 0; i <= n; ++i) {
    const int64_t w = i < n ? (t[i].n + l.chunk - 1) / l.chunk : 0;
    if (l.n > 0 && (i == n || l.n == kGradsPerLaunch || wgs + w > kMaxWorkgroups)) {
      hipLaunchKernelGGL(k_grad_norm, dim3(unsigned(wgs)), dim3(kParamThreads), 0, s, l,
                         part + done);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      done += wgs;
      l.n = 0;
      wgs = 0;
    }
    if (w == 0) continue;
    l.wg0[l.n] = int(wgs);
    l.size[l.n] = t[i].grad_bf16 ? ~t[i].n : t[i].n;
    l.grad[l.n++] = t[i].grad;
    wgs += w;
  }
  hipLaunchKernelGGL(k_grad_norm_total, dim3(1), dim3(1024), 0, s, done, part, max_norm, out);
  return hipGetLastError();
}

hipError_t launch_adamw(const ParamTensor* t, int n, const AdamArgs& a, hipStream_t s) {
  const hipError_t e = for_lists(
      t, n, kPass, [](const ParamTensor& p) { return p.m_scale == nullptr; },
      [&](const ParamList& l, unsigned wgs) {
        hipLaunchKernelGGL(k_adamw, dim3(wgs), dim3(kParamThreads), 0, s, l, a);
        return hipGetLastError();
      });
  if (e != hipSuccess) return e;
  return for_lists(
      t, n, chunk_of(t, n, kPass, kAdamChunk),
      [](const ParamTensor& p) { return p.m_scale != nullptr; },
      [&](const ParamList& l, unsigned wgs) {
        hipLaunchKernelGGL(k_adamw8, dim3(wgs), dim3(kParamThreads), 0, s, l, a);
        return hipGetLastError();
      });
}

hipError_t launch_moments8(const ParamTensor* t, int n, hipStream_t s) {
  return for_lists(
      t, n, chunk_of(t, n, kPass, kReadChunk), [](const ParamTensor&) { return true; },
      [&](const ParamList& l, unsigned wgs) {
        hipLaunchKernelGGL(k_moments8, dim3(wgs), dim3(kParamThreads), 0, s, l);
        return hipGetLastError();
      });
}

}  // namespace e3k
