// Values in 8 bits (e4m3: 4 bits of exponent, 3 of mantissa, no infinities,
// largest 448), 128 consecutive channels sharing a float32 scale:
//   scale = max(max |v| fl(1/448), 2^-126),  code = v / scale
// the product rounded once, the quotient to float32 and then to nearest in 8
// bits (ties to even).  A run that holds a value
// that is not finite has the scale NaN, and reads back as NaN.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace e3k {

constexpr int kFp8Run = 128;
constexpr float kFp8Part = 1.0f / 448.0f, kFp8Least = 0x1p-126f;

__host__ __device__ constexpr int fp8_runs(int channels) {
  return (channels + kFp8Run - 1) / kFp8Run;
}

// Largest |v|, as the largest of their bits: an infinity is above every finite
// value there, and NaN above that.
__device__ __forceinline__ float fp8_max(float a, float b) {
  return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
template <int V>
__device__ __forceinline__ float fp8_top(const float (&v)[V]) {
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) t = max(t, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return __uint_as_float(t);
}

struct Fp8Scale {
  float scale, inv;
  // top: the run's largest |v|
  __device__ __forceinline__ explicit Fp8Scale(float top) {
    scale = fmaxf(top * kFp8Part, kFp8Least);
    if (!(top < __builtin_inff())) scale = __builtin_nanf("");
    inv = 1.0f / scale;
  }
  // v / scale rounded once: the product with the reciprocal, corrected by what
  // it leaves of v (exact for quotients that 8 bits can tell from 0).
  __device__ __forceinline__ float of(float v) const {
    const float t = v * inv;
    return fmaf(fmaf(-t, scale, v), inv, t);
  }
};

// Codes of four values.
__device__ __forceinline__ uint32_t fp8_codes(float a, float b, float c, float d,
                                              const Fp8Scale& s) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(s.of(a), s.of(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(s.of(c), s.of(d), r, true);
  return uint32_t(r);
}
// V codes side by side at an address aligned to V.
template <int V, bool STREAM>
__device__ __forceinline__ void fp8_store(uint8_t* p, const float (&v)[V], const Fp8Scale& s) {
  static_assert(V == 4 || V == 8);
  if constexpr (V == 4) {
    const uint32_t c = fp8_codes(v[0], v[1], v[2], v[3], s);
    if constexpr (STREAM) __builtin_nontemporal_store(c, reinterpret_cast<uint32_t*>(p));
    else *reinterpret_cast<uint32_t*>(p) = c;
  } else {
    const uint64_t c = fp8_codes(v[0], v[1], v[2], v[3], s) |
                       uint64_t(fp8_codes(v[4], v[5], v[6], v[7], s)) << 32;
    if constexpr (STREAM) __builtin_nontemporal_store(c, reinterpret_cast<uint64_t*>(p));
    else *reinterpret_cast<uint64_t*>(p) = c;
  }
}

}  // namespace e3k
