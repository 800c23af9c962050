// Stores of 16 rows in whole 128-byte lines.  After a product lane q + 16 h
// holds 16 bytes of two neighbouring 64-byte pieces of row q, `first` and
// `second`: stored as they are, an instruction writes half lines of 16 rows.
// Trading with lane q ^ 8, a lane ends with 16 bytes of rows q & 7 and 8 + (q &
// 7), the first piece's in the lower eight lanes, and an instruction writes
// whole lines of 8 rows.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "common.h"

namespace e3k {

__device__ __forceinline__ int ror8(int v) {  // of lane ^ 8, within 16 lanes
  return __builtin_amdgcn_mov_dpp(v, 0x128, 0xF, 0xF, false);
}

struct RowHalves {
  bool low;    // q < 8
  int column;  // bytes from the first piece's start to this lane's 16
  __device__ __forceinline__ RowHalves()
      : low((threadIdx.x & 8) == 0),
        column(((threadIdx.x & 8) ? 64 : 0) + int(threadIdx.x >> 4 & 3) * 16) {}
  // a value of row q becomes those of the rows written first and second
  __device__ __forceinline__ void rows(int v, int& v0, int& v1) const {
    const int o = ror8(v);
    v0 = low ? v : o;
    v1 = low ? o : v;
  }
  template <class V>
  __device__ __forceinline__ void trade(V& first, V& second) const {
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    static_assert(sizeof(V) == 16);
    i32x4 a = __builtin_bit_cast(i32x4, first), b = __builtin_bit_cast(i32x4, second);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int got = ror8(low ? b[i] : a[i]);
      a[i] = low ? a[i] : got;
      b[i] = low ? got : b[i];
    }
    first = __builtin_bit_cast(V, a);
    second = __builtin_bit_cast(V, b);
  }
};

}  // namespace e3k
