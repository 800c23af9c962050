// Tiles of rows x 128 bytes from memory to LDS without passing through
// registers, for products whose both operands lie along k in memory: a lane
// names 16 bytes anywhere, a wavefront's 64 lanes land side by side.  The eight
// 16-byte pieces of row r lie in LDS at piece ^ (r & 7): the 16-byte reads of
// 16 lanes in consecutive rows then meet every bank alike.
//
// A workgroup of 4 wavefronts multiplies 128 rows by 128 columns, 64 x 64 a
// wavefront, in chunks of 128 bytes of k.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace e3k {

using s16x4_t = short __attribute__((ext_vector_type(4)));
using bf16x8_t = __bf16 __attribute__((ext_vector_type(8)));

constexpr int kTileRows = 128;

// What is read where a row has ended.
static __device__ const uint32_t kTileZeros[4] = {0, 0, 0, 0};

struct TileLoad {
  static constexpr int kPasses = 4;              // of 32 rows, by 256 threads
  static constexpr int kBytes = kTileRows * 128;
  int wave, row, piece;  // this lane's rows are row, row + 32, row + 64, row + 96
  __device__ __forceinline__ TileLoad()
      : wave(__builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6))),
        row(int(threadIdx.x >> 3)), piece((int(threadIdx.x) ^ int(threadIdx.x >> 3)) & 7) {}
  // asks for 16 bytes of row `row + 32 i`
  __device__ __forceinline__ void ask(const uint8_t* from, uint8_t* lds, int i) const {
    __builtin_amdgcn_global_load_lds(
        (const __attribute__((address_space(1))) void*)from,
        (__attribute__((address_space(3))) void*)(lds + (i * 4 + wave) * 1024), 16, 0, 0);
  }
};

// 16 bytes of row r.
__device__ __forceinline__ const uint8_t* tile_at(const uint8_t* lds, int r, int piece) {
  return lds + r * 128 + ((piece ^ (r & 7)) << 4);
}

// Tiles of 32 or 64 k of 128 bf16 channels that lie along the channels in
// memory: 16 pieces a k, which a transposing read turns to the order of the
// products.  A lane's pieces are of rows row, row + 16 and so on; FLIP: the bit
// of the piece at which the rows of 16 lanes part, 4 for reads of 4 channels
// out of every 8, 2 for 16 channels in a row (then 32 lanes meet no bank twice).
template <int FLIP>
struct AcrossLoad {
  int row, piece;
  __device__ __forceinline__ AcrossLoad()
      : row(int(threadIdx.x >> 4)), piece((int(threadIdx.x) & 15) ^ flip(row)) {}
  static __device__ __forceinline__ int flip(int k) {
    return FLIP == 4 ? (k & 3) << 2 : (k & 3) << 1 | (k & 8);
  }
  // 8 values along k, from 8 (lane / 16) on, of channel lane % 16 of those
  // whose fourths the lanes name: lane 4 r + c of 16 names fourth c
  static __device__ __forceinline__ bf16x8_t read(const uint8_t* lds, int kk, int piece, int half) {
    const int lane = int(threadIdx.x) & 63;
    const int k = kk * 32 + (lane >> 4) * 8 + ((lane >> 2) & 3);
    const uint8_t* at = lds + k * 256 + ((piece ^ flip(k)) << 4) + half * 8;
    using Lds = __attribute__((address_space(3))) s16x4_t;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)at);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds*)(at + 4 * 256));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// Waits for this wavefront's loads and for its reads of LDS, then for the other
// wavefronts: what it asked for is there, and nobody still reads the stage that
// is asked for next.  (The products of a turn may come after the barrier, and
// without the wait for LDS so may the last of their operands.)
__device__ __forceinline__ void tile_wait() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace e3k
