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

// Waits for this wavefront's loads, then for the other wavefronts.
__device__ __forceinline__ void tile_wait() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace e3k
