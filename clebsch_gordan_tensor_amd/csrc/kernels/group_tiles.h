// Rows of a group in tiles: which group and rows a workgroup has, found from
// the index's offsets by every wavefront for itself.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "registry.h"

namespace e3k {

struct GroupTile {
  int group;      // n_groups: rows without a group
  int64_t first;  // position in the order of the group's first row
  int64_t rows;   // of the product: the group's rows x components
  int64_t at;     // first row of the tile among them
};

// An index of other sizes than the call's is not used (its launches do nothing).
__device__ __forceinline__ bool index_matches(const int* index, int64_t n_rows, int n_groups) {
  return !index || (index[0] == kGroupMagic && index[1] == n_rows && index[2] == n_groups);
}

// Tile t when every group's rows x deg go into tiles of `size`; false past the
// last one.  A lane per group counts, the tile's group is found by a ballot.
__device__ __forceinline__ bool find_tile(const int* offsets, int n_groups, int64_t n_rows, int deg,
                                          int64_t size, int64_t t, GroupTile& tile) {
  if (!offsets) {
    tile = {0, 0, n_rows * deg, t * size};
    return tile.at < tile.rows;
  }
  const int lane = threadIdx.x & 63;
  for (int g0 = 0; g0 <= n_groups; g0 += 64) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    if (g <= n_groups) {
      lo = offsets[g];
      hi = g < n_groups ? offsets[g + 1] : n_rows;
    }
    const int n = int(((hi - lo) * deg + size - 1) / size);
    int s = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(s, o);
      if (lane >= o) s += v;
    }
    const uint64_t past = __ballot(int64_t(s) > t);
    if (past) {
      const int f = __ffsll((unsigned long long)past) - 1;
      const int before = __builtin_amdgcn_readlane(s - n, f);
      const int first = __builtin_amdgcn_readlane(int(lo), f);
      const int end = __builtin_amdgcn_readlane(int(hi), f);
      tile = {g0 + f, first, int64_t(end - first) * deg, (t - before) * size};
      return true;
    }
    t -= __builtin_amdgcn_readlane(s, 63);
  }
  return false;
}

// Most tiles that n_rows rows in n_groups groups (and some without) can fill.
inline int64_t most_tiles(int64_t n_rows, int n_groups, int deg, int64_t size, bool grouped) {
  return (n_rows * deg + size - 1) / size + (grouped ? n_groups : 0);
}

}  // namespace e3k
