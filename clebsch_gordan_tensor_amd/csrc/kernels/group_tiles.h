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
// Asked before find_tile and looked at after it, its words come with the offsets.
__device__ __forceinline__ bool index_matches(const int* index, int64_t n_rows, int n_groups) {
  if (!index) return true;
  const int magic = index[0], rows = index[1], groups = index[2];
  return (magic == kGroupMagic) & (rows == n_rows) & (groups == n_groups);
}

// Tile t when every group's rows x deg go into tiles of `size`, at least
// `least` of them; false past the last one.  A lane per group counts, the
// tile's group is found by a ballot.
__device__ __forceinline__ bool find_tile(const int* offsets, int n_groups, int64_t n_rows, int deg,
                                          int64_t size, int64_t t, GroupTile& tile, int least = 0) {
  if (!offsets) {
    tile = {0, 0, n_rows * deg, t * size};
    return tile.at < tile.rows || t < least;
  }
  const int lane = threadIdx.x & 63;
  for (int g0 = 0; g0 <= n_groups; g0 += 64) {
    const int g = g0 + lane;
    int64_t lo = 0, hi = 0;
    if (g <= n_groups) {
      lo = offsets[g];
      hi = g < n_groups ? offsets[g + 1] : n_rows;
    }
    const int n = g <= n_groups ? max(least, int(((hi - lo) * deg + size - 1) / size)) : 0;
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

// Tiles of all groups together.
__device__ __forceinline__ int count_tiles(const int* offsets, int n_groups, int64_t n_rows,
                                           int deg, int64_t size) {
  if (!offsets) return int((n_rows * deg + size - 1) / size);
  int total = 0;
  for (int g0 = 0; g0 <= n_groups; g0 += 64) {
    const int g = g0 + int(threadIdx.x & 63);
    int n = 0;
    if (g <= n_groups) {
      const int64_t lo = offsets[g], hi = g < n_groups ? offsets[g + 1] : n_rows;
      n = int(((hi - lo) * deg + size - 1) / size);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) n += __shfl_xor(n, o);
    total += n;
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// The tile of workgroup `id` where `cols` column tiles share a tile's rows:
// neighbouring workgroups run on different XCDs, and each XCD takes a stretch
// of consecutive tiles, column by column, so that a tile's rows are read once
// into its L2 and a group's weights by few of them.  The launch has
// xcd_workgroups(most_tiles) workgroups.
constexpr int kXcds = 8;
__device__ __forceinline__ bool find_tile_xcd(const int* offsets, int n_groups, int64_t n_rows,
                                              int deg, int64_t size, unsigned id, unsigned cols,
                                              GroupTile& tile, int& col) {
  const unsigned total = unsigned(count_tiles(offsets, n_groups, n_rows, deg, size));
  const unsigned per = (total + kXcds - 1) / kXcds, slot = id / kXcds, t = slot / cols;
  col = int(slot - t * cols);
  const unsigned at = id % kXcds * per + t;
  return t < per && at < total && find_tile(offsets, n_groups, n_rows, deg, size, at, tile);
}
inline int64_t xcd_workgroups(int64_t tiles, int64_t cols) {
  return (tiles + kXcds - 1) / kXcds * kXcds * cols;
}

// Rows of a group by their place in it.  Without an index the rows are their
// places; something is read all the same (`any`: memory of four bytes at
// least), so that several rows can be asked for at once.
struct RowOrder {
  const int* at;
  bool listed;
  __device__ __forceinline__ RowOrder(const int* index, int order, const GroupTile& tile,
                                      const void* any)
      : at(index ? index + order + tile.first : static_cast<const int*>(any)), listed(index) {}
  __device__ __forceinline__ int operator()(int place) const {
    const int row = at[listed ? place : 0];
    return listed ? row : place;
  }
};

// Rows of a product's tile: row r is component m of the group's row `place`.
struct TileRows {
  int from;     // place of the tile's first row
  unsigned m0;  // its component
  unsigned deg;
  __device__ __forceinline__ TileRows(int64_t first, int deg_)
      : from(int(first / deg_)), m0(unsigned(first - int64_t(from) * deg_)), deg(unsigned(deg_)) {}
  __device__ __forceinline__ int place(int r, int& m) const {
    const unsigned c = m0 + unsigned(r), d = c / deg;
    m = int(c - d * deg);
    return int(unsigned(from) + d);
  }
};

// Whether the groups have so few rows that kernels of tiles of 16 rows and
// columns answer sooner than those that keep W's columns in registers, which
// first have to fetch all of them.
inline bool few_rows(int64_t n_rows, int n_groups, const MixList& l) {
  int deg = 1;
  for (int i = 0; i < l.n_blocks; ++i) deg = l.blk[i].deg > deg ? l.blk[i].deg : deg;
  return n_rows * deg <= 16 * int64_t(n_groups) + 112;
}

// Tiles of 16 rows and columns of all blocks, a row of tiles for every group
// besides, also where there are fewer rows than groups (one row of 4096 columns
// counts 1,280 at 4 groups and goes to the large tiles in bf16, where 256 would
// do).  Kernels of such tiles fetch W for each, and yet they answer sooner than
// large tiles as long as the chip isn't full of them.  us by small tiles and by large, 1024 to 1024 channels: float32,
// one group, 512 rows 32 and 78, 1024 52 and 79, 2048 93 and 79; 16 groups,
// 1024 67 and 81, 2048 113 and 82; bf16, one group, 256 rows 11.5 and 14.8, 512
// 15.8 and 14.7; 16 groups, 128 15.5 and 15.7, 256 18.6 and 15.6; the same of
// 2048 to 512: 4,100 to 4,600 tiles 100 and 152 to 128 and 154 in float32, 1,020
// tiles 21 and 26 and 1,540 28 and 26 in bf16.
inline int64_t small_tiles(int64_t n_rows, int n_groups, const MixList& l, int cout) {
  int64_t n = 0;
  for (int i = 0; i < l.n_blocks; ++i) n += (n_rows * l.blk[i].deg + 15) / 16 + n_groups;
  return n * ((cout + 15) / 16);
}

// Most tiles that n_rows rows in n_groups groups (and some without) can fill.
inline int64_t most_tiles(int64_t n_rows, int n_groups, int deg, int64_t size, bool grouped) {
  return (n_rows * deg + size - 1) / size + (grouped ? n_groups : 0);
}

// Launches `wgs` workgroups of `threads` as go(workgroups, the first one's number).
// A launch holds fewer than 2^32 threads; more workgroups than that (a single
// column tile of 2^31 rows and components has as many) go in several, each from
// a multiple of the XCDs on.
template <class F>
hipError_t launch_tiles(int64_t wgs, int threads, F&& go) {
  const int64_t most = (int64_t(1) << 31) / threads;
  for (int64_t at = 0; at < wgs; at += most) {
    go(unsigned(wgs - at < most ? wgs - at : most), unsigned(at));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace e3k
