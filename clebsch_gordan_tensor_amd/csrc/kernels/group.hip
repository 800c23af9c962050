// Index of rows by group: `order` lists the rows of group 0, then those of
// group 1 and so on, in their own order within each, then the rows that have
// no group (an id outside [0, n_groups)); `offsets` says where each begins.
//
// A stable counting sort.  A chunk of rows is a workgroup's; each of its
// wavefronts counts its own consecutive rows per group (LDS), so a row's place
// is: where its group begins + the group's rows in earlier chunks + in earlier
// wavefronts + in earlier lanes.  The lanes of a wavefront that share a group
// find each other by one ballot per bit of the id.  Counts are whole numbers:
// the order of the LDS atomics does not show.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "registry.h"

namespace e3k {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPerLane = 8;                         // rows of a lane
constexpr int kChunk = kThreads * kPerLane;         // rows of a workgroup
constexpr int kFewCounts = 8192;                    // (groups + 1) x chunks

__device__ __forceinline__ int key_of(const int* group, int64_t r, int n_groups) {
  const int g = group[r];
  return unsigned(g) < unsigned(n_groups) ? g : n_groups;
}

// Lanes of this wavefront with the same key, the inactive ones left out.
__device__ __forceinline__ uint64_t same_key(int key, int bits, bool active) {
  uint64_t m = __ballot(active);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((key >> b) & 1);
    m &= (key >> b) & 1 ? set : ~set;
  }
  return m;
}

// Adds the wavefront's lanes to count[key], `same` being those of this lane's
// key: the first of them adds for all.
__device__ __forceinline__ void count_same(int* count, int key, uint64_t same) {
  const int lane = threadIdx.x & 63;
  if (same && lane == __ffsll((unsigned long long)same) - 1) atomicAdd(count + key, __popcll(same));
}
// The same; returns the count before this lane.
__device__ __forceinline__ int place_same(int* count, int key, uint64_t same) {
  const int lane = threadIdx.x & 63;
  const int first = same ? __ffsll((unsigned long long)same) - 1 : lane;
  int old = 0;
  if (same && lane == first) old = atomicAdd(count + key, __popcll(same));
  old = __shfl(old, first);
  return old + __popcll(same & ((uint64_t(1) << lane) - 1));
}

// Exclusive prefix sums of v[0..n) in LDS by the whole workgroup, n <= 1025;
// `part` holds a value for each wavefront.
__device__ __forceinline__ void prefix(int* v, int n, int* part) {
  const int tid = threadIdx.x, threads = blockDim.x;
  const int per = (n + threads - 1) / threads;
  int s = 0;
  for (int j = 0; j < per; ++j) {
    const int i = tid * per + j;
    if (i < n) s += v[i];
  }
  int t = s;  // inclusive over the wavefront
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(t, o);
    if ((tid & 63) >= o) t += u;
  }
  if ((tid & 63) == 63) part[tid >> 6] = t;
  __syncthreads();
  s = t - s;
  for (int j = 0; j < (tid >> 6); ++j) s += part[j];
  for (int j = 0; j < per; ++j) {
    const int i = tid * per + j;
    if (i < n) {
      const int c = v[i];
      v[i] = s;
      s += c;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void write_header(const GroupArgs& a) {
  if (threadIdx.x == 0) {
    a.index[0] = kGroupMagic;
    a.index[1] = a.n_rows;
    a.index[2] = a.n_groups;
  }
}

// hist[g][chunk]: rows of group g in the chunk.
__global__ void __launch_bounds__(kThreads) k_group_count(const GroupArgs a) {
  __shared__ int s_n[kMaxGroups + 1];
  const int G = a.n_groups;
  for (int g = threadIdx.x; g <= G; g += kThreads) s_n[g] = 0;
  __syncthreads();
  const int64_t r0 = int64_t(blockIdx.x) * kChunk;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t r = r0 + j * kThreads + threadIdx.x;
    if (r < a.n_rows) atomicAdd(s_n + key_of(a.group, r, G), 1);
  }
  __syncthreads();
  for (int g = threadIdx.x; g <= G; g += kThreads)
    a.hist[int64_t(g) * a.n_chunks + blockIdx.x] = s_n[g];
}

// A workgroup a group: hist becomes the rows of the group in earlier chunks,
// total[g] those in all.
__global__ void __launch_bounds__(kThreads) k_group_scan(const GroupArgs a) {
  __shared__ int s_part[kWaves];
  int* h = a.hist + int64_t(blockIdx.x) * a.n_chunks;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  constexpr int N = 8;  // counts of a thread, side by side
  int before = 0;
  for (int c0 = 0; c0 < a.n_chunks; c0 += N * kThreads) {
    const int c = c0 + tid * N;
    int v[N], n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c + j < a.n_chunks ? h[c + j] : 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += v[j];
    int s = n;  // inclusive over the wavefront
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int t = __shfl_up(s, o);
      if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 63) s_part[w] = s;
    __syncthreads();
    int left = before + s - n;
    for (int j = 0; j < kWaves; ++j) {
      if (j < w) left += s_part[j];
      before += s_part[j];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (c + j < a.n_chunks) h[c + j] = left;
      left += v[j];
    }
  }
  if (tid == 0) a.total[blockIdx.x] = before;
}

// The chunk is sorted in LDS first and written in runs of a group's rows: a
// store's 64 lanes then meet few lines of memory instead of 64 (4,000,003 rows
// of 118 groups: 24 us, 26 without).
// FEW: few enough counts for every workgroup to add them up for itself, which
// saves a launch.
template <bool FEW>
__global__ void __launch_bounds__(kThreads) k_group_place(const GroupArgs a) {
  __shared__ int s_at[kWaves][kMaxGroups + 1];  // next place of each group in each wavefront
  __shared__ int s_start[kMaxGroups + 1], s_local[kMaxGroups + 1];
  __shared__ int s_before[FEW ? kMaxGroups + 1 : 1];
  __shared__ int s_part[kWaves];
  __shared__ int s_sorted[kChunk];  // the chunk's rows by group: group << 16 | row
  static_assert(kMaxGroups < 1 << 15 && kChunk <= 1 << 16);
  const int G = a.n_groups, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t r0 = int64_t(blockIdx.x) * kChunk + w * 64 * kPerLane + lane;
  int key[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int64_t r = r0 + j * 64;
    key[j] = r < a.n_rows ? key_of(a.group, r, G) : -1;
  }
  for (int g = tid; g <= G; g += kThreads) {
    if (!FEW) s_start[g] = a.total[g];
    for (int j = 0; j < kWaves; ++j) s_at[j][g] = 0;
  }
  __syncthreads();
  uint64_t same[kPerLane];
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    same[j] = same_key(max(key[j], 0), a.bits, key[j] >= 0);
    count_same(s_at[w], key[j], same[j]);
  }
  if constexpr (FEW) {
    // a power of two of lanes for a group, all groups at once where they can
    // (171,895 rows of 85 groups: 29 us with 64 lanes, 16 with two)
    int log = 0;
    while (log < 6 && (G + 1) << (log + 1) <= kThreads) ++log;
    const int lanes = 1 << log, mine = tid & (lanes - 1);
    for (int g = tid >> log; g <= G; g += kThreads >> log) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int c = mine; c < a.n_chunks; c += lanes) {
        const int v = a.hist[int64_t(g) * a.n_chunks + c];
        all += v;
        before += c < int(blockIdx.x) ? v : 0;
      }
      for (int o = lanes >> 1; o; o >>= 1) {
        all += __shfl_xor(all, o);
        before += __shfl_xor(before, o);
      }
      if (mine == 0) {
        s_start[g] = all;
        s_before[g] = before;
      }
    }
    __syncthreads();
  }
  prefix(s_start, G + 1, s_part);
  if (blockIdx.x == 0) {
    for (int g = tid; g <= G; g += kThreads) a.offsets[g] = s_start[g];
    write_header(a);
  }
  // s_start: where the group's rows of this chunk go, less where they begin
  // in the sorted chunk, so that sorted row i of group g goes to s_start[g] + i
  int* s_count = s_local;
  for (int g = tid; g <= G; g += kThreads) {
    int n = 0;
    for (int j = 0; j < kWaves; ++j) n += s_at[j][g];
    s_count[g] = n;
  }
  __syncthreads();
  prefix(s_count, G + 1, s_part);
  for (int g = tid; g <= G; g += kThreads) {
    int at = s_count[g];
    s_start[g] += (FEW ? s_before[g] : a.hist[int64_t(g) * a.n_chunks + blockIdx.x]) - at;
    for (int j = 0; j < kWaves; ++j) {
      const int n = s_at[j][g];
      s_at[j][g] = at;
      at += n;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) {
    const int p = place_same(s_at[w], key[j], same[j]);
    if (key[j] >= 0) s_sorted[p] = key[j] << 16 | (w * 64 * kPerLane + j * 64 + lane);
  }
  __syncthreads();
  const int rows = int(min(int64_t(kChunk), a.n_rows - int64_t(blockIdx.x) * kChunk));
  for (int i = tid; i < rows; i += kThreads) {
    const int e = s_sorted[i];
    a.order[s_start[e >> 16] + i] = int(int64_t(blockIdx.x) * kChunk) + (e & 0xFFFF);
  }
}

// Everything in one workgroup, for few rows: one launch instead of three.
constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / 64;
constexpr int kSmallRows = 8192;
__global__ void __launch_bounds__(kSmallThreads) k_group_small(const GroupArgs a) {
  __shared__ int s_at[kSmallWaves][kMaxGroups + 1];
  __shared__ int s_start[kMaxGroups + 1];
  __shared__ int s_part[kSmallWaves];
  const int G = a.n_groups, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int g = tid; g <= G; g += kSmallThreads)
    for (int j = 0; j < kSmallWaves; ++j) s_at[j][g] = 0;
  __syncthreads();
  const int per = (a.n_rows + kSmallThreads - 1) / kSmallThreads;  // rows of a lane
  const int r0 = w * 64 * per + lane;
  for (int j = 0; j < per; ++j) {
    const int r = r0 + j * 64;
    if (r < a.n_rows) atomicAdd(&s_at[w][key_of(a.group, r, G)], 1);
  }
  __syncthreads();
  for (int g = tid; g <= G; g += kSmallThreads) {
    int n = 0;
    for (int j = 0; j < kSmallWaves; ++j) n += s_at[j][g];
    s_start[g] = n;
  }
  __syncthreads();
  prefix(s_start, G + 1, s_part);
  for (int g = tid; g <= G; g += kSmallThreads) {
    int at = s_start[g];
    a.offsets[g] = at;
    for (int j = 0; j < kSmallWaves; ++j) {
      const int n = s_at[j][g];
      s_at[j][g] = at;
      at += n;
    }
  }
  write_header(a);
  __syncthreads();
  for (int j = 0; j < per; ++j) {
    const int r = r0 + j * 64;
    const bool in = r < a.n_rows;
    const int key = in ? key_of(a.group, r, G) : 0;
    const int p = place_same(s_at[w], key, same_key(key, a.bits, in));
    if (in) a.order[p] = r;
  }
}

}  // namespace

GroupLayout group_layout(int64_t n_rows, int n_groups) {
  const auto up = [](int64_t n) { return (n + 15) / 16 * 16; };  // words of 64 bytes
  GroupLayout l;
  l.n_chunks = (n_rows + kChunk - 1) / kChunk;
  l.offsets = 16;
  l.order = l.offsets + up(n_groups + 1);
  l.total = l.order + up(n_rows);
  l.hist = l.total + up(n_groups + 1);
  l.words = l.hist + (n_rows > kSmallRows ? up(l.n_chunks * (n_groups + 1)) : 0);
  return l;
}

hipError_t launch_group_index(int n_rows, int n_groups, const int* group, int* index,
                              hipStream_t s) {
  const GroupLayout l = group_layout(n_rows, n_groups);
  GroupArgs a{};
  a.n_rows = n_rows;
  a.n_groups = n_groups;
  a.n_chunks = int(l.n_chunks);
  while ((n_groups >> a.bits) != 0) ++a.bits;
  a.group = group;
  a.index = index;
  a.offsets = index + l.offsets;
  a.order = index + l.order;
  a.total = index + l.total;
  a.hist = index + l.hist;
  if (n_rows <= kSmallRows) {
    hipLaunchKernelGGL(k_group_small, dim3(1), dim3(kSmallThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_group_count, dim3(unsigned(a.n_chunks)), dim3(kThreads), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (int64_t(a.n_chunks) * (n_groups + 1) <= kFewCounts) {
    hipLaunchKernelGGL((k_group_place<true>), dim3(unsigned(a.n_chunks)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(k_group_scan, dim3(unsigned(n_groups + 1)), dim3(kThreads), 0, s, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((k_group_place<false>), dim3(unsigned(a.n_chunks)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace e3k
