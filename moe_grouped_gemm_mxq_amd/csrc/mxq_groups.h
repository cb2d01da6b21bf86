// Per-workgroup table of ragged groups, built on the device from cumulative
// group ends (used by the grouped quantiser and the grouped GEMM schedulers).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

constexpr int kMaxGroups = 1024;

// start row and size of every group, and the exclusive prefix of
// ceil(size / unit) (bstart[G] = total units).  Group ends are clamped into
// [0, R] (R < 2^31), so a malformed array never sends an access out of
// bounds; a valid (non-decreasing, <= R) array is used unchanged.
struct GroupTable {
  int32_t start[kMaxGroups];
  int32_t size[kMaxGroups];
  int32_t bstart[kMaxGroups + 1];
};

// Clamped start row and size of group g (ends clamped into [0, R]; a group
// ending before it starts is empty).
__device__ __forceinline__ void group_span(const int32_t* __restrict__ group_end, int g, int64_t R,
                                           int32_t& start, int32_t& size) {
  int64_t e = group_end[g];
  int64_t b = g ? (int64_t)group_end[g - 1] : 0;
  e = e < 0 ? 0 : (e > R ? R : e);
  b = b < 0 ? 0 : (b > R ? R : b);
  start = (int32_t)b;
  size = e > b ? (int32_t)(e - b) : 0;
}

// All THREADS threads of the workgroup must call this; G <= 4 * THREADS.
// start / size may be null (only the block starts are written then).  With
// align > 1 a non-empty group's units start at the multiple of `align` at or
// below its first row: it counts ceil((size + start % align) / unit) units.
// The unit counts and their prefix sums are taken in 64 bits and the prefix
// saturates at INT32_MAX, so for any group_end array (even a malformed one)
// bstart is non-decreasing and bstart[g + 1] - bstart[g] never exceeds group
// g's own unit count: a position u in [bstart[g], bstart[g + 1]) always lies
// inside group g's clamped rows.
template <int THREADS>
__device__ void build_block_starts(const int32_t* __restrict__ group_end, int32_t G, int64_t R,
                                   int32_t unit, int32_t* start, int32_t* size, int32_t* bstart /* [G + 1] */,
                                   int64_t* scan_tmp /* [THREADS] */, int32_t align = 1) {
  static_assert(4 * THREADS >= kMaxGroups, "each thread owns at most four groups");
  const int t = threadIdx.x;
  int64_t local = 0;
  int64_t nb[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int g = t * 4 + j;
    nb[j] = 0;
    if (g < G) {
      int32_t b, m;
      group_span(group_end, g, R, b, m);
      if (start) start[g] = b;
      if (size) size[g] = m;
      nb[j] = m > 0 ? ((int64_t)m + b % align + unit - 1) / unit : 0;
      local += nb[j];
    }
  }
  // exclusive scan of `local` over the workgroup (Hillis-Steele in LDS)
  scan_tmp[t] = local;
  __syncthreads();
  for (int off = 1; off < THREADS; off <<= 1) {
    const int64_t v = t >= off ? scan_tmp[t - off] : 0;
    __syncthreads();
    scan_tmp[t] += v;
    __syncthreads();
  }
  constexpr int64_t kSat = 0x7FFFFFFF;
  int64_t run = scan_tmp[t] - local;
#pragma unroll
  for (int j = 0; j < 4; j++) {
    const int g = t * 4 + j;
    if (g < G) {
      bstart[g] = (int32_t)(run < kSat ? run : kSat);
      run += nb[j];
    }
  }
  if (t == THREADS - 1) bstart[G] = (int32_t)(scan_tmp[t] < kSat ? scan_tmp[t] : kSat);
  __syncthreads();
}

template <int THREADS>
__device__ void build_group_table(const int32_t* __restrict__ group_end, int32_t G, int64_t R,
                                  int32_t unit, GroupTable& gt, int64_t* scan_tmp /* [THREADS] */,
                                  int32_t align = 1) {
  build_block_starts<THREADS>(group_end, G, R, unit, gt.start, gt.size, gt.bstart, scan_tmp, align);
}

// largest g with bstart[g] <= u (u < bstart[G] assumed)
__device__ __forceinline__ int find_block_group(const int32_t* bstart, int G, int32_t u) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (bstart[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// largest g with bstart[g] <= u (u < bstart[G] assumed)
__device__ __forceinline__ int find_group(const GroupTable& gt, int G, int32_t u) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gt.bstart[mid] <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Where unit u of the ragged groups lies, when each group is cut into units of
// UNIT rows from its first one on.
struct GroupUnit {
  int g;                // its group
  int32_t start, size;  // the group's first row and rows (clamped as in group_span)
  int32_t local;        // the unit within the group
  int64_t before;       // units of the earlier groups
};
// All lanes of a wave call this with one u (no LDS, no barrier; a few hundred
// cycles for up to 64 groups).  False where u is past the last unit, with
// out.before all units.  A chunk of 64 groups holds fewer than 2^31 units for UNIT >= 64.
// SKIP: only the units past each group's first SKIP ones are counted (local counts all).
template <int UNIT, int SKIP = 0>
__device__ __forceinline__ bool find_group_unit(const int32_t* __restrict__ group_end, int G, int64_t R, int64_t u,
                                                GroupUnit& out) {
  static_assert(UNIT >= 64, "the sum of a chunk's units must fit int32");
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    int32_t start = 0, size = 0;
    if (g0 + lane < G) group_span(group_end, g0 + lane, R, start, size);
    const int32_t units = max((int32_t)(((uint32_t)size + (UNIT - 1)) / UNIT) - SKIP, 0);
    int32_t upto = units;  // units of the chunk's groups up to this lane's
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t v = __shfl_up(upto, off);
      if (lane >= off) upto += v;
    }
    const uint64_t has = __ballot(u < before + upto);
    if (has) {
      const int at = __builtin_ctzll(has);
      out.g = g0 + at;
      out.start = __builtin_amdgcn_readlane(start, at);
      out.size = __builtin_amdgcn_readlane(size, at);
      const int32_t earlier = __builtin_amdgcn_readlane(upto - units, at);
      out.before = before + earlier;
      out.local = (int32_t)(u - out.before) + SKIP;
      return true;
    }
    before += __builtin_amdgcn_readlane(upto, 63);
  }
  out.before = before;
  return false;
}

// All units of the groups, under the same conditions.
template <int UNIT>
__device__ __forceinline__ int64_t group_units(const int32_t* __restrict__ group_end, int G, int64_t R) {
  static_assert(UNIT >= 64, "the sum of a chunk's units must fit int32");
  int64_t sum = 0;
  for (int g0 = 0; g0 < G; g0 += 64) {
    int32_t start = 0, size = 0;
    if (g0 + (int)(threadIdx.x & 63) < G) group_span(group_end, g0 + (threadIdx.x & 63), R, start, size);
    int32_t units = (int32_t)(((uint32_t)size + (UNIT - 1)) / UNIT);
#pragma unroll
    for (int off = 32; off; off >>= 1) units += __shfl_xor(units, off);
    sum += __builtin_amdgcn_readfirstlane(units);
  }
  return sum;
}

}  // namespace mxq
