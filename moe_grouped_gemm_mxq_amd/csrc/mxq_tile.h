// What the tiled products share: 128-byte tile rows loaded straight into LDS,
// their swizzle, the waits around them, and the order of the output tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kXcds = 8;    // XCDs per MI355X; workgroups are dealt round robin
constexpr int kGroupM = 8;  // m-tiles per raster group

// LDS position of 16-byte chunk c of tile row r (8 chunks, 128 bytes per
// row).  A fragment read has its lanes on consecutive rows at one chunk; the
// XOR swizzle f(r) = (r & 7) ^ ((r >> 3) & 1) makes any 8 aligned consecutive
// rows land on 8 distinct 16-byte bank groups of a 128-byte bank row (32
// banks) and any 16 on 16 distinct groups of a 256-byte one (64 banks), so
// the read is conflict-free.
__device__ __forceinline__ int swz(int r, int c) {
  return r * 128 + ((c ^ ((r & 7) ^ ((r >> 3) & 1))) << 4);
}

// A direct load of a wave covers eight tile rows 8q .. 8q+7, 8 lanes a row.
// Lane l fills slot l % 8 of its row, which holds chunk slot ^ f(row); j & 1 = q & 1.
__device__ __forceinline__ int dma_chunk(int j, int lane) {
  return (lane & 7) ^ (lane >> 3) ^ (j & 1);
}

// Direct load of 16 (4) bytes a lane into LDS: lane l's go to `to` + 16 l (4 l); `to` is uniform.
__device__ __forceinline__ void load_lds16(const void* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds(from, (lds_ptr)to, 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const void* from, uint8_t* to) {
  __builtin_amdgcn_global_load_lds(from, (lds_ptr)to, 4, 0, 0);
}

// s_waitcnt with vmcnt(n) only (expcnt / lgkmcnt left at their maximum), gfx9 encoding
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(N >= 0 && N < 64, "vmcnt is 6 bits");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void wait_lgkmcnt0() { __builtin_amdgcn_s_waitcnt((15) | (3 << 14) | (0x7 << 4)); }

// Order of what follows a scheduling barrier: M matrix instructions, and between
// them, evenly, V vector instructions, D LDS reads and G global loads.
template <int M, int V, int D, int G, int m = 0>
__device__ __forceinline__ void interleave() {
  if constexpr (m < M) {
    constexpr int d = (m + 1) * D / M - m * D / M, g = (m + 1) * G / M - m * G / M, v = (m + 1) * V / M - m * V / M;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (d > 0) __builtin_amdgcn_sched_group_barrier(0x100, d, 0);
    if constexpr (g > 0) __builtin_amdgcn_sched_group_barrier(0x010, g, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    interleave<M, V, D, G, m + 1>();
  }
}

// Logical tile order: workgroups are dealt to the XCDs round robin, so remap
// blockIdx so that each XCD walks a contiguous run of the logical order (tiles
// that share operand panels then share that XCD's L2).
// (Used where every tile carries the same work; bid < n.)
__device__ __forceinline__ int xcd_remap(int bid, int n) {
  const int per = n / kXcds;
  const int x = bid % kXcds, i = bid / kXcds;
  if (i >= per) return bid;  // the last partial round stays in place
  return x * per + i;
}

// grouped raster: kGroupM m-tiles at a time, m fastest
__device__ __forceinline__ void raster(int t, int tiles_m, int tiles_n, int& mt, int& nt) {
  const int span = kGroupM * tiles_n;
  const int grp = t / span;
  const int first = grp * kGroupM;
  const int gm = min(kGroupM, tiles_m - first);
  const int r = t - grp * span;
  mt = first + r % gm;
  nt = r / gm;
}

}  // namespace mxq
