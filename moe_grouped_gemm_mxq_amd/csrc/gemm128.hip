// Products of FP8 (E4M3) operands with one fp32 scale for every block of 128
// along the reduction axis:
//   C[m][n] = sum over blocks b of sA[b][m] sB[b][n] P_b[m][n],
//   P_b[m][n] = sum over the block's k of A[m][k] B[n][k],
// A's blocks 1 x 128, B's 1 x 128 or 128 x 128 (weights).  Dense, ragged M (rows
// split into expert groups, group g times B[g]) and ragged K (one product per
// group over its padded columns).
//
// The scales are fp32, so the matrix instruction cannot apply them: each block's
// partial product starts from zero and is added to the tile's sums with one
// multiply-add an element (two where B's blocks are 1 x 128), which the vector
// units do while the matrix units work on the next block.
//
// Rounded to bf16, the partial products come from the FP8 matrix instruction,
// whose sums of eight products keep about 13 bits below the largest: off by at most
// 2^-10 of it, where the output's rounding is 2^-8 of the sum of all.  (Terms that
// cancel leave it the larger of the two; fp32 results avoid it.)  An fp32 output takes
// the codes as bf16 numbers (exact) through the bf16 instruction at half the rate: its
// products and sums are fp32's.
#include <type_traits>

#include "mxq_device.h"
#include "mxq_groups.h"
#include "mxq_host.h"
#include "mxq_internal.h"
#include "mxq_tile.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kB = 128;  // block, and the bytes of a tile row in a stage

enum Mode { kDense = 0, kRaggedM = 1, kRaggedK = 2 };

// Output tile of a workgroup: BM rows of A by BN rows of B, WAVES_M x WAVES_N
// waves, with STAGES stages in LDS.
template <int BM_, int BN_, int WAVES_M, int WAVES_N, int STAGES>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, kWavesM = WAVES_M, kStages = STAGES;
  static constexpr int kWaves = WAVES_M * WAVES_N, kThreads = 64 * kWaves;
  static constexpr int WM = BM / WAVES_M, WN = BN / WAVES_N;  // wave tile
  static constexpr int TM = WM / 16, TN = WN / 16;            // 16 x 16 blocks of a wave
  static constexpr int kLoadsA = BM / 8 / kWaves, kLoadsB = BN / 8 / kWaves;  // 1 KB loads of a wave and stage
  static constexpr int kLoads = kLoadsA + kLoadsB + 1;                        // with the scales'
  static constexpr int kCodesA = BM * kB, kCodesB = BN * kB;
  static constexpr int kStage = kCodesA + kCodesB + kWaves * 256;  // codes, then the block's scales of 64 rows a wave
  static_assert(BM / 64 + BN / 64 <= kWaves, "each wave loads the scales of at most 64 rows");
  static_assert(STAGES >= 2 && STAGES <= 4, "the stages are spelled out");
  static_assert(kLoadsA % 2 == 0 && kLoadsB % 2 == 0, "a load's parity is its place's");
};

struct Problem {
  const uint8_t* A;
  const float* sA;
  const uint8_t* B;
  const float* sB;
  void* C;
  int64_t M, N, K, ldc;
  const int32_t* group_end;
  int G;
  int tiles_m, tiles_n;
  int whole_groups;  // ragged K: an XCD takes whole groups
};

// What a workgroup computes; uniform.
struct Tile {
  int64_t m0, n0;
  int rows, cols;           // valid ones of the tile
  int64_t kb0;              // first block of the reduction
  int nkb;                  // its blocks; 0: zeros
  const uint8_t* B;         // codes and scales of the tile's expert
  const float* sB;
  int64_t c0;               // first element of its matrix in C
};

// Groups of a ragged-K product, largest first where one wave can rank them.
__device__ __forceinline__ void ragged_k_group(const int32_t* group_end, int G, int64_t K, int rank, int& g, int64_t& before,
                                               int& blocks) {
  const int lane = threadIdx.x & 63;
  if (G <= 64) {
    int32_t start = 0, size = -1;
    if (lane < G) group_span(group_end, lane, K, start, size);
    int place = 0;
    for (int h = 0; h < G; h++) {
      const int32_t other = __builtin_amdgcn_readlane(size, h);
      place += other > size || (other == size && h < lane);
    }
    const int32_t units = lane < G ? (int32_t)(((uint32_t)size + (kB - 1)) / kB) : 0;
    int32_t upto = units;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t v = __shfl_up(upto, off);
      if (lane >= off) upto += v;
    }
    g = __builtin_ctzll(__ballot(lane < G && place == rank));
    blocks = __builtin_amdgcn_readlane(units, g);
    before = __builtin_amdgcn_readlane(upto - units, g);
    return;
  }
  g = rank;
  int64_t sum = 0;
  for (int g0 = 0; g0 < g; g0 += 64) {
    int32_t start = 0, size = 0;
    if (g0 + lane < g) group_span(group_end, g0 + lane, K, start, size);
    int32_t units = (int32_t)(((uint32_t)size + (kB - 1)) / kB);
#pragma unroll
    for (int off = 32; off; off >>= 1) units += __shfl_xor(units, off);
    sum += units;
  }
  int32_t start, size;
  group_span(group_end, g, K, start, size);
  before = sum;
  blocks = __builtin_amdgcn_readfirstlane((int32_t)(((uint32_t)size + (kB - 1)) / kB));
}

// The tile of workgroup `bid`; false where there is none.
template <int MODE, class S, bool TILE128>
__device__ __forceinline__ bool find_tile(const Problem& p, int bid, Tile& t) {
  const int64_t Kb = p.K / kB;
  const int64_t scales_n = TILE128 ? (p.N + kB - 1) / kB : p.N;
  t.kb0 = 0;
  t.nkb = (int)Kb;
  t.B = p.B;
  t.sB = p.sB;
  t.c0 = 0;
  int mt, nt;
  int64_t rows;
  if constexpr (MODE == kDense) {
    raster(xcd_remap(bid, p.tiles_m * p.tiles_n), p.tiles_m, p.tiles_n, mt, nt);
    t.m0 = (int64_t)mt * S::BM;
    rows = p.M - t.m0;
  } else if constexpr (MODE == kRaggedM) {
    // (the launch has workgroups for the most tiles that any groups could have; the XCDs share the real ones)
    const int tiles_m = (int)min((int64_t)p.tiles_m, group_units<S::BM>(p.group_end, p.G, p.M));
    if (bid >= tiles_m * p.tiles_n) return false;
    raster(xcd_remap(bid, tiles_m * p.tiles_n), tiles_m, p.tiles_n, mt, nt);
    GroupUnit u;
    if (!find_group_unit<S::BM>(p.group_end, p.G, p.M, mt, u)) return false;
    t.m0 = u.start + (int64_t)u.local * S::BM;
    rows = u.size - (int64_t)u.local * S::BM;
    t.B = p.B + (int64_t)u.g * p.N * p.K;
    t.sB = p.sB + (int64_t)u.g * Kb * scales_n;
  } else {
    const int per = p.tiles_m * p.tiles_n;
    int rank, tile;
    if (p.whole_groups) {
      const int x = bid % kXcds, i = bid / kXcds, round = i / per;
      rank = round * kXcds + ((round & 1) ? kXcds - 1 - x : x);
      tile = i - round * per;
      if (rank >= p.G) return false;
    } else {
      rank = bid / per;
      tile = xcd_remap(bid - rank * per, per);
    }
    int g, blocks;
    int64_t before;
    ragged_k_group(p.group_end, p.G, p.K, rank, g, before, blocks);
    t.kb0 = min(before, Kb);
    t.nkb = (int)min((int64_t)blocks, Kb - t.kb0);
    t.c0 = (int64_t)g * p.M * p.N;
    raster(tile, p.tiles_m, p.tiles_n, mt, nt);
    t.m0 = (int64_t)mt * S::BM;
    rows = p.M - t.m0;
  }
  t.n0 = (int64_t)nt * S::BN;
  t.rows = (int)min<int64_t>(rows, S::BM);
  t.cols = (int)min<int64_t>(p.N - t.n0, S::BN);
  return true;
}

// 32 code bytes of a lane: of tile row r0 + lane % 16, the block's bytes 32g ..
// 32g + 31 (g = lane / 16).  Both operands map bytes to the instruction's k alike,
// which is all that a sum over the block asks for.
__device__ __forceinline__ v8i load_frag(const uint8_t* codes, int r0, int lane) {
  const int r = r0 + (lane & 15), c = 2 * (lane >> 4);
  const uint4 lo = *reinterpret_cast<const uint4*>(codes + swz(r, c));
  const uint4 hi = *reinterpret_cast<const uint4*>(codes + swz(r, c + 1));
  v8i f;
  f[0] = (int)lo.x; f[1] = (int)lo.y; f[2] = (int)lo.z; f[3] = (int)lo.w;
  f[4] = (int)hi.x; f[5] = (int)hi.y; f[6] = (int)hi.z; f[7] = (int)hi.w;
  return f;
}

struct AsBf16 {
  v8bf f[4];
};
// the same 32 codes as bf16 numbers (exact), eight for each of four instructions
__device__ __forceinline__ AsBf16 widen(const v8i& c) {
  AsBf16 w;
#pragma unroll
  for (int s = 0; s < 4; s++) {
    const v2bf16 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * s], 1.f, false);
    const v2bf16 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * s], 1.f, true);
    const v2bf16 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * s + 1], 1.f, false);
    const v2bf16 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * s + 1], 1.f, true);
    w.f[s] = v8bf{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
  }
  return w;
}

template <bool F32>
struct FragOf {
  typedef v8i type;
  static __device__ __forceinline__ v8i of(const v8i& c) { return c; }
};
template <>
struct FragOf<true> {
  typedef AsBf16 type;
  static __device__ __forceinline__ AsBf16 of(const v8i& c) { return widen(c); }
};

// partial product of a block: rows of n by columns (lanes) of m
__device__ __forceinline__ v4f block_product(const v8i& n, const v8i& m) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(n, m, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ v4f block_product(const AsBf16& n, const AsBf16& m) {
  v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; s++) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n.f[s], m.f[s], d, 0, 0, 0);
  return d;
}

// of TM blocks of m
template <int TM>
__device__ __forceinline__ void block_products(const v8i& n, const v8i (&m)[TM], v4f (&d)[TM]) {
#pragma unroll
  for (int j = 0; j < TM; j++) d[j] = block_product(n, m[j]);
}
template <int TM>
__device__ __forceinline__ void block_products(const AsBf16& n, const AsBf16 (&m)[TM], v4f (&d)[TM]) {
#pragma unroll
  for (int j = 0; j < TM; j++) d[j] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < 4; s++)
#pragma unroll
    for (int j = 0; j < TM; j++) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(n.f[s], m[j].f[s], d[j], 0, 0, 0);
}

__device__ __forceinline__ void store4(float* p, const v4f& v) { *reinterpret_cast<v4f*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, const v4f& v) {
  u32x2 w;
  w[0] = bf16x2_of(v[0], v[1]);
  w[1] = bf16x2_of(v[2], v[3]);
  *reinterpret_cast<u32x2*>(p) = w;
}

// One stage is one block of 128 along K: codes and scales of the tile's rows,
// loaded straight into LDS kStages - 1 stages ahead.  The stages are separate
// arrays so that the compiler can tell the one being read from those being filled.
//
// What bounds it.  bf16 C: 8192 x 18432 x 7168 takes 0.90-0.94 ms, 2300-2400 TFLOP/s (0.6 of the FP8 peak at the clock it
// runs at), where a stage of a 256 x 256 tile costs 0.9 us of matrix instructions, 0.8-1.1 us of loads (64 KB a CU from
// L2), and 1.55 us together; 131072 rows through 32 experts (7168 to 4096) 3.5-3.65 ms.  fp32 C: the vector units, which
// widen the codes (two an instruction) and apply two scales an element, have an instruction to issue in 70% of the cycles,
// the matrix units are busy in half: weight gradients of 32 experts, 131072 tokens, 7.7-7.9 ms, 1000 TFLOP/s.
template <int MODE, bool F32, bool TILE128, class S>
__global__ __launch_bounds__(S::kThreads, 2) void gemm128_kernel(Problem p) {
  typedef std::conditional_t<F32, float, uint16_t> Out;
  constexpr int TM = S::TM, TN = S::TN, NS = S::kStages;
  __shared__ __attribute__((aligned(1024))) uint8_t stage0[S::kStage], stage1[S::kStage], stage2[NS > 2 ? S::kStage : 16],
      stage3[NS > 3 ? S::kStage : 16];
  uint8_t* const stages[4] = {stage0, stage1, stage2, stage3};
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % S::kWavesM, wn = wave / S::kWavesM;
  Tile t;
  if (!find_tile<MODE, S, TILE128>(p, blockIdx.x, t)) return;

  // per-lane offsets of this wave's loads: rows past the tile read its last row
  uint32_t offA[S::kLoadsA], offB[S::kLoadsB];
#pragma unroll
  for (int j = 0; j < S::kLoadsA; j++)
    offA[j] = (uint32_t)min((wave * S::kLoadsA + j) * 8 + (lane >> 3), t.rows - 1) * (uint32_t)p.K + dma_chunk(j, lane) * 16;
#pragma unroll
  for (int j = 0; j < S::kLoadsB; j++)
    offB[j] = (uint32_t)min((wave * S::kLoadsB + j) * 8 + (lane >> 3), t.cols - 1) * (uint32_t)p.K + dma_chunk(j, lane) * 16;
  const uint8_t* const baseA = p.A + t.m0 * p.K + t.kb0 * kB;
  const uint8_t* const baseB = t.B + t.n0 * p.K + t.kb0 * kB;
  // scales: wave w those of the 64 tile rows from 64 w on, A's rows before B's (past the last: of B's last row)
  const bool of_a = wave < S::BM / 64;
  const int srow = (of_a ? wave : wave - S::BM / 64) * 64 + lane;
  const int64_t scales_n = TILE128 ? (p.N + kB - 1) / kB : p.N;
  const int64_t spitch = of_a ? p.M : scales_n;
  const int64_t sn = t.n0 + min(srow, t.cols - 1);
  const float* sp = (of_a ? p.sA + t.m0 + min(srow, t.rows - 1) : t.sB + (TILE128 ? sn / kB : sn)) + t.kb0 * spitch;

  // load n of a stage: A's codes, B's, and the scales (every wave has as many in flight)
  auto load = [&](uint8_t* st, int s, int n) {
    if (n < S::kLoadsA) {
      load_lds16(baseA + (int64_t)s * kB + offA[n], st + (wave * S::kLoadsA + n) * 1024);
    } else if (n < S::kLoadsA + S::kLoadsB) {
      load_lds16(baseB + (int64_t)s * kB + offB[n - S::kLoadsA], st + S::kCodesA + (wave * S::kLoadsB + n - S::kLoadsA) * 1024);
    } else {
      load_lds4(sp + s * spitch, st + S::kCodesA + S::kCodesB + wave * 256);
    }
  };
  auto meet = [&]() {
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  v4f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; i++)
#pragma unroll
    for (int j = 0; j < TM; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

  typedef FragOf<F32> Frag;
  // loads of each of the wave's TN row blocks of B, so that all are out by about half of the stage
  constexpr int kPer = (S::kLoads + TN / 2) / TN + 1;
  // Stage s, which is in st, while stage s + NS - 1 is loaded to next (past the last
  // one, the last again: every stage has the same loads in flight, and no branch
  // parts them from the matrix instructions).
  auto stage = [&](const uint8_t* st, uint8_t* next, int s) {
    const int ahead_s = min(s + NS - 1, t.nkb - 1);
    const float* sa_of = reinterpret_cast<const float*>(st + S::kCodesA + S::kCodesB) + wm * S::WM;
    const float* sb_of = reinterpret_cast<const float*>(st + S::kCodesA + S::kCodesB) + S::BM + wn * S::WN;
    typename Frag::type fm[TM];
    float f[TM];
#pragma unroll
    for (int j = 0; j < TM; j++) {
      fm[j] = Frag::of(load_frag(st, wm * S::WM + j * 16, lane));
      f[j] = sa_of[j * 16 + (lane & 15)];
      if constexpr (TILE128) f[j] *= sb_of[0];
    }
    // While block i's matrix instructions run, the sums of block i - 1 are taken and
    // the codes of block i + 1 widened, whose reads went out a block earlier.
    v4f d[2][TM], sb[2];
    typename Frag::type fn = Frag::of(load_frag(st + S::kCodesA, wn * S::WN, lane));
    v8i ahead = load_frag(st + S::kCodesA, wn * S::WN + (TN > 1 ? 16 : 0), lane);
    auto add = [&](int i) {
#pragma unroll
      for (int j = 0; j < TM; j++) {
        v4f v = d[i & 1][j];
        if constexpr (!TILE128) v *= sb[i & 1];
#pragma unroll
        for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(v[e], f[j], acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));  // here, not after the stage's last instruction
      }
    };
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < TN; i++) {
      if constexpr (!TILE128) sb[i & 1] = *reinterpret_cast<const v4f*>(sb_of + i * 16 + 4 * (lane >> 4));
      const v8i raw = ahead;
      if (i + 2 < TN) ahead = load_frag(st + S::kCodesA, wn * S::WN + (i + 2) * 16, lane);
      block_products(fn, fm, d[i & 1]);
      // the loads a few at a time: a wave that issues all of them at once waits for
      // the queue, and its matrix instructions with it
#pragma unroll
      for (int n = i * kPer; n < (i + 1) * kPer && n < S::kLoads; n++) load(next, ahead_s, n);
      if (i > 0) add(i - 1);
      if (i + 1 < TN) fn = Frag::of(raw);
      // one matrix instruction, then its share of the others: two waves that meet in
      // the same phase would otherwise wait for one another in both
      interleave<TM * (F32 ? 4 : 1), TM * (TILE128 ? 4 : 8) + (F32 ? 16 : 0), 2, kPer>();
      __builtin_amdgcn_sched_barrier(0);
    }
    add(TN - 1);
    wait_vmcnt<(NS - 2) * S::kLoads>();  // the next stage has landed
    wait_lgkmcnt0();
    meet();
  };
  if (t.nkb > 0) {
#pragma unroll
    for (int s = 0; s < NS - 1; s++)
#pragma unroll
      for (int n = 0; n < S::kLoads; n++) load(stages[s], min(s, t.nkb - 1), n);
    wait_vmcnt<(NS - 2) * S::kLoads>();
    meet();
    // (left from within: a way round the loop after fewer than NS stages would have
    // the compiler wait for loads that such a way would leave in flight)
    auto all_stages = [&]() {
      for (int s0 = 0;; s0 += NS) {
#pragma unroll
        for (int u = 0; u < NS; u++) {
          stage(stages[u], stages[(u + NS - 1) % NS], s0 + u);
          if (s0 + u + 1 >= t.nkb) return;
        }
      }
    };
    all_stages();
    wait_vmcnt<0>();  // the LDS is used again below
    meet();
  }

  // Lane l holds C[m = l % 16][n = 4 (l / 16) .. + 3] of each 16 x 16 block.  The
  // tile goes through LDS, every wave by itself, so that it is stored in whole lines
  // (eight columns a lane, their 16 bytes by the row's last bits).
  constexpr int WN = S::WN, kEights = WN / 8;
  constexpr int kMine = S::WM * WN * (int)sizeof(Out), kPerStage = S::kStage / kMine;
  static_assert(2 * kPerStage >= S::kWaves, "two stages hold every wave's tile");
  Out* const mine = reinterpret_cast<Out*>((wave < kPerStage ? stage0 : stage1) + wave % kPerStage * kMine);
  auto spot = [&](int m, int n) { return m * WN + (((n >> 3) ^ (m & (kEights - 1) & 7)) << 3) + (n & 7); };
#pragma unroll
  for (int j = 0; j < TM; j++)
#pragma unroll
    for (int i = 0; i < TN; i++) store4(mine + spot(j * 16 + (lane & 15), i * 16 + 4 * (lane >> 4)), acc[i][j]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  Out* C = static_cast<Out*>(p.C) + t.c0 + t.m0 * p.ldc + t.n0;
  // past the caches where the lines are whole (dense 903 -> 897 us), not where rows share them (17.4 -> 19.9 us, N = 1237)
  const bool whole_lines = (((uintptr_t)p.C | (uintptr_t)(p.ldc * sizeof(Out))) & 127) == 0;
#pragma unroll
  for (int r = 0; r < S::WM; r += 64 / kEights) {
    const int ml = r + lane / kEights, nl = lane % kEights * 8;
    const int m = wm * S::WM + ml, n = wn * WN + nl;
    if (m >= t.rows) continue;
    Out* to = C + (int64_t)m * p.ldc + n;
    const Out* from = mine + spot(ml, nl);
    if (n + 8 <= t.cols) {
#pragma unroll
      for (int k = 0; k < (int)sizeof(Out) / 2; k++) {
        const u32x4 v = *(reinterpret_cast<const u32x4*>(from) + k);
        if (whole_lines)
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(to) + k);
        else
          *(reinterpret_cast<u32x4_any*>(to) + k) = v;
      }
    } else {
      for (int e = 0; e < t.cols - n; e++) to[e] = from[e];
    }
  }
}

// Few rows of A (decoding): B is read once, straight into the lanes' registers,
// and the waves of a workgroup take different blocks of K of the same 16 NB rows
// of B by 16 MB rows of A; their sums are added through LDS in the order of
// the waves.  A comes from L2.  Bound by B's bytes: many waves with a block each in
// flight read them faster than few with several (measured 33 us against 38 for
// 132 MB, where reading alone takes 25), so registers are kept few.  Of the
// scales, lane (row, part) loads those of its row and of the part-th of the next
// kU blocks, and the lanes of the other parts get them from it.
//
// A workgroup takes at most 64 rows of a group, sixteen (MB of them) after another
// with B's rows from L2; longer groups have more workgroups (128 groups of 512 x
// 2048, 512 rows: all in one group 102 us with one workgroup for all of its rows,
// 16 so).
constexpr int kU = 4;
constexpr int kFewRows = 64;

// a lane's 32 bytes of a block: 16 of either half, so that a load covers 64 bytes of each row
__device__ __forceinline__ v8i load_lane32(const uint8_t* p) {
  const u32x4 lo = *reinterpret_cast<const u32x4*>(p), hi = *reinterpret_cast<const u32x4*>(p + 64);
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

template <int MODE, bool F32, bool TILE128, int MB, int NB, int W, int OCC>
__global__ __launch_bounds__(64 * W, OCC) void few_rows_kernel(Problem p) {
  typedef std::conditional_t<F32, float, uint16_t> Out;
  __shared__ float sums[W][NB * MB][256];
  const int lane = threadIdx.x & 63, in = lane & 15, part = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int Kb = (int)(p.K / kB);
  const int64_t scales_n = TILE128 ? (p.N + kB - 1) / kB : p.N;
  int64_t m_first = 0;
  int m_rows = (int)p.M;  // at most kFewRows
  const uint8_t* B = p.B;
  const float* sB = p.sB;
  int nt = blockIdx.x;
  if constexpr (MODE == kRaggedM) {
    // the groups' rows past their first kFewRows, then a workgroup for each group's first ones, which need no search
    const int unit = blockIdx.x / p.tiles_n, more = (int)(p.M / kFewRows);
    nt = blockIdx.x - unit * p.tiles_n;
    GroupUnit u;
    if (unit < more) {
      if (!find_group_unit<kFewRows, 1>(p.group_end, p.G, p.M, unit, u)) return;
    } else {
      u.g = unit - more;
      u.local = 0;
      group_span(p.group_end, u.g, p.M, u.start, u.size);
      if (u.size == 0) return;
    }
    m_first = u.start + (int64_t)u.local * kFewRows;
    m_rows = min(u.size - u.local * kFewRows, kFewRows);
    B += (int64_t)u.g * p.N * p.K;
    sB += (int64_t)u.g * Kb * scales_n;
  }
  const int64_t n0 = (int64_t)nt * (16 * NB);
  const uint8_t* b_row[NB];
  const float* sb_row[NB];
#pragma unroll
  for (int i = 0; i < NB; i++) {
    b_row[i] = B + min(n0 + 16 * i + in, p.N - 1) * p.K + 16 * part;
    sb_row[i] = sB + (TILE128 ? min(n0 + 16 * i, p.N - 1) / kB : min(n0 + 16 * i + in, p.N - 1));
  }

  for (int m0 = 0; m0 < m_rows; m0 += 16 * MB) {
    const uint8_t* a_row[MB];
    const float* sa_row[MB];
#pragma unroll
    for (int j = 0; j < MB; j++) {
      const int64_t m = m_first + min(m0 + 16 * j + in, m_rows - 1);
      a_row[j] = p.A + m * p.K + 16 * part;
      sa_row[j] = p.sA + m;
    }
    v4f acc[NB][MB];
#pragma unroll
    for (int i = 0; i < NB; i++)
#pragma unroll
      for (int j = 0; j < MB; j++) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave; k0 < Kb; k0 += W * kU) {
      const int64_t ks = min(k0 + part * W, Kb - 1);
      float sa[MB], sb[NB];
#pragma unroll
      for (int j = 0; j < MB; j++) sa[j] = sa_row[j][ks * p.M];
#pragma unroll
      for (int i = 0; i < NB; i++) sb[i] = sb_row[i][ks * scales_n];
#pragma unroll
      for (int u = 0; u < kU; u++) {
        const int64_t k = k0 + u * W;
        if (k >= Kb) break;
        v8i b[NB], a[MB];
#pragma unroll
        for (int i = 0; i < NB; i++) b[i] = load_lane32(b_row[i] + k * kB);
#pragma unroll
        for (int j = 0; j < MB; j++) a[j] = load_lane32(a_row[j] + k * kB);
        typename FragOf<F32>::type fm[MB];
#pragma unroll
        for (int j = 0; j < MB; j++) fm[j] = FragOf<F32>::of(a[j]);
#pragma unroll
        for (int i = 0; i < NB; i++) {
          const typename FragOf<F32>::type fn = FragOf<F32>::of(b[i]);
          v4f sbn;  // of the lane's four rows of B
          if constexpr (!TILE128) {
#pragma unroll
            for (int e = 0; e < 4; e++) sbn[e] = __shfl(sb[i], 16 * u + 4 * part + e);
          }
#pragma unroll
          for (int j = 0; j < MB; j++) {
            v4f d = block_product(fn, fm[j]);
            float f;
            if constexpr (TILE128) {
              f = __shfl(sa[j] * sb[i], 16 * u + in);
            } else {
              f = __shfl(sa[j], 16 * u + in);
              d *= sbn;
            }
#pragma unroll
            for (int e = 0; e < 4; e++) acc[i][j][e] = __builtin_fmaf(d[e], f, acc[i][j][e]);
          }
        }
      }
    }
    // [m][n] of each 16 x 16 block
#pragma unroll
    for (int i = 0; i < NB; i++)
#pragma unroll
      for (int j = 0; j < MB; j++) *reinterpret_cast<v4f*>(&sums[wave][i * MB + j][in * 16 + 4 * part]) = acc[i][j];
    __syncthreads();
    for (int at = threadIdx.x; at < NB * MB * 256; at += 64 * W) {
      const int ij = at >> 8, r = at & 255;
      float v = sums[0][ij][r];
#pragma unroll
      for (int w = 1; w < W; w++) v += sums[w][ij][r];
      const int m = m0 + 16 * (ij % MB) + (r >> 4);
      const int64_t n = n0 + 16 * (ij / MB) + (r & 15);
      if (m < m_rows && n < p.N) store_f(static_cast<Out*>(p.C), (m_first + m) * p.ldc + n, v);
    }
    if (m0 + 16 * MB < m_rows) __syncthreads();
  }
}

// Large reads the fewest bytes a product, and its registers leave room for a single factor an element; of the smaller tiles
// two are on a CU, or one with its loads three stages ahead.
typedef Shape<256, 256, 4, 2, 2> Large;
typedef Shape<128, 128, 2, 2, 2> Medium;
typedef Shape<128, 128, 2, 4, 4> Deep;
typedef Shape<64, 64, 2, 2, 4> Small;

template <int MODE, bool F32, bool TILE128, class S>
hipError_t launch_shape(Problem p, hipStream_t st) {
  p.tiles_n = (int)((p.N + S::BN - 1) / S::BN);
  const int64_t tm = (p.M + S::BM - 1) / S::BM + (MODE == kRaggedM ? p.G : 0);
  // Groups of few tiles: one XCD's L2 reads their operands once, where there are groups enough for the XCDs to share them
  // out (bf16 C, sizes even / by Zipf's law: 32 groups of 2048 rows, 512 x 1024, 55.2 / 115 us against 65.2 / 129; 128 of
  // 256 x 512 16.9 / 31 against 22.4 / 37; but 16 of 511 x 1237 17.6 / 20.7 against 19.2 / 18.2).
  p.whole_groups = MODE == kRaggedK && p.G >= 4 * kXcds && tm * p.tiles_n <= 64;
  const int64_t groups = p.whole_groups ? (p.G + kXcds - 1) / kXcds * kXcds : p.G;
  const int64_t total = tm * p.tiles_n * (MODE == kRaggedK ? groups : 1);
  if (total > INT32_MAX) return hipErrorInvalidValue;
  p.tiles_m = (int)tm;
  gemm128_kernel<MODE, F32, TILE128, S><<<(unsigned)total, S::kThreads, 0, st>>>(p);
  return hipGetLastError();
}

template <int MODE, bool F32, bool TILE128, int MB, int NB, int W, int OCC>
hipError_t launch_few(Problem p, hipStream_t st) {
  const int64_t units = MODE == kRaggedM ? p.G + p.M / kFewRows : 1;
  const int64_t tiles = (p.N + 16 * NB - 1) / (16 * NB), total = tiles * units;
  if (total > INT32_MAX) return hipErrorInvalidValue;
  p.tiles_n = (int)tiles;
  few_rows_kernel<MODE, F32, TILE128, MB, NB, W, OCC><<<(unsigned)total, 64 * W, 0, st>>>(p);
  return hipGetLastError();
}

// A launch has fewer than 2^32 threads, and few rows take 16 for each row of B, a quarter more where groups are uneven.
constexpr int64_t kMaxFewN = 1 << 27;

// Waves a workgroup, and rows of B in it, from what they measured (us; bf16 C, N x K = 4096 x 7168 / 18432 x 7168 / 32
// experts of 4096 x 7168 with 64 rows): 16 rows of B by 16 waves 8.2 / 33.4 / 102, 32 by 8 waves 11.4 / 35.2 / 97.
template <int MODE, bool F32, bool TILE128>
hipError_t launch_few_of(const Problem& p, int64_t rows, hipStream_t st) {
  const bool many = (p.N + 31) / 32 * (MODE == kRaggedM ? p.G : 1) >= 4 * (int64_t)device_cu_count();
  if (rows <= 16) {
    if (many) return launch_few<MODE, F32, TILE128, 1, 2, 8, 4>(p, st);
    return launch_few<MODE, F32, TILE128, 1, 1, 16, 8>(p, st);
  }
  if (rows <= 32) {
    if (many) return launch_few<MODE, F32, TILE128, 2, 2, 8, 4>(p, st);
    return launch_few<MODE, F32, TILE128, 2, 1, 8, 4>(p, st);
  }
  return launch_few<MODE, F32, TILE128, 4, 1, 8, 4>(p, st);
}

// tiles of side `side`
int64_t tiles_of(const Problem& p, int mode, int64_t side) {
  return (p.M + side - 1) / side * ((p.N + side - 1) / side) * (mode == kRaggedK ? p.G : 1);
}

// Measured (us; N x K = 4096 x 7168, rows 256 / 512 / 1024 / 1536 / 2048 / 4096): bf16 C: Small 26 / 35 / 62 / 82 / 116 / 225,
// Deep 40 / 40 / 44 / 76 / 80 / 156, Medium 58 / 57 / 58 / 62 / 67 / 133, Large 92 / 91 / 90 / 89 / 90 / 106; fp32 C (256 / 512
// / 1024 / 2048): Small 35 / 46 / 83 / 157, Deep 62 / 63 / 71 / 131, Medium 72 / 72 / 74 / 111.  So: Small while all of its tiles
// are in work at once (two a CU), Deep while it is alone on a CU, Large where it fills three quarters of them.  What
// bounds these sizes: one workgroup's stages follow one another (56 of Small's at 0.45 us), and K is not split.
template <int MODE, bool F32, bool TILE128>
hipError_t launch_tiles(const Problem& p, hipStream_t st) {
  const int64_t cus = device_cu_count();
  if (tiles_of(p, MODE, 64) <= 2 * cus) return launch_shape<MODE, F32, TILE128, Small>(p, st);
  if (tiles_of(p, MODE, 128) <= cus) return launch_shape<MODE, F32, TILE128, Deep>(p, st);
  if constexpr (!F32 && TILE128)
    if (4 * tiles_of(p, MODE, 256) >= 3 * cus) return launch_shape<MODE, F32, TILE128, Large>(p, st);
  return launch_shape<MODE, F32, TILE128, Medium>(p, st);
}

template <int MODE, bool TILE128>
hipError_t launch_gemm128(const Problem& p, bool f32, hipStream_t st) {
  if constexpr (MODE != kRaggedK) {
    // Rows of A, or of a larger group.  B is read again for every 64 (or 16, 32) rows; with
    // more, and with more than 16 where N alone fills the card, tiles are faster (N = 18432,
    // 64 rows: 44 us against 84; N = 4096: 26 against 20).
    const int64_t rows = MODE == kRaggedM ? 4 * p.M / p.G : p.M;
    const bool few = rows <= 16 || (rows <= 64 && p.N <= 32 * (int64_t)device_cu_count());
    if (few && p.N * p.G < kMaxFewN)
      return f32 ? launch_few_of<MODE, true, TILE128>(p, rows, st) : launch_few_of<MODE, false, TILE128>(p, rows, st);
  }
  return f32 ? launch_tiles<MODE, true, TILE128>(p, st) : launch_tiles<MODE, false, TILE128>(p, st);
}

mxq_status check(const char* who, const Problem& p, mxq_dtype cdt) {
  MXQ_REQUIRE(cdt == MXQ_DT_F32 || cdt == MXQ_DT_BF16, "%s: unknown output type %d", who, (int)cdt);
  MXQ_REQUIRE(p.M >= 0 && p.M <= INT32_MAX && p.N >= 1 && p.N <= INT32_MAX, "%s: M must be in [0, 2^31), N in [1, 2^31)", who);
  MXQ_REQUIRE(p.K >= kB && p.K % kB == 0, "%s: K must be a positive multiple of 128 (got %lld)", who, (long long)p.K);
  MXQ_REQUIRE(p.K < MXQ_GEMM_MAX_ROW_BYTES, "%s: K = %lld gives code rows of MXQ_GEMM_MAX_ROW_BYTES or more", who, (long long)p.K);
  MXQ_REQUIRE(p.ldc >= p.N, "%s: ldc < N", who);
  if (p.M == 0) return MXQ_OK;
  MXQ_REQUIRE(p.A && p.sA && p.B && p.sB && p.C, "%s: NULL operand", who);
  MXQ_REQUIRE(aligned_to(p.A, 16) && aligned_to(p.B, 16), "%s: A, B must be 16-byte aligned", who);
  MXQ_REQUIRE(aligned_to(p.sA, 4) && aligned_to(p.sB, 4), "%s: sA, sB must be 4-byte aligned", who);
  MXQ_REQUIRE(aligned_to(p.C, cdt == MXQ_DT_F32 ? 4 : 2), "%s: C must be aligned to its elements", who);
  return MXQ_OK;
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

mxq_status mxq_gemm128(const uint8_t* A, const float* sA, const uint8_t* B, const float* sB, int b_tile, void* C,
                       mxq_dtype cdt, int64_t M, int64_t N, int64_t K, int64_t ldc, hipStream_t st) {
  const Problem p{A, sA, B, sB, C, M, N, K, ldc, nullptr, 1, 0, 0, 0};
  MXQ_REQUIRE(b_tile == 1 || b_tile == 128, "mxq_gemm128: b_tile must be 1 or 128 (got %d)", b_tile);
  const mxq_status s = check("mxq_gemm128", p, cdt);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE_DEVICE();
  if (M == 0) return ok();
  const bool f32 = cdt == MXQ_DT_F32;
  return launched(b_tile == 128 ? launch_gemm128<kDense, true>(p, f32, st) : launch_gemm128<kDense, false>(p, f32, st),
                  "mxq_gemm128");
}

mxq_status mxq_grouped_gemm128(mxq_gg_mode mode, const uint8_t* A, const float* sA, const uint8_t* B, const float* sB,
                               void* C, mxq_dtype cdt, int64_t M, int64_t N, int64_t K, const int32_t* group_end,
                               int32_t G, hipStream_t st) {
  const Problem p{A, sA, B, sB, C, M, N, K, N, group_end, G, 0, 0, 0};
  MXQ_REQUIRE(mode == MXQ_GG_RAGGED_M || mode == MXQ_GG_RAGGED_K, "mxq_grouped_gemm128: bad mode");
  MXQ_REQUIRE(G >= 1 && G <= MXQ_MAX_GROUPS, "mxq_grouped_gemm128: G must be in [1, %d] (got %d)", MXQ_MAX_GROUPS, G);
  const mxq_status s = check("mxq_grouped_gemm128", p, cdt);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(group_end != nullptr && aligned_to(group_end, 4), "mxq_grouped_gemm128: group_end must be 4-byte aligned, not NULL");
  MXQ_REQUIRE_DEVICE();
  if (M == 0) return ok();
  const bool f32 = cdt == MXQ_DT_F32;
  return launched(mode == MXQ_GG_RAGGED_M ? launch_gemm128<kRaggedM, true>(p, f32, st)
                                          : launch_gemm128<kRaggedK, false>(p, f32, st),
                  "mxq_grouped_gemm128");
}

}  // extern "C"
