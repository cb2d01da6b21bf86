// Routing of tokens to experts: scores, choice and weights; the expert order
// of the chosen pairs; the gradient of the weights.
//
// The choice has to be that of exact arithmetic: two keys of a row that fp32
// cannot tell apart would come out in an order that depends on how exp is
// evaluated.  The fast kernel chooses in fp32, knows how far its keys can be
// off, and takes what that leaves open to fp64: the order of the candidates
// alone where that decides, the whole row (route_row64) where it does not.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "mxq_device.h"
#include "mxq_host.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

constexpr int kWave = 64;
constexpr double kMasked = -3.3895313892515355e38;  // lowest finite bf16: logits at or below it are masked
constexpr double kNanKey = -1e300;                  // a NaN key ranks below every number, above a masked one

struct RouteParams {
  int32_t E, K, n_group, topk_group, group_top, renorm, sigmoid;
  float scale;
};

__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// largest value of the wave and the lowest index that has it
__device__ __forceinline__ void wave_argmax(double& v, int& i) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const double u = __shfl_xor(v, o);
    const int j = __shfl_xor(i, o);
    if (u > v || (u == v && j < i)) { v = u; i = j; }
  }
}

__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return (x >= 0 ? 1.0 : e) / (1.0 + e);  // NaN: e is NaN
}

// One token by one wave in fp64.  keys: E doubles of LDS of this wave's own.
template <typename LT>
__device__ void route_row64(const LT* __restrict__ l, const float* __restrict__ bias, const RouteParams p,
                            double* keys, int32_t* __restrict__ idx, float* __restrict__ weights) {
  const int lane = threadIdx.x & (kWave - 1);
  double top = -INFINITY, total = 0;
  if (!p.sigmoid) {
    for (int e = lane; e < p.E; e += kWave) {
      const double x = load_f(l, e);
      if (!(x <= kMasked)) top = fmax(top, x);
    }
    top = wave_max(top);
    for (int e = lane; e < p.E; e += kWave) {
      const double x = load_f(l, e);
      if (!(x <= kMasked)) total += exp(x - top);
    }
    total = wave_sum(total);
  }
  auto score = [&](double x) { return p.sigmoid ? sigmoid64(x) : exp(x - top) / total; };
  auto biased = [&](int e) {
    const double x = load_f(l, e);
    if (x <= kMasked) return -(double)INFINITY;
    const double k = score(x) + (bias ? (double)bias[e] : 0.0);
    return isnan(k) ? kNanKey : k;
  };

  uint64_t kept = ~0ull;
  const int per = p.E / p.n_group;
  if (p.n_group > 1) {
    for (int e = lane; e < p.E; e += kWave) keys[e] = biased(e);
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double best = -INFINITY;
    if (lane < p.n_group) {
      double a = -INFINITY, b = -INFINITY;
      for (int j = 0; j < per; j++) {
        const double k = keys[lane * per + j];
        b = fmax(b, fmin(a, k));
        a = fmax(a, k);
      }
      best = p.group_top == 2 && b > -INFINITY ? a + b : a;
    }
    kept = 0;
    for (int r = 0; r < p.topk_group; r++) {
      double v = best;
      int g = lane;
      wave_argmax(v, g);
      if (!(v > -INFINITY)) break;
      kept |= 1ull << g;
      if (lane == g) best = -INFINITY;
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  }
  for (int e = lane; e < p.E; e += kWave) {
    double k = -INFINITY;
    if (kept >> (p.n_group > 1 ? e / per : 0) & 1) {
      if (bias) {
        k = biased(e);
      } else {
        const double x = load_f(l, e);
        k = x <= kMasked ? -(double)INFINITY : isnan(x) ? kNanKey : x;
      }
    }
    keys[e] = k;
  }
  int chosen = -1;
  for (int r = 0; r < p.K; r++) {
    double v = -INFINITY;
    int i = 0x7FFFFFFF;
    for (int e = lane; e < p.E; e += kWave) {
      const double k = keys[e];  // written by this lane
      if (k > v) { v = k; i = e; }
    }
    wave_argmax(v, i);
    if (!(v > -INFINITY)) break;
    if (lane == r) chosen = i;
    if (lane == (i & (kWave - 1))) keys[i] = -INFINITY;
  }
  double w = chosen >= 0 ? score(load_f(l, chosen)) : 0.0;
  if (p.renorm) {
    double sum = wave_sum(w);
    if (sum == 0.0) {  // scores that underflow: over the largest of their exps instead
      const double x = chosen >= 0 ? load_f(l, chosen) : -INFINITY;
      const double low = p.sigmoid ? fmin(x, 0.0) : x, m = wave_max(low);
      w = chosen >= 0 ? exp(low - m) / (p.sigmoid ? 1.0 + exp(-fabs(x)) : 1.0) : 0.0;
      sum = wave_sum(w);
    }
    w = sum == 0.0 ? 0.0 : w / sum;
  }
  if (lane < p.K) {
    idx[lane] = chosen;
    weights[lane] = (float)(w * (double)p.scale);
  }
}

constexpr int kRouteWaves = 4;

// workgroups for `units` units of work, one each while a grid can hold them
// (a grid has fewer than 2^32 threads); the kernels walk the rest
unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 20) ? units : 1 << 20); }

// one wave per token
template <typename LT>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel64(const LT* __restrict__ logits, int64_t T, int64_t ld,
                                                                    const float* __restrict__ bias, RouteParams p,
                                                                    int32_t* __restrict__ idx,
                                                                    float* __restrict__ weights) {
  extern __shared__ double lds_keys[];
  const int wave = threadIdx.x / kWave;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < T; t += (int64_t)gridDim.x * kRouteWaves)
    route_row64(logits + t * ld, bias, p, lds_keys + wave * p.E, idx + t * p.K, weights + t * p.K);
}

// ------------------------------------------------------------------ expert order
// A stable counting sort of the N = T * K pairs by expert.  The pairs are cut
// into chunks whose pairs are counted by expert (by route_fast_kernel for its own
// tokens, or by hist_kernel); order_kernel adds up the counts before its chunks
// and ranks its pairs segment by segment: within a wave by ballots over the bits
// of the expert, across waves by their counts.  No atomics order anything, so the
// result is always the same.
constexpr int kMaxOrderThreads = 1024, kMaxOrderWaves = kMaxOrderThreads / kWave;
constexpr int kMaxChunkPairs = 1 << 15;  // counts are 16-bit
// Counts of all chunks, read whole by every workgroup of order_kernel: a chunk more costs
// each of them its row.  16384 x 8 pairs of 1024 experts in 80 chunks of their own take 33 us with
// the router, in 160 36; 16384 x 256 in the router's 256 chunks 17.4, in 1024 21.7.
constexpr int64_t kCountBytes = 160 << 10;
static_assert(MXQ_MAX_GROUPS <= kMaxOrderThreads, "a thread per expert");

// elements of a chunk's row of counts: a power of two of 16-byte loads
__host__ __device__ constexpr int32_t count_stride(int32_t E) { return E <= 8 ? 8 : 1 << (32 - __builtin_clz(E - 1)); }

// LDS of the ranking: 16-bit counts of up to kMaxOrderWaves waves, rows of E rounded up to 16 bytes
__host__ __device__ constexpr int count_row(int E) { return (E + 7) / 8 * 8; }
constexpr size_t order_lds(int waves, int E) { return (size_t)waves * count_row(E) * sizeof(uint16_t); }

// Exclusive sums of one value per thread over the workgroup's waves (WAVES at most); total: of all.
// The waves' sums are read without branches between: with one, each read was waited for.
template <int WAVES>
__device__ __forceinline__ int32_t block_exclusive(int32_t v, int waves, int32_t (&part)[WAVES], int32_t& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  // inclusive over the wave: lanes 1, 2, 4, 8 below within rows of 16 (0 where there is
  // none), then the last lane of the row before, and of the 32 lanes before
  int32_t incl = v;
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xF, 0xF, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xF, 0xF, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xF, 0xF, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xF, 0xF, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xA, 0xF, false);
  incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xC, 0xF, false);
  if (lane == kWave - 1) part[wave] = incl;
  __syncthreads();
  int32_t n[WAVES], off = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) n[w] = part[w];
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) {
    off += w < wave ? n[w] : 0;
    total += w < waves ? n[w] : 0;
  }
  return off + incl - v;
}

// A segment is one pair per thread, x its expert (E: none).  rank_in_wave: how many
// earlier lanes have the same; the wave's count of each expert goes to `count`
// [waves][count_row(E)], which is zero before and read after a barrier.
__device__ __forceinline__ int rank_in_wave(int32_t x, int32_t E, uint16_t* count) {
  const int wave = threadIdx.x / kWave;
  const int bits = 32 - __builtin_clz(E);  // of 0 .. E
  uint32_t lo = ~0u, hi = ~0u;             // lanes with the same
  for (int bit = 0; bit < bits; bit++) {
    const uint32_t set = (uint32_t)((int32_t)((uint32_t)x << (31 - bit)) >> 31);
    const uint64_t m = __ballot(set != 0);
    lo &= ~((uint32_t)m ^ set);
    hi &= ~((uint32_t)(m >> 32) ^ set);
  }
  const int rank = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
  if (x < E && rank == 0) count[wave * count_row(E) + x] = (uint16_t)(__popc(lo) + __popc(hi));
  return rank;
}
// pairs of expert x (E or more: of none) in earlier waves of the segment
template <int WAVES>
__device__ __forceinline__ int32_t pairs_before(int32_t x, int32_t E, const uint16_t* count) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint16_t* c = count + min(x, E - 1);
  int32_t n[WAVES], run = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) n[w] = c[w * count_row(E)];
#pragma unroll
  for (int w = 0; w < WAVES; w++) run += w < wave ? n[w] : 0;
  return run;
}
// The segment's counts of experts 2 i and 2 i + 1, packed.
// (A segment has at most 1024 pairs, so neither half carries into the other.)
template <int WAVES>
__device__ __forceinline__ uint32_t segment_counts(int i, int32_t E, const uint16_t* count) {
  const uint32_t* c = reinterpret_cast<const uint32_t*>(count) + i;
  uint32_t run = 0;
#pragma unroll
  for (int w = 0; w < WAVES; w++) run += c[w * (count_row(E) / 2)];
  return run;
}
__device__ __forceinline__ void clear_counts(int32_t E, uint16_t* count) {
  const u32x4 zero = {0, 0, 0, 0};
  for (int i = threadIdx.x; i < (int)(blockDim.x / kWave) * count_row(E) / 8; i += blockDim.x)
    reinterpret_cast<u32x4*>(count)[i] = zero;
}
__device__ __forceinline__ int32_t expert_at(const int32_t* idx, int64_t i, int64_t e, int32_t E) {
  const int32_t x = i < e ? idx[i] : -1;
  return x >= 0 && x < E ? x : E;
}
// pair i of token `token` is the rank-th of expert x from row `first` on
__device__ __forceinline__ void put_pair(int64_t i, int64_t e, int32_t x, int32_t E, int32_t first, int rank,
                                         int32_t token, int32_t* __restrict__ row_token, int32_t* __restrict__ slot) {
  if (i >= e) return;
  int32_t row = -1;
  if (x < E) {
    row = first + rank;
    row_token[row] = token;
  }
  slot[i] = row;
}
// token of pair i (T * K < 2^31)
__device__ __forceinline__ int32_t token_of(int64_t i, int32_t K) { return (int32_t)((uint32_t)i / (uint32_t)K); }

__global__ __launch_bounds__(kMaxOrderThreads) void hist_kernel(const int32_t* __restrict__ idx, int64_t N, int64_t chunk,
                                                               int32_t E, int32_t stride,
                                                               uint16_t* __restrict__ counts) {
  __shared__ int32_t h[MXQ_MAX_GROUPS];
  for (int x = threadIdx.x; x < E; x += blockDim.x) h[x] = 0;
  __syncthreads();
  const int64_t b = blockIdx.x * chunk, e = min(b + chunk, N);
  for (int64_t i = b + threadIdx.x; i < e; i += blockDim.x) {
    const int32_t x = idx[i];
    if (x >= 0 && x < E) atomicAdd(&h[x], 1);  // a count: the order does not matter
  }
  __syncthreads();
  for (int x = threadIdx.x; x < stride; x += blockDim.x)
    counts[(int64_t)blockIdx.x * stride + x] = x < E ? (uint16_t)h[x] : 0;
}

// Sum of 16-bit pairs
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(u16x2, a) + __builtin_bit_cast(u16x2, b));
}

// Counts of a thread's chunks first, first + runs, ..: of all of them, and of those before
// chunk `mine`, eight experts each, two a word (PACKED) or one.  LOADS of them at a time, without
// branches between (past the end the last one is read and not counted).
template <bool PACKED, int LOADS>
__device__ __forceinline__ void sum_counts(const u32x4* c4, int cols, int chunks, int first, int runs, int mine,
                                           uint32_t* all, uint32_t* before) {
  for (int c0 = first; c0 < chunks; c0 += LOADS * runs) {
    u32x4 v[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; i++) v[i] = c4[(int64_t)min(c0 + i * runs, chunks - 1) * cols];
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
      const int c = c0 + i * runs;
      const uint32_t in = c < chunks ? 0xFFFFFFFFu : 0u, earlier = c < mine ? 0xFFFFFFFFu : 0u;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        if (PACKED) {
          all[j] = add2(all[j], v[i][j] & in);
          before[j] = add2(before[j], v[i][j] & earlier);
        } else {
          all[2 * j] += v[i][j] & in & 0xFFFFu;
          all[2 * j + 1] += (v[i][j] & in) >> 16;
          before[2 * j] += v[i][j] & earlier & 0xFFFFu;
          before[2 * j + 1] += (v[i][j] & earlier) >> 16;
        }
      }
    }
  }
}

// Sums over the lanes that are a multiple of cols (a power of two) apart, in each of them.
template <bool PACKED, int N>
__device__ __forceinline__ void sum_runs(int cols, uint32_t (&v)[N]) {
  auto add = [](uint32_t a, uint32_t b) { return PACKED ? add2(a, b) : a + b; };
#define MXQ_ROTATE(n)                                                                             \
  if (cols <= n)                                                                                  \
    _Pragma("unroll") for (int j = 0; j < N; j++)                                                 \
        v[j] = add(v[j], (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[j], 0x120 + n, 0xF, 0xF, true));
  MXQ_ROTATE(8)  // within rows of 16; a sum repeats every 8 lanes from here on
  MXQ_ROTATE(4)
  MXQ_ROTATE(2)
  MXQ_ROTATE(1)
#undef MXQ_ROTATE
  if (cols <= 16)
#pragma unroll
    for (int j = 0; j < N; j++) {
      const auto r = __builtin_amdgcn_permlane16_swap(v[j], v[j], false, false);
      v[j] = add(r[0], r[1]);
    }
  if (cols <= 32)
#pragma unroll
    for (int j = 0; j < N; j++) {
      const auto r = __builtin_amdgcn_permlane32_swap(v[j], v[j], false, false);
      v[j] = add(r[0], r[1]);
    }
}

constexpr int kParts = 8;  // partial sums of an expert: one of each wave, or of each run of the waves

// Workgroup b ranks chunks b * per .. (b + 1) * per - 1 of `chunk` pairs, at most `most` of them one expert's.
//
// Bound by latency: a chain of one read of the counts and four barriers.  16384 x 8 pairs of
// 256 experts take 5 us on the GPU, 5003 x 8 of 32 4, where a launch that does nothing takes 2;
// 131072 x 8 of 256 with their count 18.5.
template <int WAVES>
__global__ __launch_bounds__(WAVES* kWave) void order_kernel(const int32_t* __restrict__ idx, int64_t N, int64_t chunk,
                                                            int32_t chunks, int32_t per, int32_t E, int32_t most, int32_t K,
                                                            const uint16_t* __restrict__ counts,
                                                            int32_t* __restrict__ group_end,
                                                            int32_t* __restrict__ row_token,
                                                            int32_t* __restrict__ slot) {
  constexpr int THREADS = WAVES * kWave;  // at least E
  __shared__ __attribute__((aligned(16))) uint16_t count[WAVES * THREADS];
  __shared__ __attribute__((aligned(16))) int32_t sums[2 * kParts * THREADS];  // of all chunks, of the earlier ones
  __shared__ int32_t base[THREADS];
  __shared__ __attribute__((aligned(16))) int32_t part[WAVES];
  const int t = threadIdx.x;
  const int32_t mine = blockIdx.x * per;
  const int64_t b = mine * chunk, e = min(b + per * chunk, N);
  int32_t x = -1;
  if (N > 0) x = idx[min(b + t, N - 1)];
  int32_t token = token_of(b + t, K);
  // Eight experts' counts a load; a row of counts by stride / 8 threads, the chunks dealt to
  // as many such runs of threads as the workgroup holds.  Whole numbers: the order
  // of the additions does not matter.
  const int stride = count_stride(E), shift = __builtin_ctz(stride) - 3;
  const int cols = 1 << shift, runs = THREADS >> shift, run = t >> shift, col = t & (cols - 1);
  const int visits = (chunks + runs - 1) >> (__builtin_ctz(THREADS) - shift);
  // two sums a word where no half can carry, after the wave's runs are added up too
  const bool packed = (int64_t)most * visits * (cols < kWave ? kWave >> shift : 1) <= 0xFFFF;
  const u32x4* c4 = reinterpret_cast<const u32x4*>(counts) + col;
  uint32_t all8[8] = {}, before8[8] = {};
  if (packed) {
    uint32_t a[4] = {}, f[4] = {};
    if (visits == 1)
      sum_counts<true, 1>(c4, cols, chunks, run, runs, mine, a, f);
    else if (visits <= 4)
      sum_counts<true, 4>(c4, cols, chunks, run, runs, mine, a, f);
    else
      sum_counts<true, 16>(c4, cols, chunks, run, runs, mine, a, f);
    sum_runs<true>(cols, a);
    sum_runs<true>(cols, f);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      all8[2 * j] = a[j] & 0xFFFFu;
      all8[2 * j + 1] = a[j] >> 16;
      before8[2 * j] = f[j] & 0xFFFFu;
      before8[2 * j + 1] = f[j] >> 16;
    }
  } else {
    sum_counts<false, 8>(c4, cols, chunks, run, runs, mine, all8, before8);
    sum_runs<false>(cols, all8);
    sum_runs<false>(cols, before8);
  }
  clear_counts(E, count);
  // One of the kParts rows of the sums for each wave where a wave holds whole rows, else for each run.
  if ((t & (kWave - 1)) < cols) {
    u32x4* s = reinterpret_cast<u32x4*>(sums + (cols < kWave ? t / kWave : run) * stride + 8 * col);
    s[0] = u32x4{all8[0], all8[1], all8[2], all8[3]};
    s[1] = u32x4{all8[4], all8[5], all8[6], all8[7]};
    s += kParts * stride / 4;
    s[0] = u32x4{before8[0], before8[1], before8[2], before8[3]};
    s[1] = u32x4{before8[4], before8[5], before8[6], before8[7]};
  }
  __syncthreads();
  x = b + t < e && x >= 0 && x < E ? x : E;
  int rank = rank_in_wave(x, E, count);
  int32_t all = 0, before = 0;
  const int mine_e = min(t, E - 1);
#pragma unroll
  for (int i = 0; i < kParts; i++) {
    all += sums[i * stride + mine_e];
    before += sums[(kParts + i) * stride + mine_e];
  }
  all = t < E ? all : 0;
  int32_t total;
  const int32_t start = block_exclusive<WAVES>(all, WAVES, part, total);  // a barrier: counts of all waves
  if (t < E) {
    base[t] = start + before;
    if (blockIdx.x == 0) group_end[t] = start + all;
  }
  const int32_t earlier = pairs_before<WAVES>(x, E, count);
  __syncthreads();
  int32_t row = base[min(x, E - 1)] + earlier;
  for (int64_t s = b;;) {
    put_pair(s + t, e, x, E, row, rank, token, row_token, slot);
    s += THREADS;
    if (s >= e) break;
    const bool two = t < (E + 1) / 2;
    const uint32_t segment = two ? segment_counts<WAVES>(t, E, count) : 0;
    __syncthreads();
    if (two) {
      base[2 * t] += segment & 0xFFFFu;
      base[2 * t + 1] += segment >> 16;
    }
    clear_counts(E, count);
    x = expert_at(idx, s + t, e, E);
    token = token_of(s + t, K);
    __syncthreads();
    rank = rank_in_wave(x, E, count);
    __syncthreads();
    row = base[min(x, E - 1)] + pairs_before<WAVES>(x, E, count);
  }
  for (int64_t i = total + (int64_t)blockIdx.x * THREADS + t; i < N; i += (int64_t)gridDim.x * THREADS) row_token[i] = -1;
}

// ------------------------------------------------------------------ fast routing
// A row is held by LPR lanes (64 / LPR rows to a wave), EPL consecutive experts a
// lane, each expert group by LPG = LPR / pow2(n_group) lanes.  Keys are ordered
// 32-bit integers whose lowest bits give way to the expert's place in its lane, so
// a lane's keys differ.  A choice is a maximum over the lanes; each lane keeps its
// four largest keys in order for it.  bf16 logits without a bias leave room for the
// whole index, and keys are exact.
//
// Bound by the vector units and, up to some 16000 rows, by the latency of one pass
// (launch, read, choices one after another, write): 16384 x 256 sigmoid rows with a bias in 8
// groups take 9.7 to 10.4 us by part, 65536 in one group 20.5 (67 MB, 3.3 TB/s), 65536 x 256 bf16
// rows of a softmax 16.8.
struct Shape {
  int32_t lpg_log2;  // lanes per group
  int32_t stride;    // of the rows of counts
  int32_t full;      // every lane has EPL experts
};

struct OrderOut {
  int32_t* group_end;
  int32_t* row_token;
  int32_t* slot;
  uint16_t* counts;  // of each workgroup's pairs by expert
  int32_t mode;      // 0 none, 1 counts, 2 everything (one workgroup)
};

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp_f(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// max and sum over the LPR lanes of a row
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = quad_max_u32(v);
  v = max(v, dpp_half_mirror(v));
  v = max(v, dpp_mirror(v));
  if constexpr (LPR > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  if constexpr (LPR > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  auto f = [](uint32_t u) { return __uint_as_float(u); };
  v += f(dpp_xor1(__float_as_uint(v)));
  v += f(dpp_xor2(__float_as_uint(v)));
  v += f(dpp_half_mirror(__float_as_uint(v)));
  v += f(dpp_mirror(__float_as_uint(v)));
  if constexpr (LPR > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(r[0]) + f(r[1]);
  }
  if constexpr (LPR > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(r[0]) + f(r[1]);
  }
  return v;
}

__device__ __forceinline__ uint32_t median(uint32_t a, uint32_t b, uint32_t c) {
  return max(min(a, b), min(max(a, b), c));
}

// order-preserving integers of floats; 0 is below all of them
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
template <int LPR>
__device__ __forceinline__ float row_fmax(float v) { return unordered(row_max<LPR>(ordered(v))); }

// What a choice goes by: logits, for groups too (kLogits); logits, and scores for the
// groups (kScoredGroups); scores and a bias (kBiased).
enum Keys { kLogits, kScoredGroups, kBiased };

// weights of a row's chosen experts (one a lane, its logit v); lanes of other rows beside
template <int LPR>
__device__ __forceinline__ float weight_of(float v, bool in, const RouteParams& p, float top, float inv_total) {
  float w;
  if (p.sigmoid) {
    const float e = exp_f(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.f + e);
    if (p.renorm) {  // over the largest exp of the row, so that no score underflows
      const float low = fminf(v, 0.f);
      const float m = row_fmax<LPR>(in ? low : -INFINITY);
      w = in ? exp_f(low - m) * r : 0.f;
    } else {
      w = in ? (v >= 0.f ? 1.f : e) * r : 0.f;
    }
  } else {
    const float m = p.renorm ? row_fmax<LPR>(in ? v : -INFINITY) : top;
    w = in ? exp_f(v - m) : 0.f;
    if (!p.renorm) w *= inv_total;
  }
  if (p.renorm) {
    const float s = row_sum<LPR>(w);
    w = s > 0.f ? w / s : 0.f;
  }
  return w * p.scale;
}

template <typename LT, int LPR, int EPL, Keys KEYS>
__global__ __launch_bounds__(1024) void route_fast_kernel(const LT* __restrict__ logits, int64_t T, int64_t ld,
                                                         const float* __restrict__ bias, const RouteParams p,
                                                         const Shape sh, int32_t* idx, float* __restrict__ weights,
                                                         const OrderOut o) {
  constexpr int RPW = kWave / LPR;                 // rows of a wave
  constexpr uint32_t LOW = EPL - 1;                // a key's bits for the place in its lane
  constexpr bool EXACT = sizeof(LT) == 2 && KEYS != kBiased;
  constexpr int kSlow = 4;                         // waves that take whole rows to fp64
  constexpr uint64_t ROW = LPR == 64 ? ~0ull : (1ull << (LPR & 63)) - 1;
  extern __shared__ double lds[];                  // their keys; the ranking's counts
  __shared__ int32_t hist[MXQ_MAX_GROUPS];
  __shared__ int32_t slow_rows[16 * RPW], slow_count;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, waves = blockDim.x / kWave;
  const int sub = lane & (LPR - 1), first_lane = lane - sub;
  const int per = p.E / p.n_group;
  const bool grouped = p.n_group > 1;
  const bool stats = !p.sigmoid && (KEYS != kLogits || !p.renorm);
  const int64_t r0 = (int64_t)blockIdx.x * (waves * RPW);  // rows r0 .. r0 + waves * RPW - 1
  const int64_t t = r0 + wave * RPW + lane / LPR;
  const bool live = t < T;
  const LT* l = logits + (live ? t : r0) * ld;
  const int g = sub >> sh.lpg_log2, part = sub & ((1 << sh.lpg_log2) - 1);
  const int e0 = g * per + part * EPL;  // the lane's experts: e0 .. e0 + n - 1
  const int n = g < p.n_group ? min(max(per - part * EPL, 0), EPL) : 0;

  // logits and bias, read before the first barrier (by waves without rows too: row r0)
  float x[EPL];
  float k[EPL];  // scores + bias
  if (EPL % 4 == 0 && per % 4 == 0) {
    Raw<LT, 4> w[EPL >= 4 ? EPL / 4 : 1];
#pragma unroll
    for (int q = 0; q < EPL / 4; q++) w[q] = load_raw<4, false>(l + (4 * q < n ? e0 + 4 * q : 0));
    if (KEYS == kBiased)
#pragma unroll
      for (int q = 0; q < EPL / 4; q++) unpack(load_raw<4, false>(bias + (4 * q < n ? e0 + 4 * q : 0)), &k[4 * q]);
#pragma unroll
    for (int q = 0; q < EPL / 4; q++) unpack(w[q], &x[4 * q]);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; j++) x[j] = load_f(l, j < n ? e0 + j : 0);
    if (KEYS == kBiased)
#pragma unroll
      for (int j = 0; j < EPL; j++) k[j] = bias[j < n ? e0 + j : 0];
  }

  if (o.mode)
    for (int x = tid; x < p.E; x += blockDim.x) hist[x] = 0;
  if (tid == 0) slow_count = 0;
  __syncthreads();
  if (r0 + wave * RPW < T) {
    if (!sh.full)  // absent ones
#pragma unroll
      for (int j = 0; j < EPL; j++) x[j] = j < n ? x[j] : -INFINITY;
    float top = 0.f, inv_total = 0.f;
    if (stats) {  // masked logits add exp(-inf)
      float m = x[0];
#pragma unroll
      for (int j = 1; j < EPL; j++) m = fmaxf(m, x[j]);
      top = fmaxf(row_fmax<LPR>(m), (float)kMasked);
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; j++) s += exp_f(x[j] - top);
      s = row_sum<LPR>(s);
      inv_total = s > 0.f ? 1.f / s : 0.f;
    }
    bool odd = false;  // a NaN or an infinity that is no mask: the whole row in fp64
    if (KEYS == kLogits) {
#pragma unroll
      for (int j = 0; j < EPL; j++) odd |= !(x[j] < INFINITY);
    } else {
      // a loop each, or every step of one is a branch
      if (p.sigmoid) {  // 1 / (1 + exp(-x)) for either sign: where exp(-x) is large its relative error is that of the score
#pragma unroll
        for (int j = 0; j < EPL; j++) {
          const float s = __builtin_amdgcn_rcpf(1.f + exp_f(-x[j]));
          k[j] = KEYS == kBiased ? s + k[j] : s;
        }
      } else {
#pragma unroll
        for (int j = 0; j < EPL; j++) {
          const float s = exp_f(x[j] - top) * inv_total;
          k[j] = KEYS == kBiased ? s + k[j] : s;
        }
      }
      float zero = 0.f;  // NaN after any that is not finite
#pragma unroll
      for (int j = 0; j < EPL; j++) {
        zero = __builtin_fmaf(k[j], 0.f, zero);
        k[j] = x[j] <= (float)kMasked ? -INFINITY : k[j];
      }
      odd = zero != 0.f;
    }
    if (KEYS != kBiased)
#pragma unroll
      for (int j = 0; j < EPL; j++) x[j] = x[j] <= (float)kMasked ? -INFINITY : x[j];

    // fp64 pieces for what fp32 leaves open: the sum of a softmax, a score (+ bias)
    auto exp_sum = [&] {
      double s = 0.0;
#pragma unroll 1
      for (int j = 0; j < n; j++) {
        const float v = load_f(l, e0 + j);
        if (!(v <= (float)kMasked)) s += exp((double)v - (double)top);
      }
      for (int m = 1; m < LPR; m <<= 1) s += __shfl_xor(s, m);
      return s;
    };
    auto exact_key = [&](int e, double dsum, bool with_bias) {
      const double v = load_f(l, e);
      const double s = p.sigmoid ? sigmoid64(v) : exp(v - (double)top) / dsum;
      return with_bias ? s + (double)bias[e] : s;
    };

    bool kept = true;
    if (grouped) {
      float a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int j = 0; j < EPL; j++) {
        const float f = KEYS == kLogits ? x[j] : k[j];
        b = __builtin_amdgcn_fmed3f(a, b, f);  // a >= b: the second of the three
        a = fmaxf(a, f);
      }
      for (int m = 1; m < 1 << sh.lpg_log2; m <<= 1) {
        const float a2 = __shfl_xor(a, m), b2 = __shfl_xor(b, m);
        b = fmaxf(fminf(a, a2), fmaxf(b, b2));
        a = fmaxf(a, a2);
      }
      const bool two = p.group_top == 2 && b > -INFINITY;
      // finite keys: a sum past fp32 is still a group's total, not a masked group's -inf
      const float total = two ? fmaxf(a + b, -FLT_MAX) : a;
      if (KEYS == kLogits) {
        // A group's total is the score of its largest logit and grows with that, so logits order
        // the groups; but where the scores of the least kept and the largest not kept may be
        // one number in 64 bits, the lower group goes first, and the row is taken to fp64:
        // scores that underflow, and those apart by 2^-47 of the score or less (the
        // logits' difference times 1 - s for a sigmoid, at least min(exp(-l), 1) / 2).
        int rank = 0;
        for (int q = 0; q < p.n_group; q++) {
          const float other = __shfl(total, first_lane + (q << sh.lpg_log2));
          rank += other > total || (other == total && q < g);
        }
        kept = g < p.n_group && rank < p.topk_group && total > -INFINITY;
        const uint32_t most = row_max<LPR>(!kept && g < p.n_group && total > -INFINITY ? ordered(total) : 0u);
        const float least = unordered(~row_max<LPR>(kept ? ~ordered(total) : 0u));
        const float apart = least - unordered(most), low = p.sigmoid ? least : least - row_fmax<LPR>(total);
        odd |= most != 0 && apart != 0.f && (!(apart * (p.sigmoid ? fminf(exp_f(-least), 1.f) : 1.f) > 0x1p-46f) || low < -600.f);
      } else {
        // The largest total topk_group times over; groups of one total go together, and
        // too many of them are told apart below.  (16384 x 256 rows in 8 groups 9.6 us, by
        // comparing each group with each 10.0; 1024 experts in 64 groups 33.6 and 45.5; the bounds
        // from each group's own keys are 0.1 us of the former.)
        uint32_t left = g < p.n_group && total > -INFINITY ? ordered(total) : 0u;
        kept = false;
        for (int r = 0; r < p.topk_group; r++) {
          const uint32_t m = row_max<LPR>(left);
          if (left == m && m != 0) {  // 0: no group is left
            kept = true;
            left = 0;
          }
        }
        // A total is off by the errors of its two scores (4 half steps of 1 for a sigmoid, 42
        // for a softmax), and by the roundings of the two keys and their sum: at most two
        // half steps of |a| + |b|, which is far more than of the total where the keys have
        // opposite signs.  `error` is twice the former for two totals, `slack` twice the latter
        // for one, which leaves room for its own roundings.  Where the least total kept, lowered,
        // does not clear the largest not kept, raised, the totals are taken in fp64, from the
        // experts that can be among their groups' best two.
        const float error = p.sigmoid ? 0x1p-20f : 0x1.5p-17f;
        const float slack = fabsf(a) * 0x1p-22f + (two ? fabsf(b) * 0x1p-22f : 0.f);
        const uint32_t most = row_max<LPR>(left != 0 ? ordered(total + slack) : 0u);
        const float least = unordered(~row_max<LPR>(kept ? ~ordered(total - slack) : 0u));
        const bool many = __popcll(__ballot(kept) >> first_lane & ROW) > p.topk_group << sh.lpg_log2;
        const bool open = many || (most != 0 && !(least - unordered(most) > error));
        if (__any(open)) {
          // without a bias the sum divides all totals of the row, which matters where they underflow
          const bool divide = !p.sigmoid && (KEYS == kBiased || __any(open && least < 0x1p-100f));
          const double dsum = divide ? exp_sum() : 1.0;
          const float last = two ? b : a, from = last - (error + fabsf(last) * 0x1p-22f);
          uint32_t which = 0;
#pragma unroll
          for (int j = 0; j < EPL; j++) which |= k[j] > -INFINITY && k[j] >= from ? 1u << j : 0u;
          double da = -INFINITY, db = -INFINITY;
          while (__any(which)) {
            if (which) {
              const double s = exact_key(e0 + __ffs(which) - 1, dsum, KEYS == kBiased);
              which &= which - 1;
              db = fmax(db, fmin(da, s));
              da = fmax(da, s);
            }
          }
          for (int m = 1; m < 1 << sh.lpg_log2; m <<= 1) {
            const double a2 = __shfl_xor(da, m), b2 = __shfl_xor(db, m);
            db = fmax(fmin(da, a2), fmax(db, b2));
            da = fmax(da, a2);
          }
          const double dt = two ? da + db : da;
          int r = 0;
          for (int q = 0; q < p.n_group; q++) {
            const double other = __shfl(dt, first_lane + (q << sh.lpg_log2));
            r += other > dt || (other == dt && q < g);
          }
          kept = g < p.n_group && r < p.topk_group && dt > -INFINITY;
        }
      }
    }

    uint32_t key[EPL];
#pragma unroll
    for (int j = 0; j < EPL; j++) {
      const uint32_t u = ordered(KEYS == kBiased ? k[j] : x[j] + 0.f);  // -0 + 0 is 0: they are equal
      key[j] = EXACT ? (u & 0xFFFF0000u) | (0xFFFFu - (uint32_t)(e0 + j)) : (u & ~LOW) | (LOW - j);
    }
    constexpr uint32_t NONE = 0x007FFFFFu;   // keys of -inf and 0 lie here and below
    // The lane's largest keys in order, those that are left: a choice takes the first of
    // one lane, and a lane that has given all of its list looks through its keys for the
    // next.  (A look through them for every choice instead of the list: 65536 x 256 bf16
    // rows, top 8, 19.6 against 17.7 us; for a choice or two the list costs more than it
    // saves: top 1 of fp32 rows 13.9 against 14.6.)
    constexpr int LIST = EPL < 4 ? EPL : 4;
    uint32_t list[LIST] = {};
    if (EPL <= LIST || p.K > 2) {
#pragma unroll
      for (int j = 0; j < EPL; j++) {
#pragma unroll
        for (int i = LIST - 1; i > 0; i--) list[i] = median(list[i - 1], list[i], key[j]);
        list[0] = max(list[0], key[j]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; j++) list[0] = max(list[0], key[j]);
    }
#pragma unroll
    for (int i = 0; i < LIST; i++) list[i] = kept ? list[i] : 0u;
    int chosen_lane = 0;
    uint32_t chosen_key = 0;
    auto choose = [&](int r) {
      const uint32_t m = row_max<LPR>(list[0]);
      const uint64_t who = __ballot(list[0] == m);
      int win;
      if constexpr (LPR == 64)
        win = __ffsll((unsigned long long)who) - 1;
      else
        win = __ffs((lane < 32 ? (uint32_t)who : (uint32_t)(who >> 32)) >> (first_lane & 31)) - 1;
      if (sub == r) {
        chosen_lane = win;
        chosen_key = m;
      }
      const bool mine = sub == win;
#pragma unroll
      for (int i = 0; i + 1 < LIST; i++) list[i] = mine ? list[i + 1] : list[i];
      list[LIST - 1] = mine ? 0u : list[LIST - 1];
      if (EPL > LIST && __any(mine && list[0] == 0u && m != 0)) {  // largest below m
        uint32_t d = 0u - m;
#pragma unroll
        for (int j = 0; j < EPL; j++) d = max(d, key[j] - m);
        if (mine && list[0] == 0u && m != 0) list[0] = d + m;
      }
    };
    for (int r = 0; r < p.K; r++) choose(r);
    auto expert = [&] {
      const int e = EXACT ? 0xFFFF - (int)(chosen_key & 0xFFFFu)
                          : (chosen_lane >> sh.lpg_log2) * per + (chosen_lane & ((1 << sh.lpg_log2) - 1)) * EPL +
                                (int)(LOW - (chosen_key & LOW));
      return chosen_key > NONE ? e : -1;
    };
    int chosen = expert();
    float logit = load_f(l, max(chosen, 0));

    // Neighbours that fp32 leaves open (the same key but for the place, or scores too
    // close): they and as many more as may belong among the first K are put into the
    // order of their exact keys.
    if (!EXACT) {
      auto close = [&](uint32_t hi, uint32_t lo) {
        if (lo <= NONE) return false;
        if (KEYS != kBiased) return ((hi ^ lo) & ~LOW) == 0;
        // twice a score's error (4 or 42 half steps), the sums' roundings, the places' bits
        const float x = unordered(hi), y = unordered(lo);
        return x - y <= (p.sigmoid ? 0x1p-21f : 0x1.5p-18f) + fabsf(x) * (EPL * 0x1p-23f + 0x1p-22f);
      };
      uint32_t rest = row_max<LPR>(list[0]);
      uint32_t after = __shfl_down(chosen_key, 1);
      if (sub == p.K - 1) after = rest;
      if (__any(sub < p.K && close(chosen_key, after))) {
        int have = p.K;
        uint32_t last = __shfl(chosen_key, first_lane + have - 1);
        while (have < LPR && __any(close(last, rest))) {
          choose(have);
          have++;
          last = __shfl(chosen_key, first_lane + have - 1);
          rest = row_max<LPR>(list[0]);
        }
        odd |= close(last, rest);
        chosen = expert();
        const double dsum = KEYS == kBiased && !p.sigmoid ? exp_sum() : 1.0;
        double dk = -INFINITY;
        if (sub < have && chosen >= 0) dk = KEYS == kBiased ? exact_key(chosen, dsum, true) : (double)load_f(l, chosen);
        int rank = 0;
        for (int q = 0; q < have; q++) {
          const double v = __shfl(dk, first_lane + q);
          const int e = __shfl(chosen, first_lane + q);
          rank += v > dk || (v == dk && (e < chosen || (e == chosen && q < sub)));
        }
        chosen = __builtin_amdgcn_ds_permute((first_lane + (sub < have ? rank : sub)) * 4, chosen);
        logit = load_f(l, max(chosen, 0));
      }
    }

    const bool slow = live && (__ballot(odd) >> first_lane & ROW) != 0;
    if (slow && sub == 0) slow_rows[atomicAdd(&slow_count, 1)] = (int32_t)(t - r0);
    const float w = weight_of<LPR>(logit, sub < p.K && chosen >= 0, p, top, inv_total);
    if (live && !slow && sub < p.K) {
      idx[t * p.K + sub] = chosen;
      weights[t * p.K + sub] = w;
      if (o.mode && chosen >= 0) atomicAdd(&hist[chosen], 1);  // a count: the order does not matter
    }
  }
  __syncthreads();
  if (wave < kSlow)
    for (int q = wave; q < slow_count; q += min(kSlow, waves)) {
      const int64_t s = r0 + slow_rows[q];
      route_row64(logits + s * ld, bias, p, lds + wave * p.E, idx + s * p.K, weights + s * p.K);
      if (o.mode && lane < p.K) {
        const int32_t c = idx[s * p.K + lane];  // written by this lane
        if (c >= 0) atomicAdd(&hist[c], 1);
      }
    }
  __syncthreads();
  if (o.mode == 1) {
    for (int x = tid; x < sh.stride; x += blockDim.x)
      o.counts[(int64_t)blockIdx.x * sh.stride + x] = x < p.E ? (uint16_t)hist[x] : 0;
  } else if (o.mode == 2) {
    // all pairs here, one segment
    __shared__ __attribute__((aligned(16))) int32_t part_sums[kMaxOrderWaves];
    uint16_t* count = (uint16_t*)lds;
    clear_counts(p.E, count);
    const int32_t pairs = (int32_t)T * p.K;
    const int32_t x = expert_at(idx, tid, pairs, p.E);
    __syncthreads();
    const int rank = rank_in_wave(x, p.E, count);
    int32_t total = 0, carry = 0;
    for (int e0 = 0; e0 < p.E; e0 += blockDim.x) {
      const int e = e0 + tid;
      const int32_t c = e < p.E ? hist[e] : 0;
      const int32_t start = carry + block_exclusive<kMaxOrderWaves>(c, waves, part_sums, total);
      carry += total;
      if (e < p.E) {
        hist[e] = start;
        o.group_end[e] = start + c;
      }
      __syncthreads();
    }
    const int32_t first = hist[min(x, p.E - 1)] + pairs_before<kMaxOrderWaves>(x, p.E, count);
    put_pair(tid, pairs, x, p.E, first, rank, token_of(tid, p.K), o.row_token, o.slot);
    if (tid >= carry && tid < pairs) o.row_token[tid] = -1;
  }
}

// ------------------------------------------------------------------ launches
struct OrderPlan {
  int32_t chunks;
  int64_t chunk;  // pairs
  int32_t most;   // of them with one expert
};

// Workgroups of order_kernel at most: each reads all the counts, and there are as many CUs.
constexpr int64_t kMostOrderGroups = 256;

hipError_t launch_order(const int32_t* idx, int64_t N, int32_t K, int32_t E, OrderPlan op, int32_t* group_end,
                        int32_t* row_token, int32_t* slot, const uint16_t* counts, hipStream_t st) {
  // a thread per expert, and few waves to add up
  const int waves = E > 512 ? 16 : 8;
  const int64_t most = std::min<int64_t>(N / (waves * kWave) + 1, kMostOrderGroups);
  const int32_t per = (int32_t)((op.chunks + most - 1) / most);
  const int32_t grid = (op.chunks + per - 1) / per;
  auto f = waves == 16 ? order_kernel<16> : order_kernel<8>;
  f<<<grid, waves * kWave, 0, st>>>(idx, N, op.chunk, op.chunks, per, E, op.most, K, counts, group_end, row_token, slot);
  return hipGetLastError();
}

int64_t chunks_that_fit(int32_t E) { return kCountBytes / (count_stride(E) * (int64_t)sizeof(uint16_t)); }

// Chunks counted on their own: one for each workgroup of order_kernel, not more (320, so two
// of them for each of 160 workgroups, take 13.0 against 9.8 us for 32768 x 8 pairs of 256 experts
// and 74 against 50 for 524288 x 8).
OrderPlan order_plan(int64_t N, int32_t E) {
  const int64_t most = std::min<int64_t>(chunks_that_fit(E), kMostOrderGroups);
  const int64_t chunk = std::min<int64_t>(std::max<int64_t>((N + most - 1) / most, 512), kMaxChunkPairs);
  const int64_t c = (N + chunk - 1) / chunk;
  return {(int32_t)(c < 1 ? 1 : c), chunk, (int32_t)chunk};
}

hipError_t launch_expert_order(const int32_t* idx, int64_t N, int32_t K, int32_t E, int32_t* group_end,
                               int32_t* row_token, int32_t* slot, uint16_t* counts, hipStream_t st) {
  const OrderPlan op = order_plan(N, E);
  hist_kernel<<<op.chunks, kMaxOrderThreads, 0, st>>>(idx, N, op.chunk, E, count_stride(E), counts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_order(idx, N, K, E, op, group_end, row_token, slot, counts, st);
}

constexpr int64_t kFastRows = 1 << 25;  // of route_fast: 64 lanes each, in a grid of fewer than 2^32 threads

// Largest number of chunks that a call on these sizes cuts its pairs into: order_plan's,
// or one for each of route_fast's workgroups.
int64_t max_chunks(int64_t T, int32_t K, int32_t E) {
  const int64_t routers = std::min<int64_t>({chunks_that_fit(E), 2 * kMostOrderGroups, T / 4 + 1});
  return std::max<int64_t>(order_plan(T * K, E).chunks, routers);
}

int ceil_log2(int v) {
  int l = 0;
  while (1 << l < v) l++;
  return l;
}

// The fast kernel on a shape (LPR lanes of EPL experts) that holds the row:
// each group in its own lanes, and the chosen in one lane each.
template <typename LT, int LPR, int EPL>
bool holds(const RouteParams& p) {
  const int lanes = LPR >> ceil_log2(p.n_group);
  return lanes >= 1 && lanes * EPL >= p.E / p.n_group && p.K <= LPR;
}

constexpr int64_t kManyRows = 4096;

struct RouteArgs {
  const void* logits;
  int64_t T, ld;
  const float* bias;
  RouteParams p;
  int32_t* idx;
  float* weights;
  OrderOut o;
  hipStream_t st;
};

template <typename LT, int LPR, int EPL>
hipError_t route_fast(RouteArgs a) {
  constexpr int RPW = kWave / LPR;
  const bool order = a.o.group_end != nullptr;
  const int64_t units = (a.T + RPW - 1) / RPW;  // waves' worth of rows
  // One workgroup does it all where it holds the rows and their pairs are one segment of
  // the ranking.  Else workgroups of as few waves, from 4 to 16, as leave a chunk of counts for
  // each workgroup of order_kernel (8192 x 256: 14.0 us with 8 waves, 15.8 with 16), at
  // most two chunks with 16 waves.  Where that is not enough, the order is taken from idx
  // afterwards (65536 x 32: 20.8, in four chunks 21.8; 32768 x 256: 25.5, in two 28.5).
  const bool alone = order && units <= 16 && a.T * a.p.K <= kMaxOrderThreads;
  const int64_t pair_waves = (a.T * a.p.K + kWave - 1) / kWave;
  auto chunks = [&](int64_t waves) { return (units + waves - 1) / waves; };
  auto few = [&](int64_t waves, int64_t most) { return chunks(waves) <= std::min<int64_t>(chunks_that_fit(a.p.E), most); };
  const bool counts = order && !alone && few(16, 2 * kMostOrderGroups);
  const int waves = alone                                 ? (int)std::max<int64_t>({units, pair_waves, 1})
                    : !counts || few(4, kMostOrderGroups) ? 4
                    : few(8, kMostOrderGroups)            ? 8
                                                          : 16;
  const int64_t rows = (int64_t)waves * RPW;
  const int64_t grid = alone ? 1 : chunks(waves);
  a.o.mode = alone ? 2 : counts ? 1 : 0;
  const int groups_log2 = ceil_log2(a.p.n_group);
  const bool full = (EPL * LPR) >> groups_log2 == a.p.E / a.p.n_group && 1 << groups_log2 == a.p.n_group;
  const Shape sh = {ceil_log2(LPR) - groups_log2, count_stride(a.p.E), full};
  // 4 waves' fp64 keys, or 16 waves' 16-bit counts
  const size_t lds = std::max(order_lds(kMaxOrderWaves, a.p.E), (size_t)32 * a.p.E);
  auto f = a.bias                                  ? route_fast_kernel<LT, LPR, EPL, kBiased>
           : a.p.n_group > 1 && a.p.group_top == 2 ? route_fast_kernel<LT, LPR, EPL, kScoredGroups>
                                                   : route_fast_kernel<LT, LPR, EPL, kLogits>;
  f<<<(unsigned)grid, waves * kWave, lds, a.st>>>((const LT*)a.logits, a.T, a.ld, a.bias, a.p, sh, a.idx, a.weights, a.o);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !order || alone) return e;
  if (!counts)
    return launch_expert_order(a.idx, a.T * a.p.K, a.p.K, a.p.E, a.o.group_end, a.o.row_token, a.o.slot, a.o.counts, a.st);
  const OrderPlan op = {(int32_t)grid, rows * a.p.K, (int32_t)rows};  // a row names an expert once
  return launch_order(a.idx, a.T * a.p.K, a.p.K, a.p.E, op, a.o.group_end, a.o.row_token, a.o.slot, a.o.counts, a.st);
}

template <typename LT>
hipError_t route(const RouteArgs& a) {
  const RouteParams& p = a.p;
  // As few lanes as hold the row, since a choice costs a wave the same for one row or four.
  // But few rows of many experts take a wave each, so that a lane has no 16 experts to go
  // through: 256 experts, 256 rows 4.5 against 5.2 us, 4096 rows 6.5 against 7.0 (with the
  // expert order 14.4 against 13.7), 16384 rows 17.9 against 10.2.  (32 experts,
  // 256 rows: 3.4 by a wave each, 3.0 by 16 lanes.)
  if (a.T > 0 && a.T <= kFastRows) {  // its waves read a row before they look whether it is there
    if (holds<LT, 16, 2>(p)) return route_fast<LT, 16, 2>(a);
    if (holds<LT, 16, 4>(p)) return route_fast<LT, 16, 4>(a);
    if (a.T >= kManyRows) {
      if (holds<LT, 16, 16>(p)) return route_fast<LT, 16, 16>(a);
      if (holds<LT, 32, 16>(p)) return route_fast<LT, 32, 16>(a);
    }
    if (holds<LT, 64, 4>(p)) return route_fast<LT, 64, 4>(a);
    if (holds<LT, 64, 16>(p)) return route_fast<LT, 64, 16>(a);
  }
  // groups that do not fit 64 lanes one by one, or very many rows
  if (a.T > 0) {
    const unsigned grid = grid_of((a.T + kRouteWaves - 1) / kRouteWaves);
    route_kernel64<<<grid, kRouteWaves * kWave, (size_t)kRouteWaves * p.E * sizeof(double), a.st>>>(
        (const LT*)a.logits, a.T, a.ld, a.bias, p, a.idx, a.weights);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.o.group_end) return hipSuccess;
  return launch_expert_order(a.idx, a.T * p.K, p.K, p.E, a.o.group_end, a.o.row_token, a.o.slot, a.o.counts, a.st);
}

// ------------------------------------------------------------------ gradient
// With p = s / sum of the chosen s and c the scale:
//   sigmoid                dl_k = c g_k s_k (1 - s_k)
//   sigmoid, renormalised  dl_k = c p_k (g_k - sum_j p_j g_j) (1 - s_k)
//   softmax, renormalised  dl_k = c p_k (g_k - sum_j p_j g_j)
// for the chosen k alone, and for a plain softmax (DENSE) over all experts
//   dl_e = s_e (G_e - sum_j s_j G_j), G_e = c g_e at the chosen, else 0.
// A row is held by LPR lanes, W consecutive experts a lane and piece; the chosen
// experts' values are spread over a row of LDS, and rows are written whole.
// Bound by the launch and HBM: 16384 x 256 fp32 logits of a plain softmax (34.6 MB) take 6.6 us
// one after another, 5.2 TB/s.
template <typename LT, int LPR, int EPL, int W, bool DENSE>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_backward_kernel(const LT* __restrict__ logits, int64_t T,
                                                                           int64_t ld, RouteParams p,
                                                                           const int32_t* __restrict__ idx,
                                                                           const float* __restrict__ dweights,
                                                                           LT* __restrict__ dlogits, int64_t ldd) {
  constexpr int RPW = kWave / LPR, P = EPL / W;
  __shared__ __attribute__((aligned(16))) float lds_row[kRouteWaves * RPW][LPR * EPL];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int sub = lane & (LPR - 1);
  float* row = lds_row[wave * RPW + lane / LPR];
  for (int64_t r0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * RPW; r0 < T; r0 += (int64_t)gridDim.x * kRouteWaves * RPW) {
    const int64_t t = min(r0 + lane / LPR, T - 1);  // rows past the last repeat it
    const LT* l = logits + t * ld;
    int i = -1;
    float g = 0.f, x = 0.f;
    if (sub < p.K) {
      i = idx[t * p.K + sub];
      g = dweights[t * p.K + sub] * p.scale;
    }
    const bool named = i >= 0 && i < p.E;
    x = load_f(l, named ? i : 0);
    const bool in = named && !(x <= (float)kMasked);
    float v[P][W];
    if (DENSE) {
      Raw<LT, W> raw[P];
#pragma unroll
      for (int q = 0; q < P; q++) {
        const int e = (q * LPR + sub) * W;
        raw[q] = load_raw<W, false>(l + (e < p.E ? e : 0));
      }
#pragma unroll
      for (int q = 0; q < P; q++) unpack(raw[q], v[q]);
    }
#pragma unroll
    for (int q = 0; q < P; q++)
#pragma unroll
      for (int j = 0; j < W; j++) row[(q * LPR + sub) * W + j] = 0.f;
    g = in ? g : 0.f;

    float d = g;  // DENSE: G
    if (p.sigmoid) {
      const float ex = exp_f(-fabsf(x)), inv = __builtin_amdgcn_rcpf(1.f + ex);
      const float s = (x >= 0.f ? 1.f : ex) * inv, rest = (x >= 0.f ? ex : 1.f) * inv;  // s and 1 - s
      if (p.renorm) {  // over the largest exp of the row, so that no score underflows
        const float low = fminf(x, 0.f);
        const float m = row_fmax<LPR>(in ? low : -INFINITY);
        const float r = in ? exp_f(low - m) * inv : 0.f;
        const float total = row_sum<LPR>(r);  // all lanes take part
        const float q = in ? r / total : 0.f;
        d = q * (g - row_sum<LPR>(q * g)) * rest;
      } else {
        d = g * s * rest;
      }
    } else if (!DENSE) {
      const float m = row_fmax<LPR>(in ? x : -INFINITY);
      const float r = in ? exp_f(x - m) : 0.f;
      const float total = row_sum<LPR>(r);
      const float q = in ? r / total : 0.f;
      d = q * (g - row_sum<LPR>(q * g));
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
    if (in) row[i] = d;
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();

    float top = 0.f, scale = 0.f, dot = 0.f;
    if (DENSE) {
      top = (float)kMasked;
#pragma unroll
      for (int q = 0; q < P; q++)
#pragma unroll
        for (int j = 0; j < W; j++) {
          const bool there = (q * LPR + sub) * W < p.E && !(v[q][j] <= (float)kMasked);
          v[q][j] = there ? v[q][j] : -INFINITY;
          top = fmaxf(top, v[q][j]);
        }
      top = row_fmax<LPR>(top);
      float total = 0.f;
#pragma unroll
      for (int q = 0; q < P; q++)
#pragma unroll
        for (int j = 0; j < W; j++) {
          v[q][j] = exp_f(v[q][j] - top);  // 0 where masked
          total += v[q][j];
        }
      total = row_sum<LPR>(total);
      scale = total == 0.f ? 0.f : 1.f / total;
      dot = row_sum<LPR>(in ? exp_f(x - top) * g : 0.f) * scale;
    }
    LT* out = dlogits + t * ldd;
#pragma unroll
    for (int q = 0; q < P; q++) {
      const int e = (q * LPR + sub) * W;
      float f[W];
#pragma unroll
      for (int j = 0; j < W; j++) {
        f[j] = row[e + j];
        if (DENSE) f[j] = v[q][j] * scale * (f[j] - dot);
      }
      if (e < p.E && r0 + lane / LPR < T) store_vec<W, false>(out + e, f);
    }
    __threadfence_block();
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename LT, int LPR, int EPL>
void launch_backward(const void* logits, int64_t T, int64_t ld, const RouteParams& p, const int32_t* idx,
                     const float* dweights, void* dlogits, int64_t ldd, hipStream_t st) {
  constexpr int W = EPL < 4 ? EPL : 4;
  const bool dense = !p.sigmoid && !p.renorm;
  auto f = p.E % W == 0 ? dense ? route_backward_kernel<LT, LPR, EPL, W, true>
                                : route_backward_kernel<LT, LPR, EPL, W, false>
           : dense      ? route_backward_kernel<LT, LPR, EPL, 1, true>
                        : route_backward_kernel<LT, LPR, EPL, 1, false>;
  const int64_t rows = kRouteWaves * (kWave / LPR);
  f<<<grid_of((T + rows - 1) / rows), kRouteWaves * kWave, 0, st>>>((const LT*)logits, T, ld, p, idx, dweights, (LT*)dlogits,
                                                                   ldd);
}

// As few lanes as hold the row and the chosen, four experts each or, where rows are many, 16
// (256 experts, 16384 rows 6.6 us with 16 lanes a row, 7.2 with 64, 2048 rows 3.3 and 3.0;
// 32 experts, 16384 rows 3.1 and 5.6, 256 rows 2.5 and 2.6).
template <typename LT>
hipError_t route_backward(const void* logits, int64_t T, int64_t ld, const RouteParams& p, const int32_t* idx,
                          const float* dweights, void* dlogits, int64_t ldd, hipStream_t st) {
  auto f = p.K <= 16 && p.E <= 64                      ? launch_backward<LT, 16, 4>
           : T >= kManyRows && p.K <= 16 && p.E <= 256 ? launch_backward<LT, 16, 16>
           : p.E <= 256                                ? launch_backward<LT, 64, 4>
                                                       : launch_backward<LT, 64, 16>;
  f(logits, T, ld, p, idx, dweights, dlogits, ldd, st);
  return hipGetLastError();
}

// ------------------------------------------------------------------ checks
mxq_status check_config(const char* what, const mxq_route_config* c, int32_t E) {
  MXQ_REQUIRE(c != nullptr, "%s: config is NULL", what);
  MXQ_REQUIRE(E >= 1 && E <= MXQ_MAX_GROUPS, "%s: E must be in [1, %d] (got %d)", what, MXQ_MAX_GROUPS, E);
  MXQ_REQUIRE(c->score == MXQ_SCORE_SOFTMAX || c->score == MXQ_SCORE_SIGMOID, "%s: unknown score %d", what, c->score);
  MXQ_REQUIRE(c->top_k >= 1 && c->top_k <= MXQ_MAX_TOPK && c->top_k <= E,
              "%s: top_k must be in [1, min(E, %d)] (got %d of %d)", what, MXQ_MAX_TOPK, c->top_k, E);
  MXQ_REQUIRE(c->renormalise == 0 || c->renormalise == 1, "%s: renormalise must be 0 or 1", what);
  MXQ_REQUIRE(isfinite(c->scale), "%s: scale must be finite", what);
  return MXQ_OK;
}

mxq_status check_logits(const char* what, const void* p, mxq_dtype dt, int64_t T, int32_t E, int64_t ld) {
  MXQ_REQUIRE(dt == MXQ_DT_F32 || dt == MXQ_DT_BF16, "%s: unknown type %d", what, (int)dt);
  MXQ_REQUIRE(T >= 0, "%s: T must be >= 0", what);
  MXQ_REQUIRE(ld >= E, "%s: row stride (%lld) < E (%d)", what, (long long)ld, E);
  MXQ_REQUIRE(p != nullptr || T == 0, "%s: logits are NULL", what);
  MXQ_REQUIRE(aligned_to(p, dt == MXQ_DT_F32 ? 4 : 2), "%s: logits must be aligned to their type", what);
  return MXQ_OK;
}

bool pairs_ok(int64_t T, int32_t K) { return T <= INT32_MAX / K; }

mxq_status check_order(const char* what, int64_t T, int32_t K, int32_t E, const int32_t* group_end,
                       const int32_t* row_token, const int32_t* slot, const void* workspace, int64_t bytes) {
  MXQ_REQUIRE(group_end && (T == 0 || (row_token && slot)), "%s: group_end, row_token or slot is NULL", what);
  MXQ_REQUIRE(aligned_to(group_end, 4) && aligned_to(row_token, 4) && aligned_to(slot, 4),
              "%s: group_end, row_token and slot must be 4-byte aligned", what);
  const int64_t need = mxq_expert_order_workspace(T, K, E);
  MXQ_REQUIRE(workspace != nullptr && bytes >= need, "%s: the workspace needs %lld bytes", what, (long long)need);
  MXQ_REQUIRE(aligned_to(workspace, 16), "%s: the workspace must be 16-byte aligned", what);
  return MXQ_OK;
}

RouteParams params(const mxq_route_config* c, int32_t E) {
  return {E, c->top_k, c->n_group, c->topk_group, c->group_top, c->renormalise, c->score == MXQ_SCORE_SIGMOID, c->scale};
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

int64_t mxq_expert_order_workspace(int64_t T, int32_t top_k, int32_t E) {
  if (T < 0 || top_k < 1 || top_k > MXQ_MAX_TOPK || E < 1 || E > MXQ_MAX_GROUPS || !pairs_ok(T, top_k)) return 0;
  return (max_chunks(T, top_k, E) * count_stride(E) * (int64_t)sizeof(uint16_t) + 15) / 16 * 16;
}

mxq_status mxq_expert_order(const int32_t* idx, int64_t T, int32_t top_k, int32_t E, int32_t* group_end,
                            int32_t* row_token, int32_t* slot, void* workspace, int64_t workspace_bytes,
                            hipStream_t st) {
  MXQ_REQUIRE(T >= 0, "mxq_expert_order: T must be >= 0");
  MXQ_REQUIRE(top_k >= 1 && top_k <= MXQ_MAX_TOPK, "mxq_expert_order: top_k must be in [1, %d] (got %d)", MXQ_MAX_TOPK,
              top_k);
  MXQ_REQUIRE(E >= 1 && E <= MXQ_MAX_GROUPS, "mxq_expert_order: E must be in [1, %d] (got %d)", MXQ_MAX_GROUPS, E);
  MXQ_REQUIRE(pairs_ok(T, top_k), "mxq_expert_order: T * top_k must be < 2^31");
  MXQ_REQUIRE(idx != nullptr || T == 0, "mxq_expert_order: idx is NULL");
  MXQ_REQUIRE(aligned_to(idx, 4), "mxq_expert_order: idx must be 4-byte aligned");
  const mxq_status s = check_order("mxq_expert_order", T, top_k, E, group_end, row_token, slot, workspace, workspace_bytes);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE_DEVICE();
  return launched(launch_expert_order(idx, T * top_k, top_k, E, group_end, row_token, slot, (uint16_t*)workspace, st),
                  "mxq_expert_order");
}

mxq_status mxq_route(const void* logits, mxq_dtype dt, int64_t T, int32_t E, int64_t ld, const float* bias,
                     const mxq_route_config* cfg, int32_t* idx, float* weights, int32_t* group_end,
                     int32_t* row_token, int32_t* slot, void* workspace, int64_t workspace_bytes,
                     hipStream_t st) {
  mxq_status s = check_config("mxq_route", cfg, E);
  if (s != MXQ_OK) return s;
  s = check_logits("mxq_route", logits, dt, T, E, ld);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(cfg->n_group >= 1 && cfg->n_group <= MXQ_MAX_ROUTE_GROUPS && E % cfg->n_group == 0,
              "mxq_route: n_group must divide E and lie in [1, %d] (got %d)", MXQ_MAX_ROUTE_GROUPS, cfg->n_group);
  MXQ_REQUIRE(cfg->topk_group >= 1 && cfg->topk_group <= cfg->n_group, "mxq_route: topk_group must be in [1, n_group]");
  MXQ_REQUIRE(cfg->group_top == 1 || cfg->group_top == 2, "mxq_route: group_top must be 1 or 2");
  MXQ_REQUIRE(pairs_ok(T, cfg->top_k), "mxq_route: T * top_k must be < 2^31");
  MXQ_REQUIRE(T == 0 || (idx && weights), "mxq_route: idx or weights is NULL");
  MXQ_REQUIRE(aligned_to(idx, 4) && aligned_to(weights, 4) && aligned_to(bias, 4),
              "mxq_route: idx, weights and bias must be 4-byte aligned");
  const bool order = group_end || row_token || slot;
  if (order) {
    s = check_order("mxq_route", T, cfg->top_k, E, group_end, row_token, slot, workspace, workspace_bytes);
    if (s != MXQ_OK) return s;
  }
  MXQ_REQUIRE_DEVICE();
  if (T == 0 && !order) return ok();
  const OrderOut o = {group_end, row_token, slot, (uint16_t*)workspace, 0};
  const RouteArgs a = {logits, T, ld, bias, params(cfg, E), idx, weights, o, st};
  return launched(dt == MXQ_DT_F32 ? route<float>(a) : route<uint16_t>(a), "mxq_route");
}

mxq_status mxq_route_backward(const void* logits, mxq_dtype dt, int64_t T, int32_t E, int64_t ld,
                              const mxq_route_config* cfg, const int32_t* idx, const float* dweights,
                              void* dlogits, int64_t ldd, hipStream_t st) {
  mxq_status s = check_config("mxq_route_backward", cfg, E);
  if (s != MXQ_OK) return s;
  s = check_logits("mxq_route_backward", logits, dt, T, E, ld);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(ldd >= E, "mxq_route_backward: row stride of dlogits (%lld) < E (%d)", (long long)ldd, E);
  MXQ_REQUIRE(T == 0 || (idx && dweights && dlogits), "mxq_route_backward: idx, dweights or dlogits is NULL");
  MXQ_REQUIRE(aligned_to(idx, 4) && aligned_to(dweights, 4), "mxq_route_backward: idx and dweights must be 4-byte aligned");
  MXQ_REQUIRE(aligned_to(dlogits, dt == MXQ_DT_F32 ? 4 : 2), "mxq_route_backward: dlogits must be aligned to their type");
  MXQ_REQUIRE(pairs_ok(T, cfg->top_k), "mxq_route_backward: T * top_k must be < 2^31");
  MXQ_REQUIRE_DEVICE();
  if (T == 0) return ok();
  const RouteParams p = params(cfg, E);
  auto f = dt == MXQ_DT_F32 ? route_backward<float> : route_backward<uint16_t>;
  return launched(f(logits, T, ld, p, idx, dweights, dlogits, ldd, st), "mxq_route_backward");
}

}  // extern "C"
