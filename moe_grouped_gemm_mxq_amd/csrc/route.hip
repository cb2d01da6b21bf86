// Routing of tokens to experts: scores, choice and weights; the expert order
// of the chosen pairs; the gradient of the weights.
//
// The choice has to be that of exact arithmetic: two keys of a row that fp32
// cannot tell apart would come out in an order that depends on how exp is
// evaluated.  Keys and group totals are therefore taken in fp64.
#include <math.h>

#include "mxq_device.h"
#include "mxq_host.h"

namespace mxq {

namespace {

constexpr int kWave = 64;
constexpr double kMasked = -3.3895313892515355e38;  // lowest finite bf16: logits at or below it are masked
constexpr double kNanKey = -1e300;                  // a NaN key ranks below every number, above a masked one

struct RouteParams {
  int32_t E, K, n_group, topk_group, group_top, renorm, sigmoid;
  float scale;
};

__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(uint16_t* p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);  // to nearest even
}

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
    const double sum = wave_sum(lane < p.K ? w : 0.0);
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
__global__ __launch_bounds__(kRouteWaves* kWave) void route_kernel(const LT* __restrict__ logits, int64_t T, int64_t ld,
                                                                  const float* __restrict__ bias, RouteParams p,
                                                                  int32_t* __restrict__ idx, float* __restrict__ weights) {
  extern __shared__ double lds_keys[];
  const int wave = threadIdx.x / kWave;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < T; t += (int64_t)gridDim.x * kRouteWaves)
    route_row64(logits + t * ld, bias, p, lds_keys + wave * p.E, idx + t * p.K, weights + t * p.K);
}

// ------------------------------------------------------------------ expert order
// A stable counting sort of the N = T * K pairs by expert.  The pairs are cut
// into chunks; hist_kernel counts each chunk's pairs by expert, order_kernel
// adds up the counts before its chunk and ranks the chunk's pairs segment by
// segment: within a wave by ballots over the bits of the expert, across waves
// by their counts.  No atomics order anything, so the result is always the same.
constexpr int kOrderThreads = 1024, kOrderWaves = kOrderThreads / kWave;
constexpr int kMaxChunks = 256;

struct OrderPlan {
  int chunks;
  int64_t chunk;  // pairs per chunk, a multiple of kOrderThreads
};

OrderPlan order_plan(int64_t N) {
  int64_t per = (N + kMaxChunks - 1) / kMaxChunks;
  per = (per + kOrderThreads - 1) / kOrderThreads * kOrderThreads;
  if (per < kOrderThreads) per = kOrderThreads;
  int64_t c = (N + per - 1) / per;
  return {(int)(c < 1 ? 1 : c), per};
}

__global__ __launch_bounds__(kOrderThreads) void hist_kernel(const int32_t* __restrict__ idx, int64_t N, int64_t chunk,
                                                            int32_t E, int32_t* __restrict__ counts) {
  __shared__ int32_t h[MXQ_MAX_GROUPS];
  const int t = threadIdx.x;
  if (t < E) h[t] = 0;
  __syncthreads();
  const int64_t b = blockIdx.x * chunk, e = min(b + chunk, N);
  for (int64_t i = b + t; i < e; i += kOrderThreads) {
    const int32_t x = idx[i];
    if (x >= 0 && x < E) atomicAdd(&h[x], 1);  // a count: the order does not matter
  }
  __syncthreads();
  if (t < E) counts[(int64_t)blockIdx.x * E + t] = h[t];
}

__global__ __launch_bounds__(kOrderThreads) void order_kernel(const int32_t* __restrict__ idx, int64_t N, int64_t chunk,
                                                             int32_t E, int32_t K, const int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ group_end,
                                                             int32_t* __restrict__ row_token,
                                                             int32_t* __restrict__ slot) {
  __shared__ uint16_t wave_count[kOrderWaves][MXQ_MAX_GROUPS];
  __shared__ int32_t base[MXQ_MAX_GROUPS];
  __shared__ int32_t scan[kOrderWaves];
  const int t = threadIdx.x, lane = t & (kWave - 1), wave = t / kWave;
  // of expert t: pairs in all chunks and in those before this one
  int32_t all = 0, before = 0;
  if (t < E)
    for (int c = 0; c < (int)gridDim.x; c++) {
      const int32_t n = counts[(int64_t)c * E + t];
      all += n;
      if (c < (int)blockIdx.x) before += n;
    }
  int32_t incl = all;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int32_t v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == kWave - 1) scan[wave] = incl;
  __syncthreads();
  int32_t off = 0, total = 0;
  for (int w = 0; w < kOrderWaves; w++) {
    if (w < wave) off += scan[w];
    total += scan[w];
  }
  incl += off;
  if (t < E) {
    base[t] = incl - all + before;
    if (blockIdx.x == 0) group_end[t] = incl;
  }
  const int64_t b = blockIdx.x * chunk, e = min(b + chunk, N);
  for (int64_t s = b; s < e; s += kOrderThreads) {
    for (int i = t; i < kOrderWaves * E; i += kOrderThreads) wave_count[i / E][i % E] = 0;
    __syncthreads();
    const int64_t i = s + t;
    int32_t x = i < e ? idx[i] : -1;
    const bool in = x >= 0 && x < E;
    if (!in) x = E;  // a value of its own
    uint64_t same = ~0ull;
#pragma unroll
    for (int bit = 0; bit < 11; bit++) {
      const bool set = x >> bit & 1;
      const uint64_t m = __ballot(set);
      same &= set ? m : ~m;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) wave_count[wave][x] = (uint16_t)__popcll(same);
    __syncthreads();
    if (t < E) {  // counts -> first rows of the waves
      int32_t run = 0;
      for (int w = 0; w < kOrderWaves; w++) {
        const int32_t n = wave_count[w][t];
        wave_count[w][t] = (uint16_t)run;
        run += n;
      }
      scan[0] = 0;
      all = run;
    }
    __syncthreads();
    if (in) {
      const int32_t row = base[x] + wave_count[wave][x] + rank;
      slot[i] = row;
      row_token[row] = (int32_t)(i / K);
    } else if (i < e) {
      slot[i] = -1;
    }
    __syncthreads();
    if (t < E) base[t] += all;
  }
  for (int64_t i = total + (int64_t)blockIdx.x * kOrderThreads + t; i < N; i += (int64_t)gridDim.x * kOrderThreads)
    row_token[i] = -1;
}

hipError_t launch_expert_order(const int32_t* idx, int64_t N, int32_t K, int32_t E, int32_t* group_end,
                               int32_t* row_token, int32_t* slot, int32_t* counts, hipStream_t st) {
  const OrderPlan op = order_plan(N);
  hist_kernel<<<op.chunks, kOrderThreads, 0, st>>>(idx, N, op.chunk, E, counts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  order_kernel<<<op.chunks, kOrderThreads, 0, st>>>(idx, N, op.chunk, E, K, counts, group_end, row_token, slot);
  return hipGetLastError();
}

// ------------------------------------------------------------------ gradient
// One token by one wave; its row of gradients is gathered in LDS (`row`, E floats).
template <typename LT>
__device__ void route_backward_row(const LT* __restrict__ l, const RouteParams p, const int32_t* __restrict__ idx,
                                   const float* __restrict__ dweights, float* row, LT* __restrict__ out) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int e = lane; e < p.E; e += kWave) row[e] = 0.f;
  int i = -1;
  float g = 0.f, x = 0.f;
  if (lane < p.K) {
    i = idx[lane];
    if (i < 0 || i >= p.E) i = -1;
    if (i >= 0) {
      g = dweights[lane] * p.scale;
      x = load_f(l, i);
      if (x <= (float)kMasked) i = -1;
    }
  }
  const bool in = i >= 0;
  const bool dense = !p.sigmoid && !p.renorm;
  float top = -INFINITY;
  float d = 0.f;
  if (p.sigmoid) {
    const float ex = expf(-fabsf(x));
    const float inv = 1.f / (1.f + ex);
    const float s = in ? (x >= 0 ? inv : ex * inv) : 0.f, s1 = x >= 0 ? ex * inv : inv;  // s and 1 - s
    if (p.renorm) {
      // s of the row over the largest exp, so that no s underflows: s_k / sum s = r_k / sum r
      const float m = in ? fminf(x, 0.f) : -INFINITY;
      float mm = m;
#pragma unroll
      for (int o = 32; o; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
      const float r = in ? expf(m - mm) * inv : 0.f;
      const float sum = wave_sum(r);
      const float q = in ? r / sum : 0.f;
      const float mean = wave_sum(q * g);
      d = q * (g - mean) * s1;
    } else {
      d = g * s * s1;
    }
  } else if (p.renorm) {
    float mm = in ? x : -INFINITY;
#pragma unroll
    for (int o = 32; o; o >>= 1) mm = fmaxf(mm, __shfl_xor(mm, o));
    const float r = in ? expf(x - mm) : 0.f;
    const float sum = wave_sum(r);
    const float q = in ? r / sum : 0.f;
    const float mean = wave_sum(q * g);
    d = q * (g - mean);
  } else {
    d = g;
  }
  __threadfence_block();
  __builtin_amdgcn_wave_barrier();
  if (in) row[i] = d;
  __threadfence_block();
  __builtin_amdgcn_wave_barrier();
  if (!dense) {
    for (int e = lane; e < p.E; e += kWave) store_f(out, e, row[e]);
    return;
  }
  for (int e = lane; e < p.E; e += kWave) {
    const float v = load_f(l, e);
    if (!(v <= (float)kMasked)) top = fmaxf(top, v);
  }
#pragma unroll
  for (int o = 32; o; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  float total = 0.f, dot = 0.f;
  for (int e = lane; e < p.E; e += kWave) {
    const float v = load_f(l, e);
    const float s = v <= (float)kMasked ? 0.f : expf(v - top);
    total += s;
    dot += s * row[e];
  }
  total = wave_sum(total);
  dot = wave_sum(dot) / total;
  for (int e = lane; e < p.E; e += kWave) {
    const float v = load_f(l, e);
    const float s = v <= (float)kMasked ? 0.f : expf(v - top) / total;
    store_f(out, e, v <= (float)kMasked ? 0.f : s * (row[e] - dot));
  }
}

template <typename LT>
__global__ __launch_bounds__(kRouteWaves* kWave) void route_backward_kernel(const LT* __restrict__ logits, int64_t T,
                                                                           int64_t ld, RouteParams p,
                                                                           const int32_t* __restrict__ idx,
                                                                           const float* __restrict__ dweights,
                                                                           LT* __restrict__ dlogits, int64_t ldd) {
  extern __shared__ float lds_row[];
  const int wave = threadIdx.x / kWave;
  float* row = lds_row + wave * p.E;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave; t < T; t += (int64_t)gridDim.x * kRouteWaves)
    route_backward_row(logits + t * ld, p, idx + t * p.K, dweights + t * p.K, row, dlogits + t * ldd);
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
  return ((int64_t)order_plan(T * top_k).chunks * E * 4 + 15) / 16 * 16;
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
  return launched(launch_expert_order(idx, T * top_k, top_k, E, group_end, row_token, slot, (int32_t*)workspace, st),
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
  if (T > 0) {
    const RouteParams p = params(cfg, E);
    const unsigned grid = grid_of((T + kRouteWaves - 1) / kRouteWaves);
    const size_t lds = (size_t)kRouteWaves * E * sizeof(double);
    if (dt == MXQ_DT_F32)
      route_kernel<<<grid, kRouteWaves * kWave, lds, st>>>((const float*)logits, T, ld, bias, p, idx, weights);
    else
      route_kernel<<<grid, kRouteWaves * kWave, lds, st>>>((const uint16_t*)logits, T, ld, bias, p, idx, weights);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return launched(e, "mxq_route");
  }
  if (!order) return ok();
  return launched(launch_expert_order(idx, T * cfg->top_k, cfg->top_k, E, group_end, row_token, slot,
                                      (int32_t*)workspace, st),
                  "mxq_route(order)");
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
  const unsigned grid = grid_of((T + kRouteWaves - 1) / kRouteWaves);
  const size_t lds = (size_t)kRouteWaves * E * sizeof(float);
  if (dt == MXQ_DT_F32)
    route_backward_kernel<<<grid, kRouteWaves * kWave, lds, st>>>((const float*)logits, T, ld, p, idx, dweights,
                                                                 (float*)dlogits, ldd);
  else
    route_backward_kernel<<<grid, kRouteWaves * kWave, lds, st>>>((const uint16_t*)logits, T, ld, p, idx, dweights,
                                                                 (uint16_t*)dlogits, ldd);
  return launched(hipGetLastError(), "mxq_route_backward");
}

}  // extern "C"
