// The experts' rows back in token order (weighted combine) and its gradient,
// which is also the dispatch of tokens into expert order.
#include "mxq_device.h"
#include "mxq_host.h"

namespace mxq {

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;

// workgroups for `units` units of work, one each while a grid can hold them
// (a grid has fewer than 2^32 threads); the kernels walk the rest
unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 20) ? units : 1 << 20); }

__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(uint16_t* p, int64_t i, float v) {
  p[i] = __builtin_bit_cast(uint16_t, (__bf16)v);  // to nearest even
}

// one workgroup per token
template <typename YT, typename OT>
__global__ __launch_bounds__(kThreads) void combine_kernel(const YT* __restrict__ y, int32_t rows, int64_t ldy,
                                                          const int32_t* __restrict__ slot,
                                                          const float* __restrict__ weights, int32_t K, int64_t H,
                                                          OT* __restrict__ out, int64_t ldo, int64_t T) {
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x)
  for (int64_t h = threadIdx.x; h < H; h += kThreads) {
    float acc = 0.f;
    for (int k = 0; k < K; k++) {
      const int32_t r = slot[t * K + k];
      if (r < 0 || r >= rows) continue;
      const float w = weights ? weights[t * K + k] : 1.f;
      acc += w * load_f(y, r * ldy + h);
    }
    store_f(out, t * ldo + h, acc);
  }
}

// one workgroup per token
template <typename DT, typename YT, typename GT>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const DT* __restrict__ dout, int64_t ldd, const YT* __restrict__ y, int32_t rows, int64_t ldy,
    const int32_t* __restrict__ slot, const float* __restrict__ weights, int32_t K, int64_t H, GT* __restrict__ dy,
    int64_t lddy, float* __restrict__ dweights, int64_t T) {
  __shared__ float part[kThreads / kWave];
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x)
  for (int k = 0; k < K; k++) {
    const int32_t r = slot[t * K + k];
    const bool in = r >= 0 && r < rows;
    const float w = weights ? weights[t * K + k] : 1.f;
    float dot = 0.f;
    if (in)
      for (int64_t h = threadIdx.x; h < H; h += kThreads) {
        const float d = load_f(dout, t * ldd + h);
        if (dy) store_f(dy, r * lddy + h, w * d);
        if (dweights) dot += d * load_f(y, r * ldy + h);
      }
    if (!dweights) continue;
#pragma unroll
    for (int o = 32; o; o >>= 1) dot += __shfl_xor(dot, o);
    if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      float s = 0.f;
      for (int i = 0; i < kThreads / kWave; i++) s += part[i];
      dweights[t * K + k] = s;
    }
    __syncthreads();
  }
}

mxq_status check_rows(const char* what, const char* name, const void* p, mxq_dtype dt, int64_t ld, int64_t H,
                      bool needed) {
  MXQ_REQUIRE(dt == MXQ_DT_F32 || dt == MXQ_DT_BF16, "%s: unknown type %d of %s", what, (int)dt, name);
  MXQ_REQUIRE(p != nullptr || !needed, "%s: %s is NULL", what, name);
  MXQ_REQUIRE(p == nullptr || ld >= H, "%s: row stride of %s (%lld) < H (%lld)", what, name, (long long)ld, (long long)H);
  MXQ_REQUIRE(aligned_to(p, dt == MXQ_DT_F32 ? 4 : 2), "%s: %s must be aligned to its type", what, name);
  return MXQ_OK;
}

mxq_status check_pairs(const char* what, const int32_t* slot, const float* weights, int64_t T, int32_t K, int64_t H,
                       int64_t rows) {
  MXQ_REQUIRE(T >= 0 && T <= INT32_MAX, "%s: T must be in [0, 2^31)", what);
  MXQ_REQUIRE(rows >= 0 && rows <= INT32_MAX, "%s: rows must be in [0, 2^31)", what);
  MXQ_REQUIRE(H >= 1, "%s: H must be >= 1", what);
  MXQ_REQUIRE(K >= 1 && K <= MXQ_MAX_TOPK, "%s: top_k must be in [1, %d] (got %d)", what, MXQ_MAX_TOPK, K);
  MXQ_REQUIRE(slot != nullptr || T == 0, "%s: slot is NULL", what);
  MXQ_REQUIRE(aligned_to(slot, 4) && aligned_to(weights, 4), "%s: slot and weights must be 4-byte aligned", what);
  return MXQ_OK;
}

template <typename YT, typename OT>
hipError_t combine(const void* y, int64_t rows, int64_t ldy, const int32_t* slot, const float* weights, int64_t T,
                   int32_t K, int64_t H, void* out, int64_t ldo, hipStream_t st) {
  combine_kernel<<<grid_of(T), kThreads, 0, st>>>((const YT*)y, (int32_t)rows, ldy, slot, weights, K, H, (OT*)out, ldo, T);
  return hipGetLastError();
}

template <typename DT, typename YT, typename GT>
hipError_t combine_backward(const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* slot,
                            const float* weights, int64_t T, int32_t K, int64_t H, int64_t rows, void* dy,
                            int64_t lddy, float* dweights, hipStream_t st) {
  combine_backward_kernel<<<grid_of(T), kThreads, 0, st>>>((const DT*)dout, ldd, (const YT*)y, (int32_t)rows, ldy, slot,
                                                           weights, K, H, (GT*)dy, lddy, dweights, T);
  return hipGetLastError();
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

mxq_status mxq_combine(const void* y, mxq_dtype ydt, int64_t rows, int64_t ldy, const int32_t* slot,
                       const float* weights, int64_t T, int32_t top_k, int64_t H, void* out, mxq_dtype odt,
                       int64_t ldo, hipStream_t st) {
  mxq_status s = check_pairs("mxq_combine", slot, weights, T, top_k, H, rows);
  if (s != MXQ_OK) return s;
  s = check_rows("mxq_combine", "y", y, ydt, ldy, H, T > 0 && rows > 0);
  if (s != MXQ_OK) return s;
  s = check_rows("mxq_combine", "out", out, odt, ldo, H, T > 0);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE_DEVICE();
  if (T == 0) return ok();
  const bool yf = ydt == MXQ_DT_F32, of = odt == MXQ_DT_F32;
  auto f = yf ? (of ? combine<float, float> : combine<float, uint16_t>)
              : (of ? combine<uint16_t, float> : combine<uint16_t, uint16_t>);
  return launched(f(y, rows, ldy, slot, weights, T, top_k, H, out, ldo, st), "mxq_combine");
}

mxq_status mxq_combine_backward(const void* dout, mxq_dtype dt, int64_t ldd, const void* y, mxq_dtype ydt,
                                int64_t ldy, const int32_t* slot, const float* weights, int64_t T, int32_t top_k,
                                int64_t H, int64_t rows, void* dy, mxq_dtype dydt, int64_t lddy, float* dweights,
                                hipStream_t st) {
  mxq_status s = check_pairs("mxq_combine_backward", slot, weights, T, top_k, H, rows);
  if (s != MXQ_OK) return s;
  s = check_rows("mxq_combine_backward", "dout", dout, dt, ldd, H, T > 0);
  if (s != MXQ_OK) return s;
  s = check_rows("mxq_combine_backward", "y", y, ydt, ldy, H, dweights != nullptr && T > 0 && rows > 0);
  if (s != MXQ_OK) return s;
  s = check_rows("mxq_combine_backward", "dy", dy, dydt, lddy, H, false);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(aligned_to(dweights, 4), "mxq_combine_backward: dweights must be 4-byte aligned");
  MXQ_REQUIRE_DEVICE();
  if (T == 0 || (!dy && !dweights)) return ok();
  const int which = (dt == MXQ_DT_F32) * 4 + (ydt == MXQ_DT_F32) * 2 + (dydt == MXQ_DT_F32);
  typedef uint16_t b;
  decltype(&combine_backward<float, float, float>) const f[8] = {
      combine_backward<b, b, b>,     combine_backward<b, b, float>,     combine_backward<b, float, b>,
      combine_backward<b, float, float>, combine_backward<float, b, b>, combine_backward<float, b, float>,
      combine_backward<float, float, b>, combine_backward<float, float, float>};
  return launched(f[which](dout, ldd, y, ldy, slot, weights, T, top_k, H, rows, dy, lddy, dweights, st),
                  "mxq_combine_backward");
}

}  // extern "C"
