// The experts' rows back in token order (weighted combine) and its gradient,
// which is also the dispatch of tokens into expert order.
//
// Both stream: combine reads each row of y once and writes each token once,
// the gradient reads y and dout and writes dy.  A workgroup takes one token and
// a tile of its columns (the gradient's dot products need the whole token, so
// there it walks the tiles), a thread eight consecutive columns, and the loads
// of up to kRows rows are issued before the first of them is used.
#include "mxq_device.h"
#include "mxq_host.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

constexpr int kWave = 64;
constexpr int kThreads = 256;
constexpr int kTile = 8 * kThreads;
constexpr int kRows = 8;  // rows in flight
#ifndef NTV
#define NTV true
#endif
constexpr bool kNT = NTV;

// workgroups for `units` units of work, one each while a grid can hold them
// (a grid has fewer than 2^32 threads); the kernels walk the rest
unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 23) ? units : 1 << 23); }

// Rows k0 .. k0 + kRows - 1 of a token (uniform over the workgroup); -1: none
struct Rows {
  int32_t row[kRows];
  float w[kRows];
};
__device__ __forceinline__ Rows token_rows(const int32_t* __restrict__ slot, const float* __restrict__ weights, int64_t t,
                                           int K, int k0, int32_t rows) {
  Rows r;
#pragma unroll
  for (int j = 0; j < kRows; j++) {
    r.row[j] = -1;
    r.w[j] = 1.f;
    if (k0 + j < K) {
      const int32_t s = slot[t * K + k0 + j];
      r.row[j] = s < 0 || s >= rows ? -1 : s;
      if (weights) r.w[j] = weights[t * K + k0 + j];
    }
  }
  return r;
}

// Columns of a thread in a tile: kTile / kThreads, in pieces of W consecutive ones, so
// that each load of a wave is one unbroken run: 16 bytes a lane for fp32 (W = 4)
// and for bf16 alone (W = 8), 8 for bf16 beside fp32 (W = 4).
template <typename A, typename B>
constexpr int width() {
  return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4;
}

template <typename YT, typename OT>
__global__ __launch_bounds__(kThreads) void combine_kernel(const YT* __restrict__ y, int32_t rows, int64_t ldy,
                                                          const int32_t* __restrict__ slot,
                                                          const float* __restrict__ weights, int32_t K, int64_t H,
                                                          OT* __restrict__ out, int64_t ldo, int64_t T, uint32_t tiles) {
  constexpr int W = width<YT, OT>(), P = kTile / kThreads / W;
  for (int64_t u = blockIdx.x; u < T * tiles; u += gridDim.x) {
    const int64_t t = u / tiles;
    const int64_t h0 = (u - t * tiles) * kTile + threadIdx.x * W;
    float acc[P][W] = {};
    for (int k0 = 0; k0 < K; k0 += kRows) {
      const Rows r = token_rows(slot, weights, t, K, k0, rows);
      if (h0 + (P - 1) * kThreads * W + W <= H) {
        Raw<YT, W> v[kRows][P];
#pragma unroll
        for (int j = 0; j < kRows; j++)
          if (r.row[j] >= 0)
#pragma unroll
            for (int p = 0; p < P; p++) v[j][p] = load_raw<W, kNT>(y + r.row[j] * ldy + h0 + p * kThreads * W);
#pragma unroll
        for (int j = 0; j < kRows; j++)
          if (r.row[j] >= 0)
#pragma unroll
            for (int p = 0; p < P; p++) {
              float f[W];
              unpack(v[j][p], f);
#pragma unroll
              for (int i = 0; i < W; i++) acc[p][i] += r.w[j] * f[i];
            }
      } else {
#pragma unroll
        for (int p = 0; p < P; p++) {
          const int64_t h = h0 + p * kThreads * W;
          const int n = (int)min((int64_t)W, H - h);
          if (n > 0)
#pragma unroll
            for (int j = 0; j < kRows; j++)
              if (r.row[j] >= 0) {
                float f[W];
                load_some<W>(y + r.row[j] * ldy + h, n, f);
#pragma unroll
                for (int i = 0; i < W; i++) acc[p][i] += r.w[j] * f[i];
              }
        }
      }
    }
#pragma unroll
    for (int p = 0; p < P; p++) {
      const int64_t h = h0 + p * kThreads * W;
      const int n = (int)min((int64_t)W, H - h);
      if (n == W)
        store_vec<W, kNT>(out + t * ldo + h, acc[p]);
      else if (n > 0)
        store_some<W>(out + t * ldo + h, n, acc[p]);
    }
  }
}

// kRows columns of sums over the workgroup; the result is in the first thread
__device__ __forceinline__ void block_sums(float (&s)[kRows], float (*part)[kRows]) {
#pragma unroll
  for (int j = 0; j < kRows; j++)
#pragma unroll
    for (int o = 32; o; o >>= 1) s[j] += __shfl_xor(s[j], o);
  const int wave = threadIdx.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
    for (int j = 0; j < kRows; j++) part[wave][j] = s[j];
}

// DW: with the gradient of the weights, a token per workgroup; else a tile per workgroup
template <typename DT, typename YT, typename GT, bool DW>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const DT* __restrict__ dout, int64_t ldd, const YT* __restrict__ y, int32_t rows, int64_t ldy,
    const int32_t* __restrict__ slot, const float* __restrict__ weights, int32_t K, int64_t H, GT* __restrict__ dy,
    int64_t lddy, float* __restrict__ dweights, int64_t T, uint32_t tiles) {
  __shared__ float part[kThreads / kWave][kRows];
  constexpr int W = width<DT, YT>(), P = kTile / kThreads / W;  // dy's type has no part in the order of the dot products
  const int64_t units = DW ? T : T * tiles;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t t = DW ? u : u / tiles;
    const int64_t h0 = DW ? 0 : (u - t * tiles) * kTile, h1 = DW ? H : min(H, h0 + kTile);
    for (int k0 = 0; k0 < K; k0 += kRows) {
      const Rows r = token_rows(slot, weights, t, K, k0, rows);
      float dot[kRows] = {};
      for (int64_t hb = h0 + threadIdx.x * W; hb < h1; hb += kTile) {
        if (hb + (P - 1) * kThreads * W + W <= H) {
          Raw<DT, W> dr[P];
          Raw<YT, W> v[kRows][P];
#pragma unroll
          for (int p = 0; p < P; p++) dr[p] = load_raw<W, false>(dout + t * ldd + hb + p * kThreads * W);
          if (DW)
#pragma unroll
            for (int j = 0; j < kRows; j++)
              if (r.row[j] >= 0)
#pragma unroll
                for (int p = 0; p < P; p++) v[j][p] = load_raw<W, kNT>(y + r.row[j] * ldy + hb + p * kThreads * W);
#pragma unroll
          for (int j = 0; j < kRows; j++)
            if (r.row[j] >= 0)
#pragma unroll
              for (int p = 0; p < P; p++) {
                float d[W], f[W];
                unpack(dr[p], d);
                if (DW) {
                  unpack(v[j][p], f);
#pragma unroll
                  for (int i = 0; i < W; i++) dot[j] += d[i] * f[i];
                }
                if (dy) {
#pragma unroll
                  for (int i = 0; i < W; i++) d[i] *= r.w[j];
                  store_vec<W, kNT>(dy + r.row[j] * lddy + hb + p * kThreads * W, d);
                }
              }
        } else {
#pragma unroll
          for (int p = 0; p < P; p++) {
            const int64_t h = hb + p * kThreads * W;
            const int n = (int)min((int64_t)W, H - h);
            if (n <= 0) continue;
#pragma unroll
            for (int j = 0; j < kRows; j++)
              if (r.row[j] >= 0) {
                float d[W], f[W];
                load_some<W>(dout + t * ldd + h, n, d);
                if (DW) {
                  load_some<W>(y + r.row[j] * ldy + h, n, f);
#pragma unroll
                  for (int i = 0; i < W; i++) dot[j] += d[i] * f[i];
                }
                if (dy) {
#pragma unroll
                  for (int i = 0; i < W; i++) d[i] *= r.w[j];
                  store_some<W>(dy + r.row[j] * lddy + h, n, d);
                }
              }
          }
        }
      }
      if (DW) {
        block_sums(dot, part);
        __syncthreads();
        if (threadIdx.x < kRows && k0 + (int)threadIdx.x < K) {
          float s = 0.f;
#pragma unroll
          for (int w = 0; w < kThreads / kWave; w++) s += part[w][threadIdx.x];
          dweights[t * K + k0 + threadIdx.x] = s;
        }
        __syncthreads();
      }
    }
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
  MXQ_REQUIRE(H >= 1 && H <= INT32_MAX, "%s: H must be in [1, 2^31)", what);
  MXQ_REQUIRE(K >= 1 && K <= MXQ_MAX_TOPK, "%s: top_k must be in [1, %d] (got %d)", what, MXQ_MAX_TOPK, K);
  MXQ_REQUIRE(slot != nullptr || T == 0, "%s: slot is NULL", what);
  MXQ_REQUIRE(aligned_to(slot, 4) && aligned_to(weights, 4), "%s: slot and weights must be 4-byte aligned", what);
  return MXQ_OK;
}

uint32_t tiles_of(int64_t H) { return (uint32_t)((H + kTile - 1) / kTile); }

template <typename YT, typename OT>
hipError_t combine(const void* y, int64_t rows, int64_t ldy, const int32_t* slot, const float* weights, int64_t T,
                   int32_t K, int64_t H, void* out, int64_t ldo, hipStream_t st) {
  const uint32_t tiles = tiles_of(H);
  combine_kernel<<<grid_of(T * tiles), kThreads, 0, st>>>((const YT*)y, (int32_t)rows, ldy, slot, weights, K, H, (OT*)out,
                                                         ldo, T, tiles);
  return hipGetLastError();
}

template <typename DT, typename YT, typename GT>
hipError_t combine_backward(const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* slot,
                            const float* weights, int64_t T, int32_t K, int64_t H, int64_t rows, void* dy,
                            int64_t lddy, float* dweights, hipStream_t st) {
  const uint32_t tiles = tiles_of(H);
  if (dweights)
    combine_backward_kernel<DT, YT, GT, true><<<grid_of(T), kThreads, 0, st>>>(
        (const DT*)dout, ldd, (const YT*)y, (int32_t)rows, ldy, slot, weights, K, H, (GT*)dy, lddy, dweights, T, tiles);
  else
    combine_backward_kernel<DT, YT, GT, false><<<grid_of(T * tiles), kThreads, 0, st>>>(
        (const DT*)dout, ldd, (const YT*)y, (int32_t)rows, ldy, slot, weights, K, H, (GT*)dy, lddy, dweights, T, tiles);
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
