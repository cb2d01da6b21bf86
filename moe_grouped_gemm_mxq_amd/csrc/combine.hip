// The experts' rows back in token order (weighted combine) and its gradient,
// which is also the dispatch of tokens into expert order.
//
// Both stream and are bound by HBM: combine reads each row of y once and writes
// each token once (16384 x 8 x 4096 fp32 rows to bf16: 377 to 401 us by part, 6.05 to 5.7
// TB/s, where copies reach 6.0), the gradient reads y and dout and writes dy
// (600 to 624 us, 5.6 to 5.4 TB/s, a third of it written).  A workgroup takes one token and
// a tile of its columns (the gradient's dot products need the whole token, so
// there it walks the tiles), a thread eight consecutive columns, and the loads
// of up to kRows rows are issued before the first of them is used.
#include "mxq_device.h"
#include "mxq_host.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

constexpr int kWave = 64;
constexpr int kMaxThreads = 512;
constexpr int kCols = 8;  // columns of a thread in a tile of kCols * blockDim.x
// Rows in flight.  A thread's sums are the same few registers however many rows
// feed them, so combine takes eight; the gradient also writes eight rows then, and
// takes 635 us with eight, 624 with four (16384 x 8 x 4096, fp32 y, on one part).
constexpr int kRows = 8, kRowsBackward = 4;

// workgroups for `units` units of work, one each while a grid can hold them
// (a grid has fewer than 2^32 threads); the kernels walk the rest
unsigned grid_of(int64_t units) { return (unsigned)(units < (1 << 22) ? units : 1 << 22); }

// Rows k0 .. k0 + N - 1 of a token, uniform over the workgroup.  in[j]: pair k0 + j
// exists and names a row; where it does not, row[j] is one that the token reads
// anyway (or row 0), so that the loads need no branch between them: with one, each
// load was waited for before the next.
template <int N>
struct Rows {
  int32_t row[N];
  bool in[N];
  float w[N];
};
template <int N>
__device__ __forceinline__ Rows<N> token_rows(const int32_t* __restrict__ slot, const float* __restrict__ weights,
                                              int64_t t, int K, int k0, int32_t rows) {
  Rows<N> r;
#pragma unroll
  for (int j = 0; j < N; j++) r.row[j] = slot[t * K + min(k0 + j, K - 1)];
#pragma unroll
  for (int j = 0; j < N; j++) r.w[j] = weights ? weights[t * K + min(k0 + j, K - 1)] : 1.f;
  int32_t some = 0;
#pragma unroll
  for (int j = 0; j < N; j++) {
    r.in[j] = k0 + j < K && r.row[j] >= 0 && r.row[j] < rows;
    some = r.in[j] ? r.row[j] : some;
    r.row[j] = some;
  }
  return r;
}

// A thread's columns lie in P = kCols / W pieces of W, piece p at p * blockDim.x * W, so
// that each load of a wave is one unbroken run of 16 bytes a lane for fp32 (W = 4)
// and for bf16 alone (W = 8), 8 for bf16 beside fp32 (W = 4).  (Eight fp32
// columns as two loads 32 bytes apart from lane to lane measured 5.1 against
// 5.9 TB/s.)  A piece that would pass the row's end moves back to it; the columns
// it then shares with its neighbour are written twice with one value and counted
// once.  Rows shorter than a piece take W = 1.
constexpr int width(size_t a, size_t b) { return a == 2 && b == 2 ? 8 : 4; }

// element h of a row whose address is the same for the whole workgroup (H < 2^29: 32-bit byte offsets)
template <typename T>
__device__ __forceinline__ T* at(T* row, uint32_t h) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(row) + h * (uint32_t)sizeof(T));
}

template <typename YT, typename OT, int W, int N>
__global__ __launch_bounds__(kMaxThreads) void combine_kernel(const YT* __restrict__ y, int32_t rows, int64_t ldy,
                                                             const int32_t* __restrict__ slot,
                                                             const float* __restrict__ weights, int32_t K, uint32_t H,
                                                             OT* __restrict__ out, int64_t ldo, int64_t T,
                                                             uint32_t tiles) {
  constexpr int P = kCols / W;
  const uint32_t step = blockDim.x * W;
  for (int64_t u = blockIdx.x; u < T * tiles; u += gridDim.x) {
    const int64_t t = u / tiles;
    const uint32_t h0 = (uint32_t)(u - t * tiles) * (P * step) + threadIdx.x * W;
    uint32_t h[P];
#pragma unroll
    for (int p = 0; p < P; p++) h[p] = min(h0 + p * step, H - W);
    float acc[P][W] = {};
    if (rows > 0)
      for (int k0 = 0; k0 < K; k0 += N) {
        const Rows<N> r = token_rows<N>(slot, weights, t, K, k0, rows);
        Raw<YT, W> v[N][P];
#pragma unroll
        for (int j = 0; j < N; j++)
#pragma unroll
          for (int p = 0; p < P; p++) v[j][p] = load_raw<W, true>(at(y + r.row[j] * ldy, h[p]));
#pragma unroll
        for (int j = 0; j < N; j++)
          if (r.in[j])
#pragma unroll
            for (int p = 0; p < P; p++) {
              float f[W];
              unpack(v[j][p], f);
#pragma unroll
              for (int i = 0; i < W; i++) acc[p][i] += r.w[j] * f[i];
            }
      }
#pragma unroll
    for (int p = 0; p < P; p++)
      if (h0 + p * step < H) store_vec<W, true>(at(out + t * ldo, h[p]), acc[p]);
  }
}

// DW: with the gradient of the weights, whose dot products need a whole token per
// workgroup; else a tile per workgroup.
template <typename DT, typename YT, typename GT, int W, int N, bool DW>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
    const DT* __restrict__ dout, int64_t ldd, const YT* __restrict__ y, int32_t rows, int64_t ldy,
    const int32_t* __restrict__ slot, const float* __restrict__ weights, int32_t K, uint32_t H, GT* __restrict__ dy,
    int64_t lddy, float* __restrict__ dweights, int64_t T, uint32_t tiles) {
  constexpr int P = kCols / W;
  __shared__ float part[kMaxThreads / kWave][N];
  const uint32_t step = blockDim.x * W;
  const int64_t units = DW ? T : T * tiles;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t t = DW ? u : u / tiles;
    const uint32_t first = DW ? 0 : (uint32_t)(u - t * tiles) * (P * step), last = DW ? H : min(H, first + P * step);
    for (int k0 = 0; k0 < K; k0 += N) {
      const Rows<N> r = token_rows<N>(slot, weights, t, K, k0, rows);
      float dot[N] = {};
      if (rows > 0)
      for (uint32_t h0 = first + threadIdx.x * W; h0 < last; h0 += P * step) {
        uint32_t h[P];
#pragma unroll
        for (int p = 0; p < P; p++) h[p] = min(h0 + p * step, H - W);
        Raw<DT, W> dr[P];
        Raw<YT, W> v[N][P];
#pragma unroll
        for (int p = 0; p < P; p++) dr[p] = load_raw<W, false>(at(dout + t * ldd, h[p]));
        if (DW)
#pragma unroll
          for (int j = 0; j < N; j++)
#pragma unroll
            for (int p = 0; p < P; p++) v[j][p] = load_raw<W, true>(at(y + r.row[j] * ldy, h[p]));
        float d[P][W];
#pragma unroll
        for (int p = 0; p < P; p++) unpack(dr[p], d[p]);
#pragma unroll
        for (int j = 0; j < N; j++)
          if (r.in[j])
#pragma unroll
            for (int p = 0; p < P; p++) {
              float f[W];
              if (DW) {
                unpack(v[j][p], f);
#pragma unroll
                for (int i = 0; i < W; i++)
                  if (h[p] + i >= h0 + p * step) dot[j] += d[p][i] * f[i];
              }
              if (dy && h0 + p * step < H) {
#pragma unroll
                for (int i = 0; i < W; i++) f[i] = d[p][i] * r.w[j];
                store_vec<W, true>(at(dy + r.row[j] * lddy, h[p]), f);
              }
            }
      }
      if (DW) {  // sums over the workgroup, always in the same order
#pragma unroll
        for (int j = 0; j < N; j++)
#pragma unroll
          for (int o = 32; o; o >>= 1) dot[j] += __shfl_xor(dot[j], o);
        if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
          for (int j = 0; j < N; j++) part[threadIdx.x / kWave][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < N && k0 + (int)threadIdx.x < K) {
          float s = 0.f;
          for (int w = 0; w < (int)blockDim.x / kWave; w++) s += part[w][threadIdx.x];
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
  MXQ_REQUIRE(H >= 1 && H < (1 << 29), "%s: H must be in [1, 2^29)", what);
  MXQ_REQUIRE(K >= 1 && K <= MXQ_MAX_TOPK, "%s: top_k must be in [1, %d] (got %d)", what, MXQ_MAX_TOPK, K);
  MXQ_REQUIRE(slot != nullptr || T == 0, "%s: slot is NULL", what);
  MXQ_REQUIRE(aligned_to(slot, 4) && aligned_to(weights, 4), "%s: slot and weights must be 4-byte aligned", what);
  return MXQ_OK;
}

// Tiles of a row and threads of a workgroup.  As few tiles as up to 512 threads
// allow (16384 x 8 x 4096 fp32 rows, 512 threads against 256 and two tiles: the gradient
// 624 against 649 us, combine 401 against 399), then as few whole waves as the
// tiles need, so that most threads have all their columns inside the row.  Few
// tokens: half as large, to reach more CUs.
struct Shape {
  unsigned threads;
  uint32_t tiles;
};
Shape shape_of(int64_t T, int64_t H) {
  const int64_t most = T >= 256 ? kMaxThreads : kMaxThreads / 2;
  const int64_t tiles = (H + most * kCols - 1) / (most * kCols);
  const int64_t waves = (H + tiles * kWave * kCols - 1) / (tiles * kWave * kCols);
  return {(unsigned)waves * kWave, (uint32_t)tiles};
}

// The K rows in as few passes of at most `most` as hold them, and those of one size: rows that
// a pass lacks are loads of the last one again.  8192 tokens of 4096 fp32 columns: one row in
// a pass of one 35 us (the gradient 47), in a pass of two 43 (61); five in the
// gradient in passes of three 201, of four 224.
int rows_at_a_time(int32_t K, int most) {
  const int passes = (K + most - 1) / most;
  return (K + passes - 1) / passes;
}

template <typename YT, typename OT>
hipError_t combine(const void* y, int64_t rows, int64_t ldy, const int32_t* slot, const float* weights, int64_t T,
                   int32_t K, int64_t H, void* out, int64_t ldo, hipStream_t st) {
  const Shape s = shape_of(T, H);
  constexpr int W = width(sizeof(YT), sizeof(OT));
  const int n = rows_at_a_time(K, kRows);
  auto f = H < W    ? combine_kernel<YT, OT, 1, 2>
           : n == 1 ? combine_kernel<YT, OT, W, 1>
           : n == 2 ? combine_kernel<YT, OT, W, 2>
           : n <= 4 ? combine_kernel<YT, OT, W, 4>
           : n <= 6 ? combine_kernel<YT, OT, W, 6>
                    : combine_kernel<YT, OT, W, kRows>;
  f<<<grid_of(T * s.tiles), s.threads, 0, st>>>((const YT*)y, (int32_t)rows, ldy, slot, weights, K, (uint32_t)H, (OT*)out,
                                                ldo, T, s.tiles);
  return hipGetLastError();
}

template <typename DT, typename YT, typename GT>
hipError_t combine_backward(const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* slot,
                            const float* weights, int64_t T, int32_t K, int64_t H, int64_t rows, void* dy,
                            int64_t lddy, float* dweights, hipStream_t st) {
  const Shape s = shape_of(T, H);
  // dy's type has no part in W, hence none in the order of the dot products
  constexpr int W = width(sizeof(DT), sizeof(YT));
  const int n = rows_at_a_time(K, kRowsBackward);
  auto f = dweights ? (H < W    ? combine_backward_kernel<DT, YT, GT, 1, 2, true>
                       : n == 1 ? combine_backward_kernel<DT, YT, GT, W, 1, true>
                       : n == 2 ? combine_backward_kernel<DT, YT, GT, W, 2, true>
                       : n == 3 ? combine_backward_kernel<DT, YT, GT, W, 3, true>
                                : combine_backward_kernel<DT, YT, GT, W, kRowsBackward, true>)
                    : (H < W ? combine_backward_kernel<DT, YT, GT, 1, kRowsBackward, false>
                             : combine_backward_kernel<DT, YT, GT, W, kRowsBackward, false>);
  f<<<grid_of(dweights ? T : T * s.tiles), s.threads, 0, st>>>((const DT*)dout, ldd, (const YT*)y, (int32_t)rows, ldy, slot,
                                                              weights, K, (uint32_t)H, (GT*)dy, lddy, dweights, T, s.tiles);
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
