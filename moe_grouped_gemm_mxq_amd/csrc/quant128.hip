// FP8 (E4M3) quantisation with one fp32 scale for every block of 128: blocks of
// 1 x 128 along the reduction axis (activations, gradients) or of 128 x 128
// (weights), of a matrix, of its transpose, or of both from one read; the
// transposed copy may restart its blocks with each group of rows.
//
// With amax the largest magnitude of the block (no less than 2^-100, so that
// scales and their reciprocals stay normal):  scale = amax / 448,
// code = e4m3(448 x / amax) to nearest even.  The quotient is (7/8 x) / (amax / 512):
// a bf16 x times 7/8 and amax / 512 are exact, y0 = 7/8 x * r with r the rounded
// 512 / amax is off by a few units of the last place, and one step
// y = y0 + (7/8 x - y0 amax / 512) * r gives the correctly rounded quotient, which
// for bf16 x has the exact quotient's E4M3 rounding (a quotient of an 11-bit and
// an 8-bit number that is not half way between two codes is at least 2^-14 away).
// The division would cost about ten instructions an element where this takes four.
//
// Both kernels stream and are bound by HBM: 131072 x 4096 bf16 both ways, grouped, 0.43 ms (2.2 GB at 5.1 TB/s; 0.78 with
// the elements held as fp32), 32 matrices 7168 x 4096 both ways in 128 x 128 blocks 0.72 ms (3.8 GB at 5.2 TB/s); rows
// alone 131072 x 7168 0.53 ms from bf16, 0.94 from fp32 (2.8 and 4.7 GB at 5.3 and 5.0 TB/s).  A copy of 2 GB runs at
// 4.9-6.0 TB/s.
#include "mxq_device.h"
#include "mxq_groups.h"
#include "mxq_host.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

constexpr int kB = 128;          // block
constexpr int kThreads = 256;
constexpr int kLanes = 16;       // lanes of a row's block, eight elements each
constexpr float kMaxCode = 448.f;
constexpr uint32_t kAmaxFloor = 0x0D800000u;  // 2^-100
constexpr uint32_t kInf = 0x7F800000u;
constexpr int64_t kMaxGrid = (1 << 24) - 1;  // workgroups of a launch: a grid has fewer than 2^32 threads

// Eight consecutive elements as they lie in memory, zero from the n-th on.
template <typename T>
struct Eight;
template <>
struct Eight<uint16_t> {
  u32x4 a;
  __device__ __forceinline__ float at(int j) const { return __uint_as_float((j & 1) ? a[j >> 1] & 0xFFFF0000u : a[j >> 1] << 16); }
};
template <>
struct Eight<float> {
  u32x4 a, b;
  __device__ __forceinline__ float at(int j) const { return __uint_as_float(j < 4 ? a[j & 3] : b[j & 3]); }
};
__device__ __forceinline__ Eight<float> load8(const float* p, int n) {
  Eight<float> v;
  if (n >= 8) {
    v.a = load_raw<4, false>(p).a;
    v.b = load_raw<4, false>(p + 4).a;
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v.a[j] = j < n ? __float_as_uint(p[j]) : 0u;
      v.b[j] = j + 4 < n ? __float_as_uint(p[j + 4]) : 0u;
    }
  }
  return v;
}
__device__ __forceinline__ Eight<uint16_t> load8(const uint16_t* p, int n) {
  Eight<uint16_t> v;
  if (n >= 8) {
    v.a = load_raw<8, false>(p).a;
  } else {
#pragma unroll
    for (int j = 0; j < 4; j++)
      v.a[j] = (2 * j < n ? (uint32_t)p[2 * j] : 0u) | (2 * j + 1 < n ? (uint32_t)p[2 * j + 1] << 16 : 0u);
  }
  return v;
}

// Magnitudes as integers, which order them with NaN above infinity.  Of eight
// columns: their largest so far, two to a register for bf16.
template <typename T>
struct Largest;
template <>
struct Largest<float> {
  uint32_t m[8];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = 0;
  }
  __device__ __forceinline__ void take(const Eight<float>& v) {
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = max(m[j], __float_as_uint(v.at(j)) & 0x7FFFFFFFu);
  }
  __device__ __forceinline__ void fold(int lanes) {  // with those of the lane `lanes` away
#pragma unroll
    for (int j = 0; j < 8; j++) m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], lanes));
  }
  __device__ __forceinline__ uint32_t of(int j) const { return m[j]; }
  __device__ __forceinline__ uint32_t all() const {
    return max(max(max(m[0], m[1]), max(m[2], m[3])), max(max(m[4], m[5]), max(m[6], m[7])));
  }
};
template <>
struct Largest<uint16_t> {
  uint32_t m[4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int j = 0; j < 4; j++) m[j] = 0;
  }
  __device__ __forceinline__ void take(const Eight<uint16_t>& v) {
#pragma unroll
    for (int j = 0; j < 4; j++) m[j] = pkmax_u16(m[j], v.a[j] & 0x7FFF7FFFu);
  }
  __device__ __forceinline__ void fold(int lanes) {
#pragma unroll
    for (int j = 0; j < 4; j++) m[j] = pkmax_u16(m[j], (uint32_t)__shfl_xor((int)m[j], lanes));
  }
  __device__ __forceinline__ uint32_t of(int j) const { return (j & 1) ? m[j >> 1] & 0xFFFF0000u : m[j >> 1] << 16; }
  __device__ __forceinline__ uint32_t all() const { return hmax_u16x2(pkmax_u16(pkmax_u16(m[0], m[1]), pkmax_u16(m[2], m[3]))) << 16; }
};
template <typename T>
__device__ __forceinline__ uint32_t largest_of(const Eight<T>& v) {
  Largest<T> l;
  l.clear();
  l.take(v);
  return l.all();
}

// largest of 16 lanes of a DPP row
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = max(v, dpp_xor1(v));
  v = max(v, dpp_xor2(v));
  v = max(v, dpp_half_mirror(v));
  return max(v, dpp_mirror(v));
}

// What a block's elements are divided by: d = amax / 512 and its reciprocal, both
// rounded to nearest.  With an infinite amax (r = 0) the step must not see d: the
// finite elements' quotients are 0 then, and the infinities' 0 x inf, a NaN.
struct Divisor {
  float amax, d, r;
  __device__ __forceinline__ explicit Divisor(uint32_t m) {
    amax = __uint_as_float(max(m, kAmaxFloor));
    const float whole = amax * 0x1p-9f;
    r = 1.f / whole;
    d = m >= kInf ? 0.f : whole;
  }
  __device__ __forceinline__ float of(float x) const {
    const float xs = x * 0.875f;
    const float y0 = xs * r;
    const float y = __builtin_fmaf(__builtin_fmaf(-y0, d, xs), r, y0);
    return __builtin_copysignf(y, x);  // (the step loses a zero's sign)
  }
  __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float e) const {
    const int v = __builtin_amdgcn_cvt_pk_fp8_f32(of(a), of(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(of(c), of(e), v, true);
  }
  template <typename T>
  __device__ __forceinline__ uint2 codes8(const Eight<T>& v) const {
    return make_uint2(codes4(v.at(0), v.at(1), v.at(2), v.at(3)), codes4(v.at(4), v.at(5), v.at(6), v.at(7)));
  }
};

// Row copy with 1 x 128 blocks.  16 lanes take a block; the workgroup's 16
// groups take 16 rows, so that their scales, which lie next to each other
// (scales[block][row]), are written together.
constexpr int kPerChunk = 4;  // blocks of a row that a workgroup takes
template <typename T>
__global__ __launch_bounds__(kThreads) void rows_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                        int64_t x_stride, uint8_t* __restrict__ q,
                                                        float* __restrict__ s, int64_t first, int64_t chunks) {
  const int64_t Cb = (C + kB - 1) / kB, Cp = Cb * kB;
  const int64_t bid = first + blockIdx.x, rt = bid / chunks, chunk = bid - rt * chunks;
  const int64_t row = rt * 16 + threadIdx.x / kLanes;
  if (row >= R) return;
  const int c = (threadIdx.x % kLanes) * 8;
  const T* xr = x + blockIdx.y * x_stride + row * ldx;
  uint8_t* qr = q + ((int64_t)blockIdx.y * R + row) * Cp;
  float* sr = s + (int64_t)blockIdx.y * Cb * R + row;
  const int64_t last = min((chunk + 1) * kPerChunk, Cb);
  for (int64_t b = chunk * kPerChunk; b < last; b++) {
    const int64_t col = b * kB + c;
    const Eight<T> v = load8(xr + col, (int)min<int64_t>(C - col, 8));
    const Divisor by(max16(largest_of(v)));
    *reinterpret_cast<uint2*>(qr + col) = by.codes8(v);
    if (c == 0) sr[b * R] = by.amax / kMaxCode;
  }
}

// One 128 x 128 tile of x: any of the copies from one read.  Thread (i, c) holds
// rows 8i .. 8i+7 and columns 8c .. 8c+7 of the tile, so a row's block is 16
// lanes, and a column's codes come in runs of eight, which go through LDS
// ([column][16 runs], run i of column 8c + j at i ^ c: sixteen lanes with one i
// write to all banks) into whole 128-byte lines of the transpose.
template <typename T, bool TILE128, bool ROW, bool COLT, bool GROUPED>
__global__ __launch_bounds__(kThreads) void tile_kernel(const T* __restrict__ x, int64_t R, int64_t C, int64_t ldx,
                                                        int64_t x_stride, const int32_t* __restrict__ group_end,
                                                        int G, int64_t ldq, uint8_t* __restrict__ q_row,
                                                        float* __restrict__ s_row, uint8_t* __restrict__ q_colT,
                                                        float* __restrict__ s_colT, int64_t first, int64_t tiles_c) {
  __shared__ uint2 turned[COLT ? kB * 16 : 1];
  __shared__ uint32_t part[4][kB];
  const int t = threadIdx.x, wave = t >> 6;
  const int c = t & 15, i = t >> 4;
  const int64_t bid = first + blockIdx.x, rt = bid / tiles_c, ct = bid - rt * tiles_c;
  const int64_t Cb = tiles_c, Cp = Cb * kB;
  const int64_t Rb = (R + kB - 1) / kB;
  int64_t row0 = rt * kB, out0 = rt * kB;  // first row, and its place along the transpose's rows
  int64_t rows = R - row0;
  bool turn = COLT;
  if constexpr (GROUPED) {
    GroupUnit u;
    if (find_group_unit<kB>(group_end, G, R, rt, u)) {
      row0 = u.start + (int64_t)u.local * kB;
      rows = u.size - (int64_t)u.local * kB;
      out0 = (u.before + u.local) * kB;
      turn = out0 + kB <= ldq;
    } else {  // rows past the last group: in the row copy alone
      if constexpr (!ROW) return;
      turn = false;
      row0 = min(max((int64_t)group_end[G - 1], (int64_t)0), R) + (rt - u.before) * kB;
      rows = R - row0;
      if (rows <= 0) return;
    }
  }
  const int nrows = (int)min<int64_t>(rows, kB);
  const int64_t col0 = ct * kB;
  const int ncols = (int)min<int64_t>(C - col0, kB);
  x += (int64_t)blockIdx.y * x_stride;

  Eight<T> v[8];
  const int n = min(max(ncols - 8 * c, 0), 8);
  const T* xp = x + row0 * ldx + col0 + 8 * c;
#pragma unroll
  for (int p = 0; p < 8; p++) v[p] = load8(xp + (int64_t)(8 * i + p) * ldx, 8 * i + p < nrows ? n : 0);

  Largest<T> cm;  // of the thread's columns
  cm.clear();
#pragma unroll
  for (int p = 0; p < 8; p++) cm.take(v[p]);
  uint32_t tile_max = 0;
  if constexpr (TILE128) {
    uint32_t m = max16(cm.all());
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if ((t & 63) == 0) part[wave][0] = m;
    __syncthreads();
    tile_max = max(max(part[0][0], part[1][0]), max(part[2][0], part[3][0]));
    if (t == 0) {
      const float scale = __uint_as_float(max(tile_max, kAmaxFloor)) / kMaxCode;
      if constexpr (ROW) s_row[((int64_t)blockIdx.y * Cb + ct) * Rb + rt] = scale;
      if constexpr (COLT) s_colT[((int64_t)blockIdx.y * Rb + rt) * Cb + ct] = scale;
    }
  } else if constexpr (COLT) {
    cm.fold(16);
    cm.fold(32);
    if ((t & 63) < 16) {
#pragma unroll
      for (int j = 0; j < 8; j++) part[wave][8 * c + j] = cm.of(j);
    }
  }

  uint2 code[TILE128 ? 8 : 1];
  if constexpr (ROW || TILE128) {
    const Divisor tile_by(tile_max);
    uint8_t* qp = q_row + ((int64_t)blockIdx.y * R + row0) * Cp + col0 + 8 * c;
#pragma unroll
    for (int p = 0; p < 8; p++) {
      const int r = 8 * i + p;
      const Divisor by = TILE128 ? tile_by : Divisor(max16(largest_of(v[p])));
      const uint2 w = by.codes8(v[p]);
      if constexpr (TILE128) code[p] = w;  // the same codes both ways
      if (ROW && r < nrows) {
        *reinterpret_cast<uint2*>(qp + (int64_t)r * Cp) = w;
        if (!TILE128 && c == 0) s_row[((int64_t)blockIdx.y * Cb + ct) * R + row0 + r] = by.amax / kMaxCode;
      }
    }
  }
  if constexpr (COLT) {
    const int64_t Rp = GROUPED ? ldq : Rb * kB;
    if constexpr (!TILE128) __syncthreads();  // the waves' columns are in
#pragma unroll
    for (int j = 0; j < 8; j++) {
      uint2 w;
      if constexpr (TILE128) {  // byte j of the rows' codes
        const uint32_t sel = (uint32_t)(j & 3);
        auto two = [&](int p) {
          const uint32_t a = j < 4 ? code[p].x : code[p].y, b = j < 4 ? code[p + 1].x : code[p + 1].y;
          return __builtin_amdgcn_perm(b, a, 0x0c0c0000u | sel | ((4u + sel) << 8));
        };
        w = make_uint2(two(0) | (two(2) << 16), two(4) | (two(6) << 16));
      } else {
        const int k = 8 * c + j;
        const Divisor by(max(max(part[0][k], part[1][k]), max(part[2][k], part[3][k])));
        w = make_uint2(by.codes4(v[0].at(j), v[1].at(j), v[2].at(j), v[3].at(j)),
                       by.codes4(v[4].at(j), v[5].at(j), v[6].at(j), v[7].at(j)));
      }
      turned[(8 * c + j) * 16 + (i ^ c)] = w;
    }
    __syncthreads();
    if (!turn) return;
    uint8_t* qp = q_colT + (int64_t)blockIdx.y * C * Rp + out0;
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const int col = 32 * k + (t >> 3), pair = t & 7;
      const int cc = col >> 3;
      const uint2 a = turned[col * 16 + ((2 * pair) ^ cc)], b = turned[col * 16 + ((2 * pair + 1) ^ cc)];
      if (col < ncols)
        *reinterpret_cast<uint4*>(qp + (col0 + col) * Rp + 16 * pair) = make_uint4(a.x, a.y, b.x, b.y);
    }
    if constexpr (!TILE128) {
      if (t < ncols) {
        const uint32_t m = max(max(part[0][t], part[1][t]), max(part[2][t], part[3][t]));
        s_colT[((int64_t)blockIdx.y * (Rp / kB) + out0 / kB) * C + col0 + t] = __uint_as_float(max(m, kAmaxFloor)) / kMaxCode;
      }
    }
  }
}

struct Args {
  int64_t batch, R, C, ldx, x_stride;
  const int32_t* group_end;
  int G;
  int64_t ldq;
  uint8_t* q_row;
  float* s_row;
  uint8_t* q_colT;
  float* s_colT;
};

template <typename T, bool TILE128, bool ROW, bool COLT>
void launch_tile(const T* x, const Args& a, dim3 grid, int64_t first, int64_t tiles_c, hipStream_t st) {
  if constexpr (!TILE128 && COLT) {
    if (a.group_end) {
      tile_kernel<T, TILE128, ROW, COLT, true><<<grid, kThreads, 0, st>>>(x, a.R, a.C, a.ldx, a.x_stride, a.group_end, a.G,
                                                                          a.ldq, a.q_row, a.s_row, a.q_colT, a.s_colT, first, tiles_c);
      return;
    }
  }
  tile_kernel<T, TILE128, ROW, COLT, false><<<grid, kThreads, 0, st>>>(x, a.R, a.C, a.ldx, a.x_stride, nullptr, 0, 0,
                                                                       a.q_row, a.s_row, a.q_colT, a.s_colT, first, tiles_c);
}

template <typename T>
hipError_t launch(const T* x, int tile, bool row, bool col, const Args& a, hipStream_t st) {
  const int64_t Cb = (a.C + kB - 1) / kB, chunks = (Cb + kPerChunk - 1) / kPerChunk;
  const bool by_rows = tile == 1 && !col;
  const int64_t all = by_rows ? (a.R + 15) / 16 * chunks : ((a.R + kB - 1) / kB + (a.group_end ? a.G + 1 : 0)) * Cb;
  for (int64_t first = 0; first < all; first += kMaxGrid) {
    const dim3 grid((unsigned)(all - first < kMaxGrid ? all - first : kMaxGrid), (unsigned)a.batch);
    if (by_rows)
      rows_kernel<T><<<grid, kThreads, 0, st>>>(x, a.R, a.C, a.ldx, a.x_stride, a.q_row, a.s_row, first, chunks);
    else if (tile == 1 && row)
      launch_tile<T, false, true, true>(x, a, grid, first, Cb, st);
    else if (tile == 1)
      launch_tile<T, false, false, true>(x, a, grid, first, Cb, st);
    else if (row && col)
      launch_tile<T, true, true, true>(x, a, grid, first, Cb, st);
    else if (row)
      launch_tile<T, true, true, false>(x, a, grid, first, Cb, st);
    else
      launch_tile<T, true, false, true>(x, a, grid, first, Cb, st);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

hipError_t launch_any(const void* x, mxq_dtype dt, int tile, bool row, bool col, const Args& a, hipStream_t st) {
  if (a.R == 0) return hipSuccess;
  if (dt == MXQ_DT_F32) return launch(static_cast<const float*>(x), tile, row, col, a, st);
  return launch(static_cast<const uint16_t*>(x), tile, row, col, a, st);
}

mxq_status check(const char* who, const void* x, mxq_dtype dt, int64_t R, int64_t C, int64_t ldx, int axis_mask,
                 const Args& a) {
  MXQ_REQUIRE(dt == MXQ_DT_F32 || dt == MXQ_DT_BF16, "%s: unknown type %d", who, (int)dt);
  MXQ_REQUIRE(R >= 0 && R <= INT32_MAX, "%s: the rows must be in [0, 2^31) (got %lld)", who, (long long)R);
  MXQ_REQUIRE(C >= 1 && C <= INT32_MAX - kB, "%s: the columns must be in [1, 2^31 - 128) (got %lld)", who, (long long)C);
  MXQ_REQUIRE(ldx >= C, "%s: ldx (%lld) < C (%lld)", who, (long long)ldx, (long long)C);
  MXQ_REQUIRE(axis_mask >= 1 && axis_mask <= 3, "%s: axis_mask must be ROW, COLT or ROW|COLT", who);
  if (R == 0 || a.batch == 0) return MXQ_OK;
  const bool row = axis_mask & MXQ_AXIS_ROW, col = axis_mask & MXQ_AXIS_COLT;
  MXQ_REQUIRE(x != nullptr, "%s: x is NULL", who);
  MXQ_REQUIRE(!row || (a.q_row && a.s_row), "%s: row outputs are NULL", who);
  MXQ_REQUIRE(!col || (a.q_colT && a.s_colT), "%s: colT outputs are NULL", who);
  MXQ_REQUIRE(aligned_to(x, dt == MXQ_DT_F32 ? 4 : 2), "%s: x must be aligned to its elements", who);
  MXQ_REQUIRE((!row || aligned_to(a.q_row, 16)) && (!col || aligned_to(a.q_colT, 16)),
              "%s: code outputs must be 16-byte aligned", who);
  MXQ_REQUIRE((!row || aligned_to(a.s_row, 4)) && (!col || aligned_to(a.s_colT, 4)),
              "%s: scale outputs must be 4-byte aligned", who);
  return MXQ_OK;
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

int64_t mxq_grouped128_cols_max(int64_t T, int32_t G) {
  if (T < 0 || G < 0 || T > INT32_MAX) return 0;
  return ((T + 127 * (int64_t)G + kB - 1) / kB | 1) * kB;
}

mxq_status mxq_quantize128(const void* x, mxq_dtype dt, int64_t batch, int64_t R, int64_t C, int64_t ldx,
                           int64_t x_stride, int tile, int axis_mask, uint8_t* q_row, float* s_row, uint8_t* q_colT,
                           float* s_colT, hipStream_t st) {
  const Args a{batch, R, C, ldx, x_stride, nullptr, 0, 0, q_row, s_row, q_colT, s_colT};
  MXQ_REQUIRE(tile == 1 || tile == 128, "mxq_quantize128: tile must be 1 or 128 (got %d)", tile);
  MXQ_REQUIRE(batch >= 0 && batch <= 65535, "mxq_quantize128: batch must be in [0, 65535] (got %lld)", (long long)batch);
  const mxq_status s = check("mxq_quantize128", x, dt, R, C, ldx, axis_mask, a);
  if (s != MXQ_OK) return s;
  // (R - 1) ldx + C may be past 64 bits
  MXQ_REQUIRE(batch <= 1 || R == 0 || (x_stride >= C && (R == 1 || (x_stride - C) / (R - 1) >= ldx)),
              "mxq_quantize128: x_stride (%lld) smaller than one matrix", (long long)x_stride);
  MXQ_REQUIRE_DEVICE();
  if (batch == 0) return ok();
  return launched(launch_any(x, dt, tile, axis_mask & MXQ_AXIS_ROW, axis_mask & MXQ_AXIS_COLT, a, st), "mxq_quantize128");
}

mxq_status mxq_quantize128_grouped(const void* x, mxq_dtype dt, int64_t T, int64_t C, int64_t ldx,
                                   const int32_t* group_end, int32_t G, int64_t ldq, int axis_mask, uint8_t* q_row,
                                   float* s_row, uint8_t* q_colT, float* s_colT, hipStream_t st) {
  const bool col = axis_mask & MXQ_AXIS_COLT;
  const Args a{1, T, C, ldx, 0, col ? group_end : nullptr, G, ldq, q_row, s_row, q_colT, s_colT};
  const mxq_status s = check("mxq_quantize128_grouped", x, dt, T, C, ldx, axis_mask, a);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(group_end != nullptr && aligned_to(group_end, 4), "mxq_quantize128_grouped: group_end must be 4-byte aligned, not NULL");
  MXQ_REQUIRE(G >= 1 && G <= MXQ_MAX_GROUPS, "mxq_quantize128_grouped: G must be in [1, %d] (got %d)", MXQ_MAX_GROUPS, G);
  MXQ_REQUIRE(!col || (ldq >= kB && ldq % kB == 0), "mxq_quantize128_grouped: ldq must be a positive multiple of 128");
  MXQ_REQUIRE_DEVICE();
  return launched(launch_any(x, dt, 1, axis_mask & MXQ_AXIS_ROW, col, a, st), "mxq_quantize128_grouped");
}

}  // extern "C"
