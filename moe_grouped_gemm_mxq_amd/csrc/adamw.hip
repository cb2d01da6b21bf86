// AdamW step of many tensors in one launch per kTensors of them, with the
// states in fp32 or in MXFP8 blocks.
//
// One pass, bound by HBM: 940M fp32 weights with MXFP8 states and a bf16 copy take 2.90 ms
// (5.9 TB/s), 147M bf16 weights with fp32 states 558 us (5.8).  With MXFP8 states and
// both weights and gradients in bf16 the vector units bind it (200M: 414 us, 4.9 TB/s), and small
// tensors the chain of reads: 48 of them with 120000 elements take 5.6 us.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "mxq_device.h"
#include "mxq_host.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;
// A workgroup takes one tile: kPieces pieces of four elements a thread, so that a wave's
// loads are unbroken runs.  Neighbouring workgroups run together, so short tiles keep
// what is touched at a time close together, but each pays a table of scales (150
// instructions a thread).  940M fp32 weights with MXFP8 states and a copy / 147M bf16
// weights with fp32 states / 200M bf16 weights and gradients with MXFP8 states, on
// one part (before the last steps): 2048 elements in two pieces 2.93 ms / 554 / 422 us, in two passes of
// one piece 3.03 / 562 / 423, by 512 threads 2.85 / 550 / 487, 4096 in four pieces
// 3.01 / 554 / 411; runs of 8192 or more lose 5 to 10%.  Ordinary instead of
// non-temporal stores lose 13% (200M fp32 weights, MXFP8 states: 609 against 689 us).
constexpr int kPieces = 2;
constexpr int kTile = kPieces * 4 * kThreads;
// Tensors of a launch: as many descriptors as fit the 4 KB of a kernel's arguments, in which they
// travel.  (At most 64: a wave looks its workgroup's tensor up, a tensor per lane.)  50 small
// tensors take 3.2 us on the GPU in a graph, 51 in two launches 5.9.
constexpr int kTensors = 50;
constexpr size_t kArgumentBytes = 4096;
constexpr int64_t kMaxGrid = (1 << 24) - 1;  // workgroups of a launch: a grid has fewer than 2^32 threads
constexpr int kLine = 32;  // fp32 states in a cache line
constexpr int64_t kMaxRun = 32 * kTile, kMaxElements = kMaxGrid * kMaxRun - kLine;

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  uint16_t* copy;
  int64_t n;
  float decay;          // weight decay of this tensor
  uint32_t first_wg;    // of the launch
  uint32_t index;       // in the call
};

// Tiles of fp32 states begin where a cache line of m does, so many elements before the first
// (and where lines of the other arrays do, if they lie alike, as views of flat buffers do): lines
// that two waves share are written twice.  200M fp32 weights in 3 tensors packed without
// gaps and a copy 1260 us with tiles from the first element, 1095 so.  MXFP8 states
// have their tiles at blocks of the tensor.
__host__ __device__ inline int32_t lead_of(const void* m, bool mx) {
  return mx ? 0 : (int32_t)((uintptr_t)m / sizeof(float) % kLine);
}

struct Hyper {
  float b1, c1, b2, c2;  // betas and 1 - betas
  float eps, grad_scale;
  float rs, alpha;       // 1 / sqrt(1 - beta2^step), lr / (1 - beta1^step)
  double lr;
  uint32_t key;          // seed + 0x9E3779B9 * step
};

struct Args {
  Tensor t[kTensors];
  int32_t count;
  int32_t chunk;  // elements of a workgroup, a multiple of kTile
  Hyper h;
  double log2_b1, log2_b2;
  const mxq_adamw_control* control;
};
static_assert(kTensors <= 64 && sizeof(Args) <= kArgumentBytes && sizeof(Args) + sizeof(Tensor) > kArgumentBytes,
              "as many tensors as fit");

// ------------------------------------------------------------------ random bits
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;  // odd fractions of sqrt 2 and sqrt 3
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

// Element pair q of a tensor with this key -> 64 bits: element 2q takes bits
// 0-15 for m and 16-31 for r, element 2q + 1 bits 32-47 and 40-55 (the top
// byte of a product's high word is not uniform).
__device__ __forceinline__ uint64_t pair_bits(uint32_t key, int64_t q) {
  uint32_t x = key + (uint32_t)q * 0x9E3779B9u + (uint32_t)(q >> 32) * 0x243F6A89u;
  x = (x ^ (x >> 15)) * 0x6A09E667u;
  x = x ^ (x >> 13);
  return (uint64_t)x * 0xBB67AE85u;
}

// ------------------------------------------------------------------ MXFP8 states
// Stochastic rounding to E4M3 by the conversion instruction: it adds the top 20
// random bits below the kept mantissa bits, so 16 of them and a half stand for
// u = (u16 + 1/2) / 65536.  Checked against floor(y / step + u) over 2^24 values and
// numbers of each range: equal from 2^-6 to 448; below, where E4M3 is
// subnormal, the two differ where y has bits below 2^-29 that decide.
__device__ __forceinline__ uint32_t above(uint32_t u16_in_the_top) { return (u16_in_the_top & 0xFFFF0000u) | 0x8000u; }

// four codes times their scale
__device__ __forceinline__ void e4m3_decode4(uint32_t c, float scale, float (&f)[4]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const f2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, false);
  const f2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c, scale, true);
  f[0] = lo[0];
  f[1] = lo[1];
  f[2] = hi[0];
  f[3] = hi[1];
}

// Square root rounded to nearest: the hardware's is off by at most one step, and
// the residuals at its neighbours say which way.  Equal to sqrtf for every x
// from 2^-96 up (all of them compared), within a step below; 0, infinity and NaN pass.
__device__ __forceinline__ float sqrt_rn(float x) {
  const float s = __builtin_amdgcn_sqrtf(x);
  const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(__float_as_uint(s) + 1);
  const float r = __builtin_fmaf(-down, s, x) <= 0.f ? down : s;
  return __builtin_fmaf(-up, s, x) > 0.f ? up : r;
}

// scale byte of a block whose largest finite magnitude has these bits:
// smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), at least byte 1
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)((amax + 0x1FFFFFu) >> 23) - 8;
  return e < 1 ? 1u : (uint32_t)e;
}
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }

// largest of the eight lanes that hold a block
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  v = quad_max_u32(v);
  return max(v, dpp_half_mirror(v));
}

template <typename PT, typename GT, bool MX>
struct Step {
  PT* p;
  const GT* g;
  void *m, *v;
  uint8_t *ms, *vs;
  uint16_t* copy;
  int64_t n;
  float keep;
  uint32_t key;

  // Elements i0 + 1024 j + 4 threadIdx.x .. + 3 for j < kPieces.  INSIDE: all of them are
  // elements of the tensor, so the loads are whole and need no branch between them.
  template <bool INSIDE>
  __device__ __forceinline__ void tile(int64_t i0, const Hyper& h, const float* inverse) const {
#pragma clang fp contract(off)
    float pr[kPieces][4], gr[kPieces][4], mr[kPieces][4], vr[kPieces][4];
    uint32_t mc[kPieces], vc[kPieces], mb[kPieces], vb[kPieces];
    Raw<PT, 4> pw[kPieces];
    Raw<GT, 4> gw[kPieces];
    Raw<float, 4> mw[kPieces], vw[kPieces];
    int64_t at[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; j++) at[j] = i0 + j * 4 * kThreads + threadIdx.x * 4;
    if constexpr (INSIDE) {
#pragma unroll
      for (int j = 0; j < kPieces; j++) {
        const int64_t i = at[j];
        gw[j] = load_raw<4, true>(g + i);
        pw[j] = load_raw<4, true>(p + i);
        if constexpr (MX) {
          mc[j] = load_u32((const uint8_t*)m + i);
          vc[j] = load_u32((const uint8_t*)v + i);
          mb[j] = ms[i >> 5];
          vb[j] = vs[i >> 5];
        } else {
          mw[j] = load_raw<4, true>((const float*)m + i);
          vw[j] = load_raw<4, true>((const float*)v + i);
        }
      }
#pragma unroll
      for (int j = 0; j < kPieces; j++) {
        unpack(gw[j], gr[j]);
        unpack(pw[j], pr[j]);
        if constexpr (!MX) {
          unpack(mw[j], mr[j]);
          unpack(vw[j], vr[j]);
        }
      }
    } else {
      // one by one, elements that are not there from the nearest that is, without branches between
      uint32_t m1[kPieces][4], v1[kPieces][4];
#pragma unroll
      for (int j = 0; j < kPieces; j++) {
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const int64_t i = min(max(at[j] + k, (int64_t)0), n - 1);
          gr[j][k] = load_f(g, i);
          pr[j][k] = load_f(p, i);
          if constexpr (MX) {
            m1[j][k] = ((const uint8_t*)m)[i];
            v1[j][k] = ((const uint8_t*)v)[i];
          } else {
            mr[j][k] = ((const float*)m)[i];
            vr[j][k] = ((const float*)v)[i];
          }
        }
        if constexpr (MX) {
          mb[j] = ms[min(at[j], n - 1) >> 5];
          vb[j] = vs[min(at[j], n - 1) >> 5];
        }
      }
#pragma unroll
      for (int j = 0; j < kPieces; j++) {
        mc[j] = vc[j] = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          const bool in = (uint64_t)(at[j] + k) < (uint64_t)n;
          gr[j][k] = in ? gr[j][k] : 0.f;
          pr[j][k] = in ? pr[j][k] : 0.f;
          if constexpr (MX) {
            mc[j] |= in ? m1[j][k] << (8 * k) : 0u;
            vc[j] |= in ? v1[j][k] << (8 * k) : 0u;
          } else {
            mr[j][k] = in ? mr[j][k] : 0.f;
            vr[j][k] = in ? vr[j][k] : 0.f;
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; j++) {
      const int64_t i = at[j];
      if constexpr (MX) {
        e4m3_decode4(mc[j], scale_value(mb[j]), mr[j]);
        e4m3_decode4(vc[j], scale_value(vb[j]), vr[j]);
#pragma unroll
        for (int k = 0; k < 4; k++) vr[j][k] = vr[j][k] * vr[j][k];
      }
      // The moments' products and sums are rounded one by one, as documented.  The
      // parameter's may be contracted and its quotient is m times a reciprocal
      // (one step): neither feeds a state.
      float rr[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float gs = gr[j][k] * h.grad_scale;
        mr[j][k] = mr[j][k] * h.b1 + gs * h.c1;
        vr[j][k] = vr[j][k] * h.b2 + gs * h.c2 * gs;
        rr[k] = sqrt_rn(vr[j][k]);
        const float den = __builtin_fmaf(rr[k], h.rs, h.eps);
        pr[j][k] = __builtin_fmaf(pr[j][k], keep, -(h.alpha * mr[j][k]) * __builtin_amdgcn_rcpf(den));
      }
      if constexpr (MX) {
        uint32_t ma = 0, ra = 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          ma = max(ma, __float_as_uint(mr[j][k]) & 0x7FFFFFFFu);
          ra = max(ra, __float_as_uint(rr[k]) & 0x7FFFFFFFu);
        }
        ma = block_max(ma);
        ra = block_max(ra);
        const bool odd = max(ma, ra) >= 0x7F800000u;  // an infinity or NaN in the block
        if (__builtin_expect(__any(odd), 0)) {          // leave those out of the largest magnitudes
          ma = ra = 0;
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const uint32_t x = __float_as_uint(mr[j][k]) & 0x7FFFFFFFu, y = __float_as_uint(rr[k]) & 0x7FFFFFFFu;
            ma = max(ma, x < 0x7F800000u ? x : 0u);
            ra = max(ra, y < 0x7F800000u ? y : 0u);
          }
          ma = block_max(ma);
          ra = block_max(ra);
        }
        mb[j] = scale_byte(ma);
        vb[j] = scale_byte(ra);
        const float mi = inverse[mb[j]], vi = inverse[vb[j]];
        int mw4 = 0, vw4 = 0;
        const uint64_t b0 = pair_bits(key, i >> 1), b1 = pair_bits(key, (i >> 1) + 1);
        const uint32_t w[4] = {(uint32_t)b0, (uint32_t)(b0 >> 32), (uint32_t)b1, (uint32_t)(b1 >> 32)};
        // m: between -448 and 448; r: not below the least E4M3 value unless it is 0
        auto put = [&](auto byte) {
          constexpr int k = decltype(byte)::value;
          const float x = __builtin_amdgcn_fmed3f(mr[j][k] * mi, -448.f, 448.f);
          const float y = __builtin_amdgcn_fmed3f(rr[k] * vi, fminf(rr[k] * 0x1p100f, 0x1p-9f), 448.f);
          mw4 = __builtin_amdgcn_cvt_sr_fp8_f32(x, (int)above(w[k] << 16), mw4, k);
          vw4 = __builtin_amdgcn_cvt_sr_fp8_f32(y, (int)above(k & 1 ? w[k] << 8 : w[k]), vw4, k);
        };
        put(std::integral_constant<int, 0>{});
        put(std::integral_constant<int, 1>{});
        put(std::integral_constant<int, 2>{});
        put(std::integral_constant<int, 3>{});
        mc[j] = (uint32_t)mw4;
        vc[j] = (uint32_t)vw4;
        if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
          for (int k = 0; k < 4; k++) {
            if ((__float_as_uint(mr[j][k]) & 0x7FFFFFFFu) >= 0x7F800000u) mc[j] |= 0x7Fu << (8 * k);
            if ((__float_as_uint(rr[k]) & 0x7FFFFFFFu) >= 0x7F800000u) vc[j] |= 0x7Fu << (8 * k);
          }
        }
      }
      if constexpr (INSIDE) {
        store_vec<4, true>(p + i, pr[j]);
        if (copy) store_vec<4, true>(copy + i, pr[j]);
        if constexpr (MX) {
          store_u32((uint8_t*)m + i, mc[j]);
          store_u32((uint8_t*)v + i, vc[j]);
        } else {
          store_vec<4, true>((float*)m + i, mr[j]);
          store_vec<4, true>((float*)v + i, vr[j]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; k++)
          if ((uint64_t)(i + k) < (uint64_t)n) {
            store_f(p, i + k, pr[j][k]);
            if (copy) copy[i + k] = bf16_of(pr[j][k]);
            if constexpr (MX) {
              ((uint8_t*)m)[i + k] = (uint8_t)(mc[j] >> (8 * k));
              ((uint8_t*)v)[i + k] = (uint8_t)(vc[j] >> (8 * k));
            } else {
              ((float*)m)[i + k] = mr[j][k];
              ((float*)v)[i + k] = vr[j][k];
            }
          }
      }
      if (MX && (threadIdx.x & 7) == 0 && (INSIDE || i < n)) {
        ms[i >> 5] = (uint8_t)mb[j];
        vs[i >> 5] = (uint8_t)vb[j];
      }
    }
  }

  static __device__ __forceinline__ uint32_t load_u32(const uint8_t* q) {
    typedef uint32_t u32_any __attribute__((aligned(1)));
    return __builtin_nontemporal_load(reinterpret_cast<const u32_any*>(q));
  }
  static __device__ __forceinline__ void store_u32(uint8_t* q, uint32_t x) {
    typedef uint32_t u32_any __attribute__((aligned(1)));
    __builtin_nontemporal_store(x, reinterpret_cast<u32_any*>(q));
  }
};

template <typename PT, typename GT, bool MX>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Args a) {
  __shared__ float inverse[MX ? 256 : 1];
  Hyper h = a.h;
  if (a.control) {
    const mxq_adamw_control c = *a.control;
    if (c.step < 1 || !isfinite(c.lr)) return;  // as the host refuses them in the config
    h.lr = c.lr;
    h.grad_scale = c.grad_scale;
    h.key = c.seed + 0x9E3779B9u * (uint32_t)c.step;
    h.rs = (float)(1.0 / sqrt(1.0 - exp2(c.step * a.log2_b2)));
    h.alpha = (float)(h.lr / (1.0 - exp2(c.step * a.log2_b1)));
  }
  if (!isfinite(h.grad_scale)) return;
  // 2^(127 - byte) by powf, which on this GPU is off by one step of fp32 for some
  // exponents.  torch.ldexp and torch.pow take it the same way, so the states are
  // bit for bit those of these formulas in torch operations.  A scaled value is then off by at
  // most three steps of fp32 (this one, doubled where the value's mantissa is near 2, and the
  // product's), 3 * 2^-20 of an E4M3 step: it rounds the other way where u lies
  // within that of the border, for some of the exponents 1 element in 10^6, and a value that
  // E4M3 holds stays (u is 2^-17 or more from 0 and 1).  The exact power is a shift of
  // the exponent and needs no table: 200M bf16 weights and gradients 391 against 434 us, but
  // other bits in the states.
  if constexpr (MX) {
    static_assert(kThreads == 256, "one entry per thread");
    inverse[threadIdx.x] = powf(2.0f, 127.0f - (float)threadIdx.x);
    __syncthreads();
  }
  const int lane = threadIdx.x & 63;
  const bool before = lane < a.count && a.t[lane < a.count ? lane : 0].first_wg <= blockIdx.x;
  const int k = __popcll(__ballot(before)) - 1;  // workgroups of the tensors follow one another
  const Tensor& t = a.t[k];
  const Step<PT, GT, MX> s = {(PT*)t.p, (const GT*)t.g, t.m, t.v, t.ms, t.vs, t.copy, t.n, (float)(1.0 - h.lr * t.decay),
                              mix(h.key + 0xBB67AE85u * (t.index + 1))};
  const int64_t begin = (int64_t)(blockIdx.x - t.first_wg) * a.chunk - lead_of(t.m, MX);
  const int64_t end = min(begin + a.chunk, t.n);
  int64_t i = begin;
  if (i >= 0)
    for (; i + kTile <= end; i += kTile) s.template tile<true>(i, h, inverse);
  for (; i < end; i += kTile) s.template tile<false>(i, h, inverse);
}

template <typename PT, typename GT>
void launch(bool mx, unsigned grid, const Args& a, hipStream_t st) {
  if (mx)
    adamw_kernel<PT, GT, true><<<grid, kThreads, 0, st>>>(a);
  else
    adamw_kernel<PT, GT, false><<<grid, kThreads, 0, st>>>(a);
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

mxq_status mxq_adamw(const mxq_adamw_tensor* tensors, int32_t n_tensors, mxq_dtype param_dt, mxq_dtype grad_dt,
                     mxq_adamw_format format, const mxq_adamw_config* cfg, const mxq_adamw_control* control,
                     hipStream_t st) {
  MXQ_REQUIRE(n_tensors >= 0 && (tensors || n_tensors == 0), "mxq_adamw: tensors is NULL or n_tensors negative");
  MXQ_REQUIRE(cfg != nullptr, "mxq_adamw: config is NULL");
  MXQ_REQUIRE(param_dt == MXQ_DT_F32 || param_dt == MXQ_DT_BF16, "mxq_adamw: unknown parameter type %d", (int)param_dt);
  MXQ_REQUIRE(grad_dt == MXQ_DT_F32 || grad_dt == MXQ_DT_BF16, "mxq_adamw: unknown gradient type %d", (int)grad_dt);
  MXQ_REQUIRE(format == MXQ_ADAMW_F32 || format == MXQ_ADAMW_MXFP8, "mxq_adamw: unknown state format %d", (int)format);
  MXQ_REQUIRE(cfg->beta1 >= 0 && cfg->beta1 < 1 && cfg->beta2 >= 0 && cfg->beta2 < 1, "mxq_adamw: betas must be in [0, 1)");
  // in fp32: an eps that is 0 or subnormal there makes 0 / (0 + eps) a NaN
  MXQ_REQUIRE((float)cfg->eps >= FLT_MIN && isfinite(cfg->eps), "mxq_adamw: eps must be finite and at least 2^-126");
  MXQ_REQUIRE(isfinite(cfg->lr) && isfinite(cfg->weight_decay), "mxq_adamw: lr and weight_decay must be finite");
  MXQ_REQUIRE(control != nullptr || cfg->step >= 1, "mxq_adamw: step must be >= 1");
  MXQ_REQUIRE(aligned_to(control, 16), "mxq_adamw: control must be 16-byte aligned");
  const bool mx = format == MXQ_ADAMW_MXFP8;
  const uintptr_t pa = param_dt == MXQ_DT_F32 ? 4 : 2, ga = grad_dt == MXQ_DT_F32 ? 4 : 2;
  for (int32_t i = 0; i < n_tensors; i++) {
    const mxq_adamw_tensor& t = tensors[i];
    MXQ_REQUIRE(t.n >= 0, "mxq_adamw: tensor %d: n must be >= 0", i);
    MXQ_REQUIRE(isfinite(t.decay_scale), "mxq_adamw: tensor %d: decay_scale must be finite", i);
    if (t.n == 0) continue;
    MXQ_REQUIRE(t.param && t.grad && t.m && t.v, "mxq_adamw: tensor %d: NULL pointer", i);
    MXQ_REQUIRE(!mx || (t.m_scale && t.v_scale), "mxq_adamw: tensor %d: MXFP8 states need m_scale and v_scale", i);
    MXQ_REQUIRE(aligned_to(t.param, pa) && aligned_to(t.grad, ga) && aligned_to(t.copy, 2) &&
                    (mx || (aligned_to(t.m, 4) && aligned_to(t.v, 4))),
                "mxq_adamw: tensor %d: a pointer is not aligned to its type", i);
    MXQ_REQUIRE(t.n <= kMaxElements, "mxq_adamw: tensor %d has too many elements", i);
  }
  MXQ_REQUIRE_DEVICE();
  if (!control && !isfinite(cfg->grad_scale)) return ok();
  Args a;
  a.control = control;
  a.log2_b1 = log2(cfg->beta1);
  a.log2_b2 = log2(cfg->beta2);
  a.h.b1 = (float)cfg->beta1;
  a.h.c1 = (float)(1.0 - cfg->beta1);
  a.h.b2 = (float)cfg->beta2;
  a.h.c2 = (float)(1.0 - cfg->beta2);
  a.h.eps = (float)cfg->eps;
  a.h.grad_scale = (float)cfg->grad_scale;
  a.h.lr = cfg->lr;
  a.h.rs = (float)(1.0 / sqrt(1.0 - pow(cfg->beta2, (double)cfg->step)));
  a.h.alpha = (float)(cfg->lr / (1.0 - pow(cfg->beta1, (double)cfg->step)));
  a.h.key = cfg->seed + 0x9E3779B9u * (uint32_t)cfg->step;
  auto workgroups = [&](const mxq_adamw_tensor& t, int64_t chunk) {
    return t.n == 0 ? 0 : (t.n + lead_of(t.m, mx) + chunk - 1) / chunk;
  };
  int32_t i = 0;
  while (i < n_tensors) {
    int32_t end = i;  // the launch takes tensors i .. end - 1
    int64_t runs = 0;
    for (int32_t count = 0; end < n_tensors && count < kTensors; end++) {
      const int64_t r = workgroups(tensors[end], kMaxRun);
      if (runs + r > kMaxGrid) break;
      runs += r;
      count += r > 0;
    }
    a.chunk = kTile;  // more only where the grid would not hold the workgroups
    auto fits = [&] {
      int64_t w = 0;
      for (int32_t j = i; j < end; j++) w += workgroups(tensors[j], a.chunk);
      return w <= kMaxGrid;
    };
    while (!fits()) a.chunk *= 2;
    int64_t wgs = 0;
    a.count = 0;
    for (; i < end; i++) {
      const mxq_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      a.t[a.count++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, (uint16_t*)t.copy, t.n,
                        (float)(cfg->weight_decay * t.decay_scale), (uint32_t)wgs, (uint32_t)i};
      wgs += workgroups(t, a.chunk);
    }
    if (a.count == 0) continue;
    const unsigned grid = (unsigned)wgs;
    if (param_dt == MXQ_DT_F32)
      grad_dt == MXQ_DT_F32 ? launch<float, float>(mx, grid, a, st) : launch<float, uint16_t>(mx, grid, a, st);
    else
      grad_dt == MXQ_DT_F32 ? launch<uint16_t, float>(mx, grid, a, st) : launch<uint16_t, uint16_t>(mx, grid, a, st);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return launched(e, "mxq_adamw");
  }
  return ok();
}

}  // extern "C"
