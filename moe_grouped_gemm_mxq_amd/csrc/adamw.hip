// AdamW step of many tensors in one launch per kTensors of them, with the
// states in fp32 or in MXFP8 blocks.
#include <math.h>

#include "mxq_device.h"
#include "mxq_host.h"

namespace mxq {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;   // elements per workgroup, a multiple of the 32-element blocks
constexpr int64_t kMaxGrid = (1 << 24) - 1;  // workgroups of a launch: a grid has fewer than 2^32 threads
constexpr int kTensors = 40;   // per launch: the descriptors travel as a kernel argument (< 4 KB)

struct Tensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* ms;
  uint8_t* vs;
  uint16_t* copy;
  int64_t n;
  double decay;         // weight decay of this tensor
  uint32_t first_wg;    // of the launch
  uint32_t index;       // in the call
};

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
  Hyper h;
  double log2_b1, log2_b2;
  const mxq_adamw_control* control;
};

__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }
__device__ __forceinline__ uint16_t bf16_of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(uint16_t* p, int64_t i, float v) { p[i] = bf16_of(v); }

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
// y >= 0, y <= 448, with 16 random bits -> E4M3 magnitude code.  Times 2^-120
// an fp32 number's exponent field is the E4M3 one and its top three mantissa
// bits the E4M3 mantissa, subnormals included, so adding u below bit 20
// carries into the code exactly when y is rounded up.
__device__ __forceinline__ uint32_t e4m3_stochastic(float y, uint32_t u16) {
  const uint32_t b = __float_as_uint(y * 0x1p-120f);
  return (b + (u16 << 4) + 8u) >> 20;
}

__device__ __forceinline__ float e4m3_decode(uint32_t c) {
  if ((c & 0x7F) == 0x7F) return NAN;
  const float a = __uint_as_float((c & 0x7F) << 20) * 0x1p120f;
  return c & 0x80 ? -a : a;
}

// scale byte of a block whose largest finite magnitude has these bits:
// smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8), at least byte 1
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax == 0) return 0;
  const int e = (int)((amax + 0x1FFFFFu) >> 23) - 8;
  return e < 1 ? 1u : (uint32_t)e;
}
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }
// 2^(127 - byte) by powf, which on this GPU is off by one step for some
// exponents.  torch.ldexp and torch.pow take it the same way, so the states are
// bit for bit those of this formula in torch operations; one step of the scaled
// value changes a probability of rounding up by at most 2^-20.
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return powf(2.0f, 127.0f - (float)byte); }

__device__ __forceinline__ uint32_t half_wave_max(uint32_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
  return v;
}

// one element per lane, 32 lanes per block
template <typename PT, typename GT, bool MX>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Args a) {
#pragma clang fp contract(off)
  Hyper h = a.h;
  if (a.control) {
    const mxq_adamw_control c = *a.control;
    if (c.step < 1) return;
    h.lr = c.lr;
    h.grad_scale = c.grad_scale;
    h.key = c.seed + 0x9E3779B9u * (uint32_t)c.step;
    h.rs = (float)(1.0 / sqrt(1.0 - exp2(c.step * a.log2_b2)));
    h.alpha = (float)(h.lr / (1.0 - exp2(c.step * a.log2_b1)));
  }
  if (!isfinite(h.grad_scale)) return;
  int k = 0;
  while (k + 1 < a.count && a.t[k + 1].first_wg <= blockIdx.x) k++;
  const Tensor& t = a.t[k];
  const int64_t begin = (int64_t)(blockIdx.x - t.first_wg) * kChunk;
  const int64_t end = min(begin + kChunk, t.n);
  const float keep = (float)(1.0 - h.lr * t.decay);
  const uint32_t key = mix(h.key + 0xBB67AE85u * (t.index + 1));
  PT* p = (PT*)t.p;
  const GT* g = (const GT*)t.g;
  for (int64_t i0 = begin; i0 < end; i0 += kThreads) {
    const int64_t i = i0 + threadIdx.x;
    const bool in = i < end;
    float m = 0.f, v = 0.f, gr = 0.f, pr = 0.f;
    if (in) {
      gr = load_f(g, i) * h.grad_scale;
      pr = load_f(p, i);
      if constexpr (MX) {
        m = e4m3_decode(((const uint8_t*)t.m)[i]) * scale_value(t.ms[i >> 5]);
        const float r = e4m3_decode(((const uint8_t*)t.v)[i]) * scale_value(t.vs[i >> 5]);
        v = r * r;
      } else {
        m = ((const float*)t.m)[i];
        v = ((const float*)t.v)[i];
      }
    }
    m = m * h.b1 + gr * h.c1;
    v = v * h.b2 + gr * h.c2 * gr;
    const float r = sqrtf(v);
    pr = pr * keep - h.alpha * (m / (r * h.rs + h.eps));
    if constexpr (MX) {
      const uint32_t mb = __float_as_uint(m) & 0x7FFFFFFFu, rb = __float_as_uint(r) & 0x7FFFFFFFu;
      const bool mf = mb < 0x7F800000u, rf = rb < 0x7F800000u;
      const uint32_t mscale = scale_byte(half_wave_max(in && mf ? mb : 0));
      const uint32_t rscale = scale_byte(half_wave_max(in && rf ? rb : 0));
      if (in) {
        const uint64_t bits = pair_bits(key, i >> 1);
        const uint32_t um = (uint32_t)(bits >> (i & 1 ? 32 : 0)) & 0xFFFFu;
        const uint32_t ur = (uint32_t)(bits >> (i & 1 ? 40 : 16)) & 0xFFFFu;
        uint32_t mc = mf ? e4m3_stochastic(fabsf(m) * scale_inverse(mscale), um) : 0x7Fu;
        mc |= (__float_as_uint(m) >> 24) & 0x80u;
        uint32_t rc = rf ? e4m3_stochastic(r * scale_inverse(rscale), ur) : 0x7Fu;
        if (rc == 0 && r > 0.f) rc = 1;
        ((uint8_t*)t.m)[i] = (uint8_t)mc;
        ((uint8_t*)t.v)[i] = (uint8_t)rc;
        if ((i & 31) == 0) {
          t.ms[i >> 5] = (uint8_t)mscale;
          t.vs[i >> 5] = (uint8_t)rscale;
        }
      }
    } else if (in) {
      ((float*)t.m)[i] = m;
      ((float*)t.v)[i] = v;
    }
    if (in) {
      store_f(p, i, pr);
      if (t.copy) t.copy[i] = bf16_of(pr);
    }
  }
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
  MXQ_REQUIRE(cfg->eps > 0 && isfinite(cfg->eps), "mxq_adamw: eps must be positive");
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
    MXQ_REQUIRE((t.n - 1) / kChunk < kMaxGrid, "mxq_adamw: tensor %d has too many elements", i);
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
  int32_t i = 0;
  while (i < n_tensors) {
    int64_t wgs = 0;
    a.count = 0;
    for (; i < n_tensors && a.count < kTensors; i++) {
      const mxq_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      const int64_t w = (t.n + kChunk - 1) / kChunk;
      if (wgs + w > kMaxGrid) break;
      a.t[a.count++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, (uint16_t*)t.copy, t.n,
                        cfg->weight_decay * t.decay_scale, (uint32_t)wgs, (uint32_t)i};
      wgs += w;
    }
    if (a.count == 0) break;
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
