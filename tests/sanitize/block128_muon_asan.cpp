// Drives the block-128 quantisers and products and the Muon entry points with
// arguments their host-side checks must reject and with well-formed ones, in a
// build of their host code under AddressSanitizer / UndefinedBehaviorSanitizer.
// Without a usable gfx950 device every well-formed call must stop at the device
// gate.  Prints "ok".
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/mxq.h"
#include "../../moe_grouped_gemm_mxq_amd/csrc/mxq_internal.h"

namespace mxq {
static void reached(const char* what) {
  std::fprintf(stderr, "kernel launcher %s reached without a device\n", what);
  std::exit(3);
}
hipError_t launch_quant_row(const uint16_t*, int64_t, int64_t, int64_t, uint8_t*, uint8_t*, hipStream_t, int,
                            BatchStrides) { reached("quant_row"); return hipSuccess; }
hipError_t launch_quant_tile(const uint16_t*, int64_t, int64_t, int64_t, const int32_t*, int32_t, int64_t,
                             uint8_t*, uint8_t*, uint8_t*, uint8_t*, hipStream_t, int, BatchStrides) {
  reached("quant_tile"); return hipSuccess;
}
hipError_t launch_gemm(int, bool, const uint8_t*, const uint8_t*, const uint8_t*, const uint8_t*, float*, int64_t,
                       int64_t, int64_t, int64_t, const int32_t*, int32_t, hipStream_t) {
  reached("gemm"); return hipSuccess;
}
}  // namespace mxq

static int fails = 0;
#define EXPECT(call, want)                                                                      \
  do {                                                                                          \
    mxq_status _s = (call);                                                                     \
    if (_s != (want)) {                                                                         \
      std::fprintf(stderr, "line %d: %s gave %d, want %d (%s)\n", __LINE__, #call, (int)_s, (int)(want), \
                   mxq_last_error());                                                           \
      fails++;                                                                                  \
    } else if (_s != MXQ_OK && std::strlen(mxq_last_error()) == 0) {                            \
      std::fprintf(stderr, "line %d: no error message\n", __LINE__);                            \
      fails++;                                                                                  \
    }                                                                                           \
  } while (0)

int main() {
  alignas(256) static uint8_t buf[1 << 12];
  uint8_t* p = buf;  // 256-byte aligned stand-in, never dereferenced
  float* f = reinterpret_cast<float*>(buf);
  int32_t* i = reinterpret_cast<int32_t*>(buf);
  uint16_t* h = reinterpret_cast<uint16_t*>(buf);
  const mxq_status INV = MXQ_ERR_INVALID_ARGUMENT, DEV = MXQ_ERR_DEVICE;
  const mxq_dtype F32 = MXQ_DT_F32, BF16 = MXQ_DT_BF16;
  const int64_t M31 = INT32_MAX;

  // sizes: every corner of the arguments
  const int64_t corners[] = {INT64_MIN, INT32_MIN, -1, 0, 1, 127, 128, 1 << 20, (1 << 20) + 1, M31, M31 + 1, INT64_MAX};
  for (int64_t T : corners)
    for (int32_t G : {INT32_MIN, -1, 0, 1, 1024, INT32_MAX}) {
      const int64_t n = mxq_grouped128_cols_max(T, G);
      const bool good = T >= 0 && T <= M31 && G >= 0;
      if (good ? n < T + 127 * (int64_t)G || n % 256 != 128 : n != 0) fails++;
    }
  for (int64_t batch : corners)
    for (int64_t R : corners)
      for (int64_t C : corners)
        for (int dt = -1; dt <= 2; dt++) {
          const int64_t n = mxq_orthogonalize_workspace(batch, R, C, (mxq_dtype)dt);
          const bool good = batch >= 0 && batch <= 65535 && R >= 1 && R <= 1 << 20 && C >= 1 && C <= 1 << 20 && (dt == 0 || dt == 1);
          if (n < 0 || (!good && n != 0) || (good && batch > 0 && n > 0 && n / batch < R * C * 2)) fails++;
        }

  // quantisers: well-formed calls of both extremes, and every size out of range
  for (int64_t R : corners)
    for (int64_t C : corners) {
      const bool good = R >= 0 && R <= M31 && C >= 1 && C <= M31 - 128;
      for (int tile : {1, 128})
        for (int axes : {1, 2, 3}) EXPECT(mxq_quantize128(p, BF16, 1, R, C, C, 0, tile, axes, p, f, p, f, nullptr), good ? DEV : INV);
      EXPECT(mxq_quantize128_grouped(p, F32, R, C, C, i, 7, 1280, 3, p, f, p, f, nullptr), good ? DEV : INV);
    }
  EXPECT(mxq_quantize128(p, F32, 65535, M31, 128, INT64_MAX / M31, INT64_MAX, 1, 3, p, f, p, f, nullptr), DEV);
  EXPECT(mxq_quantize128(p, F32, INT64_MAX, 4, 4, 4, 16, 1, 3, p, f, p, f, nullptr), INV);
  EXPECT(mxq_quantize128(p, F32, 2, 4, 4, 4, INT64_MIN, 1, 3, p, f, p, f, nullptr), INV);
  EXPECT(mxq_quantize128(p, F32, 1, 4, 4, INT64_MIN, 0, 1, 3, p, f, p, f, nullptr), INV);
  EXPECT(mxq_quantize128(p, F32, 2, M31, 4, INT64_MAX, INT64_MAX, 1, 3, p, f, p, f, nullptr), INV);
  for (int bad : {INT32_MIN, -1, 0, 2, 127, INT32_MAX}) EXPECT(mxq_quantize128(p, F32, 1, 4, 4, 4, 0, bad, 3, p, f, p, f, nullptr), INV);
  for (int64_t ldq : {INT64_MIN, (int64_t)-128, (int64_t)0, (int64_t)64, INT64_MAX})
    EXPECT(mxq_quantize128_grouped(p, F32, 4, 4, 4, i, 1, ldq, 2, nullptr, nullptr, p, f, nullptr), INV);
  EXPECT(mxq_quantize128_grouped(p, F32, 4, 4, 4, i, INT32_MAX, 128, 2, nullptr, nullptr, p, f, nullptr), INV);

  // products
  for (int64_t M : corners)
    for (int64_t N : corners)
      for (int64_t K : corners) {
        const bool good = M >= 0 && M <= M31 && N >= 1 && N <= M31 && (K == 128 || K == 1 << 20);
        for (int tile : {1, 128}) EXPECT(mxq_gemm128(p, f, p, f, tile, p, BF16, M, N, K, N, nullptr), good ? DEV : INV);
        for (mxq_gg_mode mode : {MXQ_GG_RAGGED_M, MXQ_GG_RAGGED_K})
          EXPECT(mxq_grouped_gemm128(mode, p, f, p, f, p, F32, M, N, K, i, 1024, nullptr), good ? DEV : INV);
      }
  EXPECT(mxq_gemm128(p, f, p, f, 128, p, (mxq_dtype)INT32_MAX, 4, 4, 128, 4, nullptr), INV);
  EXPECT(mxq_gemm128(p, f, p, f, 128, p, F32, 4, 4, 128, INT64_MIN, nullptr), INV);
  EXPECT(mxq_grouped_gemm128((mxq_gg_mode)7, p, f, p, f, p, F32, 4, 4, 128, i, 2, nullptr), INV);
  EXPECT(mxq_grouped_gemm128(MXQ_GG_RAGGED_M, p, f, p, f, p, F32, 4, 4, 128, i, INT32_MIN, nullptr), INV);

  // orthogonalised updates
  const mxq_newton_schulz ns = {3.4445, -4.7750, 2.0315, 1e-7, 5};
  const int64_t ws = mxq_orthogonalize_workspace(3, 40, 50, F32);
  EXPECT(mxq_orthogonalize(p, BF16, 3, 40, 50, &ns, p, F32, p, ws, nullptr), DEV);
  EXPECT(mxq_orthogonalize(p, BF16, 3, 40, 50, &ns, p, F32, p, ws - 1, nullptr), INV);
  EXPECT(mxq_orthogonalize(nullptr, BF16, 0, 40, 50, &ns, nullptr, F32, nullptr, 0, nullptr), DEV);
  EXPECT(mxq_orthogonalize(p, BF16, 3, INT64_MAX, INT64_MIN, &ns, p, F32, p, INT64_MAX, nullptr), INV);
  EXPECT(mxq_orthogonalize(p, BF16, 3, 40, 50, nullptr, p, F32, p, ws, nullptr), INV);
  mxq_muon_config c = {ns, 1e-3, 0.95, 0.1, 0.2, 1.0, 1};
  EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &c, nullptr, p, ws, nullptr), DEV);
  EXPECT(mxq_muon(p, F32, p, BF16, f, nullptr, 3, 40, 50, nullptr, nullptr, p, ws, nullptr), INV);
  const double odd[] = {NAN, INFINITY, -INFINITY, 1e300, -1e300};
  for (double bad : odd) {
    for (int field = 0; field < 4; field++) {
      mxq_muon_config d = c;
      (&d.ns.a)[field] = bad;
      const bool huge_eps = field == 3 && bad == 1e300;  // eps is used in 64 bits
      EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &d, nullptr, p, ws, nullptr), huge_eps ? DEV : INV);
    }
    mxq_muon_config m = c, w = c, s = c, l = c;
    m.momentum = w.weight_decay = s.scale = l.lr = bad;
    EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &m, nullptr, p, ws, nullptr), INV);
    EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &w, nullptr, p, ws, nullptr), INV);
    EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &s, nullptr, p, ws, nullptr), INV);
    EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &l, nullptr, p, ws, nullptr), DEV);  // a step to skip, on a device
  }
  for (int32_t bad : {INT32_MIN, -1, 0, 33, INT32_MAX}) {
    mxq_muon_config d = c;
    d.ns.steps = bad;
    EXPECT(mxq_muon(p, F32, p, BF16, f, h, 3, 40, 50, &d, nullptr, p, ws, nullptr), INV);
  }
  if (fails) return 1;
  std::puts("ok");
  return 0;
}
