// Drives the router, expert order, combine and AdamW entry points with
// arguments their host-side checks must reject and with well-formed ones, in a
// build of their host code under AddressSanitizer / UndefinedBehaviorSanitizer.
// Without a usable gfx950 device every well-formed call must stop at the device
// gate.  Prints "ok".
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

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
  void* p = buf;  // 256-byte aligned stand-in, never dereferenced
  float* f = reinterpret_cast<float*>(buf);
  int32_t* i = reinterpret_cast<int32_t*>(buf);
  const mxq_status INV = MXQ_ERR_INVALID_ARGUMENT, DEV = MXQ_ERR_DEVICE;
  const mxq_dtype F32 = MXQ_DT_F32, BF16 = MXQ_DT_BF16;

  // sizes: every corner of the arguments, the workspace of a well-formed call positive
  for (int64_t T : {(int64_t)0, (int64_t)1, (int64_t)4096, (int64_t)1 << 25, (int64_t)INT32_MAX, INT64_MAX, INT64_MIN})
    for (int32_t K : {INT32_MIN, 0, 1, 8, 32, 33, INT32_MAX})
      for (int32_t E : {INT32_MIN, 0, 1, 32, 1023, 1024, 1025, INT32_MAX}) {
        const bool good = T >= 0 && K >= 1 && K <= 32 && E >= 1 && E <= 1024 && T <= INT32_MAX / K;
        if ((mxq_expert_order_workspace(T, K, E) > 0) != good) fails++;
      }

  mxq_route_config c = {MXQ_SCORE_SIGMOID, 8, 8, 4, 2, 1, 2.5f};
  const int64_t ws = mxq_expert_order_workspace(100, 8, 256);
  EXPECT(mxq_route(p, F32, 100, 256, 256, f, &c, i, f, i, i, i, p, ws, nullptr), DEV);
  EXPECT(mxq_route(p, BF16, 100, 256, 300, nullptr, &c, i, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), DEV);
  EXPECT(mxq_route(nullptr, F32, 0, 256, 256, f, &c, nullptr, nullptr, i, nullptr, nullptr, p, ws, nullptr), DEV);
  EXPECT(mxq_route(p, F32, 100, 256, 256, f, &c, i, f, i, i, i, p, ws - 1, nullptr), INV);
  EXPECT(mxq_route(p, F32, INT64_MAX, 256, 256, f, &c, i, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), INV);
  EXPECT(mxq_route(p, F32, 100, INT32_MAX, INT64_MAX, f, &c, i, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), INV);
  EXPECT(mxq_route(p, (mxq_dtype)-5, 100, 256, 256, f, &c, i, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), INV);
  for (int field = 0; field < 6; field++)
    for (int32_t bad : {INT32_MIN, -1, INT32_MAX}) {
      mxq_route_config d = c;
      (&d.score)[field] = bad;
      EXPECT(mxq_route(p, F32, 100, 256, 256, f, &d, i, f, nullptr, nullptr, nullptr, nullptr, 0, nullptr), INV);
    }
  EXPECT(mxq_route_backward(p, F32, 100, 256, 256, &c, i, f, p, 256, nullptr), DEV);
  EXPECT(mxq_route_backward(p, F32, 100, 256, 256, &c, i, f, p, 255, nullptr), INV);
  EXPECT(mxq_route_backward(p, F32, 100, 256, 256, nullptr, i, f, p, 256, nullptr), INV);
  EXPECT(mxq_expert_order(i, 100, 8, 256, i, i, i, p, ws, nullptr), DEV);
  EXPECT(mxq_expert_order(i, INT64_MAX, 8, 256, i, i, i, p, INT64_MAX, nullptr), INV);

  EXPECT(mxq_combine(p, F32, 800, 512, i, f, 100, 8, 512, p, BF16, 512, nullptr), DEV);
  EXPECT(mxq_combine(nullptr, F32, 0, 512, i, f, 100, 8, 512, p, BF16, 512, nullptr), DEV);
  EXPECT(mxq_combine(p, F32, INT64_MAX, 512, i, f, 100, 8, 512, p, BF16, 512, nullptr), INV);
  EXPECT(mxq_combine(p, F32, 800, INT64_MIN, i, f, 100, 8, 512, p, BF16, 512, nullptr), INV);
  EXPECT(mxq_combine(p, F32, 800, INT64_MAX, i, f, 100, 8, (int64_t)1 << 29, p, BF16, INT64_MAX, nullptr), INV);
  EXPECT(mxq_combine_backward(p, BF16, 512, p, F32, 512, i, f, 100, 8, 512, 800, p, BF16, 512, f, nullptr), DEV);
  EXPECT(mxq_combine_backward(p, BF16, 512, nullptr, F32, 0, i, nullptr, 100, 8, 512, 800, p, BF16, 512, nullptr, nullptr), DEV);
  EXPECT(mxq_combine_backward(p, BF16, 512, nullptr, F32, 0, i, f, 100, 8, 512, 800, p, BF16, 512, f, nullptr), INV);

  mxq_adamw_config h = {1e-3, 0.9, 0.999, 1e-8, 0.01, 1.0, 1, 7};
  std::vector<mxq_adamw_tensor> t(100, mxq_adamw_tensor{p, p, p, p, buf, buf, p, 1000, 1.0});
  EXPECT(mxq_adamw(t.data(), 100, F32, BF16, MXQ_ADAMW_MXFP8, &h, nullptr, nullptr), DEV);
  EXPECT(mxq_adamw(t.data(), 100, F32, BF16, MXQ_ADAMW_F32, &h, nullptr, nullptr), DEV);
  EXPECT(mxq_adamw(nullptr, 0, F32, BF16, MXQ_ADAMW_F32, &h, nullptr, nullptr), DEV);
  t[99].n = INT64_MAX;
  EXPECT(mxq_adamw(t.data(), 100, F32, BF16, MXQ_ADAMW_F32, &h, nullptr, nullptr), INV);
  t[99].n = INT64_MIN;
  EXPECT(mxq_adamw(t.data(), 100, F32, BF16, MXQ_ADAMW_F32, &h, nullptr, nullptr), INV);
  t[99].n = 0;
  EXPECT(mxq_adamw(t.data(), -1, F32, BF16, MXQ_ADAMW_F32, &h, nullptr, nullptr), INV);
  EXPECT(mxq_adamw(t.data(), 100, F32, BF16, (mxq_adamw_format)INT32_MAX, &h, nullptr, nullptr), INV);
  for (double bad : {(double)NAN, (double)INFINITY, -1.0, 1.0, 2.0}) {
    mxq_adamw_config d = h;
    d.beta1 = bad;
    EXPECT(mxq_adamw(t.data(), 100, F32, BF16, MXQ_ADAMW_F32, &d, nullptr, nullptr), INV);
  }
  if (fails) return 1;
  std::puts("ok");
  return 0;
}
