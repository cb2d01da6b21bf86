// Orthogonalised updates of weight matrices: Newton-Schulz iterations
//   X <- u / (|u|_F + eps),   X <- a X + (b A + c A^2) X  with  A = X X^T,
// and the Muon step around them (momentum, decayed weights).
//
// X is the matrix or its transpose, so that A is the smaller of the two Gram
// matrices: lo x lo, X lo x hi.  An iteration is three products on fp16
// operands with fp32 sums:
//   gram    A = X X^T, and square  B = b A + c A^2 + (a - e) I: symmetric, so only
//           the tiles on and above the diagonal are computed and each is stored
//           twice;
//   update  X' = e X + B X, from rows of B and columns of X, which the LDS reads
//           turn (four rows of sixteen numbers at a time), so that X is kept once.
// Splitting a into e and a - e changes nothing but the rounding: e = a while the
// iteration grows X, and less in the last two, where B is near its diagonal.
//
// Precision.  The iteration multiplies small singular values by up to a = 3.4
// each time, and rounding errors in their directions with them, so X itself is
// kept in two fp16 numbers (22 bits).  The operands of the products are fp16: its
// 11 bits put five steps' result within 2e-3 of itself (2-norm) where there are 64
// rows and more, about bf16's own rounding, and within 1e-2 where so few elements
// make up the result that their roundings do not average out; bf16 operands would be
// off by 1e-2 to 2e-1 (gradients of low rank).  Results kept in fp32 take each product
// three times, high x high, high x low and low x high: as near as fp32 operands (2e-6
// for noise, 6e-5 for low rank).
// fp16's range is kept by powers of two: X is stored times 2^15, A times 2^14, B
// times a power that its coefficients allow.  X's singular values, and with them its
// elements, stay within 1.25, so 1.25 x 2^15 is the largest number; any smaller power
// would put more of the low halves of small elements under fp16's smallest step, and
// they are what an outlier row or column leaves of the others (16 x 64 with a row and a
// column 1000 times the rest, fp32 result: off by 5e-7, with 2^5 by 1.2e-5).
//
// What bounds it.  Large matrices: the matrix units and what feeds them; four 7168 x 4096 with fp32 weights 22.5 ms (three
// products each: 1150 TFLOP/s, 66-73% of the cycles in matrix instructions), with bf16 weights 9.5 ms (900; 45-61%: of an
// update's 1.06 ms about 0.2 are X read and written by all CUs at the same time).  An fp16 product of 8192^3 by the vendor's
// library runs at 1400 TFLOP/s on such numbers.  Small ones (32 times 512 x 256: 174 us): 17 dependent launches of 8 to
// 18 us, each some stages' latency and the traffic of its operands.
#include <cmath>

#include "mxq_device.h"
#include "mxq_host.h"
#include "mxq_internal.h"
#include "mxq_tile.h"
#include "mxq_vec.h"

namespace mxq {

namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kScaleX = 32768.f, kScaleA = 16384.f;
constexpr int kMaxSide = 1 << 20;
constexpr int kThreads = 256;
constexpr int kMaxParts = 256;  // partial sums of squares of a matrix

int64_t up64(int64_t n) { return (n + 63) / 64 * 64; }

// An operand's row of K numbers in fp16.  Where products are taken three times
// (SPLIT), the high and the low halves of 32 numbers lie side by side in a
// 128-byte line, so that a stage's line feeds all three; else it is the high halves.
template <bool SPLIT>
struct Row {
  static constexpr int kWide = SPLIT ? 2 : 1;  // fp16 numbers an element takes
  static __host__ __device__ __forceinline__ int64_t at(int64_t k) { return SPLIT ? (k >> 5) * 64 + (k & 31) : k; }
  static constexpr int kLow = 32;  // from a high half to its low one
};

// Where a matrix's operands lie.
struct Space {
  int64_t lo, hi, Lp, Hp;  // sides, and rounded up to 64 (zeros there)
  _Float16 *x, *x2;        // [batch][Lp] rows of Hp: this iteration's X and the next one's
  _Float16* xl;            // what fp16 leaves of X, [batch][Lp][Hp], where the rows do not hold it
  _Float16 *a, *b;         // [batch][Lp] rows of Lp
  double* parts;           // [batch][kMaxParts]
};

// total bytes; fills sp where base is given
int64_t lay_out(Space* sp, uint8_t* base, int64_t batch, int64_t R, int64_t C, bool split) {
  const int64_t lo = R < C ? R : C, hi = R < C ? C : R;
  const int64_t Lp = up64(lo), Hp = up64(hi), wide = split ? 2 : 1;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return base ? base + here : nullptr;
  };
  auto half = [&](int64_t n) { return reinterpret_cast<_Float16*>(take(batch * n * 2)); };
  Space s;
  s.lo = lo, s.hi = hi, s.Lp = Lp, s.Hp = Hp;
  s.x = half(Lp * Hp * wide), s.x2 = half(Lp * Hp * wide);
  s.xl = split ? nullptr : half(Lp * Hp);
  s.a = half(Lp * Lp * wide), s.b = half(Lp * Lp * wide);
  s.parts = reinterpret_cast<double*>(take(batch * kMaxParts * 8));
  if (sp) *sp = s;
  return at;
}

// What an update's matrix is made of: the momentum's combination with the
// gradient, or the matrix given.
struct Source {
  const void* grad;
  float* m;          // fp32 [batch][n] or null: the update is the gradient itself
  int64_t n;         // elements of a matrix
  float beta, keep;  // m' = beta m + keep g
  float grad_scale;
  int nesterov;
  const mxq_adamw_control* control;
};

// learning rate and gradient scale of this step; false: skip it
__device__ __forceinline__ bool step_of(const mxq_adamw_control* control, float& lr, float& grad_scale) {
  if (control) {
    lr = control->lr;
    grad_scale = control->grad_scale;
  }
  return fabsf(lr) < __builtin_inff() && fabsf(grad_scale) < __builtin_inff();
}

// W elements of the momentum's update and of u, from W gradients; m advances where FIRST
template <typename G, bool MOMENTUM, bool FIRST, int W>
__device__ __forceinline__ void update_of(const G* grad, float* m, const Source& s, float scale, float* u) {
  Raw<G, W> g = load_raw<W, false>(grad);
  float gf[W];
  unpack(g, gf);
  if constexpr (!MOMENTUM) {
#pragma unroll
    for (int j = 0; j < W; j++) u[j] = gf[j];
    return;
  }
  float mf[W];
  unpack(load_raw<W, false>(m), mf);
#pragma unroll
  for (int j = 0; j < W; j++) {
    const float gj = gf[j] * scale;
    if constexpr (FIRST) mf[j] = __builtin_fmaf(s.beta, mf[j], s.keep * gj);
    u[j] = s.nesterov ? __builtin_fmaf(s.beta, mf[j], s.keep * gj) : mf[j];
  }
  if constexpr (FIRST) store_vec<W, false>(m, mf);
}

// Momentum, and the sums of squares of u: one partial sum a workgroup, in 64 bits
// (fp32 squares of gradients below 2^-63 or above 2^63 would leave its range).
template <typename G, bool MOMENTUM>
__global__ __launch_bounds__(kThreads) void momentum_kernel(Source s, double* __restrict__ parts) {
  float lr = 0.f, scale = s.grad_scale;
  if (!step_of(s.control, lr, scale)) return;
  const int64_t base = blockIdx.y * s.n;
  const G* g = static_cast<const G*>(s.grad) + base;
  float* m = MOMENTUM ? s.m + base : nullptr;
  double sum = 0.0;
  const int64_t quads = s.n / 4, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < quads; i += stride) {
    float u[4];
    update_of<G, MOMENTUM, true, 4>(g + 4 * i, MOMENTUM ? m + 4 * i : nullptr, s, scale, u);
#pragma unroll
    for (int j = 0; j < 4; j++) sum = __builtin_fma((double)u[j], (double)u[j], sum);
  }
  if (blockIdx.x == 0 && (int64_t)threadIdx.x < s.n - 4 * quads) {
    const int64_t i = 4 * quads + threadIdx.x;
    float u[1];
    update_of<G, MOMENTUM, true, 1>(g + i, MOMENTUM ? m + i : nullptr, s, scale, u);
    sum = __builtin_fma((double)u[0], (double)u[0], sum);
  }
  __shared__ double waves[kThreads / 64];
#pragma unroll
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) parts[blockIdx.y * (int64_t)kMaxParts + blockIdx.x] = (waves[0] + waves[1]) + (waves[2] + waves[3]);
}

__device__ __forceinline__ void split_half(float v, _Float16& hi, _Float16& lo) {
  hi = (_Float16)v;
  lo = (_Float16)(v - (float)hi);
}

// X = u / (|u| + eps) times kScaleX from 64 x 64 of u [R][C]; X's rows are u's columns
// where it is tall.  low: where the low halves go that X's rows do not hold.
template <typename G, bool MOMENTUM, bool SPLIT>
__global__ __launch_bounds__(kThreads) void start_kernel(Source s, int64_t R, int64_t C, int64_t Rp, int64_t Cp, int nparts,
                                                         double eps, const double* __restrict__ parts, int tall,
                                                         _Float16* __restrict__ x, _Float16* __restrict__ low) {
  typedef Row<SPLIT> L;
  __shared__ float tile[64][65];
  __shared__ double waves[kThreads / 64];
  float lr = 0.f, scale = s.grad_scale;
  const bool run = step_of(s.control, lr, scale);
  const int t = threadIdx.x;
  double sum = run && t < nparts ? parts[blockIdx.y * (int64_t)kMaxParts + t] : 0.0;
#pragma unroll
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
  if ((t & 63) == 0) waves[t >> 6] = sum;
  __syncthreads();
  const double squares = (waves[0] + waves[1]) + (waves[2] + waves[3]);
  const double inv = squares == 0 ? 0 : (double)kScaleX / (sqrt(squares) + eps);  // (may be past fp32's range; zeros stay zeros without an eps)
  const int64_t tiles_c = Cp / 64;
  const int64_t r0 = blockIdx.x / tiles_c * 64, c0 = blockIdx.x % tiles_c * 64;
  const int64_t base = blockIdx.y * s.n;
  const int c = (t & 15) * 4;
#pragma unroll
  for (int k = 0; k < 4; k++) {
    const int64_t r = r0 + 16 * k + (t >> 4);
    float u[4] = {0.f, 0.f, 0.f, 0.f};
    if (run && r < R) {
      const int64_t i = base + r * C + c0 + c;
      const G* g = static_cast<const G*>(s.grad) + i;
      float* m = MOMENTUM ? s.m + i : nullptr;
      if (c0 + c + 4 <= C) {
        update_of<G, MOMENTUM, false, 4>(g, m, s, scale, u);
      } else {
        for (int e = 0; e < 4 && c0 + c + e < C; e++) update_of<G, MOMENTUM, false, 1>(g + e, MOMENTUM ? m + e : nullptr, s, scale, u + e);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; e++) tile[16 * k + (t >> 4)][c + e] = (float)(u[e] * inv);
  }
  __syncthreads();
  // rows of X, eight numbers a lane
  const int64_t x0 = tall ? c0 : r0, k0 = tall ? r0 : c0, width = tall ? Rp : Cp, out = blockIdx.y * Rp * Cp;
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int row = 32 * k + (t >> 3), at = (t & 7) * 8;
    v8h h, l;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      _Float16 hi, lo;
      split_half(tall ? tile[at + e][row] : tile[row][at + e], hi, lo);
      h[e] = hi;
      l[e] = lo;
    }
    const int64_t begin = out + (x0 + row) * width;
    *reinterpret_cast<v8h*>(x + begin * L::kWide + L::at(k0 + at)) = h;
    if constexpr (SPLIT) *reinterpret_cast<v8h*>(x + begin * L::kWide + L::at(k0 + at) + L::kLow) = l;
    else *reinterpret_cast<v8h*>(low + begin + k0 + at) = l;
  }
}

enum Product { kGram, kSquare, kUpdate, kLast };

// D[p][q] = sum_k P[p][k] Q[q][k] (gram, square), or sum_k P[k][p] Q[q][k] (update,
// last); rows, columns and K of one matrix, in elements.
struct Args {
  const _Float16 *P, *Q;  // operands
  int64_t rows_p, rows_q, K;
  int tiles_p, tiles_q;   // of one matrix
  int first, parts;       // workgroup i does tile first + i, or of that many tiles a quarter each (parts = 2)
  // gram, square: A (read by square) and the result
  const _Float16* a;
  float of_sum, of_a, on_diag;  // result = of_sum * sum + of_a * A + on_diag on the diagonal
  _Float16* out;  // (update: the next X)
  // update, last: X's low halves where its rows do not hold them (read and written)
  float e;
  _Float16* xl;
  // last: the result's matrix
  void* param;
  uint16_t* copy;
  int64_t n, lo, hi;  // elements of a matrix, its sides
  int tall;           // it is [hi][lo]
  float from_x;       // result = from_x * X'
  float lr, decay, scale, grad_scale;
  const mxq_adamw_control* control;
};

// Output tile of a workgroup: BP rows of P by BQ rows of Q, WAVES_P x WAVES_Q waves,
// STAGES stages in LDS.
template <int BP, int BQ, int WAVES_P, int WAVES_Q, int STAGES>
struct Shape {
  static constexpr int kP = BP, kQ = BQ, kWavesP = WAVES_P, kStages = STAGES;
  static_assert(BP % 64 == 0 && BQ % 64 == 0, "operands' rows come in multiples of 64");
  static constexpr int kWaves = WAVES_P * WAVES_Q, kThreads = 64 * kWaves;
  static constexpr int WP = BP / WAVES_P, WQ = BQ / WAVES_Q;
  static constexpr int TP = WP / 32, TQ = WQ / 32;  // 32 x 32 blocks of a wave
  static constexpr int kLoadsP = BP / 8 / kWaves, kLoadsQ = BQ / 8 / kWaves, kLoads = kLoadsP + kLoadsQ;
  static constexpr int kBytesP = BP * 128, kBytesQ = BQ * 128, kStage = kBytesP + kBytesQ;
  static_assert(STAGES >= 2 && STAGES <= 4, "the stages are spelled out");
  static_assert(kLoadsP % 2 == 0 && kLoadsQ % 2 == 0, "a load's parity is its place's");
};

// eight numbers of a lane for a 32 x 32 x 16 instruction: row r0 + lane % 32, 16-byte chunk c + lane / 32
__device__ __forceinline__ v8h load_half8(const uint8_t* st, int r0, int c, int lane) {
  return *reinterpret_cast<const v8h*>(st + swz(r0 + (lane & 31), c + (lane >> 5)));
}

// The same where a stage holds rows of k, `row_bytes` of numbers p each, in chunks
// of 64 bytes (32 numbers) of which row k has chunk c at turned_chunk(c, k): chunk
// c, rows k0 + 8 (lane / 32) .. + 7, number lane % 32.  An instruction takes eight
// bytes of a lane and gives lane i of sixteen the i-th numbers of four rows.
template <int ROW_BYTES>
__device__ __forceinline__ int turned_chunk(int c, int k) {  // four rows' chunks lie in different banks
  return c ^ (ROW_BYTES >= 256 ? k & 3 : (k >> 1) & 1);
}
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;
template <int ROW_BYTES>
__device__ __forceinline__ v8h load_turned8(const uint8_t* st, int k0, int c, int lane) {
  const int k = (lane & 15) >> 2;
  const uint8_t* at = st + (k0 + 8 * (lane >> 5) + k) * ROW_BYTES + turned_chunk<ROW_BYTES>(c, k) * 64 + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)at), b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(at + 4 * ROW_BYTES));
  return __builtin_bit_cast(v8h, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// T: the last product's parameter (float or bf16's bits); STEP: it is updated
// rather than overwritten.  A stage is a 128-byte line of every row of the tile:
// 64 numbers, or the halves of 32; of a turned P as many rows of k.
template <int WHAT, bool SPLIT, class S, typename T = float, bool STEP = false>
__global__ __launch_bounds__(S::kThreads, 2) void product_kernel(Args p) {
  typedef Row<SPLIT> L;
  constexpr int TP = S::TP, TQ = S::TQ, NS = S::kStages;
  __shared__ __attribute__((aligned(1024))) uint8_t stage0[S::kStage], stage1[S::kStage], stage2[NS > 2 ? S::kStage : 16],
      stage3[NS > 3 ? S::kStage : 16];
  uint8_t* const stages[4] = {stage0, stage1, stage2, stage3};
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave % S::kWavesP, wq = wave / S::kWavesP;
  const int quarters = p.parts * p.parts;
  const int tile = p.first + xcd_remap(blockIdx.x / quarters, gridDim.x / quarters), quarter = blockIdx.x % quarters;
  const int tiles = WHAT == kGram || WHAT == kSquare ? p.tiles_p * (p.tiles_p + 1) / 2 : p.tiles_p * p.tiles_q;
  const int64_t b = tile / tiles;
  int at = tile - (int)b * tiles, pt, qt;
  if constexpr (WHAT == kGram || WHAT == kSquare) {  // row pt of the upper triangle has tiles_p - pt tiles
    pt = 0;
    while (at >= p.tiles_p - pt) at -= p.tiles_p - pt++;
    qt = pt + at;
  } else {
    raster(at, p.tiles_p, p.tiles_q, pt, qt);
  }
  const int64_t p0 = (int64_t)(pt * p.parts + quarter / p.parts) * S::kP, q0 = (int64_t)(qt * p.parts + quarter % p.parts) * S::kQ;
  if (p0 >= p.rows_p || q0 >= p.rows_q || ((WHAT == kGram || WHAT == kSquare) && p0 > q0)) return;
  const int np = (int)min<int64_t>(S::kP, p.rows_p - p0), nq = (int)min<int64_t>(S::kQ, p.rows_q - q0);

  constexpr bool kTurn = WHAT == kUpdate || WHAT == kLast;
  constexpr int kRowP = S::kP * 2 * L::kWide, kRowsP = 64 / L::kWide;  // a turned stage's rows
  const uint32_t ld = (uint32_t)p.K * 2 * L::kWide, ldp = kTurn ? (uint32_t)p.rows_p * 2 * L::kWide : ld;
  uint32_t offP[S::kLoadsP], offQ[S::kLoadsQ];
#pragma unroll
  for (int j = 0; j < S::kLoadsP; j++) {
    if constexpr (kTurn) {  // past the tile: its last chunk
      constexpr int lanes = kRowP / 16;  // of a row
      const int k = (wave * S::kLoadsP + j) * (64 / lanes) + lane / lanes, pos = lane % lanes;
      offP[j] = (uint32_t)k * ldp + min(turned_chunk<kRowP>(pos / 4, k), np * L::kWide / 32 - 1) * 64 + pos % 4 * 16;
    } else {
      offP[j] = (uint32_t)min((wave * S::kLoadsP + j) * 8 + (lane >> 3), np - 1) * ld + dma_chunk(j, lane) * 16;
    }
  }
#pragma unroll
  for (int j = 0; j < S::kLoadsQ; j++)
    offQ[j] = (uint32_t)min((wave * S::kLoadsQ + j) * 8 + (lane >> 3), nq - 1) * ld + dma_chunk(j, lane) * 16;
  const uint8_t* const baseP =
      reinterpret_cast<const uint8_t*>(p.P) + (kTurn ? b * p.K * ldp + p0 * 2 * L::kWide : (b * p.rows_p + p0) * ld);
  const int64_t stepP = kTurn ? (int64_t)kRowsP * ldp : 128;
  const uint8_t* const baseQ = reinterpret_cast<const uint8_t*>(p.Q) + (b * p.rows_q + q0) * ld;
  const int ns = (int)(ld / 128);
  auto load = [&](uint8_t* st, int s, int n) {
    if (n < S::kLoadsP)
      load_lds16(baseP + s * stepP + offP[n], st + (wave * S::kLoadsP + n) * 1024);
    else
      load_lds16(baseQ + (int64_t)s * 128 + offQ[n - S::kLoadsP], st + S::kBytesP + (wave * S::kLoadsQ + n - S::kLoadsP) * 1024);
  };
  auto meet = [&]() {
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  v16f acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; i++)
#pragma unroll
    for (int j = 0; j < TQ; j++)
#pragma unroll
      for (int e = 0; e < 16; e++) acc[i][j][e] = 0.f;

  auto read = [&](const uint8_t* st, int chunk, v8h (&fp)[TP], v8h (&fq)[TQ]) {
#pragma unroll
    for (int i = 0; i < TP; i++) {
      if constexpr (kTurn)  // (the halves of 32 numbers are chunks side by side)
        fp[i] = load_turned8<kRowP>(st, 8 * (SPLIT ? chunk & 3 : chunk), (wp * TP + i) * L::kWide + (SPLIT ? chunk >> 2 : 0), lane);
      else
        fp[i] = load_half8(st, wp * S::WP + 32 * i, chunk, lane);
    }
#pragma unroll
    for (int j = 0; j < TQ; j++) fq[j] = load_half8(st + S::kBytesP, wq * S::WQ + 32 * j, chunk, lane);
  };
  auto multiply = [&](const v8h (&fp)[TP], const v8h (&fq)[TQ]) {
#pragma unroll
    for (int i = 0; i < TP; i++)
#pragma unroll
      for (int j = 0; j < TQ; j++) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fp[i], fq[j], acc[i][j], 0, 0, 0);
  };
  // Stage s, which is in st, while stage s + NS - 1 is loaded to next (past the last
  // one, the last again: every stage has the same loads in flight, and no branch
  // parts them from the matrix instructions).  Each part's numbers are read while the
  // part before it multiplies.
  constexpr int kM = TP * TQ, kD = TP * (kTurn ? 2 : 1) + TQ, kG = (S::kLoads + 1) / 2;
  auto stage = [&](const uint8_t* st, uint8_t* next, int s) {
    const int ahead = min(s + NS - 1, ns - 1);
    auto load_half_of = [&](int which) {
#pragma unroll
      for (int n = which * kG; n < (which + 1) * kG && n < S::kLoads; n++) load(next, ahead, n);
    };
    if constexpr (SPLIT) {
      v8h hp[2][TP], hq[2][TQ], lp[TP], lq[TQ];
      read(st, 0, hp[0], hq[0]);
      __builtin_amdgcn_sched_barrier(0);
      read(st, 4, lp, lq);
      multiply(hp[0], hq[0]);
      load_half_of(0);
      interleave<kM, 0, kD, kG>();
      __builtin_amdgcn_sched_barrier(0);
      read(st, 2, hp[1], hq[1]);
      multiply(hp[0], lq);
      multiply(lp, hq[0]);
      load_half_of(1);
      interleave<2 * kM, 0, kD, S::kLoads - kG>();
      __builtin_amdgcn_sched_barrier(0);
      read(st, 6, lp, lq);
      multiply(hp[1], hq[1]);
      interleave<kM, 0, kD, 0>();
      __builtin_amdgcn_sched_barrier(0);
      multiply(hp[1], lq);
      multiply(lp, hq[1]);
    } else {
      v8h fp[2][TP], fq[2][TQ];
      read(st, 0, fp[0], fq[0]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        if (k < 3) read(st, 2 * k + 2, fp[(k + 1) & 1], fq[(k + 1) & 1]);
        multiply(fp[k & 1], fq[k & 1]);
        if (k == 0) {
          load_half_of(0);
          interleave<kM, 0, kD, kG>();
        } else if (k == 1) {
          load_half_of(1);
          interleave<kM, 0, kD, S::kLoads - kG>();
        } else if (k == 2) {
          interleave<kM, 0, kD, 0>();
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    wait_vmcnt<(NS - 2) * S::kLoads>();  // the next stage has landed
    wait_lgkmcnt0();
    meet();
  };
#pragma unroll
  for (int s = 0; s < NS - 1; s++)
#pragma unroll
    for (int n = 0; n < S::kLoads; n++) load(stages[s], min(s, ns - 1), n);
  wait_vmcnt<(NS - 2) * S::kLoads>();
  meet();
  // (left from within: a way round the loop after fewer than NS stages would have the
  // compiler wait for loads that such a way would leave in flight)
  auto all_stages = [&]() {
    for (int s0 = 0;; s0 += NS) {
#pragma unroll
      for (int u = 0; u < NS; u++) {
        stage(stages[u], stages[(u + NS - 1) % NS], s0 + u);
        if (s0 + u + 1 >= ns) return;
      }
    }
  };
  all_stages();
  wait_vmcnt<0>();  // the LDS is used again below
  meet();

  // The sums go through LDS (every wave by itself, kP2 x 32 TQ numbers at a time) so
  // that what they are combined with, and where they go, is read and written in whole
  // lines both ways round.
  float rate = 0.f, decay = 0.f;
  if constexpr (WHAT == kLast && STEP) {
    float lr = p.lr, unused = p.grad_scale;
    if (!step_of(p.control, lr, unused)) return;
    rate = lr * p.scale;
    decay = 1.f - lr * p.decay;
  }
  constexpr int kI = TP < 2 ? 1 : 2, kPw = 32 * kI, kQw = 32 * TQ;
  constexpr int kPerStage = S::kStage / (kPw * kQw * 4);
  static_assert(2 * kPerStage >= S::kWaves, "two stages hold every wave's numbers");
  float* const mine = reinterpret_cast<float*>((wave < kPerStage ? stage0 : stage1) + wave % kPerStage * (kPw * kQw * 4));
  // element (row, col) of rows of `width`: 16-byte chunks by the row's last bits
  auto spot = [&](int row, int col, int width) { return row * width + (((col >> 2) ^ (row & (width / 4 - 1) & 15)) << 2) + (col & 3); };
  // rows of `width`, eight numbers of one a lane
  auto each_row = [&](int rows, int width, auto&& body) {
    const int per = width / 8, step = 64 / per;
#pragma unroll
    for (int r = 0; r < rows; r += step) body(r + lane / per, lane % per * 8);
  };
  auto get8 = [&](int row, int col, int width, float* v) {
    const v4f a = *reinterpret_cast<const v4f*>(mine + spot(row, col, width)), c = *reinterpret_cast<const v4f*>(mine + spot(row, col + 4, width));
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = a[e], v[e + 4] = c[e];
  };
  auto between = [&]() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
  // eight halves of a row of an operand, from element k on; those of large matrices past the caches, which the operands
  // need (four times 4096 x 4096 x 7168: update 1090 -> 1060 us; 32 times 256 x 256 x 512 174 -> 192 us in all if they were too)
  const bool past = S::kP == 256 || (S::kP == 128 && p.parts == 2);
  auto put = [&](v8h v, _Float16* to) {
    if (past) __builtin_nontemporal_store(v, reinterpret_cast<v8h*>(to));
    else *reinterpret_cast<v8h*>(to) = v;
  };
  auto store_halves = [&](_Float16* row, _Float16* low, int64_t k, const float* v) {
    v8h h, l;
#pragma unroll
    for (int e = 0; e < 8; e++) {
      _Float16 hi, lo;
      split_half(v[e], hi, lo);
      h[e] = hi;
      l[e] = lo;
    }
    put(h, row + L::at(k));
    if constexpr (SPLIT) put(l, row + L::at(k) + L::kLow);
    else if (low) put(l, low + k);
  };
  auto load_halves = [&](const _Float16* row, const _Float16* low, int64_t k, float* v) {
    const v8h h = *reinterpret_cast<const v8h*>(row + L::at(k));
    v8h l = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (SPLIT) l = *reinterpret_cast<const v8h*>(row + L::at(k) + L::kLow);
    else if (low) l = past ? __builtin_nontemporal_load(reinterpret_cast<const v8h*>(low + k)) : *reinterpret_cast<const v8h*>(low + k);
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = (float)h[e] + (float)l[e];
  };
  // eight results of one row of the parameter, from column k on
  auto finish = [&](int64_t row, int64_t k, int64_t rows, int64_t width, const float* x) {
    if (row >= rows || k >= width) return;
    T* param = static_cast<T*>(p.param) + b * p.n + row * width + k;
    uint16_t* copy = STEP && p.copy ? p.copy + b * p.n + row * width + k : nullptr;
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; e++) y[e] = x[e] * p.from_x;
    if (k + 8 <= width) {
      if constexpr (STEP) {
        float old[8];
        constexpr int W = sizeof(T) == 4 ? 4 : 8;
#pragma unroll
        for (int e = 0; e < 8; e += W) unpack(load_raw<W, false>(param + e), old + e);
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] = __builtin_fmaf(old[e], decay, -rate * y[e]);
      }
      store_vec<8, false>(param, y);
      if (STEP && copy) store_vec<8, false>(copy, y);
    } else {
      for (int e = 0; e < width - k; e++) {
        if constexpr (STEP) y[e] = __builtin_fmaf(load_f(param, e), decay, -rate * y[e]);
        store_f(param, e, y[e]);
        if (STEP && copy) store_f(copy, e, y[e]);
      }
    }
  };
  const int64_t x_stride = p.rows_p * p.rows_q;  // (of a square matrix: gram, square)
  auto row_of = [&](auto* of, int64_t row, int wide) { return of + (b * x_stride + row * p.rows_p) * wide; };
#pragma unroll
  for (int i0 = 0; i0 < TP; i0 += kI) {
    const int pp = wp * S::WP + 32 * i0, qq = wq * S::WQ;
    if (pp >= np || qq >= nq) continue;  // (rows come in multiples of 64)
    const int64_t row_p = p0 + pp, row_q = q0 + qq;
    between();
    // along P: rows of Q
    if constexpr (WHAT != kGram) {
      each_row(kQw, kPw, [&](int r, int c) {
        float v[8];
        if constexpr (WHAT == kSquare)
          load_halves(row_of(p.a, row_q + r, L::kWide), nullptr, row_p + c, v);
        else
          load_halves(row_of(p.P, row_q + r, L::kWide), SPLIT ? nullptr : row_of(p.xl, row_q + r, 1), row_p + c, v);
        *reinterpret_cast<v4f*>(mine + spot(r, c, kPw)) = v4f{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<v4f*>(mine + spot(r, c + 4, kPw)) = v4f{v[4], v[5], v[6], v[7]};
      });
      between();
    }
    // lane l holds D[8 (e / 4) + 4 (l / 32) + e % 4][l % 32] of each 32 x 32 block
#pragma unroll
    for (int i = i0; i < i0 + kI; i++)
#pragma unroll
      for (int j = 0; j < TQ; j++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
          const int row = 32 * j + (lane & 31), col = 32 * (i - i0) + 8 * r + 4 * (lane >> 5);
          v4f* at = reinterpret_cast<v4f*>(mine + spot(row, col, kPw));
          v4f v;
#pragma unroll
          for (int e = 0; e < 4; e++) v[e] = p.of_sum * acc[i][j][4 * r + e];
          if constexpr (WHAT != kGram) {
            const v4f with = *at;
            const float times = WHAT == kSquare ? p.of_a : p.e;
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] = __builtin_fmaf(times, with[e], v[e]);
          }
          if constexpr (WHAT == kSquare) {
#pragma unroll
            for (int e = 0; e < 4; e++) v[e] += row_p + col + e == row_q + row ? p.on_diag : 0.f;
          }
          if (!(WHAT == kLast && p.tall)) *at = v;
#pragma unroll
          for (int e = 0; e < 4; e++) acc[i][j][4 * r + e] = v[e];
        }
    between();
    if (WHAT != kLast || !p.tall) {
      each_row(kQw, kPw, [&](int r, int c) {
        float v[8];
        get8(r, c, kPw, v);
        if constexpr (WHAT == kLast)
          finish(row_q + r, row_p + c, p.lo, p.hi, v);
        else
          store_halves(row_of(p.out, row_q + r, L::kWide), !SPLIT && WHAT == kUpdate ? row_of(p.xl, row_q + r, 1) : nullptr, row_p + c, v);
      });
    }
    if ((WHAT == kLast && p.tall) || ((WHAT == kGram || WHAT == kSquare) && p0 != q0)) {  // along Q: rows of P
      between();
#pragma unroll
      for (int i = i0; i < i0 + kI; i++)
#pragma unroll
        for (int j = 0; j < TQ; j++)
#pragma unroll
          for (int e = 0; e < 16; e++)
            mine[spot(32 * (i - i0) + 8 * (e / 4) + 4 * (lane >> 5) + e % 4, 32 * j + (lane & 31), kQw)] = acc[i][j][e];
      between();
      each_row(kPw, kQw, [&](int r, int c) {
        float v[8];
        get8(r, c, kQw, v);
        if constexpr (WHAT == kLast)
          finish(row_p + r, row_q + c, p.hi, p.lo, v);
        else
          store_halves(row_of(p.out, row_p + r, L::kWide), nullptr, row_q + c, v);
      });
    }
  }
}

typedef Shape<256, 256, 2, 4, 2> Large;
typedef Shape<128, 128, 4, 2, 2> Medium;  // (eight waves: update of 32 times 256 x 256 x 512 14.4 us against 16.1 with four)
typedef Shape<64, 64, 2, 2, 4> Small;

// what the host has checked
struct Plan {
  int64_t batch, R, C;
  int steps;
  double a, b, c, eps;
};

// tiles of side `side` of all matrices
template <int WHAT>
int64_t tiles_of(const Args& p, int64_t batch, int64_t side) {
  const int64_t tp = (p.rows_p + side - 1) / side, tq = (p.rows_q + side - 1) / side;
  return batch * (WHAT == kGram || WHAT == kSquare ? tp * (tp + 1) / 2 : tp * tq);
}

// `count` tiles of side `side` from `first` on, in workgroup tiles of shape S
template <int WHAT, bool SPLIT, class S, typename T, bool STEP>
hipError_t launch_shape(Args p, int64_t side, int64_t first, int64_t count, hipStream_t st) {
  p.tiles_p = (int)((p.rows_p + side - 1) / side);
  p.tiles_q = (int)((p.rows_q + side - 1) / side);
  p.parts = (int)(side / S::kP);
  p.first = (int)first;
  if (first + count > INT32_MAX / 4) return hipErrorInvalidValue;
  product_kernel<WHAT, SPLIT, S, T, STEP><<<(unsigned)(count * p.parts * p.parts), S::kThreads, 0, st>>>(p);
  return hipGetLastError();
}

// 64 x 64 tiles where 128 x 128 ones leave CUs without work (32 times 256 x 256 x 512, fp32 weights: gram 10.4 us against
// 18.1 with 96 of them; update 19.0 against 14.4 with 256), 256 x 256 ones where there are two a CU (four times 4096 x 4096
// x 7168: update 2.36 ms against 2.53), but for a last round that would leave more than half of the CUs idle.
template <int WHAT, bool SPLIT, typename T = float, bool STEP = false>
hipError_t launch_product(const Args& p, int64_t batch, hipStream_t st) {
  const int64_t cus = device_cu_count(), large = tiles_of<WHAT>(p, batch, 256), medium = tiles_of<WHAT>(p, batch, 128);
  if (large >= 2 * cus) {
    const int64_t rest = 2 * (large % cus) <= cus ? large % cus : 0;
    const hipError_t err = launch_shape<WHAT, SPLIT, Large, T, STEP>(p, 256, 0, large - rest, st);
    if (err != hipSuccess || rest == 0) return err;
    return launch_shape<WHAT, SPLIT, Medium, T, STEP>(p, 256, large - rest, rest, st);
  }
  if (medium >= cus) return launch_shape<WHAT, SPLIT, Medium, T, STEP>(p, 128, 0, medium, st);
  return launch_shape<WHAT, SPLIT, Small, T, STEP>(p, 64, 0, tiles_of<WHAT>(p, batch, 64), st);
}

template <typename G, bool MOMENTUM, bool SPLIT>
void launch_start(const Source& s, const Plan& pl, Space& sp, hipStream_t st) {
  const int64_t per = 4 * kThreads;
  int64_t parts = (s.n + per - 1) / per;
  if (parts > kMaxParts) parts = kMaxParts;
  momentum_kernel<G, MOMENTUM><<<dim3((unsigned)parts, (unsigned)pl.batch), kThreads, 0, st>>>(s, sp.parts);
  const int64_t Rp = up64(pl.R), Cp = up64(pl.C);
  start_kernel<G, MOMENTUM, SPLIT><<<dim3((unsigned)(Rp / 64 * (Cp / 64)), (unsigned)pl.batch), kThreads, 0, st>>>(
      s, pl.R, pl.C, Rp, Cp, (int)parts, pl.eps, sp.parts, pl.R > pl.C, sp.x, sp.xl);
}

template <bool SPLIT, typename T, bool STEP>
hipError_t iterate(const Plan& pl, Space& sp, Args last, hipStream_t st) {
  // B = b A + c A^2 + (a - e) I with A's eigenvalues in [0, 1.25^2]
  const double reach = std::fabs(pl.b) * 1.5625 + std::fabs(pl.c) * 1.5625 * 1.5625 + std::fabs(pl.a);
  const float scale_b = std::ldexp(1.f, 15 - (int)std::ceil(std::log2(reach > 1.0 ? reach : 1.0)));
  for (int i = 0; i < pl.steps; i++) {
    const int left = pl.steps - 1 - i;
    const float e = (float)(pl.a * (left == 0 ? 0.4375 : left == 1 ? 0.71875 : 1.0));
    Args g{};
    g.P = g.Q = sp.x, g.rows_p = g.rows_q = sp.Lp, g.K = sp.Hp;
    g.of_sum = kScaleA / (kScaleX * kScaleX), g.out = sp.a;
    hipError_t err = launch_product<kGram, SPLIT>(g, pl.batch, st);
    if (err != hipSuccess) return err;
    Args q{};
    q.P = q.Q = sp.a, q.rows_p = q.rows_q = q.K = sp.Lp, q.a = sp.a;
    q.of_sum = (float)(pl.c * scale_b / ((double)kScaleA * kScaleA)), q.of_a = (float)(pl.b * scale_b / kScaleA);
    q.on_diag = (float)((pl.a - e) * scale_b), q.out = sp.b;
    err = launch_product<kSquare, SPLIT>(q, pl.batch, st);
    if (err != hipSuccess) return err;
    Args u = last;
    u.P = sp.x, u.Q = sp.b, u.rows_p = sp.Hp, u.rows_q = u.K = sp.Lp;
    u.of_sum = 1.f / scale_b, u.e = e, u.xl = sp.xl, u.out = sp.x2;
    if (left) {
      err = launch_product<kUpdate, SPLIT>(u, pl.batch, st);
      _Float16* v = sp.x;
      sp.x = sp.x2, sp.x2 = v;
    } else {
      err = launch_product<kLast, SPLIT, T, STEP>(u, pl.batch, st);
    }
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

// u from s, orthogonalised into last.param
template <bool STEP>
hipError_t run(const Plan& pl, const Source& s, mxq_dtype gdt, mxq_dtype odt, Args last, uint8_t* workspace, hipStream_t st) {
  const bool split = odt == MXQ_DT_F32;
  Space sp;
  lay_out(&sp, workspace, pl.batch, pl.R, pl.C, split);
  if (gdt == MXQ_DT_F32) {
    if (split) launch_start<float, STEP, true>(s, pl, sp, st);
    else launch_start<float, STEP, false>(s, pl, sp, st);
  } else {
    if (split) launch_start<uint16_t, STEP, true>(s, pl, sp, st);
    else launch_start<uint16_t, STEP, false>(s, pl, sp, st);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  last.n = pl.R * pl.C, last.lo = sp.lo, last.hi = sp.hi, last.tall = pl.R > pl.C, last.from_x = 1.f / kScaleX;
  if (split) return iterate<true, float, STEP>(pl, sp, last, st);
  return iterate<false, uint16_t, STEP>(pl, sp, last, st);
}

// largest |a s + b s^3 + c s^5| for s in [0, 1.25]
double reach_of(double a, double b, double c) {
  auto at = [&](double s) { return std::fabs(((c * s * s + b) * s * s + a) * s); };
  double most = at(1.25);
  const double d = 9 * b * b - 20 * a * c;  // 5 c t^2 + 3 b t + a = 0 for t = s^2
  if (d >= 0) {
    const double q = -0.5 * (3 * b + std::copysign(std::sqrt(d), b));  // (no difference of near numbers where c is tiny)
    for (double t : {q / (5 * c), a / q})
      if (t > 0) most = std::fmax(most, at(std::fmin(1.25, std::sqrt(t))));
  }
  return most;
}

// Largest |a + b s^2 + c s^4| for s in [1.25, 1.255]: by what an iteration multiplies a singular value that roundings
// have put past 1.25.  Above 1 it would grow from there, and X leave fp16's range (a rank-1 matrix of 128 x 256 did so in
// 8 steps with -4.125, 11.375, -6).
double growth_past_reach(double a, double b, double c) {
  auto at = [&](double t) { return std::fabs((c * t + b) * t + a); };
  const double from = 1.25 * 1.25, to = 1.255 * 1.255;
  double most = std::fmax(at(from), at(to));
  if (c != 0 && -b / (2 * c) > from && -b / (2 * c) < to) most = std::fmax(most, at(-b / (2 * c)));
  return most;
}

mxq_status check(const char* who, int64_t batch, int64_t R, int64_t C, const mxq_newton_schulz* ns, mxq_dtype gdt, mxq_dtype odt,
                 const void* workspace, int64_t bytes) {
  MXQ_REQUIRE(gdt == MXQ_DT_F32 || gdt == MXQ_DT_BF16, "%s: unknown type %d", who, (int)gdt);
  MXQ_REQUIRE(odt == MXQ_DT_F32 || odt == MXQ_DT_BF16, "%s: unknown type %d", who, (int)odt);
  MXQ_REQUIRE(batch >= 0 && batch <= 65535, "%s: batch must be in [0, 65535] (got %lld)", who, (long long)batch);
  MXQ_REQUIRE(R >= 1 && R <= kMaxSide && C >= 1 && C <= kMaxSide, "%s: R and C must be in [1, %d]", who, kMaxSide);
  MXQ_REQUIRE(ns != nullptr, "%s: config is NULL", who);
  MXQ_REQUIRE(ns->steps >= 1 && ns->steps <= MXQ_MAX_NS_STEPS, "%s: steps must be in [1, %d] (got %d)", who, MXQ_MAX_NS_STEPS, ns->steps);
  MXQ_REQUIRE(std::isfinite(ns->a) && std::isfinite(ns->b) && std::isfinite(ns->c), "%s: coefficients must be finite", who);
  MXQ_REQUIRE(std::fabs(ns->a) <= 64 && std::fabs(ns->b) <= 64 && std::fabs(ns->c) <= 64 && reach_of(ns->a, ns->b, ns->c) <= 1.25,
              "%s: coefficients must keep singular values in [0, 1.25] there", who);
  MXQ_REQUIRE(growth_past_reach(ns->a, ns->b, ns->c) <= 1, "%s: coefficients must not let singular values grow from 1.25 on", who);
  MXQ_REQUIRE(std::isfinite(ns->eps) && ns->eps >= 0, "%s: eps must be finite and not negative", who);
  if (batch == 0) return MXQ_OK;
  MXQ_REQUIRE(workspace != nullptr && aligned_to(workspace, 256), "%s: workspace must be 256-byte aligned, not NULL", who);
  MXQ_REQUIRE(bytes >= mxq_orthogonalize_workspace(batch, R, C, odt), "%s: workspace is too small (%lld bytes)", who, (long long)bytes);
  return MXQ_OK;
}

Plan plan_of(int64_t batch, int64_t R, int64_t C, const mxq_newton_schulz& ns) {
  return Plan{batch, R, C, ns.steps, ns.a, ns.b, ns.c, ns.eps};
}

}  // namespace

}  // namespace mxq

using namespace mxq;

extern "C" {

int64_t mxq_orthogonalize_workspace(int64_t batch, int64_t R, int64_t C, mxq_dtype odt) {
  if (batch < 0 || batch > 65535 || R < 1 || R > kMaxSide || C < 1 || C > kMaxSide) return 0;
  if (odt != MXQ_DT_F32 && odt != MXQ_DT_BF16) return 0;
  const int64_t one = lay_out(nullptr, nullptr, 1, R, C, odt == MXQ_DT_F32);
  if (batch > INT64_MAX / one) return 0;
  return lay_out(nullptr, nullptr, batch, R, C, odt == MXQ_DT_F32);
}

mxq_status mxq_orthogonalize(const void* x, mxq_dtype dt, int64_t batch, int64_t R, int64_t C, const mxq_newton_schulz* cfg,
                             void* out, mxq_dtype odt, void* workspace, int64_t workspace_bytes, hipStream_t st) {
  const mxq_status s = check("mxq_orthogonalize", batch, R, C, cfg, dt, odt, workspace, workspace_bytes);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(batch == 0 || (x && out), "mxq_orthogonalize: NULL matrix");
  MXQ_REQUIRE(aligned_to(x, dt == MXQ_DT_F32 ? 4 : 2) && aligned_to(out, odt == MXQ_DT_F32 ? 4 : 2),
              "mxq_orthogonalize: x and out must be aligned to their elements");
  MXQ_REQUIRE_DEVICE();
  if (batch == 0) return ok();
  const Source src{x, nullptr, R * C, 0.f, 0.f, 1.f, 0, nullptr};
  Args last{};
  last.param = out;
  return launched(run<false>(plan_of(batch, R, C, *cfg), src, dt, odt, last, static_cast<uint8_t*>(workspace), st),
                  "mxq_orthogonalize");
}

mxq_status mxq_muon(void* param, mxq_dtype param_dt, const void* grad, mxq_dtype grad_dt, float* m, uint16_t* copy,
                    int64_t batch, int64_t R, int64_t C, const mxq_muon_config* cfg, const mxq_adamw_control* control,
                    void* workspace, int64_t workspace_bytes, hipStream_t st) {
  MXQ_REQUIRE(cfg != nullptr, "mxq_muon: config is NULL");
  const mxq_status s = check("mxq_muon", batch, R, C, &cfg->ns, grad_dt, param_dt, workspace, workspace_bytes);
  if (s != MXQ_OK) return s;
  MXQ_REQUIRE(batch == 0 || (param && grad && m), "mxq_muon: NULL tensor");
  MXQ_REQUIRE(aligned_to(param, param_dt == MXQ_DT_F32 ? 4 : 2) && aligned_to(grad, grad_dt == MXQ_DT_F32 ? 4 : 2) &&
                  aligned_to(m, 4) && aligned_to(copy, 2),
              "mxq_muon: tensors must be aligned to their elements");
  MXQ_REQUIRE(cfg->momentum >= 0 && cfg->momentum < 1, "mxq_muon: momentum must be in [0, 1)");
  MXQ_REQUIRE(cfg->nesterov == 0 || cfg->nesterov == 1, "mxq_muon: nesterov must be 0 or 1");
  MXQ_REQUIRE(std::isfinite((float)cfg->weight_decay) && std::isfinite((float)cfg->scale), "mxq_muon: weight_decay and scale must be finite in fp32");
  MXQ_REQUIRE(aligned_to(control, 16), "mxq_muon: control must be 16-byte aligned");
  MXQ_REQUIRE_DEVICE();
  if (batch == 0) return ok();
  const Source src{grad, m, R * C, (float)cfg->momentum, (float)(1 - cfg->momentum), (float)cfg->grad_scale, cfg->nesterov, control};
  Args last{};
  last.param = param, last.copy = copy;
  last.lr = (float)cfg->lr, last.decay = (float)cfg->weight_decay, last.scale = (float)cfg->scale;
  last.grad_scale = (float)cfg->grad_scale, last.control = control;
  if (!control && !(std::isfinite(last.lr) && std::isfinite(last.grad_scale))) return ok();  // (a step to skip)
  return launched(run<true>(plan_of(batch, R, C, cfg->ns), src, grad_dt, param_dt, last, static_cast<uint8_t*>(workspace), st),
                  "mxq_muon");
}

}  // extern "C"
