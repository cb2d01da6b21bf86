/*
 * mxq.h -- C ABI of libmxq: MX microscaling quantisation and block-scaled
 * GEMMs for AMD Instinct MI355X (gfx950).
 *
 * The operations follow these web pages:
 *  - torchtitan-npu feature guide "低精度训练特性（MXFP8 / HiFloat8）",
 *    sections "线性层低精度" (MXFP8 linear: per-block quantisation with 32
 *    elements sharing one scale, forward, input-gradient and weight-gradient
 *    GEMMs in FP8, output returned at higher precision) and "MoE 专家层低精度"
 *    (grouped expert GEMMs; grouped per-block quantisation of the
 *    weight-gradient operands).
 *  - MindSpeed pull request 3852 (--fp8-quant-fb-split), "主要改动": expert
 *    weights quantised on both axes at once in the forward pass, or on the
 *    forward reduction axis only with the backward axis re-quantised later.
 *  - "AMCT FakeQuant 模拟伪量化工具包：MXFP4 推理精度验证与 QAT 训练实践",
 *    section 2 "MXFP4 数值模型" and section 3.3 (MXFP4 quant-dequant).
 * The pages leave the MXFP8 shared-exponent rule open; the library uses the
 * OCP MX v1.0 rule (shared = floor(log2(amax)) - 8, elements rounded to
 * nearest-even and saturated at +-448, all-zero block -> scale byte 0).
 *
 * Conventions shared by every entry point
 *  - Tensors are row-major and live in device memory of the current HIP
 *    device; host pointers are never accepted for tensor arguments.
 *  - Ownership: the caller allocates and frees every buffer.  The library
 *    never allocates or frees device memory, never synchronises, never copies
 *    group sizes back to the host and keeps no per-call state; it only caches
 *    the per-device architecture check and a thread-local error message.
 *  - Work is enqueued on the caller's stream `st` (0 = the null stream) as
 *    kernel launches only (no memset, copy or synchronisation), so a
 *    sequence of calls can be recorded into a HIP graph and replayed.
 *    Outputs must not alias inputs.  Code arrays (quantiser outputs, GEMM
 *    operands) must be 16-byte aligned; each entry point states what it
 *    requires of its other pointers (bf16 inputs 2 bytes, fp32 data and
 *    packed scale arrays that are written as dwords 4 bytes) and rejects a
 *    pointer that breaks it with MXQ_ERR_INVALID_ARGUMENT.
 *  - A quantised MXFP8 operand is `codes[rows][Kp]` (one E4M3 byte per
 *    element, the reduction axis K contiguous, Kp = ceil32(K), padding codes
 *    0x00) plus its scales: one E8M0 byte (value 2^(byte-127)) per row and
 *    block of 32, in 128-row groups -- the scale of row r, block b is byte
 *    (((r/128) * (Kp/32) + b) * 32 + r%32) * 4 + (r/32)%4 of an array of
 *    ceil128(rows) * (Kp/32) bytes ("scales[ceil128(rows)/128][Kp/32][32][4]").
 *    A dword holds the scales of rows r, r+32, r+64, r+96 of a group for one
 *    block, and a group's blocks are 128 bytes apart, which is how a GEMM
 *    tile fetches them.  Bytes of rows past `rows` are not written.  A row
 *    range whose first row is a multiple of 128 is itself a valid operand
 *    (its scale array starts at byte first_row * (Kp/32)).
 *  - "row" copy: blocks along the contiguous dim of the input.  "colT" copy:
 *    the quantised transpose, blocks running down the columns of the input.
 *  - Errors: every entry point validates its host-visible arguments first
 *    and returns a status (never aborts); on failure `mxq_last_error()`
 *    describes it.  Faults inside kernels surface at the caller's next
 *    synchronisation of the stream.  Group ends live on the device and are a
 *    precondition (non-decreasing, last <= rows); kernels clamp them so that a
 *    malformed array never makes them access memory out of bounds, and
 *    `mxq_validate_group_end` checks them on the device.
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MXQ_ABI_VERSION 9
#define MXQ_BLOCK 32          /* elements per MX block; fixed */
#define MXQ_MAX_GROUPS 1024   /* largest G the grouped entry points accept */
/* E4M3 GEMM reductions of at most this many elements (dense and ragged M: K;
 * ragged K: an expert's token count) run with exact 8-product MFMA groups;
 * see mxq_gemm. */
#define MXQ_EXACT_GROUPS_MAX_K 1024
/* Code bytes per operand row the GEMMs address (K for E4M3, K/2 for E2M1)
 * must stay below this: a 256-row tile of codes is addressed with 32-bit
 * offsets.  So K <= 2^23 - 32 (E4M3) and K <= 2^24 - 32 (E2M1). */
#define MXQ_GEMM_MAX_ROW_BYTES (1 << 23)

typedef enum {
    MXQ_OK = 0,
    MXQ_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, misaligned pointer, bad enum */
    MXQ_ERR_UNSUPPORTED = 2,      /* valid request the library does not implement */
    MXQ_ERR_DEVICE = 3,           /* no HIP device, or the current device is not gfx950 */
    MXQ_ERR_LAUNCH = 4,           /* the HIP runtime rejected a kernel launch */
    MXQ_STATUS_MAX_ENUM = 0x7FFFFFFF
} mxq_status;

/* Every enum of this header spans the int32 range (its *_MAX_ENUM member), so
 * a caller passing any int32 value (for instance through a foreign-function
 * binding) passes a valid value of the type; values outside the listed ones
 * are rejected with MXQ_ERR_INVALID_ARGUMENT or MXQ_ERR_UNSUPPORTED. */

/* axis bitmask for the quantisers; ROW|COLT is the dual-axis quantisation
 * (both copies from one read of the input). */
enum { MXQ_AXIS_ROW = 1, MXQ_AXIS_COLT = 2 };

/* element format of a GEMM operand: E4M3 codes (one byte each, written by
 * the MXFP8 quantisers) or E2M1 codes (two per byte, element 2j in the low
 * nibble of byte j, written by mxq_quantize_fp4) */
typedef enum { MXQ_FMT_E4M3 = 0, MXQ_FMT_E2M1 = 1, MXQ_FMT_MAX_ENUM = 0x7FFFFFFF } mxq_fmt;

/* grouped GEMM modes */
typedef enum {
    MXQ_GG_RAGGED_M = 0, /* expert forward / input gradient: rows split into groups */
    MXQ_GG_RAGGED_K = 1, /* expert weight gradient: reduction axis split into groups */
    MXQ_GG_MAX_ENUM = 0x7FFFFFFF
} mxq_gg_mode;

/* Version of this ABI (MXQ_ABI_VERSION of the built library). */
int mxq_abi_version(void);

/* Message for the last failed call on this thread ("" if none). Owned by the
 * library; valid until the next call on the same thread. */
const char* mxq_last_error(void);

/* MXQ_OK iff HIP device `device` exists and is gfx950. */
mxq_status mxq_device_check(int device);

/* Row pitch (ldq) for a grouped token-axis copy of T rows in G groups: at
 * least T + 31 G, an upper bound of sum_g ceil32(m_g), rounded up to an odd
 * multiple of 256.  Rows then start on 128-byte lines (E4M3 rows of ldq
 * bytes, E2M1 rows of ldq/2), which the weight-gradient GEMM loads whole,
 * and consecutive rows do not fall in the same memory channels (a pitch of
 * 2^10 x 129 bytes measured 1.2x slower).  Any ldq that is a multiple of 32
 * and at least sum_g ceil32(m_g) stays valid.  Pure host arithmetic. */
int64_t mxq_grouped_cols_max(int64_t T, int32_t G);

/* Bytes of a quantised GEMM operand of `rows` rows and reduction length K in
 * format fmt (MXQ_FMT_E4M3 or MXQ_FMT_E2M1), Kp = ceil32(K): *code_bytes =
 * rows * Kp (E4M3) or rows * Kp / 2 (E2M1); *scale_bytes = ceil128(rows) *
 * Kp / 32 (the operand scale layout below).  The row copy of an R x C matrix
 * is (R, C), its colT copy (C, R), a grouped token-axis copy (C, ldq), an
 * MXFP4 operand (rows, L).  The shape-only counterpart of the quantisers, so
 * a caller can allocate their outputs.  Pure host arithmetic; rows, K >= 1,
 * outputs non-NULL, else MXQ_ERR_INVALID_ARGUMENT. */
mxq_status mxq_operand_sizes(int64_t rows, int64_t K, int fmt, int64_t* code_bytes, int64_t* scale_bytes);

/*
 * MXFP8 quantisation of a bf16 matrix x [R][ldx] (R x C used), the per-block
 * quantisation of activations and weights of the torchtitan-npu guide
 * ("线性层低精度"), with the axis choice of MindSpeed PR 3852 ("主要改动").
 *   axis_mask & MXQ_AXIS_ROW : q_row [R][Cp], s_row (R rows, Cp/32 blocks,
 *                              operand layout), Cp = ceil32(C)
 *   axis_mask & MXQ_AXIS_COLT: q_colT [C][Rp], s_colT (C rows, Rp/32 blocks,
 *                              operand layout), Rp = ceil32(R)
 * Pointers for an axis not requested may be NULL.  Both axes together read
 * x once (dual-axis quantisation).  R, C >= 1; ldx >= C.  x 2-byte aligned
 * (16-byte alignment with ldx % 8 == 0 takes the vector load path), q_row
 * and q_colT 16-byte, s_row 4-byte aligned; s_colT any alignment.
 */
mxq_status mxq_quantize(const uint16_t* x, int64_t R, int64_t C, int64_t ldx, int axis_mask,
                        uint8_t* q_row, uint8_t* s_row, uint8_t* q_colT, uint8_t* s_colT,
                        hipStream_t st);

/*
 * mxq_quantize over `batch` matrices in one launch: matrix b is
 * x + b * x_stride (bf16 elements), each [R][ldx] (R x C used) -- the
 * per-expert weights [G][K][N] of the MoE layer (torchtitan-npu guide,
 * "MoE 专家层低精度"; MindSpeed PR 3852, "主要改动").  The outputs of
 * matrix b are exactly what mxq_quantize writes for it, back to back:
 * q_row + b*R*Cp, s_row + b*ceil128(R)*(Cp/32), q_colT + b*C*Rp,
 * s_colT + b*ceil128(C)*(Rp/32) (each scale array the full operand scale
 * layout of its matrix).  1 <= batch <= 65535;
 * x_stride >= (R-1)*ldx + C when batch > 1.
 */
mxq_status mxq_quantize_batched(const uint16_t* x, int64_t batch, int64_t R, int64_t C, int64_t ldx,
                                int64_t x_stride, int axis_mask, uint8_t* q_row, uint8_t* s_row,
                                uint8_t* q_colT, uint8_t* s_colT, hipStream_t st);

/*
 * Grouped token-axis MXFP8 quantisation for the expert weight gradient
 * (torchtitan-npu guide, "MoE 专家层低精度").  x bf16 [T][ldx] (T x C used);
 * group g owns rows [end_{g-1}, end_g) with end_g = group_end[g] (device
 * int32 [G], cumulative, end_{-1} = 0).
 *   MXQ_AXIS_COLT: q_colT [C][ldq], s_colT (C rows, ldq/32 blocks,
 *     operand layout).  Blocks restart at
 *     each group start; group g occupies columns [P_g, P_g + ceil32(m_g)),
 *     P_g = sum_{j<g} ceil32(m_j), its tail zero-padded.  Columns at and past
 *     P_G are not written.  ldq % 32 == 0; ldq >= sum_g ceil32(m_g) is a
 *     precondition (mxq_grouped_cols_max(T, G) always suffices); blocks that
 *     would fall past ldq are dropped.
 *   MXQ_AXIS_ROW: q_row [T][Cp], s_row (T rows, operand layout), identical to
 *     mxq_quantize's row copy; with COLT the input is read once.
 * 1 <= G <= MXQ_MAX_GROUPS; T, C >= 1.
 */
mxq_status mxq_quantize_grouped(const uint16_t* x, int64_t T, int64_t C, int64_t ldx,
                                const int32_t* group_end, int32_t G, int64_t ldq, int axis_mask,
                                uint8_t* q_row, uint8_t* s_row, uint8_t* q_colT, uint8_t* s_colT,
                                hipStream_t st);

/*
 * MXFP4 quantise-dequantise of the AMCT FakeQuant article (section 2 and
 * section 3.3).  x, y fp32 [rows][L], L = last dim of the caller's tensor.
 * Each row is zero-padded to Lp = ceil32(L) on its own, so rows never share a
 * block.  Per block: scale = 2^round(log2(max|x|/6)) with the raw scale
 * max|x|/6 clamped at 2^-30 (round taken exactly); each element becomes the
 * E2M1 codebook value {0,0.5,1,1.5,2,3,4,6} nearest to |x|/scale, ties to the
 * larger magnitude, everything from 5 up saturating to 6; y = sign(x) * code
 * * scale (the sign of x is kept also when the code is 0).
 * Optional outputs (NULL to skip): codes [rows][Lp/2] E2M1 nibbles, element
 * 2j in the low nibble of byte j, nibble = sign<<3 | codebook index (the OCP
 * E2M1 bit pattern); scales [rows][Lp/32] E8M0 bytes, row-major (these are
 * not GEMM operands).  NaN/Inf inputs are outside the contract.  rows, L >= 1.
 */
mxq_status mxq_qdq_fp4(const float* x, float* y, int64_t rows, int64_t L,
                       uint8_t* codes, uint8_t* scales, hipStream_t st);

/*
 * MXFP4 quantise-dequantise with a runtime scale factor and the clipped-STE
 * saturation mask (AMCT FakeQuant article: scale_factor among the section 2
 * parameters, passed to the op as 6 / scale_factor in section 3.3; the
 * clipped straight-through estimator of section 4.1).  As mxq_qdq_fp4, with
 * scale = 2^round(log2(max|x| / scale_factor)) (raw scale clamped at 2^-30,
 * round taken exactly); scale_factor = 6 gives mxq_qdq_fp4's results.
 * scale_factor must be a normal fp32 value in [2^-64, 2^64), else
 * MXQ_ERR_INVALID_ARGUMENT.  Blocks whose scale would exceed 2^127, or whose
 * dequantised values overflow fp32, are outside the contract (only possible
 * for scale_factor < 6 and inputs near the fp32 maximum).
 * sat_mask (optional, NULL to skip; 4-byte aligned): device bytes
 * [rows][Lp/8]; bit j of byte k is element 8k + j of the row, set iff
 * |x| > 6 * scale (the element was clipped to the largest code); bits of the
 * padding past L are 0.  codes and scales as for mxq_qdq_fp4.
 */
mxq_status mxq_qdq_fp4_ex(const float* x, float* y, int64_t rows, int64_t L, float scale_factor,
                          uint8_t* codes, uint8_t* scales, uint8_t* sat_mask, hipStream_t st);

/*
 * Clipped-STE backward of the MXFP4 quantiser (AMCT FakeQuant article,
 * section 4.1): grad_x = 0 where the forward clipped the element (its
 * sat_mask bit, as written by mxq_qdq_fp4_ex for the same rows and L, is
 * set), grad_x = grad_y elsewhere.  grad_y, grad_x fp32 [rows][L] on the
 * device; grad_x may be grad_y (in place) but must not partly overlap it.
 * All three pointers 4-byte aligned; rows, L >= 1.
 */
mxq_status mxq_ste_backward_fp4(const float* grad_y, const uint8_t* sat_mask, float* grad_x,
                                int64_t rows, int64_t L, hipStream_t st);

/*
 * Host only (no device needed): the exponent threshold mxq_qdq_fp4_ex uses
 * for a scale factor.  With scale_factor * sqrt(2) = (1 + t) * 2^F, a block's
 * exponent is E - F + (m >= T) for max|x| = (1 + m / 2^23) * 2^E, where
 * T = ceil(t * 2^23) (T = 2^23: never).  Writes F and T; rejects factors
 * outside [2^-64, 2^64) with MXQ_ERR_INVALID_ARGUMENT.
 */
mxq_status mxq_fp4_scale_threshold(float scale_factor, int32_t* F, uint32_t* T);

/*
 * MXFP4 GEMM operand quantisation: the same block rule and element rounding
 * as mxq_qdq_fp4_ex (AMCT FakeQuant article, section 2; scale_factor 6 is the
 * default) without the dequantised output, with the scales in the layout
 * the GEMMs read.  x fp32 [rows][L] device, 4-byte aligned; each row zero-
 * padded to Lp = ceil32(L).  codes: device bytes [rows][Lp/2], 16-byte
 * aligned, E2M1 nibbles as for mxq_qdq_fp4 (element 2j in the low nibble of
 * byte j).  scales: E8M0 bytes in the GEMM operand layout of the MXFP8
 * quantisers (row r, block b at byte (((r/128)*(Lp/32) + b)*32 + r%32)*4 +
 * (r/32)%4 of a ceil128(rows)*(Lp/32)-byte array; bytes of rows past `rows`
 * are not written).  A GEMM operand with K = Lp.  scale_factor as for
 * mxq_qdq_fp4_ex.  rows, L >= 1.
 */
mxq_status mxq_quantize_fp4(const float* x, int64_t rows, int64_t L, float scale_factor, uint8_t* codes,
                            uint8_t* scales, hipStream_t st);

/*
 * Grouped token-axis MXFP4 GEMM operands for the expert weight gradient (the
 * optional MXFP4 of routed experts, torchao_npu RFC section 3.4, with the
 * numeric model of the AMCT FakeQuant article, section 2): x fp32 [T][ldx]
 * (T x C used) on the device, 4-byte aligned; group_end as for
 * mxq_quantize_grouped.  Blocks of 32 run down the token axis within each
 * group and restart at each group start; group g occupies padded positions
 * [P_g, P_g + ceil32(m_g)), P_g = sum_{j<g} ceil32(m_j), its tail zero.  The
 * block rule and element rounding are mxq_quantize_fp4's (scale_factor 6 by
 * default, same range).  codes: device bytes [C][ldq/2], 16-byte aligned,
 * E2M1 nibbles with position 2j in the low nibble of byte j; scales: E8M0
 * bytes in the GEMM operand layout (C rows, ldq/32 blocks).  Positions at
 * and past P_G are not written.  ldq % 32 == 0; ldq >= sum_g ceil32(m_g) is
 * a precondition (mxq_grouped_cols_max(T, G) suffices); blocks past ldq are
 * dropped.  1 <= G <= MXQ_MAX_GROUPS; T, C >= 1.  The operands of
 * mxq_grouped_gemm(MXQ_GG_RAGGED_K, .., MXQ_FMT_E2M1).
 */
mxq_status mxq_quantize_fp4_grouped(const float* x, int64_t T, int64_t C, int64_t ldx,
                                    const int32_t* group_end, int32_t G, int64_t ldq, float scale_factor,
                                    uint8_t* codes, uint8_t* scales, hipStream_t st);

/*
 * Block-scaled GEMM C[m][n] = sum_k deq(A)[m][k] * deq(B)[n][k] (the FP8
 * linear GEMMs of the torchtitan-npu guide, "线性层低精度"), fp32
 * accumulation and fp32 output.  A codes [M][K] + scales (M rows);
 * B codes [N][K] + scales (N rows), scales in the operand layout; C fp32 [M][ldc].
 * Forward Y = X W: A = row copy of X, B = colT copy of W [K][N].
 * Input gradient dX = dY W^T: A = row copy of dY, B = row copy of W.
 * Weight gradient dW = X^T dY: A = colT copy of X, B = colT copy of dY.
 * fmt MXQ_FMT_E2M1 (MXFP4 operands: the optional MXFP4 of routed experts in
 * the torchao_npu RFC's "mix" recipe, section 3.4, with the AMCT article's
 * numeric model, taken as a GEMM on the codes): A codes [M][K/2], B codes
 * [N][K/2] as written by mxq_quantize_fp4 (rows of K elements), scales in
 * the same operand layout.
 * M, N >= 1; K >= 32, K % 32 == 0; code bytes per row (K, or K/2 for
 * E2M1) below MXQ_GEMM_MAX_ROW_BYTES; ldc >= N.  A, B 16-byte aligned, sA,
 * sB and C 4-byte aligned (else MXQ_ERR_INVALID_ARGUMENT).  Unknown fmt:
 * MXQ_ERR_UNSUPPORTED.
 */
mxq_status mxq_gemm(const uint8_t* A, const uint8_t* sA, const uint8_t* B, const uint8_t* sB,
                    float* C, int64_t M, int64_t N, int64_t K, int64_t ldc, mxq_fmt fmt,
                    hipStream_t st);

/*
 * Grouped block-scaled GEMM over ragged expert groups (torchtitan-npu guide,
 * "MoE 专家层低精度"); group_end device int32 [G] as for mxq_quantize_grouped.
 *   MXQ_GG_RAGGED_M: A [M][K] (+ scales of M rows); B [G][N][K] with G
 *     scale arrays of N rows each, expert g's at byte g * ceil128(N) * (K/32);
 *     C fp32 [M][N].  Rows of group g use expert B[g]; rows at or past
 *     group_end[G-1] are not written.  K >= 32, K % 32 == 0.
 *     Expert forward: A = row copy of X, B[g] = colT copy of W[g] [K][N].
 *     Expert input gradient: A = row copy of dY, B[g] = row copy of W[g].
 *   MXQ_GG_RAGGED_K: A [M][K] and B [N][K] are grouped token-axis copies
 *     (K = their ldq); C fp32 [G][M][N] with
 *     C[g] = sum over group g's padded columns of deq(A) deq(B);
 *     an empty group gets exact zeros.  Expert weight gradient:
 *     A = grouped copy of X (M = hidden), B = grouped copy of dY (N = ffn).
 *     The kernel reads each group's rows from the 128-byte line at or below
 *     its first column and zeroes the columns before it, so the columns
 *     before P_g must hold quantised data (the earlier groups' blocks, as the
 *     grouped quantisers write them: no positions lie between groups).
 * fmt MXQ_FMT_E2M1: MXFP4 operands as for mxq_gemm (codes K/2 bytes per row,
 * expert g's B codes at byte g * N * K/2); for MXQ_GG_RAGGED_K the grouped
 * token-axis copies of mxq_quantize_fp4_grouped (K = their ldq).
 * M, N >= 1; K >= 32, K % 32 == 0; code bytes per row below
 * MXQ_GEMM_MAX_ROW_BYTES (as for mxq_gemm); 1 <= G <= MXQ_MAX_GROUPS.  A, B
 * 16-byte aligned, sA, sB and C 4-byte aligned (else
 * MXQ_ERR_INVALID_ARGUMENT).
 */
mxq_status mxq_grouped_gemm(mxq_gg_mode mode, const uint8_t* A, const uint8_t* sA,
                            const uint8_t* B, const uint8_t* sB, float* C,
                            int64_t M, int64_t N, int64_t K,
                            const int32_t* group_end, int32_t G, mxq_fmt fmt, hipStream_t st);

/*
 * Device-side check of a group_end array: writes 0 to *flag (device int32)
 * if group_end is non-decreasing, starts >= 0 and ends <= T, else 1 + the
 * index of the first offending entry.  Enqueued on `st`; read *flag after
 * synchronising.  1 <= G <= MXQ_MAX_GROUPS.
 */
mxq_status mxq_validate_group_end(const int32_t* group_end, int32_t G, int64_t T,
                                  int32_t* flag, hipStream_t st);

/* ------------------------------------------------------------------ around the expert GEMMs
 * Routing, the move between token order and expert order, and the optimiser
 * step of an MoE layer.  T = 0 tokens (and tensors without elements) are
 * valid; pointers of empty arrays may then be NULL. */

/* element type of a float tensor argument (this and the enums below span every int32) */
typedef enum {
    MXQ_DT_F32 = 0,
    MXQ_DT_BF16 = 1,
    MXQ_DT_MIN_ENUM = -0x7FFFFFFF - 1,
    MXQ_DT_MAX_ENUM = 0x7FFFFFFF
} mxq_dtype;

typedef enum {
    MXQ_SCORE_SOFTMAX = 0,
    MXQ_SCORE_SIGMOID = 1,
    MXQ_SCORE_MIN_ENUM = -0x7FFFFFFF - 1,
    MXQ_SCORE_MAX_ENUM = 0x7FFFFFFF
} mxq_score;

#define MXQ_MAX_TOPK 32          /* largest top_k */
#define MXQ_MAX_ROUTE_GROUPS 64  /* largest n_group */

/* How a token's experts are chosen among E (<= MXQ_MAX_GROUPS) experts.
 *  - score: s = softmax of the row's logits, or their sigmoid.
 *  - A logit at or below the lowest finite bf16 value (-3.3895314e38, so
 *    -inf and both types' lowest values) masks its expert: score 0, never
 *    chosen, not counted by a softmax.
 *  - An expert ranks by its key: s + bias[e], or its logit where bias is
 *    NULL.  A NaN key ranks below every number, and one of -inf (a bias that
 *    bars its expert) is not chosen.  (Rows with keys that are not finite take
 *    several times as long as others, so a bias of -inf costs all rows; masked
 *    logits cost nothing.)
 *  - n_group > 1 splits the experts into n_group equal runs; a group's total
 *    is the sum of its best `group_top` (1 or 2) s + bias (s without bias)
 *    over unmasked experts; only the topk_group best groups' experts can be
 *    chosen.  E must be a multiple of n_group.  (Totals are of scores also where
 *    experts rank by logits: groups whose scores are one number in 64 bits, as
 *    sigmoids of 40 and 45 are, tie.)
 *  - The top_k largest keys are chosen, largest first; ties go to the lowest
 *    index (experts and groups).  Order is that of the keys and totals in
 *    64-bit arithmetic.  A row with fewer available experts than top_k ends
 *    in index -1 with weight 0.
 *  - The weight of a chosen expert is scale * s, or with renormalise
 *    scale * s / (sum of the chosen s), taken so that scores which underflow
 *    still have their ratio.  The bias has no part in it.  NaN and +inf logits follow the arithmetic. */
typedef struct {
    int32_t score;       /* mxq_score */
    int32_t top_k;       /* 1 .. min(E, MXQ_MAX_TOPK) */
    int32_t n_group;     /* 1 .. MXQ_MAX_ROUTE_GROUPS */
    int32_t topk_group;  /* 1 .. n_group */
    int32_t group_top;   /* 1 or 2 */
    int32_t renormalise; /* 0 or 1 */
    float scale;         /* finite */
} mxq_route_config;

/* Workspace bytes of mxq_route with expert order, or of mxq_expert_order.
 * Pure host arithmetic; 0 for arguments those would refuse.  The workspace
 * needs no initialisation and holds nothing between calls. */
int64_t mxq_expert_order_workspace(int64_t T, int32_t top_k, int32_t E);

/* Route T tokens: logits [T][E] (type dt, row stride ld >= E elements) ->
 * idx int32 [T][top_k] and weights fp32 [T][top_k].  bias fp32 [E] or NULL.
 * group_end, row_token, slot: all NULL, or all given (then also a 16-byte
 * aligned workspace of mxq_expert_order_workspace bytes) to have the expert
 * order of mxq_expert_order too.  T * top_k < 2^31. */
mxq_status mxq_route(const void* logits, mxq_dtype dt, int64_t T, int32_t E, int64_t ld, const float* bias,
                     const mxq_route_config* cfg, int32_t* idx, float* weights, int32_t* group_end,
                     int32_t* row_token, int32_t* slot, void* workspace, int64_t workspace_bytes,
                     hipStream_t st);

/* Expert order of a routing: the pairs (t, k) sorted by expert, pairs of one
 * expert in the order of t * top_k + k (so the result does not depend on
 * timing).  idx int32 [T][top_k]; entries outside [0, E) are dropped.
 *  group_end int32 [E]: the cumulative ends that the grouped entry points take.
 *  row_token int32 [T * top_k]: the token of each expert-ordered row, -1 for
 *    rows past the last.
 *  slot int32 [T][top_k]: the row of each pair, -1 for a dropped one. */
mxq_status mxq_expert_order(const int32_t* idx, int64_t T, int32_t top_k, int32_t E, int32_t* group_end,
                            int32_t* row_token, int32_t* slot, void* workspace, int64_t workspace_bytes,
                            hipStream_t st);

/* Gradient of the weights of mxq_route with respect to the logits for the
 * chosen experts idx (entries of a row distinct; outside [0, E): no
 * gradient): dweights fp32 [T][top_k] -> dlogits [T][E] (type dt, row stride
 * ldd), every element written, 0 at masked experts.  cfg: score, top_k,
 * renormalise and scale are used. */
mxq_status mxq_route_backward(const void* logits, mxq_dtype dt, int64_t T, int32_t E, int64_t ld,
                              const mxq_route_config* cfg, const int32_t* idx, const float* dweights,
                              void* dlogits, int64_t ldd, hipStream_t st);

/* out[t] = sum_k weights[t][k] * y[slot[t][k]]: the experts' rows back in
 * token order.  y [rows][H] (row stride ldy), slot int32 [T][top_k] (entries
 * outside [0, rows) take no part; a token with none gets zeros), weights fp32
 * [T][top_k] or NULL for 1 (then also the gradient of a dispatch), out
 * [T][H] (row stride ldo).  Sums in fp32 in the order of k, rounded once.
 * top_k <= MXQ_MAX_TOPK, T and rows < 2^31, H < 2^29. */
mxq_status mxq_combine(const void* y, mxq_dtype ydt, int64_t rows, int64_t ldy, const int32_t* slot,
                       const float* weights, int64_t T, int32_t top_k, int64_t H, void* out, mxq_dtype odt,
                       int64_t ldo, hipStream_t st);

/* Gradient of mxq_combine: dy[slot[t][k]] = weights[t][k] * dout[t] and
 * dweights[t][k] = <dout[t], y[slot[t][k]]> (0 for a dropped pair; sums in
 * fp32, in an order that does not depend on timing).  weights NULL: 1.
 * dweights NULL: not computed, y is not read and may be NULL.  dy NULL: not
 * computed.  No two pairs may share a row; rows that no pair names are not
 * written.  With weights and dweights NULL this is the dispatch of tokens
 * into expert order: dy[slot[t][k]] = dout[t]. */
mxq_status mxq_combine_backward(const void* dout, mxq_dtype dt, int64_t ldd, const void* y, mxq_dtype ydt,
                                int64_t ldy, const int32_t* slot, const float* weights, int64_t T, int32_t top_k,
                                int64_t H, int64_t rows, void* dy, mxq_dtype dydt, int64_t lddy, float* dweights,
                                hipStream_t st);

/* State format of mxq_adamw: fp32, or MXFP8: E4M3 codes with an E8M0 scale
 * byte for every 32 consecutive elements of the tensor. */
typedef enum {
    MXQ_ADAMW_F32 = 0,
    MXQ_ADAMW_MXFP8 = 1,
    MXQ_ADAMW_MIN_ENUM = -0x7FFFFFFF - 1,
    MXQ_ADAMW_MAX_ENUM = 0x7FFFFFFF
} mxq_adamw_format;

/* One tensor of n contiguous elements.  fp32 arrays 4-byte aligned, bf16 2. */
typedef struct {
    void* param;           /* fp32 or bf16, updated */
    const void* grad;      /* fp32 or bf16 */
    void* m;               /* first moment: fp32 [n], or E4M3 codes [n]; updated */
    void* v;               /* second moment v: fp32 [n], or E4M3 codes of sqrt(v) [n]; updated */
    uint8_t* m_scale;      /* MXFP8: E8M0 bytes [ceil(n / 32)], else NULL */
    uint8_t* v_scale;      /* likewise */
    void* copy;            /* bf16 [n]: the new parameters rounded to bf16, or NULL */
    int64_t n;             /* elements, >= 0 */
    double decay_scale;    /* times weight_decay (0: none for this tensor) */
} mxq_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay; /* 0 <= beta < 1, eps >= 2^-126 (normal in fp32) */
    double grad_scale;                          /* multiplies every gradient */
    int64_t step;                               /* of this update, 1 for the first */
    uint32_t seed;                              /* of the stochastic rounding */
} mxq_adamw_config;

/* What changes from step to step, in device memory (16 bytes, 16-byte aligned), so that a
 * captured step can be replayed with new values: where given to mxq_adamw, it
 * replaces the config's lr, grad_scale, step and seed.  An lr or a grad_scale
 * that is not finite, or a step below 1, skips the step: nothing changes. */
typedef struct {
    float lr;
    float grad_scale;
    int32_t step;
    uint32_t seed;
} mxq_adamw_control;

/* One AdamW step of n_tensors tensors (a host array, read before the call
 * returns), all of one parameter, gradient and state type:
 *   g' = grad_scale g;  m' = beta1 m + (1 - beta1) g';  v' = beta2 v + (1 - beta2) g'^2
 *   p' = p (1 - lr wd) - lr / (1 - beta1^step) * m' / (sqrt(v') / sqrt(1 - beta2^step) + eps)
 * in fp32.  The products and sums of the moments are rounded one by one in this
 * order, without contraction; those of p' may be contracted and its quotient is
 * m' times a reciprocal (the update is within 2^-20 of itself).  p' is
 * rounded to nearest for bf16.  A grad_scale that is not finite (a gradient
 * norm or loss scale that overflowed) skips the step: nothing changes.
 * MXFP8 states hold m and r = sqrt(v); the block's scale is the smallest
 * power of two (2^(byte-127), byte >= 1) that keeps its largest finite
 * magnitude at or below 448, 0 for a block of zeros; elements are rounded
 * stochastically, y -> step * floor(y / step + u) with u in (0, 1) from a
 * counter hash of (seed, step, index of the tensor in the call, element), so
 * that moments whose change in one step is below half an E4M3 step still
 * move.  y is the element times 2^(127-byte), off by at most 2^-18 of a step
 * (u comes in steps of 2^-16, and a y that E4M3 holds stays what it is).  A positive
 * r stays positive; a moment that is not finite becomes NaN.  Zero codes
 * and scales are the state before the first step. */
mxq_status mxq_adamw(const mxq_adamw_tensor* tensors, int32_t n_tensors, mxq_dtype param_dt, mxq_dtype grad_dt,
                     mxq_adamw_format format, const mxq_adamw_config* cfg, const mxq_adamw_control* control,
                     hipStream_t st);

/* ------------------------------------------------------------------ FP8 with a scale for each block of 128
 * E4M3 codes with one fp32 scale for each block of 1 x 128 elements along the
 * reduction axis (activations, gradients) or of 128 x 128 (weights).  An
 * operand is `codes[rows][Kp]` (Kp = ceil128(K), codes past K 0x00, or NaN in a
 * block that holds a NaN) plus its scales, block by block:
 * `scales[Kp/128][rows]` (1 x 128) or `scales[Kp/128][ceil(rows/128)]` (128 x 128).
 * R = 0 (M = 0) rows are valid. */

/* Row pitch (ldq) for a grouped token-axis copy of T rows in G groups: at
 * least T + 127 G, an upper bound of sum_g ceil128(m_g), rounded up to an odd
 * multiple of 128.  Any multiple of 128 that is at least sum_g ceil128(m_g) is
 * valid.  Pure host arithmetic; 0 for bad arguments. */
int64_t mxq_grouped128_cols_max(int64_t T, int32_t G);

/* Quantise `batch` matrices x + b * x_stride, each [R][ldx] of type dt (R x C
 * used), in blocks of `tile` x 128, tile 1 or 128:
 *   amax = max(largest |x| of the block, 2^-100), scale = amax / 448,
 *   code = e4m3(448 x / amax), to nearest even (exact for bf16 x; for fp32 x the
 *   quotient is off by at most 2^-23 of itself).  A block with a NaN has a NaN
 *   scale and NaN codes; one with an infinity has an infinite scale, NaN for its
 *   infinities and 0 elsewhere.
 *   axis_mask & MXQ_AXIS_ROW : q_row [batch][R][Cp], s_row [batch][Cp/128][R]
 *                              (tile 1) or [batch][Cp/128][ceil(R/128)]
 *   axis_mask & MXQ_AXIS_COLT: the same of the transposes: q_colT [batch][C][Rp],
 *                              s_colT [batch][Rp/128][C] or [batch][Rp/128][ceil(C/128)]
 * Pointers for an axis not requested may be NULL; both axes read x once.
 * 0 <= R < 2^31, 1 <= C < 2^31 - 128, ldx >= C, 0 <= batch <= 65535,
 * x_stride >= (R-1)*ldx + C when batch > 1.  x aligned to its elements, codes
 * to 16 bytes, scales to 4. */
mxq_status mxq_quantize128(const void* x, mxq_dtype dt, int64_t batch, int64_t R, int64_t C, int64_t ldx,
                           int64_t x_stride, int tile, int axis_mask, uint8_t* q_row, float* s_row, uint8_t* q_colT,
                           float* s_colT, hipStream_t st);

/* The same in 1 x 128 blocks for one matrix x [T][ldx] whose rows are in groups
 * (group_end as for mxq_quantize_grouped):
 *   MXQ_AXIS_COLT: q_colT [C][ldq], s_colT [ldq/128][C]: blocks restart at each
 *     group start; group g occupies columns [P_g, P_g + ceil128(m_g)), P_g =
 *     sum_{j<g} ceil128(m_j), its tail zero (NaN in a block that holds a NaN).
 *     Columns at and past P_G are not written.  ldq % 128 == 0; blocks that would
 *     fall past ldq are dropped.
 *   MXQ_AXIS_ROW: as mxq_quantize128's, of all T rows.
 * 1 <= G <= MXQ_MAX_GROUPS. */
mxq_status mxq_quantize128_grouped(const void* x, mxq_dtype dt, int64_t T, int64_t C, int64_t ldx,
                                   const int32_t* group_end, int32_t G, int64_t ldq, int axis_mask, uint8_t* q_row,
                                   float* s_row, uint8_t* q_colT, float* s_colT, hipStream_t st);

/* C[m][n] = sum_k deq(A)[m][k] deq(B)[n][k] for A codes [M][K] with 1 x 128
 * blocks (sA [K/128][M]) and B codes [N][K] with blocks of b_tile x 128 (sB
 * [K/128][N] for b_tile 1, [K/128][ceil(N/128)] for 128); C [M][ldc] of type cdt.
 * fp32 C: products exact, sums in fp32.  bf16 C: a block's products are summed by
 * the FP8 matrix instruction (each group of eight keeps about 13 bits below its
 * largest product: what terms that cancel leave is off by that much of the terms),
 * the blocks in fp32.  A product of two scales below 2^-126 loses bits as fp32
 * subnormals do, and one past fp32's range is infinite (NaN where the block's
 * products add to 0); with b_tile 1 the same goes for the products' sum times sB.
 * K a positive multiple of 128 below MXQ_GEMM_MAX_ROW_BYTES; 0 <= M < 2^31,
 * 1 <= N < 2^31, ldc >= N.  A, B 16-byte aligned, scales 4-byte, C to its
 * elements. */
mxq_status mxq_gemm128(const uint8_t* A, const float* sA, const uint8_t* B, const float* sB, int b_tile, void* C,
                       mxq_dtype cdt, int64_t M, int64_t N, int64_t K, int64_t ldc, hipStream_t st);

/* Grouped products (group_end as for mxq_grouped_gemm).
 *   MXQ_GG_RAGGED_M: A [M][K] with sA [K/128][M]; B [G][N][K] in 128 x 128
 *     blocks, sB [G][K/128][ceil(N/128)]; C [M][N].  Rows of group g use B[g];
 *     rows at or past group_end[G-1] are not written.
 *   MXQ_GG_RAGGED_K: A [M][K] and B [N][K] are grouped token-axis copies (K =
 *     their ldq) in 1 x 128 blocks, sA [K/128][M], sB [K/128][N]; C [G][M][N],
 *     C[g] the sum over group g's columns, zeros for an empty group.
 * As for mxq_gemm128 otherwise; 1 <= G <= MXQ_MAX_GROUPS. */
mxq_status mxq_grouped_gemm128(mxq_gg_mode mode, const uint8_t* A, const float* sA, const uint8_t* B, const float* sB,
                               void* C, mxq_dtype cdt, int64_t M, int64_t N, int64_t K, const int32_t* group_end,
                               int32_t G, hipStream_t st);

/* ------------------------------------------------------------------ orthogonalised updates (Muon)
 * Newton-Schulz iterations on matrices u [R][C]:
 *   X = u / (|u|_F + eps), then `steps` times X = a X + (b A + c A^2) X, A = X X^T
 * (the same for u and its transpose).  a s + b s^3 + c s^5 must stay within 1.25
 * in magnitude for s in [0, 1.25], and within s for s in [1.25, 1.255], where
 * roundings may put a singular value; 3.4445, -4.7750, 2.0315 and 5 steps bring singular
 * values from 1/500 of the norm up to between 0.68 and 1.21.
 * The products are taken on fp16 operands with fp32 sums, X being kept in 22 bits.
 * How far a result is from the exact one, in the 2-norm and relative to it, before
 * it is rounded, with these coefficients and 5 steps:
 *   bf16: 2^-9 for matrices of 64 rows and columns and more; up to 2^-6 for smaller
 *     ones (the roundings of a few elements do not average out) and for those with
 *     a row or column 100 times the others and more;
 *   fp32 (every product is taken in three): about as far as the same iteration in
 *     fp32; 2^-18 for noise, 2^-14 where nearly all of a matrix lies in few directions.
 * The iteration does not converge with these coefficients, and where the polynomial's
 * slope is above 1 a step multiplies what is off: noise of 128 x 256 is off by 4e-3
 * (bf16) and 4e-6 (fp32) after 12 steps, by 1e-2 and 7e-6 after 32, matrices of a few
 * rows by up to 0.2 then (bf16).  A norm far below eps loses bits (u/eps is then small
 * in fp16).
 * A matrix with a NaN or an infinity becomes NaN; one of zeros stays zero, whatever eps. */
#define MXQ_MAX_NS_STEPS 32
typedef struct {
    double a, b, c; /* each at most 64 in magnitude */
    double eps;     /* >= 0 */
    int32_t steps;  /* 1 .. MXQ_MAX_NS_STEPS */
} mxq_newton_schulz;

/* Workspace bytes of mxq_orthogonalize with a result, or mxq_muon with parameters,
 * of type odt.  Pure host arithmetic; 0 for arguments those would refuse.  It needs
 * no initialisation and holds nothing between calls. */
int64_t mxq_orthogonalize_workspace(int64_t batch, int64_t R, int64_t C, mxq_dtype odt);

/* x [batch][R][C] of type dt, contiguous -> out [batch][R][C] of type odt, each
 * matrix by itself.  0 <= batch <= 65535; 1 <= R, C <= 2^20.  workspace 256-byte
 * aligned. */
mxq_status mxq_orthogonalize(const void* x, mxq_dtype dt, int64_t batch, int64_t R, int64_t C, const mxq_newton_schulz* cfg,
                             void* out, mxq_dtype odt, void* workspace, int64_t workspace_bytes, hipStream_t st);

typedef struct {
    mxq_newton_schulz ns;
    double lr, momentum, weight_decay; /* 0 <= momentum < 1 */
    double scale;                      /* times the orthogonalised update */
    double grad_scale;                 /* multiplies every gradient */
    int32_t nesterov;                  /* 0 or 1 */
} mxq_muon_config;

/* One Muon step of `batch` matrices [R][C], contiguous:
 *   g' = grad_scale g;  m' = momentum m + (1 - momentum) g'
 *   u = (1 - momentum) g' + momentum m' (nesterov), or m'
 *   p' = p (1 - lr wd) - lr scale orthogonalised(u)
 * param fp32 or bf16 (rounded to nearest), grad fp32 or bf16, m fp32; copy: bf16,
 * gets p' too, or NULL.  control: as for mxq_adamw, its lr and grad_scale replace
 * the config's; where one of the two is not finite, nothing changes. */
mxq_status mxq_muon(void* param, mxq_dtype param_dt, const void* grad, mxq_dtype grad_dt, float* m, uint16_t* copy,
                    int64_t batch, int64_t R, int64_t C, const mxq_muon_config* cfg, const mxq_adamw_control* control,
                    void* workspace, int64_t workspace_bytes, hipStream_t st);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H */
