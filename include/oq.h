/*
 * oq.h -- C ABI of the rotated low-bit linear layer for AMD MI355X (gfx950).
 *
 * The layer (CentriQ, arXiv 2610.06260, Sec. 4.2 Eq. 5 and App. B.2 Eq. 9;
 * OrbitQuant PR #25, "Default changes" and "Runtime work"):
 *
 *     y_t = alpha_t * sum_g s_w[o,g] * (q_a . q_w)_g  +  m_t * w1[o]  +  b[o]
 *     q_a = Q_a( R (x_t - m_t 1) )
 *
 * R is a randomised permuted block-Hadamard rotation (one or two rounds of
 * gather -> +-1 signs -> normalised Sylvester blocks of h = 32..1024) or a set
 * of dense per-32-block transforms (WUSH review, "Core claim"); Q_a is the
 * per-token absmax quantizer of CentriQ Eq. 1 (8, 6 or 4 bits) or MXFP4
 * (E2M1 elements, one E8M0 scale per 32); weights are symmetric INT4 with
 * one fp32 scale per row and group of input columns, or MXFP4.
 *
 * Conventions shared by every call
 *   - Return value: OQ_OK (0) or one of the OQ_ERR_* codes.  On error nothing
 *     has been enqueued; oq_last_error() returns a message for the calling
 *     thread.  There is no fallback path: an unsupported request fails
 *     (model card FLUX.1-schnell-OrbitQuant-W4A4, "Limitations": the fused
 *     runtime fails loudly when its kernel is unavailable).
 *   - Every data pointer is device memory owned by the caller.  The library
 *     allocates no device memory except where a call says so
 *     (oq_linear_fused with ws == NULL is rejected, not allocated).
 *     Descriptor structs (oq_rot) are host memory, read during the call only.
 *   - Calls are asynchronous on the caller's stream; none synchronises.
 *   - Matrices are row-major.  Leading dimensions are in elements unless the
 *     name ends in _bytes.  bfloat16 values are passed as uint16_t bits.
 *   - Alignment: x, y and code/weight pointers 16 bytes; leading dimensions
 *     such that every row starts 16-byte aligned.  Violations give
 *     OQ_ERR_ALIGNMENT.
 *   - Thread safety: calls may be made from several host threads; calls on
 *     one stream execute in order.
 */
#ifndef OQ_H
#define OQ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  OQ_OK = 0,
  OQ_ERR_INVALID_ARG = 1,   /* null pointer, bad size, bad enum value       */
  OQ_ERR_UNSUPPORTED = 2,   /* well-formed request this library does not run */
  OQ_ERR_ALIGNMENT = 3,     /* pointer or leading dimension misaligned      */
  OQ_ERR_WORKSPACE = 4,     /* workspace missing or too small               */
  OQ_ERR_HIP = 5            /* the HIP runtime reported a launch error      */
};

/* rotation kinds */
enum { OQ_ROT_RPBH = 1, OQ_ROT_DENSE32 = 2, OQ_ROT_KRON = 3 };

/* activation code formats (the value is the bit width for integer codes) */
enum { OQ_A8 = 8, OQ_A6 = 6, OQ_A4 = 4, OQ_MXFP4 = 0x104 };

/* weight formats for oq_quant_weight */
enum { OQ_W4 = 4, OQ_W_MXFP4 = 0x104 };

/*
 * Operand layout flag, OR-ed into afmt (OQ_A4 | OQ_TILED, OQ_A6 | OQ_TILED):
 * codes are stored as FP6 E2M3 values of the integer codes (exact for
 * |q| <= 7) in the MFMA-tiled layout below, the layout the fast GEMM reads.
 *   rows padded to a multiple of 32, K a multiple of 64; tile (r/32, kg =
 *   k / 64) is 1536 bytes at ((r/32) * (K/64) + kg) * 1536.  Within it, the
 *   32 codes of row r and k-half h (k = 64 kg + 32 h + j, j = 0..31) form a
 *   192-bit string with code j in bits [6j, 6j+6); with l = 32 h + r % 32,
 *   its bytes 0..15 sit at tile + 16 l and bytes 16..23 at tile + 1024 + 8 l.
 *   One plane is oq_tiled_bytes(rows, K) bytes.  OQ_A6 uses two planes:
 *   q = 8 qh + ql with qh = floor(q / 8) in plane 0 and ql = q - 8 qh in
 *   plane 1 (each in [-4, 7]).
 * Weights for tiled GEMMs come from oq_prepack_w4 (same layout, one plane,
 * plus scales transposed to [K/64][N_padded]).  The per-token scale
 * (a_scale) and mean arrays are unchanged.  Tiled GEMMs require group == 64.
 *
 * OQ_MXFP4 | OQ_TILED (K a multiple of 128): the MXFP4 codes and E8M0 scales
 * in the layout the MXFP4 GEMM copies whole:
 *   codes: rows padded to 32; tile (r/32, kg = k / 64) is 1024 bytes at
 *     ((r/32) * (K/64) + kg) * 1024; the 16 bytes of row r and k-half h (32
 *     E2M1 codes, code j in bits [4j, 4j+4), the bytes of the row-major
 *     layout) sit at tile + 16 (32 h + r % 32).  oq_tiled_mx_bytes(rows, K).
 *   scales: one 32-bit word per (128-wide k-slice s, row r) at byte
 *     (s * rows_padded + r) * 4, holding the E8M0 bytes of the blocks
 *     4s .. 4s+3 in order; oq_tiled_mx_bytes(rows, K) / 16 bytes, 4-byte
 *     aligned.  Padding rows carry zero codes.
 * Weights come from oq_prepack_mx.
 */
enum { OQ_TILED = 0x10000 };

/*
 * Scale flag, OR-ed into afmt for integer activation codes (OQ_A8, OQ_A6,
 * OQ_A4, tiled or not) in oq_quant_act and oq_linear_fused -- CentriQ Sec.
 * 4.2 "Scale and grid" and App. B.3 Table 3: the token's range is
 *   r = RN32((q * 2.5591) / Phi^-1(0.99975))      (evaluated in float64),
 * q the 0.9995-quantile of the d rotated magnitudes, interpolated linearly
 * between the order statistics floor(0.9995 (d - 1)) and the next one
 * (ascending); then alpha = RN32(r / qmax) and codes clip to +-qmax as in
 * Eq. 1.  Needs d % 16 == 0 and 16 <= d <= 4096; not for MXFP4.
 */
enum { OQ_SCALE_PCTL = 0x20000 };

/* Bytes of one plane of the tiled FP6 layout for `rows` rows of width K. */
size_t oq_tiled_bytes(int64_t rows, int32_t K);

/* Bytes of the tiled MXFP4 codes for `rows` rows of width K (the scale words
 * take a sixteenth of that). */
size_t oq_tiled_mx_bytes(int64_t rows, int32_t K);

/*
 * Rotation descriptor (host struct, device arrays).
 *
 * OQ_ROT_RPBH -- OrbitQuant PR #25 "Default changes" (independent extra
 *   rounds); CentriQ related-work paragraph (randomly permuted block-Hadamard
 *   basis); model card "Artifact Files" (stored deterministic rotation
 *   metadata).  Round r maps v to B_h D_{s_r} P_{pi_r} v:
 *     u[i] = signs[r][i] * v[perm[r][i]]    (gather over the whole width d)
 *     v    = (1/sqrt h) H_h u  per block of h consecutive coordinates.
 *   block: power of two in [32, 1024]; d % block == 0; rounds in {1, 2};
 *   perm: int32 [rounds][d], each row a permutation of 0..d-1 (not checked);
 *   signs: int8 [rounds][d] in {-1, +1}.
 *   The float32 results follow one fixed order: butterfly stages of stride
 *   1, 2, ..., h/2, each add/subtract rounded once, then a multiply by
 *   RN32(1/sqrt h).
 *
 * OQ_ROT_DENSE32 -- WUSH review "Core claim": one transform per 32-block,
 *   activations take T_b and weights its inverse-transpose T_b^{-T}.
 *   mats: bfloat16 [d/32][32][32] row-major, v_b = T_b x_b, 16-byte aligned.
 *   d % 32 == 0.  Weights (oq_quant_weight) use the same mats: the library
 *   forms T_b^{-T} itself in float64 (Gauss-Jordan with partial pivoting);
 *   every T_b must be invertible.
 *   Activation-side float32 results are T_b x_b rounded once to float32,
 *   the bf16 x bf16 products summed in float64 (exact whenever the products
 *   of one output span at most 32 binades, as ordinary activations do).
 */
typedef struct {
  int32_t kind;
  int32_t d;
  int32_t block;
  int32_t rounds;
  const int32_t *perm;
  const int8_t *signs;
  const uint16_t *mats;
} oq_rot;

/* Message of the last failed call on this thread ("" if none). */
const char *oq_last_error(void);

/*
 * oq_center -- CentriQ Sec. 4.2 Eq. 4: per-token mean and centered token.
 *   mean[t] = RN32(RN64(sum_j x[t][j]) / d), the sum formed in float64
 *             (exact whenever the row's exponent spread allows, which holds
 *             for ordinary activations);
 *   xc[t][j] = RN32(x[t][j] - mean[t]).
 * x: bf16 [M][ldx]; xc: float32 [M][ldxc] (may be NULL to compute the mean
 * only); mean: float32 [M].  M >= 0 (M == 0 enqueues nothing); 1 <= d <= 16384.
 */
int oq_center(const uint16_t *x, int64_t M, int32_t d, int64_t ldx,
              float *xc, int64_t ldxc, float *mean, hipStream_t stream);

/*
 * oq_rotate -- the rotation of the online activation path (OrbitQuant PR #25
 * "Runtime work": the whole pre-rotation in one kernel) with float32 output,
 * optionally after centering (CentriQ Eq. 4-5: rotate the centered token).
 * rot: required (RPBH or DENSE32); rot->d is the width.
 * x: bf16 [M][ldx]; y: float32 [M][ldy]; mean: float32 [M], required iff
 * center != 0 (DENSE32 does not support centering).
 */
int oq_rotate(const oq_rot *rot, const uint16_t *x, int64_t M, int64_t ldx,
              int center, float *mean, float *y, int64_t ldy, hipStream_t stream);

/*
 * oq_quant_act -- fused (center) -> rotate -> quantize -> pack for the
 * activations: CentriQ Eq. 1 (symmetric per-token absmax, alpha_t = r_t/qmax,
 * qmax = 2^{b-1}-1) and OrbitQuant's absmax A8; MXFP4 per WUSH review.
 *   codes for q = clamp(RNE(RN32(v * RN32(qmax / a))), -qmax, qmax) with
 *   a = max(max_j |v_tj|, RN32(1e-10)) (model card: activation normalization
 *   epsilon 1e-10); scale[t] = RN32(a / qmax).
 * afmt OQ_A8, OQ_A6: int8 codes [M][ldc_bytes]; OQ_A4: two codes per byte,
 *   element 2i in bits 3..0, two's complement, [M][ldc_bytes >= d/2];
 *   scale float32 [M]; e8m0 must be NULL.
 * afmt OQ_A4 | OQ_TILED, OQ_A6 | OQ_TILED: codes in the tiled FP6 layout
 *   (planes * oq_tiled_bytes(M, d) bytes; d % 64 == 0; ldc_bytes ignored).
 * afmt OQ_MXFP4 (rot->kind must be OQ_ROT_DENSE32, center == 0): E2M1 codes
 *   two per byte as above, sign in bit 3; e8m0 uint8 [M][d/32] with
 *   e = clamp(floor(log2 amax) - 2, -127, 127), byte = e + 127; scale NULL.
 * rot may be NULL (no rotation; integer formats only, d = ldx's row width
 *   given by the d argument).  mean: float32 [M], required iff center != 0.
 */
int oq_quant_act(const uint16_t *x, int64_t M, int32_t d, int64_t ldx,
                 const oq_rot *rot, int center, int afmt,
                 void *codes, int64_t ldc_bytes, float *scale, uint8_t *e8m0,
                 float *mean, hipStream_t stream);

/*
 * oq_quant_weight -- offline weight path (CentriQ Sec. 3 "Hadamard
 * rotation": W x = (W H^T)(H x); App. B.1: the weight absorbs P^T H^T;
 * Eq. 4: w1 = W 1 in float32 from the unquantized weight).
 *   Each row w of W [N][ldw] (float32) becomes R w (the same rotation as the
 *   activations; for DENSE32 the inverse-transposes of rot->mats, applied in
 *   float64 with one rounding to float32), then:
 *   wfmt OQ_W4: symmetric absmax INT4 per (row, group of `group` input
 *     columns), codes packed two per byte [N][K/2], scales float32 [N][K/group];
 *   wfmt OQ_W_MXFP4: E2M1 codes [N][K/2] and E8M0 bytes [N][K/32] (group 32).
 *   w1 (nullable): float32 [N], RN32 of the row sum of the input W (float64
 *   accumulation).  rot may be NULL (no rotation).
 * group: multiple of 32 dividing K (OQ_W4); K % 32 == 0.
 */
int oq_quant_weight(const float *w, int32_t N, int32_t K, int64_t ldw,
                    const oq_rot *rot, int wfmt, int32_t group,
                    uint8_t *codes, void *scales, float *w1, hipStream_t stream);

/*
 * oq_gemm_w4a8 -- int8-coded activations (OQ_A8 or OQ_A6 codes) times packed
 * INT4 weights with the fp32 epilogue of CentriQ Eq. 5 / Eq. 9:
 *   y[t][o] = bf16_RNE( a_scale[t] * sum_g w_scale[o][g] * acc_g[t][o]
 *                       + mean[t] * w1[o] + bias[o] )
 *   acc_g = exact int32 sum over the group's input columns.
 * qa int8 [M][lda]; a_scale float32 [M]; w uint8 [N][K/2] (canonical
 * nibbles); w_scale float32 [N][K/group]; mean and w1 both NULL or both set;
 * bias nullable; y bf16 [M][ldy].  group: multiple of 32 dividing K.
 * A product of fewer than 128 output tiles of 128 x 128 with K <= 4096 runs
 * one 4-wavefront workgroup per 32 x 32 output tile (operands staged through
 * LDS from coalesced loads), with no scratch and the one-pass kernel's
 * arithmetic: the two give identical bits.  OQ_INT_SMALL=0 in the
 * environment turns this routing off.
 * ws/ws_bytes: optional device scratch (16-byte aligned, else
 * OQ_ERR_ALIGNMENT).  Another product of fewer than 128 such tiles (K >
 * 4096, or the routing above turned off) given at least
 * oq_workspace_bytes(OQ_OP_GEMM_W4A8, M, K, N, 0) bytes runs split across K
 * on more workgroups: each writes the float32 sum of its groups' s_g acc_g
 * to ws, and a second launch adds those sums in split order and applies the
 * epilogue (a different float32 summation order from the one-pass kernel,
 * within the same rounding bound).  Without scratch, or with less, the
 * product runs in one pass; the result is deterministic either way.
 */
int oq_gemm_w4a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int32_t K,
                 const uint8_t *w, const float *w_scale, int32_t N, int32_t group,
                 const float *mean, const float *w1, const float *bias,
                 uint16_t *y, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * oq_gemm_w4a4 -- 4-bit activations times 4-bit weights.
 *   afmt OQ_A4: qa nibbles [M][lda_bytes], a_scale float32 [M]; w canonical
 *     INT4 nibbles [N][K/2], w_scale float32 [N][K/group]; epilogue as
 *     oq_gemm_w4a8.
 *   afmt OQ_A4 | OQ_TILED or OQ_A6 | OQ_TILED: qa in the tiled layout (from
 *     oq_quant_act with the same afmt; lda_bytes ignored), w and w_scale
 *     from oq_prepack_w4, group 64; output bit-identical to the canonical
 *     path on the same codes.  The library picks the workgroup shape from
 *     M, N and the CU count; the environment variable OQ_FP6_TILE forces
 *     one, for tuning: 256x256, 256x192, 256x128w8 (eight waves), 256x128
 *     (four waves) or 128x192 for OQ_A4; 256x192 or 256x128w8 for OQ_A6.
 *     The result does not depend on the shape.  One activation plane
 *     (oq_tiled_bytes(M, K)) and the weights (oq_tiled_bytes(N, K)) must each
 *     stay below 4 GiB (the kernel's 32-bit operand offsets); larger requests
 *     fail with OQ_ERR_UNSUPPORTED (split M or N).
 *   afmt OQ_MXFP4: qa E2M1 nibbles, a_scale uint8 E8M0 [M][K/32]; w E2M1
 *     nibbles [N][K/2], w_scale uint8 E8M0 [N][K/32]; group must be 32;
 *     y = bf16_RNE( sum_blocks 2^(ea+ew) sum_k fp4(a) fp4(w) + bias[o] );
 *     mean/w1 must be NULL.
 */
int oq_gemm_w4a4(int afmt, const uint8_t *qa, int64_t lda_bytes, const void *a_scale,
                 int64_t M, int32_t K, const uint8_t *w, const void *w_scale,
                 int32_t N, int32_t group, const float *mean, const float *w1,
                 const float *bias, uint16_t *y, int64_t ldy,
                 void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * oq_linear_fused -- the whole layer: oq_quant_act into the workspace, then
 * the matching GEMM, on one stream (CentriQ App. B.2: prologue quantizes
 * each token tile once; rank-1 term and bias in the GEMM epilogue).
 * afmt OQ_A8/OQ_A6/OQ_A4 with an RPBH rotation (or NULL), optional centering
 * (then w1 is required); OQ_MXFP4 with a DENSE32 rotation and E8M0 w_scale.
 * afmt OQ_A4 | OQ_TILED or OQ_A6 | OQ_TILED: w/w_scale from oq_prepack_w4
 * (group 64); activations are quantized straight into the tiled layout.
 * ws: device scratch of at least oq_workspace_bytes(OQ_OP_LINEAR, M, K, N, afmt).
 */
int oq_linear_fused(const uint16_t *x, int64_t M, int32_t K, int64_t ldx,
                    const oq_rot *rot, int center, int afmt,
                    const uint8_t *w, const void *w_scale, int32_t N, int32_t group,
                    const float *w1, const float *bias, uint16_t *y, int64_t ldy,
                    void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * oq_linear_fused_noalloc -- oq_linear_fused for callers that cannot allocate
 * device memory or pass a workspace: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.  Same arguments, formats
 * and result as oq_linear_fused (bit for bit), without ws / ws_bytes: the
 * codes, scales and means go to a static scratch array of
 * OQ_NOALLOC_SCRATCH_BYTES (32 MiB) that the library holds on every GPU it
 * runs on until the process ends (its device address is looked up once per
 * device, on the first call there).  A layer whose
 * oq_workspace_bytes(OQ_OP_LINEAR, M, K, N, afmt) exceeds that size fails
 * with OQ_ERR_WORKSPACE before anything is enqueued.  The call allocates
 * nothing.  Every call on one GPU shares that GPU's scratch, which keeps the
 * last call's contents (nothing in it needs to start at zero): calls that
 * overlap on one GPU (several streams or host threads at once) race; serialise
 * them, for instance on one stream.
 */
#define OQ_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int oq_linear_fused_noalloc(const uint16_t *x, int64_t M, int32_t K, int64_t ldx,
                            const oq_rot *rot, int center, int afmt,
                            const uint8_t *w, const void *w_scale, int32_t N, int32_t group,
                            const float *w1, const float *bias, uint16_t *y, int64_t ldy,
                            hipStream_t stream);

/*
 * oq_prepack_w4 -- repack canonical INT4 weights (oq_quant_weight OQ_W4
 * output: codes [N][K/2], scales float32 [N][K/64]) into the tiled FP6
 * layout for OQ_TILED GEMMs.  Values are unchanged (every INT4 code is an
 * exact FP6 E2M3 value).  w_tiled: oq_tiled_bytes(N, K) bytes; w_scale_t:
 * float32 [K/64][N rounded up to 32] (padding columns get scale 0).
 * group must be 64.
 */
int oq_prepack_w4(const uint8_t *w, const float *w_scale, int32_t N, int32_t K, int32_t group,
                  uint8_t *w_tiled, float *w_scale_t, hipStream_t stream);

/*
 * oq_prepack_mx -- repack canonical MXFP4 weights (oq_quant_weight
 * OQ_W_MXFP4 output: codes [N][K/2], E8M0 [N][K/32]) into the tiled MXFP4
 * layout for OQ_MXFP4 | OQ_TILED GEMMs.  Values are unchanged.  w_tiled:
 * oq_tiled_mx_bytes(N, K) bytes; w_e8m0_tiled: a sixteenth of that, 4-byte
 * aligned (padding rows get zero codes and the unit scale 127).
 * K must be a multiple of 128.
 */
int oq_prepack_mx(const uint8_t *w, const uint8_t *w_e8m0, int32_t N, int32_t K,
                  uint8_t *w_tiled, uint8_t *w_e8m0_tiled, hipStream_t stream);

/*
 * Lloyd-Max activation path (OrbitQuant PR #25, "Default changes": Lloyd-Max
 * codes are the method's activation quantizer below 8 bits, with codebooks
 * built per layer width by a Newton solver; CentriQ Sec. 2 "Related work":
 * the codebook comes from the post-rotation marginal; model card
 * FLUX.1-schnell-OrbitQuant-W4A4, "Quantization": codebook lloyd_max,
 * activation normalization epsilon 1e-10).
 *
 * The marginal is that of one coordinate T of a point uniform on the unit
 * sphere S^{d-1}, density proportional to (1 - t^2)^((d-3)/2); tokens are
 * normalised by their RMS, so levels are for U = sqrt(d) T (variance 1).
 */

/*
 * oq_lloyd_max_levels -- host function, no device work.  levels: host
 * float64 [2^bits], ascending: the minimum-MSE quantizer levels of U (every
 * level the mean of U over its cell, every boundary the midpoint of its two
 * levels), solved by Newton's method on those conditions.  d >= 3,
 * bits in [1, 8].  OQ_ERR_UNSUPPORTED if the solve does not converge.
 */
int oq_lloyd_max_levels(int32_t d, int32_t bits, double *levels);

/*
 * oq_lloyd_max_tables -- host function: the stored codebook the kernels use.
 * levels_f16: host uint16 [2^bits], the levels rounded to float16 (RNE);
 * thresholds: host float32 [2^bits - 1], the exact midpoints of adjacent
 * float16 levels (so a code is the nearest stored level).  Copy both to the
 * device for oq_quant_act_lm / oq_gemm_lm.
 */
int oq_lloyd_max_tables(int32_t d, int32_t bits, uint16_t *levels_f16, float *thresholds);

/* bytes of the tiled float16 operand layout for `rows` rows (K % 16 == 0) */
size_t oq_tiled_f16_bytes(int64_t rows, int32_t K);

/*
 * oq_quant_act_lm -- fused (center) -> RPBH rotate -> Lloyd-Max codes.
 *   rho_t = max(RN32(sqrt(S_t / d)), RN32(1e-10)), S_t the float64 sum of
 *   squares of the rotated float32 values; u = RN32(v RN32(1 / rho_t));
 *   code = number of thresholds strictly below u (ties go to the lower level).
 *   scale[t] = rho_t (float32 [M]).
 * tiled == 0: codes are level indices, two per byte (element 2i in bits
 *   3..0) for bits <= 4, else one byte each, rows of ldc_bytes (multiple of 16).
 * tiled != 0: codes receives the float16 levels themselves in the tiled
 *   float16 layout (oq_tiled_f16_bytes(M, d) bytes; ldc_bytes ignored), the
 *   operand oq_gemm_lm takes directly.
 * levels_f16 / thresholds: device copies of oq_lloyd_max_tables' output for
 * the same bits.  rot: RPBH or NULL; d <= 4096.  mean as in oq_quant_act.
 */
int oq_quant_act_lm(const uint16_t *x, int64_t M, int32_t d, int64_t ldx, const oq_rot *rot, int center,
                    int32_t bits, int tiled, const uint16_t *levels_f16, const float *thresholds,
                    void *codes, int64_t ldc_bytes, float *scale, float *mean, hipStream_t stream);

/*
 * oq_prepack_w16 -- dequantize canonical INT4 weights (oq_quant_weight OQ_W4
 * output) to W16[o][k] = RN16(w_scale[o][k / group] * q[o][k]) (the exact
 * product rounded once) in the tiled float16 layout: oq_tiled_f16_bytes(N, K)
 * bytes, padding rows zero.  K % 32 == 0; group a multiple of 32 dividing K.
 */
int oq_prepack_w16(const uint8_t *w, const float *w_scale, int32_t N, int32_t K, int32_t group,
                   uint16_t *w16_tiled, hipStream_t stream);

/*
 * oq_gemm_lm -- Lloyd-Max activations times dequantized weights:
 *   y[t][o] = bf16_RNE( a_scale[t] * sum_k A16[t][k] W16[o][k]
 *                       + mean[t] * w1[o] + bias[o] )
 *   A16 the float16 level of each code; products exact in float32, summed in
 *   float32 on the float16 matrix cores.
 * tiled != 0: qa is oq_quant_act_lm's tiled output (lda_bytes, levels_f16 and
 *   ws unused).  tiled == 0: qa holds level indices as oq_quant_act_lm writes
 *   them for `bits`, rows of lda_bytes; levels_f16 (device) expands them into
 *   ws, which needs oq_workspace_bytes(OQ_OP_GEMM_LM, M, K, N, 0) bytes.
 * w16_tiled from oq_prepack_w16; a_scale float32 [M]; mean and w1 both NULL
 * or both set; bias nullable; y bf16 [M][ldy].  K % 32 == 0.
 * The workgroup shape (256 x 384, 256 x 256 or 256 x 192 outputs) follows M, N and the
 * CU count; OQ_F16_TILE=256x384, 256x256 or 256x192 in the environment forces
 * one.
 * The result does not depend on the shape.
 */
int oq_gemm_lm(int32_t bits, int tiled, const void *qa, int64_t lda_bytes, const float *a_scale, int64_t M,
               int32_t K, const uint16_t *levels_f16, const uint16_t *w16_tiled, int32_t N, const float *mean,
               const float *w1, const float *bias, uint16_t *y, int64_t ldy, void *ws, size_t ws_bytes,
               hipStream_t stream);

/*
 * Asymmetric grouped INT4 weights (CentriQ Sec. 3 Eq. 2: W_g = sigma (Q - z),
 * Q in 0..15, per-(row, group) scale sigma and shift z stored in 16 bits, RTN
 * from the group minimum and maximum; App. B.2: codes stored as Q - 8, the
 * correction C = sigma (z - 8) per row and 64-column group weighted by the
 * group sums p of the activation codes).
 */

/*
 * oq_quant_weight_asym -- offline: rotate each row as oq_quant_weight does,
 * then per group of `group` columns sigma = RNbf16(RN32((max - min) / 15))
 * (1 for a constant group), z = RNbf16(RN32(-min / sigma)),
 * Q = clamp(RNE(RN32(RN32(w / sigma) + z)), 0, 15).
 * codes: Q - 8 as 4-bit two's complement, [N][K/2]; sigma, zero: bfloat16
 * bits [N][K/group]; w1 (nullable) as oq_quant_weight.  K % 64 == 0.
 */
int oq_quant_weight_asym(const float *w, int32_t N, int32_t K, int64_t ldw, const oq_rot *rot, int32_t group,
                         uint8_t *codes, uint16_t *sigma, uint16_t *zero, float *w1, hipStream_t stream);

/*
 * oq_prepack_w4_asym -- repack asymmetric weights for oq_gemm_w4a4_asym:
 * w_tiled (oq_tiled_bytes(N, K) bytes) holds q'/2 for q' = Q - 8 in the tiled
 * FP6 layout; w_scale_t float32 [K/64][N rounded up to 32] = sigma;
 * corr [K/64][N rounded up to 32] pairs of uint32 (8 bytes, 8-byte aligned):
 * C = RN32(sigma RN32(z - 8)) as the three bfloat16 pieces of its truncation
 * split C = c1 + c2 + c3 (each exactly a bfloat16), stored negated as
 * (-c1 | -c2 << 16, -c3); C = -(c1' + c2' + c3') recovers it exactly.
 * (Both tables are group-major so that a row of outputs reads them as one run.)
 * Padding rows get zeros.  group must be 64.
 */
int oq_prepack_w4_asym(const uint8_t *w, const uint16_t *sigma, const uint16_t *zero, int32_t N, int32_t K,
                       int32_t group, uint8_t *w_tiled, float *w_scale_t, uint32_t *corr, hipStream_t stream);

/*
 * oq_quant_act_gsum -- oq_quant_act for afmt OQ_A4 | OQ_TILED or
 * OQ_A6 | OQ_TILED (OQ_SCALE_PCTL allowed), which also writes gsum uint32
 * [d/64][M] (group-major): the sum p of the codes of every 64-wide group
 * (an integer, |p| < 2048) as the operand word of oq_gemm_w4a4_asym, two
 * bfloat16 values whose sum is p exactly: p1 = 8 floor(p / 8) in bits 0-15
 * and p2 = p - p1 (0..7) in bits 16-31.
 * d % 64 == 0, d <= 4096.
 */
int oq_quant_act_gsum(const uint16_t *x, int64_t M, int32_t d, int64_t ldx, const oq_rot *rot, int center, int afmt,
                      void *codes, float *scale, uint32_t *gsum, float *mean, hipStream_t stream);

/*
 * oq_gemm_w4a4_asym -- tiled 4-bit activations times asymmetric weights:
 *   y[t][o] = bf16_RNE( a_scale[t] * sum_g (sigma[o][g] acc_g[t][o]
 *                        - corr[g][o] gsum[g][t]) + mean[t] w1[o] + bias[o] )
 *   acc_g = exact sum over the group of q_a (Q - 8).
 * afmt must be OQ_A4 | OQ_TILED; qa, a_scale, gsum (the packed group sums
 * described above) from oq_quant_act_gsum;
 * w_tiled, w_scale_t, corr from oq_prepack_w4_asym; K % 64 == 0.
 */
int oq_gemm_w4a4_asym(int afmt, const uint8_t *qa, const float *a_scale, const uint32_t *gsum, int64_t M, int32_t K,
                      const uint8_t *w_tiled, const float *w_scale_t, const uint32_t *corr, int32_t N, const float *mean,
                      const float *w1, const float *bias, uint16_t *y, int64_t ldy, hipStream_t stream);

/*
 * Factorised Paley x Sylvester rotation (CentriQ Sec. 4.2 "Rotation", App.
 * B.1): H = (H_m (x) H_b) / sqrt(m b) with H_b Sylvester (b = 2^k) and H_m
 * a Paley matrix (m = 12, 44: type I with q = 11, 43; m = 36: type II with
 * q = 17; m = 1: none), applied as vec(H_b X H_m^T) to the token reshaped
 * column-major to X in R^{b x m}; a row of native width n < m b is centred
 * over its n coordinates and then zero-padded to m b (centering precedes
 * padding).  Descriptor: oq_rot{kind = OQ_ROT_KRON, d = n, block = b,
 * rounds = m, perm = signs = mats = NULL}.  Every output of the rotation,
 * and every code and weight column, has the padded width m b; the GEMMs take
 * K = m b.  oq_rotate, oq_quant_act (integer formats, tiled or not, absmax
 * scale) and oq_quant_weight / oq_quant_weight_asym accept it;
 * oq_linear_fused, group sums, Lloyd-Max codes and the percentile scale do not.
 * Float32 order: un-normalised Sylvester stages on each block, then the
 * m-term sums in increasing c, then one multiply by RN32(1/sqrt(m b)).
 */

/*
 * oq_kron_plan -- host function: the smallest admissible padded width
 * n_pad = m * block >= n with m in {1, 12, 36, 44} and block a power of two
 * of at least 16 (one thread's share of coordinates).  n <= 16384.
 */
int oq_kron_plan(int32_t n, int32_t *m, int32_t *block, int32_t *n_pad);

/*
 * 8-bit weights: layers that do not tolerate 4 bits keep int8 codes with one
 * scale per output row, behind the same rotation, centering and activation
 * codes (oq_quant_act OQ_A8 or OQ_A6) as the INT4 layers.
 */

/*
 * oq_quant_weight_w8 -- offline: rotate each row as oq_quant_weight does, then
 * symmetric absmax INT8 per row: scale[o] = RN32(a / 127) with a = max(max_j
 * |v_oj|, RN32(1e-10)), codes clamp(RNE(RN32(v RN32(127 / a))), -127, 127).
 * codes int8 [N][ldc_bytes], rows of the rotated width (padded for the
 * Kronecker rotation), 16-byte aligned; scales float32 [N]; w1 (nullable) as
 * oq_quant_weight.  rot: RPBH, Kronecker or NULL.  K % 16 == 0.
 */
int oq_quant_weight_w8(const float *w, int32_t N, int32_t K, int64_t ldw, const oq_rot *rot, int8_t *codes,
                       int64_t ldc_bytes, float *scales, float *w1, hipStream_t stream);

/*
 * oq_gemm_w8a8 -- int8 activations times int8 weights:
 *   y[t][o] = bf16_RNE( a_scale[t] * w_scale[o] * acc[t][o] + mean[t] * w1[o] + bias[o] )
 *   acc = exact int32 sum over K, converted to float32 with one rounding.
 * qa int8 [M][lda]; a_scale float32 [M]; w int8 [N][ldw]; w_scale float32 [N];
 * mean and w1 both NULL or both set; bias nullable; y bf16 [M][ldy].
 * 0 <= M <= 2^30, any N >= 0 (zero enqueues nothing); K a multiple of 16, 16 <= K <=
 * 131056 (the int32 sum cannot overflow, codes of -128 included); lda, ldw
 * multiples of 16, at most 2^23; qa and w 16-byte aligned.  No scratch.  The result does
 * not depend on the tile that the library picks from M, N, K and the CU count.
 */
int oq_gemm_w8a8(const int8_t *qa, int64_t lda, const float *a_scale, int64_t M, int32_t K, const int8_t *w,
                 int64_t ldw, const float *w_scale, int32_t N, const float *mean, const float *w1, const float *bias,
                 uint16_t *y, int64_t ldy, hipStream_t stream);

/*
 * Between the projections of an attention layer: per-head norm and rotary
 * embedding of queries and keys, a paged cache of keys and values, and
 * attention over it.  Heads are bfloat16 vectors of d consecutive elements;
 * element (token t, head h) of a tensor starts at base + t ld + h hs
 * (elements; every start 16-byte aligned, so ld, hs and d multiples of 8).
 * ld and hs are at least d; heads of an output must not overlap.
 */

/*
 * Rotary embedding (host struct, device arrays): the pair (a, b) of a head at
 * position p becomes (a cos[p][i] - b sin[p][i], b cos[p][i] + a sin[p][i]),
 * i = 0 .. dim/2 - 1, on elements (i, i + dim/2), or (2i, 2i + 1) with
 * interleaved != 0; elements dim .. d - 1 stay.  cos, sin: float32
 * [rows][dim/2], 4-byte aligned.  dim even, 2 <= dim <= d.
 */
typedef struct {
  const float *cos;
  const float *sin;
  int64_t rows;
  int32_t dim;
  int32_t interleaved;
} oq_rope;

/*
 * Paged cache (host struct, device arrays): page p of k and of v starts at
 * base + p page_stride (elements, a multiple of 8, >= heads * page * d) and
 * holds [heads][page][d].  page: a power of two in [8, 1024].  k and v may be
 * parts of one allocation (pages of both interleaved); a cache may pass 4 GiB.
 */
typedef struct {
  uint16_t *k;
  uint16_t *v;
  int64_t page_stride;
  int32_t pages;
  int32_t page;
  int32_t heads;
  int32_t d;
} oq_kv;

/*
 * oq_qk_norm_rope -- for every head x of every token, query and key heads in
 * one launch:  n = x / sqrt(mean(x^2) + eps) * w  (w float32 [d]; NULL: n = x),
 * then the rotary embedding at position pos[t] (pos int32 [T]; NULL: t; rope
 * NULL: none), rounded once to bfloat16 (float32 inside).
 * q: heads_q heads of T tokens (heads_q 0: none, q NULL); k the same.  Outputs
 * have their own strides; out == in with the same strides works in place.
 * A position outside [0, rope->rows) gives NaN in that token's rows.
 * d a multiple of 8, 8 <= d <= 512.  eps >= 0, finite.
 */
int oq_qk_norm_rope(const uint16_t *q, int64_t q_ld, int64_t q_hs, int32_t heads_q, const uint16_t *k, int64_t k_ld,
                    int64_t k_hs, int32_t heads_k, int64_t T, int32_t d, const float *w_q, const float *w_k, float eps,
                    const oq_rope *rope, const int32_t *pos, uint16_t *q_out, int64_t qo_ld, int64_t qo_hs,
                    uint16_t *k_out, int64_t ko_ld, int64_t ko_hs, hipStream_t stream);

/*
 * oq_kv_append -- token t's keys, through the norm (w_k NULL: none) and rotary
 * embedding (rope NULL: none) of oq_qk_norm_rope, and its values as they are,
 * go to slot[t] of the cache: page slot / page, place slot % page, all
 * kv->heads heads of kv->d.  slot int64 [T]; a slot outside [0, pages * page)
 * writes nothing (padding tokens carry -1).  Two tokens of one call must not
 * share a slot.  kv->d <= 512.
 */
int oq_kv_append(const uint16_t *k, int64_t k_ld, int64_t k_hs, const uint16_t *v, int64_t v_ld, int64_t v_hs,
                 int64_t T, const float *w_k, float eps, const oq_rope *rope, const int32_t *pos, const int64_t *slot,
                 const oq_kv *kv, hipStream_t stream);

/*
 * oq_attn_prefix -- attention of B sequences that share prefix_len cached
 * tokens, each followed by a suffix of its own.  Sequence b has n_q query
 * tokens t = b n_q + i (decode: n_q = 1), the last tokens of its suffix:
 * token i sees the whole prefix and the suffix places j < lens[b] - n_q + 1 + i.
 *   o[t][h] = sum_j p_j v_j,  p = softmax_j(scale q[t][h] . k_j)
 * over the seen keys of key head h / (heads_q / kv->heads); a row that sees
 * no key, or whose every score is -inf, gives zeros and lse -inf.  lse (nullable) float32 [B n_q][heads_q]:
 * log sum_j exp(scale q . k_j).
 * prefix_table int32 [ceil(prefix_len / page)], tables int32 [B][table_ld]:
 * page numbers in order; lens int32 [B], at most table_ld * page places are
 * read.  Keys on a page number outside [0, pages) are left out.  Cache places
 * that a row does not see (past its sequence's length, or of a later query
 * token) may hold anything, NaN included, without a trace in that row.
 * NaN in a query, or in a key or value that a row sees, gives NaN there; an
 * infinite value gives infinity, or NaN where its weight is too small for
 * float32.  A row's bits do not depend on the contents of other rows.
 * The prefix is read once for all rows of a tile; scores, statistics and sums
 * are float32; softmax numerators enter the value product as bfloat16 (their
 * sum is of the float32 values), an error of about the output's own rounding.
 * d (kv->d) 64 or 128; heads_q a multiple of kv->heads; scale log2(e) finite.
 * ws: device scratch of oq_attn_prefix_ws_bytes(B, n_q, heads_q, kv,
 * prefix_len, table_ld) bytes, 16-byte aligned (may be 0).
 */
int oq_attn_prefix(const uint16_t *q, int64_t q_ld, int64_t q_hs, int32_t B, int32_t n_q, int32_t heads_q,
                   const oq_kv *kv, const int32_t *prefix_table, int32_t prefix_len, const int32_t *tables,
                   int32_t table_ld, const int32_t *lens, float scale, uint16_t *o, int64_t o_ld, int64_t o_hs,
                   float *lse, void *ws, size_t ws_bytes, hipStream_t stream);

/* Scratch bytes of oq_attn_prefix (0 for arguments it refuses).  Pure host
 * function of the sizes and the device's CU count.  It does not grow with the
 * arguments: the number of parts follows from how the work fills the CUs, so a
 * shorter prefix can take more than a longer one.  A caller whose sizes change
 * asks for each, or keeps the largest of those that come. */
size_t oq_attn_prefix_ws_bytes(int32_t B, int32_t n_q, int32_t heads_q, const oq_kv *kv, int32_t prefix_len,
                               int32_t table_ld);

/*
 * The feed-forward half of a sparse (mixture-of-experts) layer on int8 codes,
 * and the answer behind the last layer: routing, the experts' products, the
 * residual stream with its norms, log probabilities.  An entry i = t k + j is
 * the j-th choice of token t; entries are the rows of everything that the
 * experts compute.
 */

/* element types of logits and of the residual stream */
enum { OQ_F32 = 1, OQ_BF16 = 2 };

/* scores of a router */
enum { OQ_SCORE_SOFTMAX = 1, OQ_SCORE_SIGMOID = 2 };

/*
 * A router (host struct, bias device float32 [experts] or NULL).  For the
 * logits l of a token: s = softmax(l) or sigmoid(l), element by element;
 *   c = s + bias (without a bias experts are compared by l itself);
 *   the experts lie in `groups` equal runs; a run's score is the sum of its
 *   group_best (1 or 2) best c (without a bias: of the best l, or of the two best
 *   s), and the top_groups best runs are open (groups 1: all);
 *   chosen are the k best c of the open runs, in falling order;
 *   weight = factor s, divided by the sum of the chosen s if renorm is not 0.
 * Equal ones go to the lowest index, runs and experts alike.  Choices are those
 * of the exact values: where float32 cannot tell neighbours apart, float64
 * decides.  A NaN ranks below all numbers (in a run's score it counts as -inf);
 * ids are valid whatever the logits hold, weights follow the formula (a softmax over
 * NaN or +inf is NaN throughout, whoever is chosen).
 * 1 <= experts <= 1024 (512 with groups); groups <= 64 divides experts; group_best <= experts /
 * groups; 1 <= k <= 32, k <= top_groups experts / groups; factor finite.
 */
typedef struct {
  const float *bias;
  int32_t experts;
  int32_t k;
  int32_t score;
  int32_t groups;
  int32_t top_groups;
  int32_t group_best;
  int32_t renorm;
  float factor;
} oq_router;

/*
 * oq_route -- logits [T][ld] (dtype OQ_F32 or OQ_BF16, ld >= experts) to
 * ids int32 [T][k], weights float32 [T][k] and, where offsets and order are
 * given (both or neither), the lists that oq_gemm_w8a8_experts reads: order
 * int32 [T k] holds the entries by expert, those of one expert in rising
 * order, expert e's at offsets[e] .. offsets[e + 1] - 1 (int32 [experts + 1]).
 * mask uint8 [T] (nullable): a token of 0 gets ids -1 and weights 0 and is in
 * no list; places of order behind offsets[experts] get -1.
 * T k <= 2^28.  ws: device scratch of oq_route_ws_bytes(T, r) bytes, 16-byte
 * aligned (not read without lists; may be 0).
 */
int oq_route(const void *logits, int dtype, int64_t ld, int64_t T, const uint8_t *mask, const oq_router *r, int32_t *ids,
             float *weights, int32_t *offsets, int32_t *order, void *ws, size_t ws_bytes, hipStream_t stream);

/* Scratch bytes of oq_route (0 for arguments it refuses).  Pure host function. */
size_t oq_route_ws_bytes(int64_t T, const oq_router *r);

/* what the experts' product does with its outputs */
enum { OQ_ACT_NONE = 0, OQ_ACT_SWIGLU = 1 };

/*
 * oq_gemm_w8a8_experts -- the product of oq_gemm_w8a8 for every entry with the
 * weights of its expert: for entry i = order[p], offsets[e] <= p < offsets[e + 1],
 * on activation row i / per,
 *   v[o] = a_scale[row] * w_scale[e][o] * acc + mean[row] * w1[e][o] + bias[e][o]
 *   y[i][o] = bf16_RNE(v[o])                                  OQ_ACT_NONE, N outputs
 *   y[i][o] = bf16_RNE(v[o] / (1 + exp(-v[o])) * v[N/2 + o])  OQ_ACT_SWIGLU, N/2 outputs
 * (N even; the first half of the weight rows is the gate; below a gate of -174 the product
 * may be 0, and NaN with an infinite v[N/2 + o]).
 * per = k: entries of a token share its activation row (up projections); per =
 * 1: every entry has a row of its own (down projections).
 * qa int8 [rows][lda], a_scale and mean float32 [rows]; w int8 [E][N][ldw], an
 * expert's rows w_stride bytes behind the last one's; w_scale, w1, bias float32
 * [E][N]; mean and w1 both NULL or both set, bias nullable; offsets int32 [E + 1]
 * and order int32 [n] as from oq_route; y bf16 [n][ldy].
 * An entry may be in the lists once; rows of y whose entry is in no list stay
 * as they are.  List values outside their range are ignored (offsets are cut to
 * 0 .. n, an order outside 0 .. n - 1 has no row).
 * 0 <= n <= 2^28, per >= 1, rows >= ceil(n / per); 1 <= E <= 1024; K, lda, ldw,
 * alignment as oq_gemm_w8a8, w_stride a multiple of 16 and at least N ldw.
 * N <= 2^20.  No scratch.  A row's bits do not depend on the other entries.
 */
int oq_gemm_w8a8_experts(const int8_t *qa, int64_t lda, const float *a_scale, int64_t rows, int32_t K, const int8_t *w,
                         int64_t ldw, int64_t w_stride, const float *w_scale, int32_t N, int32_t E,
                         const int32_t *offsets, const int32_t *order, int64_t n, int32_t per, int act,
                         const float *mean, const float *w1, const float *bias, uint16_t *y, int64_t ldy,
                         hipStream_t stream);

/*
 * A norm over the d elements of a row (host struct; w, b device float32 [d] or
 * NULL):  OQ_NORM_RMS    x / sqrt(mean(x^2) + eps) * w + b
 *         OQ_NORM_LAYER  (x - mean(x)) / sqrt(mean((x - mean(x))^2) + eps) * w + b
 */
enum { OQ_NORM_RMS = 1, OQ_NORM_LAYER = 2 };
typedef struct {
  const float *w;
  const float *b;
  int32_t kind;
  float eps;
} oq_norm;

/*
 * Modulation (host struct, device arrays): gate, scale, shift bfloat16
 * [rows][ld] (each nullable; they may be columns of one table); token t uses
 * row row[t] (int32 [T]; NULL: row 0 of a single one, else row t).  A row
 * outside [0, rows) gives NaN in that token's outputs.
 */
typedef struct {
  const uint16_t *gate;
  const uint16_t *scale;
  const uint16_t *shift;
  const int32_t *row;
  int64_t ld;
  int64_t rows;
} oq_mod;

/*
 * oq_residual_norm -- from the end of one block to the start of the next, one
 * pass over each row:
 *   u = sum_j weights[t][j] y[t k + j]    (weights NULL: k = 1 and u = y[t])
 *   R = r_scale r + y_scale gate post(u)  (r NULL: without it; post, gate: as given)
 *   h = pre(R) (1 + scale) + shift        (pre, scale, shift: as given)
 * Stored are r_out = R and h, each nullable, each rounded once from float32; h
 * is formed of R before its rounding.  y NULL: R = r_scale r (no post, no gate).
 * A row of y whose weight is 0 is not read (an entry that has no expert, say).
 * y, h bf16; r, r_out of type r_type (OQ_F32 or OQ_BF16).  r_out may be r (same
 * ld); other outputs must not overlap inputs or each other.
 * Sums are float32, the norms' squares included (elements below 2^63).
 * d a multiple of 8, 8 <= d <= 16384; 1 <= k <= 64; T k < 2^31; every row
 * 16-byte aligned; y_scale, r_scale finite; eps finite, >= 0.
 */
int oq_residual_norm(const uint16_t *y, int64_t y_ld, int32_t k, const float *weights, float y_scale, const void *r,
                     int64_t r_ld, float r_scale, int r_type, int64_t T, int32_t d, const oq_norm *post,
                     const oq_norm *pre, const oq_mod *mod, void *r_out, int64_t ro_ld, uint16_t *h, int64_t h_ld,
                     hipStream_t stream);

/*
 * oq_logprobs -- of each row x of logits [T][ld] (dtype OQ_F32 or OQ_BF16, V
 * wide), with p = softmax(scale x):
 *   logprob[t][i] = log p[tokens[t][i]]      (n tokens a row, int32 [T][n])
 *   rank[t][i]    = how many of the row come before that token (0: the first)
 *   entropy[t]    = -sum_v p log p,  lse[t] = log sum_v exp(scale x)
 *   top_id[t][j], top_logprob[t][j], j < top: the first `top` of the row
 * The order is that of falling logits, equal ones by rising index; NaN comes
 * behind all numbers.  A token outside [0, V) (padding) gives NaN and rank -1.
 * Masked logits (-inf, or the type's lowest value) take no part.  A row of nothing
 * but -inf has lse -inf and NaN for all other values; a row with NaN or +inf has NaN
 * for all of them.  Ranks and top_id are in order in such rows as well.
 * Sums are float32, of the others beside the largest logit alone: a log probability is off
 * by at most some 100 units of 2^-24 (3 more for each unit of scale x that the others lie
 * below the largest logit on average) of itself, however near 0 it is, and never above 0;
 * an entropy likewise, and never below 0.  (Terms below 2^-126 of the largest may count as 0.)
 * Each output nullable but logprob and rank with n > 0, and the top pair with
 * top > 0.  Rows need the alignment of their element only.
 * T <= 2^24, 1 <= V <= 2^21, 0 <= n <= 64, 0 <= top <= 32, top <= V, scale > 0 and its
 * product with log2(e) finite.
 * ws: device scratch of oq_logprobs_ws_bytes(T, V, n, top) bytes, 16-byte
 * aligned (may be 0).
 */
int oq_logprobs(const void *logits, int dtype, int64_t ld, int64_t T, int32_t V, float scale, const int32_t *tokens,
                int32_t n, int32_t top, float *logprob, int32_t *rank, float *entropy, float *lse, int32_t *top_id,
                float *top_logprob, void *ws, size_t ws_bytes, hipStream_t stream);

/* Scratch bytes of oq_logprobs for either dtype (0 for arguments it refuses).
 * Pure host function of the sizes and the device's CU count; not monotonic. */
size_t oq_logprobs_ws_bytes(int64_t T, int32_t V, int32_t n, int32_t top);

/*
 * oq_probe_mfma -- measurement helper, not part of the layer: the rate one
 * matrix-core instruction sustains on the calling device at its current clock
 * (a roofline denominator beside the published dense peak, which assumes the
 * top clock).  Launches, on `stream`, two workgroups of four wavefronts per
 * CU that each issue iters x 32 independent instructions of the kind
 * (four accumulator chains, operands in registers, no memory traffic), and
 * returns in *ops the operation count of that launch (2 M N K per
 * instruction); the caller times the launch (for instance with events on the
 * stream) and divides.  sink: device float32 buffer of at least
 * oq_probe_sink_elems() elements (written, values meaningless).  Kinds:
 * OQ_PROBE_FP6 and OQ_PROBE_FP4 (v_mfma_scale_f32_32x32x64_f8f6f4 with both
 * operands FP6 E2M3 / FP4 E2M1, unit scales: the instructions of the tiled
 * INT4 and MXFP4 GEMMs), OQ_PROBE_FP8 (the same instruction on FP8 E4M3),
 * OQ_PROBE_I8 (v_mfma_i32_32x32x32_i8), OQ_PROBE_BF16, OQ_PROBE_F16
 * (v_mfma_f32_32x32x16_bf16 / _f16), and OQ_PROBE_FP6_UPDATE: the tiled INT4
 * GEMM's arithmetic without memory traffic, each FP6 MFMA followed by the 16
 * float32 group-scale updates of the previous tile (8 MFMAs per iteration and
 * wavefront; *ops counts 2 M N K of the MFMAs), the rate the fp32 update
 * leaves to that GEMM.  1 <= iters <= 2^20 (a launch of 2^20 iterations runs
 * for about a second), else OQ_ERR_INVALID_ARG.
 */
enum { OQ_PROBE_FP6 = 1, OQ_PROBE_FP4 = 2, OQ_PROBE_FP8 = 3, OQ_PROBE_I8 = 4, OQ_PROBE_BF16 = 5, OQ_PROBE_F16 = 6,
       OQ_PROBE_FP6_UPDATE = 7 };
int oq_probe_mfma(int kind, int32_t iters, float *sink, double *ops, hipStream_t stream);
size_t oq_probe_sink_elems(void);

enum { OQ_OP_GEMM_W4A8 = 1, OQ_OP_GEMM_W4A4 = 2, OQ_OP_LINEAR = 3, OQ_OP_GEMM_LM = 4 };

/* Scratch bytes a call needs (0 if none).  Pure host function.  For
 * OQ_OP_GEMM_LM, afmt is OQ_TILED for tiled activations, else 0.  For
 * OQ_OP_GEMM_W4A8 (afmt ignored), the optional scratch of the split
 * product, enough for any group size (0 when the product runs in one pass
 * or on the 32 x 32 tile kernel). */
size_t oq_workspace_bytes(int op, int64_t M, int32_t K, int32_t N, int afmt);

#ifdef __cplusplus
}
#endif

#endif /* OQ_H */
