/*
 * fq.h -- blockwise FP4 fake quantization on AMD Instinct MI355X (gfx950).
 *
 * C ABI of libfq.so.  Every call validates its arguments on the host, then
 * enqueues hand-written HIP kernels on the caller's stream and returns.  The
 * library allocates no device memory and keeps no state between calls other
 * than a thread-local error message; scratch memory comes from the caller's
 * workspace argument.
 *
 * Sources for the operations (cited by page title and section):
 *  - "Como o Treinamento com Quantizacao Detecta e Recupera Precisao em
 *    Inferencia de Baixa Precisao" (brainai.pro), "Detalhes tecnicos ou
 *    Implementacao": QAT fake-quantizes weights and activations in the
 *    forward pass (quantize then dequantize inside a wider type) and passes
 *    gradients through the quantizer with the straight-through estimator,
 *    exposing rounding and clipping effects.
 *  - "Aprimorando gpt-oss para Precisao e Desempenho com Treinamento
 *    Consciente a Quantizacao" (brainai.pro), "O que ha de novo", and the
 *    gpt-oss QAT tutorial (thakicloud), "NVFP4: The Next Generation": MXFP4
 *    and NVFP4 targets, NVFP4's FP8 E4M3 block scale, switching between the
 *    two formats as a one-line configuration change.
 *  - "Resumo Tecnico: TetraJet-v2" (gist.science), sec. 2.A: NVFP4 groups of
 *    16 elements with an 8-bit scale; a 128-element outer block with its own
 *    scale over 16-element inner blocks instead of a tensor-wide maximum;
 *    stochastic rounding with E[round(x)] = x in the backward pass; 1x16
 *    weight groups with the transposed weight aligned accordingly; linear
 *    layers whose activations and weights are all quantized.
 *  - Format definitions: OCP Microscaling Formats (MX) v1.0 (FP4 E2M1
 *    element, E8M0 scale 2^(floor(log2 amax) - 2)); OCP OFP8 v1.0 (E4M3,
 *    bias 7, max 448, no infinities).  Philox4x32-10: Salmon et al., "Parallel
 *    Random Numbers: As Easy as 1, 2, 3", SC'11.
 *
 * Numerics (identical, bit for bit, on every call):
 *  - E2M1 codes: bit 3 sign, magnitudes {0, .5, 1, 1.5, 2, 3, 4, 6}; the sign
 *    of x is kept, so a negative value that rounds to zero is code 8 and
 *    dequantizes to -0.0.
 *  - MXFP4 block scale: E8M0 code clamp(floor(log2 amax) - 2, -127, 127) + 127
 *    (an all-zero block gets code 0).
 *  - NVFP4 outer scale s = RN(amax_outer / 2688) in FP32 (2688 = 6 * 448),
 *    amax_outer over the whole tensor (FQ_OUTER_TENSOR) or over each
 *    128-element outer block (FQ_OUTER_BLOCK128).  Block scale code
 *    e4 = E4M3_RNE_sat(RN(RN(amax_b / 6) / s)) (0 if s = 0); effective scale
 *    s_eff = RN(e4m3(e4) * s).
 *  - Scaled magnitude a = RN(|x| / s_eff), correctly rounded FP32 (0 when
 *    s_eff = 0).
 *  - FQ_ROUND_RNE: a rounds to the nearest grid value, ties to the even
 *    code, saturating at 6.  FQ_ROUND_SR: a >= 6 gives 6; otherwise with
 *    g_k <= a < g_{k+1}, T = floor((a - g_k) / (g_{k+1} - g_k) * 65536) and
 *    the element rounds up iff r16(n) < T, where r16(n) is 16-bit half
 *    (n & 1) of word ((n >> 1) & 3) of Philox4x32-10 with key (seed low word,
 *    seed high word) and counter (low word of n >> 3, high word of n >> 3,
 *    0, 0), and n is the element's row-major index in the orientation being
 *    quantized (r * cols + c for FQ_AXIS_ROW, c * rows + r for FQ_AXIS_COL).
 *  - Dequantized value y = BF16_RNE(RN(+-g * s_eff)).
 *  - A value is clipped when a > 6.
 *
 * Layouts (all row-major, contiguous):
 *  - x, y, dy, dx: BF16 [rows, cols].
 *  - FQ_AXIS_ROW (1xB groups along each row, the contiguous axis):
 *      codes [rows, cols/2] bytes (element 2j in the low nibble),
 *      scales [rows, cols/B] bytes, outer: 1 float (TENSOR) or
 *      [rows, cols/128] floats (BLOCK128).
 *  - FQ_AXIS_COL (groups of B consecutive rows in each column, i.e. 1xB
 *    groups along the rows of x^T): codes [cols, rows/2], scales
 *    [cols, rows/B], outer 1 float or [cols, rows/128] -- the layout of x^T;
 *    y stays in the layout of x.
 *
 * Pointers: x, y, dy, dx, codes and scales are device pointers aligned to
 * 16 bytes; outer is a device pointer aligned to 4 bytes; descriptors are
 * host pointers read only during the call.  The caller owns all memory.
 *
 * Asynchrony: calls return after enqueueing on `stream` (a hipStream_t, NULL
 * for the default stream).  Results are ready when the stream reaches them.
 * A call that returns an error other than FQ_ERR_DEVICE has enqueued nothing
 * and written nothing.
 *
 * Limits: 1 <= rows, cols < 2^31 and rows * cols <= 2^34 elements.
 */
#ifndef FQ_H
#define FQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FQ_OK = 0,
    FQ_ERR_NULL = 1,       /* a required pointer is NULL */
    FQ_ERR_DESC = 2,       /* unsupported descriptor combination */
    FQ_ERR_SHAPE = 3,      /* sizes out of range or not divisible by the block */
    FQ_ERR_ALIGN = 4,      /* a pointer is not aligned as documented */
    FQ_ERR_WORKSPACE = 5,  /* workspace missing or smaller than required */
    FQ_ERR_DEVICE = 6      /* a HIP launch or query failed */
} fq_status;

enum { FQ_SCALE_E8M0 = 0, FQ_SCALE_E4M3 = 1 };
enum { FQ_OUTER_NONE = 0, FQ_OUTER_TENSOR = 1, FQ_OUTER_BLOCK128 = 2 };
enum { FQ_ROUND_RNE = 0, FQ_ROUND_SR = 1 };
enum { FQ_AXIS_ROW = 0, FQ_AXIS_COL = 1 };

/* Quantization format and rounding.  Valid combinations:
 *   MXFP4: {block_size 32, FQ_SCALE_E8M0, FQ_OUTER_NONE}
 *   NVFP4: {block_size 16, FQ_SCALE_E4M3, FQ_OUTER_TENSOR or FQ_OUTER_BLOCK128}
 * with any rounding and axis.  seed is read only for FQ_ROUND_SR. */
typedef struct {
    int32_t block_size;
    int32_t scale_type;
    int32_t outer;
    int32_t rounding;
    int32_t axis;
    int32_t reserved;      /* must be 0 */
    uint64_t seed;
} fq_desc;

/* Presets: the one-line switch between the two formats.
 * fq_desc_mxfp4() = {32, E8M0, NONE, RNE, ROW, 0, seed 0}
 * fq_desc_nvfp4() = {16, E4M3, TENSOR, RNE, ROW, 0, seed 0} */
fq_desc fq_desc_mxfp4(void);
fq_desc fq_desc_nvfp4(void);

/* Bytes of workspace that fq_quantize / fq_fake_quant need for this
 * descriptor and shape: 4096 for FQ_OUTER_TENSOR (partial maxima of the
 * per-tensor reduction), 0 otherwise.  Contents need no initialization and
 * are not meaningful after the call.  Returns 0 for an invalid descriptor. */
size_t fq_workspace_size(const fq_desc *desc, int64_t rows, int64_t cols);

/* Quantize: x -> codes, scales and (NVFP4) outer scales.
 * codes, scales must be non-NULL; outer must be non-NULL for NVFP4 and is
 * ignored for MXFP4.  ws / ws_bytes: see fq_workspace_size (ws may be NULL
 * when 0 bytes are needed).  Source: the quantize half of fake quantization
 * ("Como o Treinamento ...", "Detalhes tecnicos"); format per the header. */
fq_status fq_quantize(const fq_desc *desc, const void *x_bf16, int64_t rows,
                      int64_t cols, void *codes, void *scales, float *outer,
                      void *ws, size_t ws_bytes, void *stream);

/* Dequantize: codes, scales, outer -> y [rows, cols] BF16, where rows x cols
 * is the shape of the original x and desc->axis says which layout codes and
 * scales are in: y = BF16_RNE(RN(+-g * s_eff)) per element, the value the
 * quantized element stands for.  Rounding and seed are ignored.  codes and
 * scales are required, outer for NVFP4; shape rules as fq_quantize.  Source:
 * the dequantize half of fake quantization, which brings the quantized
 * values back into the wider type the forward pass computes in ("Como o
 * Treinamento ...", "Detalhes tecnicos ou Implementacao"); for the formats,
 * OCP MX v1.0 (an element's value is its E2M1 value times the block scale)
 * and, for NVFP4, the E4M3 block scale times the FP32 outer scale
 * ("Resumo Tecnico: TetraJet-v2", sec. 2.A). */
fq_status fq_dequantize(const fq_desc *desc, const void *codes, const void *scales,
                        const float *outer, int64_t rows, int64_t cols,
                        void *y_bf16, void *stream);

/* Fake quantization: y = dequantize(quantize(x)) in one pass over x.
 * y must be non-NULL; codes, scales and outer may each be NULL to skip that
 * output.  Source: "Como o Treinamento ...", "Detalhes tecnicos" (fake
 * quantization in the forward pass); TetraJet-v2 sec. 2.A for the double
 * block and stochastic rounding. */
fq_status fq_fake_quant(const fq_desc *desc, const void *x_bf16, int64_t rows,
                        int64_t cols, void *y_bf16, void *codes, void *scales,
                        float *outer, void *ws, size_t ws_bytes, void *stream);

/* Straight-through estimator with clipping: dx = dy where the forward did
 * not clip x (a <= 6), else +0.  a is recomputed from x and the forward's
 * stored scales (and outer scales) in the forward's layout (desc->axis).
 * Source: "Como o Treinamento ...", "Detalhes tecnicos" (gradients through
 * the quantizer by STE; clipping effects). */
fq_status fq_ste_backward(const fq_desc *desc, const void *x_bf16,
                          const void *scales, const float *outer,
                          const void *dy_bf16, int64_t rows, int64_t cols,
                          void *dx_bf16, void *stream);

/* fq_fake_quant for callers that cannot allocate or pass a workspace (code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation): the same computation and outputs, with the per-tensor
 * maximum's partials (the only scratch any format needs, at most 4096 bytes
 * whatever the shape) in a 4 KB device array the library owns, one per GPU,
 * instead of ws.  The call allocates nothing.  Calls on one GPU share that
 * array: calls that overlap on one GPU (different streams, or different
 * threads) race and must be serialized by the caller.  Arguments and errors
 * otherwise as fq_fake_quant; FQ_ERR_DEVICE if the array's address cannot be
 * looked up on the current device. */
fq_status fq_fake_quant_noalloc(const fq_desc *desc, const void *x_bf16, int64_t rows,
                                int64_t cols, void *y_bf16, void *codes, void *scales,
                                float *outer, void *stream);

/* Fake quantization that also writes the STE keep mask: as fq_fake_quant,
 * plus keep [rows, cols / 8] uint8 in the layout of x (row-major, whatever
 * desc->axis is): bit (c mod 8) of byte (r, c / 8) is 1 where element (r, c)
 * was kept (a = RN(|x| / s_eff) <= 6) and 0 where the forward clipped it.
 * The backward then needs neither x nor the scales (fq_ste_backward_mask):
 * the clipped STE reads 2 B of dy and 1/8 B of mask per element instead of
 * 2 B of x plus the scales.  cols must be a multiple of 8; keep must be
 * non-NULL, 16-byte aligned, and must not overlap the other buffers.  Errors
 * as fq_fake_quant.  Source: TetraJet-v2 sec. 2.A (the backward passes
 * gradients through the quantizer where it did not clip); "Como o
 * Treinamento ...", "Detalhes tecnicos" (STE, clipping effects). */
fq_status fq_fake_quant_mask(const fq_desc *desc, const void *x_bf16, int64_t rows,
                             int64_t cols, void *y_bf16, void *codes, void *scales,
                             float *outer, void *keep, void *ws, size_t ws_bytes,
                             void *stream);

/* Fake quantization of the random Hadamard rotation of x along the
 * quantization axis, in one pass: y = dequantize(quantize(H x)), codes and
 * scales of H x.  H is blockwise H_n (n = rht_block, 16 or 128) with the
 * Philox sign vector of rht_seed, exactly as fq_hadamard computes it
 * (including the BF16 rounding of the rotated values), so the result equals
 * fq_fake_quant applied to fq_hadamard's output.  desc: MXFP4 or NVFP4
 * FQ_OUTER_BLOCK128 (the per-tensor scale would need the rotated tensor's
 * maximum first), either axis, RNE or SR; the quantized axis a multiple of
 * rht_block.  y required; codes, scales, outer optional.  Source: "Resumo
 * Tecnico: TetraJet-v2", sec. 2.C (the rotation ahead of the backward's FP4
 * quantization). */
fq_status fq_fake_quant_rht(const fq_desc *desc, const void *x_bf16, int64_t rows, int64_t cols,
                            int32_t rht_block, uint64_t rht_seed, void *y_bf16, void *codes,
                            void *scales, float *outer, void *stream);

/* Clipped straight-through estimator from a keep mask written by
 * fq_fake_quant_mask: dx = dy where the element's keep bit is set, else +0.
 * keep [rows, cols / 8] (layout above), dy and dx [rows, cols] BF16, all
 * device pointers, 16-byte aligned; dx may alias dy.  rows >= 1, cols >= 8,
 * cols a multiple of 8.  Format independent.  Source: as fq_ste_backward. */
fq_status fq_ste_backward_mask(const void *keep, const void *dy_bf16, int64_t rows,
                               int64_t cols, void *dx_bf16, void *stream);

/* Workspace for fq_qlinear_fwd: the dequantized X_hat [M, K] BF16 at offset
 * 0, the dequantized and transposed W_hat^T [N, K] BF16 at offset
 * round_up(M * K * 2, 256), then 8192 bytes of reduction scratch.  When both
 * descriptors are MXFP4, the operands stay encoded instead: X's codes [M, K/2] at 0, X's E8M0 scales [M, K/32] at
 * c1 = round_up(M * K / 2, 256), W's codes in the transposed layout [N, K/2]
 * at c2 = c1 + round_up(M * K / 32, 256), W's scales [N, K/32] at
 * c2 + round_up(N * K / 2, 256) (same total size).  0 for dimensions outside
 * the limits of fq_qlinear_fwd. */
size_t fq_qlinear_workspace_size(const fq_desc *desc_x, const fq_desc *desc_w,
                                 int64_t M, int64_t K, int64_t N);

/* QAT linear forward: Y [M, N] BF16 = FQ(X) [M, K] x FQ(W) [K, N] with FP32
 * accumulation on the matrix cores.  X is quantized in groups along K (its
 * rows: desc_x->axis must be FQ_AXIS_ROW), W in groups along K (its
 * columns: desc_w->axis must be FQ_AXIS_COL), so both operands are blocked
 * along the contraction.  Shapes: M, N >= 1; K a multiple of 64 (the
 * matrix-core kernels step through K 64 elements at a time and have no
 * partial step; this also covers both block sizes), and of 128 for
 * FQ_OUTER_BLOCK128; N a multiple of 8 (W is quantized along its columns,
 * whose kernels move 8 columns at a time); M, K, N < 2^31 and M * K, K * N
 * and M * N <= 2^34.
 * Otherwise FQ_ERR_SHAPE.
 * Source: gpt-oss QAT tutorial, "NVFP4: The Next Generation"
 * (weight-activation quantization of the MLP); TetraJet-v2 sec. 2 (NVFP4
 * activations and weights in every linear layer).  MXFP4 x MXFP4 multiplies the E2M1 codes with their E8M0 block scales on the scaled FP4
 * matrix cores (OCP Microscaling v1.0 block scaling), which is the same
 * product of the same dequantized values. */
fq_status fq_qlinear_fwd(const fq_desc *desc_x, const fq_desc *desc_w,
                         const void *x_bf16, const void *w_bf16, int64_t M,
                         int64_t K, int64_t N, void *y_bf16, void *ws,
                         size_t ws_bytes, void *stream);

/* Random Hadamard transform: y = BF16_RNE(RN32(c_n * H_n (s o x))) in
 * blocks of n = 16 or 128 consecutive elements along `axis` (FQ_AXIS_ROW:
 * along each row; FQ_AXIS_COL: down each column), where H_n is the Hadamard
 * matrix in Sylvester order applied by radix-2 FP32 butterflies (half-widths
 * 1, 2, ..., n/2; a pair (a, b) becomes (a + b, a - b)), c_n the FP32 value
 * nearest to 1/sqrt(n), and s_j = -1 where bit (j mod 128) of
 * Philox4x32-10(key = seed, counter = (j / 128, 0, 0, 0)) is set (bit t of
 * output word w counts as bit 32w + t), j the position along the axis.
 * x, y: device [rows, cols] BF16, 16-byte aligned, not overlapping.  The
 * transformed axis must be a multiple of n; FQ_AXIS_COL needs cols % 8 == 0.
 * Source: "Resumo Tecnico: TetraJet-v2", sec. 2.C (OutControl: a random
 * Hadamard transform on the backward's products spreads outlier energy). */
fq_status fq_hadamard(const void *x_bf16, int64_t rows, int64_t cols, int32_t axis,
                      int32_t block, uint64_t seed, void *y_bf16, void *stream);

/* Workspace for fq_qlinear_bwd (internal layout; the size depends only on
 * the arguments). */
size_t fq_qlinear_bwd_workspace_size(const fq_desc *desc_x, const fq_desc *desc_w,
                                     const fq_desc *desc_g, int32_t rht_block, int64_t M,
                                     int64_t K, int64_t N);

/* QAT linear backward of fq_qlinear_fwd (Y = FQ(X) x FQ(W), X [M, K],
 * W [K, N]), given dY [M, N]:
 *   dX [M, K] = STE_X( Q(dY) x Q(W_hat)^T ),  Q along N for both operands,
 *   dW [K, N] = STE_W( Q(X_hat)^T x Q(dY) ),  Q along M for both operands,
 * where X_hat = FQ(X, desc_x) and W_hat = FQ(W, desc_w) are the forward's
 * fake-quantized operands (recomputed here), Q quantizes with desc_g's
 * format and rounding along the contraction axis of each product, and
 * STE_X / STE_W pass a gradient entry where the forward did not clip that
 * entry of X / W (a <= 6) and write +0 where it did.  The four Q draws use
 * Philox keys desc_g->seed + 0 (dY along N), + 1 (W_hat along N), + 2 (X_hat
 * along M), + 3 (dY along M); desc_g->axis is ignored.  rht_block = 16 or
 * 128 first rotates both operands of each product along its contraction axis
 * by the random Hadamard transform of fq_hadamard with seed rht_seed (which
 * cancels in the exact product); 0 leaves them as they are (with an MXFP4 or
 * double-block desc_g the rotation runs inside the quantizers, as in
 * fq_fake_quant_rht).  Products accumulate in FP32 on the matrix cores and are
 * rounded to BF16 before the STE, which is applied as the product is stored.
 * With an MXFP4 desc_g both products run on the scaled FP4 matrix cores from
 * the gradient operands' codes and E8M0 scales.
 * Shapes: K a multiple of 8 and of desc_x's and desc_w's block sizes (128
 * for FQ_OUTER_BLOCK128); M and N multiples of 64 and of desc_g's block size
 * (128 for FQ_OUTER_BLOCK128) and of rht_block; desc_x->axis FQ_AXIS_ROW,
 * desc_w->axis FQ_AXIS_COL as in the forward.
 * Pointers x, w, dy, dx, dw, ws: device, 16-byte aligned, caller-owned; ws
 * at least fq_qlinear_bwd_workspace_size bytes.  Errors as fq_qlinear_fwd.
 * Source: TetraJet-v2, sec. 2.A (the backward computes on the aligned X_hat,
 * with stochastic rounding so that E[round(x)] = x, and 1x16 weight groups
 * realigned for the transposed weight) and sec. 2.C (random Hadamard
 * transform of the backward's products); "Como o Treinamento ...",
 * "Detalhes tecnicos" (gradients pass the quantizer by STE, clipping
 * effects). */
fq_status fq_qlinear_bwd(const fq_desc *desc_x, const fq_desc *desc_w,
                         const fq_desc *desc_g, int32_t rht_block, uint64_t rht_seed,
                         const void *x_bf16, const void *w_bf16, const void *dy_bf16,
                         int64_t M, int64_t K, int64_t N, void *dx_bf16, void *dw_bf16,
                         void *ws, size_t ws_bytes, void *stream);

/* ---- TetraJet-v2 OsciReset ("Resumo Tecnico: TetraJet-v2", sec. 2.B) ----
 * Per-element state of n weights, all device arrays the caller owns: w_prev
 * and dist_m, dist_q FP32 [n], q_prev BF16 [n].  w is the FP32 master weight,
 * q the BF16 fake-quantized weight the forward pass used.  n >= 4, n a
 * multiple of 4; every pointer 16-byte aligned (q, q_prev: 8-byte).
 *
 * fq_osci_track: one training step.  dist_m += |w - w_prev| and dist_q +=
 * |q - q_prev| (FP32, one rounding per operation), then w_prev = w and
 * q_prev = q.  first != 0 starts the trajectory: records w and q and zeroes
 * the distances (no memset: safe inside a captured graph). */
fq_status fq_osci_track(const float *w, const void *q_bf16, float *w_prev, void *q_prev_bf16,
                        float *dist_m, float *dist_q, int64_t n, int32_t first, void *stream);

/* fq_osci_reset: the check, called when the learning rate is low.  The
 * oscillation risk is dist_q / dist_m; an element with dist_q > RN(tau *
 * dist_m) is reset, all others keep w.  Then every element starts a new
 * window: w_prev = w, q_prev = q, distances 0.  tau is the risk threshold
 * (finite, >= 0).  w, q and the state are [rows, cols] row-major (n =
 * rows * cols), cols a multiple of 4.
 * target FQ_OSCI_BIN_CENTRE (sec. 2.B, "Mecanismo": the master weight goes
 * to the centre of its current quantization bin): w = sign * RN(c_m * s_eff)
 * for the element's current E2M1 code (sign, magnitude m) and effective
 * block scale s_eff, read from codes / scales / outer, the fq_quantize or
 * fq_fake_quant outputs of the quantization that gave q, in desc's format
 * and axis layout (rows x cols is the shape of that quantization's input).
 * c_m is the centre of the interval of scaled magnitudes that round to grid
 * value g_m: 0, 0.5, 1, 1.5, 2.125, 3, 4.25, 6 for g = 0, 0.5, 1, 1.5, 2, 3,
 * 4, 6 (the bins of 2 and 4, [1.75, 2.5] and [3.5, 5], are lopsided; the top
 * bin, from 5, is read as closing at 7, midway to 8, the next value of the
 * E2M1 exponent progression, so its centre is 6).  desc, codes, scales
 * (16-byte aligned) are required, outer (4-byte aligned) for NVFP4; desc's
 * shape rules are those of fq_quantize.
 * target FQ_OSCI_GRID_VALUE: w = q (its quantized value); desc, codes,
 * scales and outer are not read and may be NULL. */
enum { FQ_OSCI_BIN_CENTRE = 0, FQ_OSCI_GRID_VALUE = 1 };
fq_status fq_osci_reset(const fq_desc *desc, float *w, const void *q_bf16, const void *codes,
                        const void *scales, const float *outer, int64_t rows, int64_t cols,
                        float *w_prev, void *q_prev_bf16, float *dist_m, float *dist_q,
                        float tau, int32_t target, void *stream);

/* ---- TetraJet-v2 static outlier-channel retention (sec. 2.C) ----
 * Calibration: fq_channel_absmax folds max |x[:, c]| of a BF16 [rows, cols]
 * tensor into amax [cols] (uint32, the BF16 magnitude bits; zero it once before
 * the first batch), by integer atomic maximum, so the result does not depend
 * on order.  cols a multiple of 8; x 16-byte and amax 4-byte aligned. */
fq_status fq_channel_absmax(const void *x_bf16, int64_t rows, int64_t cols, uint32_t *amax,
                            void *stream);

/* Selection: the k channels with the largest amax (ties: lower index first)
 * are retained.  Writes retain [cols / 8] (bit c mod 8 of byte c / 8 set for a
 * retained channel) and chan_scale [cols] FP32 = amax_c / 448 (the largest
 * E4M3 value; 0 for other channels).  0 <= k <= cols, cols a multiple of 8. */
fq_status fq_select_channels(const uint32_t *amax, int64_t cols, int64_t k, void *retain,
                             float *chan_scale, void *stream);

/* Fake quantization with retained channels, along either axis: the columns
 * of x whose retain bit is set (the activation's channels) are FP8 E4M3
 * fake-quantized under chan_scale (|x| / s in FP32, nearest-even, saturating
 * at 448, times s, sign kept; s = 0 gives +-0) and carry FP4 code 0; every
 * FP4 block, 128-element outer and per-tensor maximum is taken over the other
 * elements only.  That is the plain fake quantization of x with the retained
 * columns set to +0, the FP8 values in their place.  FQ_AXIS_ROW: the
 * retained columns drop out of the 1xB groups they share; FQ_AXIS_COL: every
 * group of a retained column is empty.  desc: any format, rounding and axis;
 * cols a multiple of 8; y required, codes, scales, outer optional (as
 * fq_fake_quant); retain and chan_scale as written by fq_select_channels,
 * chan_scale 16-byte aligned; ws / ws_bytes as fq_fake_quant (per-tensor
 * NVFP4: 4096 bytes).  Source: "Resumo Tecnico: TetraJet-v2", sec. 2.C
 * (OutControl, "Retencao Estatica de Outliers": the top p % channels stay in
 * FP8 in the forward and the backward pass, the rest in FP4). */
fq_status fq_fake_quant_retain(const fq_desc *desc, const void *x_bf16, int64_t rows,
                               int64_t cols, void *y_bf16, void *codes, void *scales,
                               float *outer, const void *retain, const float *chan_scale,
                               void *ws, size_t ws_bytes, void *stream);

/* fq_qlinear_fwd with the activation's retained channels (columns of X, as
 * fq_fake_quant_retain along the row axis) kept in FP8: Y = FQ_retain(X) x
 * FQ(W) on the BF16 matrix cores (whatever the formats).  Arguments and
 * workspace as fq_qlinear_fwd, plus retain [K/8] and chan_scale [K]; K a
 * multiple of 8.  Source: "Resumo Tecnico: TetraJet-v2", sec. 2.C (forward
 * pass). */
fq_status fq_qlinear_fwd_retain(const fq_desc *desc_x, const fq_desc *desc_w, const void *x_bf16,
                                const void *w_bf16, int64_t M, int64_t K, int64_t N,
                                const void *retain, const float *chan_scale, void *y_bf16,
                                void *ws, size_t ws_bytes, void *stream);

/* fq_qlinear_bwd (without the rotation) with the activation's retained
 * channels kept in FP8: X_hat is fq_fake_quant_retain of X along the row
 * axis, X_hat's quantization along M for dW keeps the same channels in FP8
 * (fq_fake_quant_retain along the column axis with desc_g's format, rounding
 * and key seed + 2), and STE_X passes a retained entry where |x| / s <= 448
 * (the FP8 format's clip).  Both products run on the BF16 matrix cores.
 * Arguments and workspace as fq_qlinear_bwd with rht_block = 0, plus retain
 * [K/8] and chan_scale [K]; K a multiple of 8.  Source: "Resumo Tecnico:
 * TetraJet-v2", sec. 2.C (forward and backward pass). */
fq_status fq_qlinear_bwd_retain(const fq_desc *desc_x, const fq_desc *desc_w,
                                const fq_desc *desc_g, const void *x_bf16, const void *w_bf16,
                                const void *dy_bf16, int64_t M, int64_t K, int64_t N,
                                const void *retain, const float *chan_scale, void *dx_bf16,
                                void *dw_bf16, void *ws, size_t ws_bytes, void *stream);

/* ---- Around the linears of a training step ------------------------------------
 * Operators that a quantization-aware training step runs beside its quantized
 * products: the norm in front of a linear, the sorting of tokens by expert
 * around the experts' linears, and the optimizer behind them.  Unlike the
 * quantizers they accept infinities and NaN, as described at each.
 *
 * 8-bit rows (FQ_F8_*), elements E4M3 (OCP OFP8 v1.0), scales rounded up so
 * that no value saturates (so the straight-through gradient passes everywhere):
 *   FQ_F8_MX   per 32 consecutive elements the smallest power of two 2^e with
 *              amax <= 448 * 2^e, as E8M0 code clamp(e, -127, 127) + 127 (OCP
 *              MX v1.0's MXFP8 layout): scales uint8 [rows, cols / 32].
 *   FQ_F8_ROW  per row s = max(RN(amax * RN(1 / 448)), 2^-126): scales FP32
 *              [rows]; the scaled value is RN(x * RN(1 / s)) clamped to +-448.
 * Codes are nearest even.  A block (row) whose amax is infinite or NaN gets
 * scale code 255 (scale NaN) and codes 0x7F, and stands for NaN.  cols must be
 * a multiple of 32. */
enum { FQ_F8_NONE = 0, FQ_F8_MX = 1, FQ_F8_ROW = 2 };
enum { FQ_TYPE_BF16 = 0, FQ_TYPE_F32 = 1 };

/* Residual addition and root-mean-square norm:
 *   h = x + res   rounded once to the stream's type (nearest even);
 *   r = 1 / sqrt(mean(h^2) + eps) over each row, FP32;
 *   n = (h * r) * gamma, FP32;   y = BF16_RNE(n).
 * The norm is that of the stored h, the value the backward reads.  Without a
 * residual (res NULL, then h NULL too) h is x and stream_type is not used.
 * With f8 != FQ_F8_NONE n goes to 8 bits instead (above): codes [rows, cols]
 * and scales, and y, if given, holds the values they stand for (for
 * FQ_F8_ROW rounded to BF16).
 * x BF16 [rows, cols]; res and h of stream_type (FQ_TYPE_*), h may be res;
 * gamma [cols] of gamma_type; rstd FP32 [rows] receives r (may be NULL).  y is
 * required without f8; with it at least one of y and codes, and scales with
 * codes.  rows >= 1, 1 <= cols <= 32768 (any, a multiple of 32 with f8), rows *
 * cols <= 2^34.  All pointers 16-byte aligned, rstd 4-byte.  A NaN in
 * a row makes all of its n NaN; an infinity makes r 0, so n is NaN there and 0
 * elsewhere in the row. */
fq_status fq_rmsnorm_fwd(const void *x_bf16, const void *res, int32_t stream_type,
                         const void *gamma, int32_t gamma_type, float eps, int64_t rows,
                         int64_t cols, int32_t f8, void *h, void *y_bf16, void *codes,
                         void *scales, float *rstd, void *stream);

/* Bytes of workspace of fq_rmsnorm_bwd (column sums of groups of rows); 0 for
 * a shape outside its limits. */
size_t fq_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols);

/* Backward of fq_rmsnorm_fwd.  With xh = h * r and g = dy * gamma:
 *   dh = r * (g - xh * mean(g * xh)) + dres,   dgamma = sum over rows of dy * xh.
 * h of stream_type is the forward's h (x in BF16 where it had no residual),
 * rstd the forward's r.  dres (same type, may be NULL) is the gradient that
 * reaches h from elsewhere; dh (same type, may be dres, h or dy) is the gradient
 * of both x and res; dx, if given, receives it rounded to BF16 (the gradient of x
 * beside an FP32 stream).  dgamma FP32 [cols] may be NULL, then no workspace
 * is needed.  FP32 sums in a fixed order: equal calls give equal bits.  The
 * rounding to 8 bits is passed straight through. */
fq_status fq_rmsnorm_bwd(const void *dy_bf16, const void *h, int32_t stream_type,
                         const void *gamma, int32_t gamma_type, const float *rstd,
                         const void *dres, int64_t rows, int64_t cols, void *dh, void *dx_bf16,
                         float *dgamma, void *ws, size_t ws_bytes, void *stream);

/* Tokens sorted by expert.  experts_of [tokens, k] int32 names the experts of
 * every token; assignment a = t * k + j.  Expert e's assignments, in ascending
 * order, take rows offsets[e], offsets[e] + 1, ... of the sorted order; each
 * segment is padded to a multiple of `align` rows (fq_qlinear_bwd takes
 * multiples of 64 or 128).  An id outside [0, experts) is no expert: such an
 * assignment has no row.
 *   offsets [experts + 1] int32: segment starts, then the number of rows used;
 *   pos [tokens, k] int32: row of each assignment, -1 without one;
 *   src [rows] int32: assignment of each row, -1 for padding and unused rows.
 * rows, the length of the sorted order's buffers, is at least fq_moe_rows
 * (what the segments take at most, whatever the ids; 0 for arguments outside
 * the limits).  1 <= k <= 64, 1 <= experts <= 1024, tokens * k <= 2^30, 1 <=
 * align <= 1024.  ws: fq_moe_sort_workspace_size bytes (0: may be NULL). */
enum { FQ_MOE_MAX_K = 64, FQ_MOE_MAX_ALIGN = 1024 };
int64_t fq_moe_rows(int64_t tokens, int64_t k, int64_t experts, int64_t align);
size_t fq_moe_sort_workspace_size(int64_t tokens, int64_t k, int64_t experts);
fq_status fq_moe_sort(const int32_t *experts_of, int64_t tokens, int64_t k, int64_t experts,
                      int64_t align, int64_t rows, int32_t *offsets, int32_t *pos, int32_t *src,
                      void *ws, size_t ws_bytes, void *stream);

/* Rows of the tokens in the sorted order: y[pos[t, j]] = x[t], +0 in rows
 * without an assignment.  y BF16 [rows, cols]; x BF16 [tokens, cols], or with
 * f8 the codes and scales of fq_rmsnorm_fwd, decoded on the way (rounded to
 * BF16).  cols a multiple of 8 (32 with f8) below 2^31, rows below 2^31, rows *
 * cols and tokens * cols at most 2^34, here and in the next two; tokens and k as
 * for fq_moe_sort.  pos and src as fq_moe_sort wrote them; entries outside [0,
 * rows) or [0, tokens * k) count as -1.  Its backward is fq_moe_combine without
 * weights. */
fq_status fq_moe_dispatch(const void *x, int32_t f8, const void *scales, int64_t tokens,
                          int64_t k, int64_t cols, int64_t rows, const int32_t *pos,
                          const int32_t *src, void *y_bf16, void *stream);

/* Back to the tokens: out[t] = BF16_RNE(sum over j of weights[t, j] *
 * y[pos[t, j]]), summed in FP32 in the order of j over the assignments that
 * have a row (+0 for a token with none); weights FP32 [tokens, k], NULL for
 * ones. */
fq_status fq_moe_combine(const void *y_bf16, const float *weights, int64_t tokens, int64_t k,
                         int64_t cols, int64_t rows, const int32_t *pos, void *out_bf16,
                         void *stream);

/* Backward of fq_moe_combine: dy[pos[t, j]] = BF16_RNE(weights[t, j] *
 * dout[t]), +0 in rows without an assignment; dweights[t, j] = <dout[t],
 * y[pos[t, j]]> in FP32, 0 without a row. */
fq_status fq_moe_combine_bwd(const void *dout_bf16, const void *y_bf16, const float *weights,
                             int64_t tokens, int64_t k, int64_t cols, int64_t rows,
                             const int32_t *pos, const int32_t *src, void *dy_bf16,
                             float *dweights, void *stream);

/* One AdamW step over `count` tensors:
 *   g' = g * grad_scale;  m = beta1 m + (1 - beta1) g';
 *   v = beta2 v + (1 - beta2) g'^2;  l = lr * lr_mult;
 *   w = w (1 - l * weight_decay)
 *       - l / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps);
 *   w_bf16 = BF16_RNE(w),
 * in FP32.  w is the FP32 master weight (as for fq_osci_track), w_bf16 (may be
 * NULL) the copy that the linears read, g BF16 or FP32.
 * state_type FQ_STATE_F32: m, v FP32 [n].  FQ_STATE_F8: m E4M3 and v E5M2
 * codes [n], m_scale and v_scale FP32 [ceil(n / 128)], a scale per 128
 * consecutive elements: s = max(RN(amax * RN(1 / 448)), 2^-126) for m (57344 for v)
 * with amax over the block's finite values, a = min(|x| RN(1 / s), largest),
 * rounded stochastically: up to the next value exactly when r16 <
 * floor(2^16 * fraction of the way to it), with r16 the low (m) or high (v)
 * half of word n mod 4 of Philox4x32-10 with key seed and counter (low and
 * high word of n / 4, number of the tensor in the list, step), n the element.
 * A positive v gets at least code 1; infinities and NaN get code 0x7F, NaN (m
 * with its sign).
 * Rounding to nearest would keep an 8-bit v where it is for ever, because
 * 1 - beta2 is far below half a step of the format.  All-zero codes and scales
 * are the state before the first step.
 * step counts from 1.  lr and eps are rounded to FP32, where lr is finite and eps 0
 * or positive and finite (with eps 0 an element whose m and v are 0 becomes NaN,
 * 0 / 0).  grad_scale: device scalar (a clipping factor), NULL for
 * 1.  lr and step are read by the call: a captured call keeps them.  w, w_bf16,
 * g, m, v 16-byte aligned, scales 4-byte; n <= 2^34, n = 0 is skipped;
 * `tensors` is read during the call only.  No workspace. */
enum { FQ_STATE_F32 = 0, FQ_STATE_F8 = 1 };
typedef struct {
    float *w;
    void *w_bf16;
    const void *g;
    void *m;
    void *v;
    float *m_scale;
    float *v_scale;
    int64_t n;
    int32_t g_type;
    int32_t reserved;      /* must be 0 */
    float lr_mult;
    float weight_decay;
} fq_adamw_tensor;
typedef struct {
    double lr, beta1, beta2, eps;
    int64_t step;
    uint64_t seed;
    const float *grad_scale;
    int32_t state_type;
    int32_t reserved;      /* must be 0 */
} fq_adamw_hyper;
fq_status fq_adamw_step(const fq_adamw_hyper *hyper, const fq_adamw_tensor *tensors,
                        int64_t count, void *stream);

/* The same list for many steps, in one launch a step whatever its length
 * (fq_adamw_step launches once per 32 tensors).  fq_adamw_plan checks the
 * tensors as fq_adamw_step does and writes fq_adamw_plan_size bytes to `plan`
 * (host memory, 16-byte aligned); the caller keeps them and copies them to
 * device memory once (16-byte aligned).  fq_adamw_step_plan takes both copies;
 * hyper->state_type must be the plan's.  A plan holds the tensors' addresses:
 * their contents may change between steps, where they are may not.  A plan has
 * at most 2^31 tiles (of 4096 elements of a tensor, 2048 with 8-bit moments). */
size_t fq_adamw_plan_size(int64_t count);
fq_status fq_adamw_plan(const fq_adamw_tensor *tensors, int64_t count, int32_t state_type,
                        void *plan, size_t plan_bytes);
fq_status fq_adamw_step_plan(const fq_adamw_hyper *hyper, const void *plan,
                             const void *plan_device, void *stream);

/* ---- The feed-forward products of a training step ---------------------------------
 * In BF16 with FP32 sums on the matrix cores: for layers that are not quantized,
 * and for operands that are fake-quantized already (fq_fake_quant's y and
 * fq_moe_dispatch's rows are BF16 tensors).
 *
 * One product, or one per expert: with offsets (int32 [experts + 1], device, as
 * fq_moe_sort wrote them) rows offsets[e] .. offsets[e + 1] meet the weight and
 * bias of expert e, whatever the segments' lengths, none included; rows past the
 * last segment are neither read nor written.  Entries are brought into 0 .. rows;
 * where they do not ascend the results of the rows concerned are unspecified.
 * Without offsets (NULL) experts is 0 and weights and biases have no expert axis.
 *
 * Layouts, row-major: activations [rows, ...]; weights BF16 [experts, k, n] (as
 * fq_qlinear_fwd's); bias BF16 or FP32 [experts, n], may be NULL.
 * Shapes: 1 <= rows <= 2^30; k and n multiples of 8 from 8 to 2^20 (of 32 where an
 * operand of that width is held in 8 bits); rows * k, rows * columns and experts
 * * k * columns at most 2^34; experts <= 1024.  Tensors 16-byte aligned, offsets
 * 4-byte.  Outputs overlap no other operand except where it is said.
 *
 * Activations a(z), FP32: FQ_ACT_RELU max(z, 0); FQ_ACT_SILU z / (1 + exp(-z));
 * FQ_ACT_GELU z (1 + erf(z / sqrt 2)) / 2.  An infinite z may give NaN with the
 * last two (infinity times zero).  ReLU's derivative is 0 at 0.
 *
 * Checkpoints: what a forward keeps for its backward, in BF16 or in 8 bits
 * (FQ_F8_*, above).  `pre` receives the values before the activation, rounded to
 * BF16 (FQ_F8_NONE) or as codes and scales (FQ_F8_MX), from FP32 in both; where
 * an expert's rows end it is left as it was, as y.  A backward takes x in BF16 or as
 * 8-bit rows (FQ_F8_MX or FQ_F8_ROW, as fq_rmsnorm_fwd or fq_f8_encode wrote them):
 * the values that codes and scales stand for.  FQ_F8_MX's are exact in BF16 (but below
 * its normal range).  FQ_F8_ROW's are rounded to it where dz is dy; else dw is made of
 * the codes times a power of two of their scale and of d times its mantissa (at most 1
 * for scales below 2^100), that product rounded to BF16. */
enum { FQ_ACT_NONE = 0, FQ_ACT_RELU = 1, FQ_ACT_SILU = 2, FQ_ACT_GELU = 3 };

/* 8-bit rows of x BF16 [rows, cols] and back: codes uint8 [rows, cols], scales as
 * FQ_F8_MX or FQ_F8_ROW has them (above).  y BF16 [rows, cols] is each code's
 * value times its scale, rounded to BF16 (exact for FQ_F8_MX unless it falls
 * below BF16's normal range).  cols a multiple of 32, below 2^31 and for
 * fq_f8_encode with FQ_F8_ROW at most 32768; rows * cols <= 2^34.  A block or row
 * with an infinity or NaN stands for NaN.  All pointers 16-byte aligned. */
fq_status fq_f8_encode(const void *x_bf16, int32_t f8, int64_t rows, int64_t cols, void *codes,
                       void *scales, void *stream);
fq_status fq_f8_decode(const void *codes, const void *scales, int32_t f8, int64_t rows,
                       int64_t cols, void *y_bf16, void *stream);

/* Matrix product with bias, activation and residual:
 *   z = x w + bias;   y = a(z) + res.
 * x BF16 [rows, k], w [experts, k, n], y of y_type [rows, n] rounded once, res
 * (may be NULL, may be y) of y's type.  pre (may be NULL) [rows, n] receives z as
 * pre_f8 says, pre_scales its scales.  ws: fq_linear_fwd_workspace_size bytes (0:
 * may be NULL). */
size_t fq_linear_fwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts);
fq_status fq_linear_fwd(const void *x_bf16, const void *w_bf16, const void *bias,
                        int32_t bias_type, const void *res, int64_t rows, int64_t k, int64_t n,
                        int64_t experts, const int32_t *offsets, int32_t act, void *pre,
                        int32_t pre_f8, void *pre_scales, void *y, int32_t y_type, void *ws,
                        size_t ws_bytes, void *stream);

/* Backward of fq_linear_fwd for the gradient dy BF16 [rows, n] of y (which is also
 * the gradient of res):
 *   d = dy a'(z);  dz = BF16_RNE(d);  dx = BF16_RNE(dz w^T);  dw = x^T dz;
 *   dbias = sum over rows of d,
 * z read from pre (not read with FQ_ACT_NONE), dw of dw_type [experts, k, n],
 * dbias FP32 [experts, n], both 0 for an expert without rows.  dx, dw and dbias
 * may each be NULL, not all; x is read for dw only, w for dx only.  Sums have a
 * fixed order: equal calls give equal bits. */
size_t fq_linear_bwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts,
                                    int32_t x_f8);
fq_status fq_linear_bwd(const void *dy_bf16, const void *x, int32_t x_f8, const void *x_scales,
                        const void *w_bf16, const void *pre, int32_t pre_f8,
                        const void *pre_scales, int64_t rows, int64_t k, int64_t n,
                        int64_t experts, const int32_t *offsets, int32_t act, void *dx_bf16,
                        void *dw, int32_t dw_type, float *dbias, void *ws, size_t ws_bytes,
                        void *stream);

/* Gated feed-forward block, both projections, the activation and the product in
 * one kernel:
 *   [g, u] = x w + bias (the first and the last n columns);
 *   h = a(min(g, limit)) * (min(max(u, -limit), limit) + shift),
 * a(v) = v / (1 + exp(-alpha v)) for FQ_ACT_SILU, else as above (alpha 1).
 * {FQ_ACT_SILU, 1, INFINITY, 0} is the usual block.  limit > 0, may be infinite.
 * x BF16 [rows, k], w [experts, k, 2 n], bias [experts, 2 n], h BF16 [rows, n], pre
 * (may be NULL) [rows, 2 n] as for fq_linear_fwd. */
typedef struct {
    int32_t act;
    float alpha, limit, shift;
} fq_gate;
size_t fq_glu_fwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts);
fq_status fq_glu_fwd(const fq_gate *gate, const void *x_bf16, const void *w_bf16,
                     const void *bias, int32_t bias_type, int64_t rows, int64_t k, int64_t n,
                     int64_t experts, const int32_t *offsets, void *pre, int32_t pre_f8,
                     void *pre_scales, void *h_bf16, void *ws, size_t ws_bytes, void *stream);

/* Its backward for the gradient dh BF16 [rows, n], from pre:
 *   dg = dh (u' + shift) a'(g') where g <= limit, else 0;
 *   du = dh a(g') where -limit <= u <= limit, else 0;   d = [dg, du],
 * and dz, dx, dw [experts, k, 2 n], dbias [experts, 2 n] of d as in fq_linear_bwd.
 * h, if given, receives the block's output again, from pre: BF16 [rows, n], what
 * the next product's backward takes as its x. */
size_t fq_glu_bwd_workspace_size(int64_t rows, int64_t k, int64_t n, int64_t experts,
                                 int32_t x_f8);
fq_status fq_glu_bwd(const fq_gate *gate, const void *dh_bf16, const void *x, int32_t x_f8,
                     const void *x_scales, const void *w_bf16, const void *pre, int32_t pre_f8,
                     const void *pre_scales, int64_t rows, int64_t k, int64_t n, int64_t experts,
                     const int32_t *offsets, void *dx_bf16, void *dw, int32_t dw_type,
                     float *dbias, void *h_bf16, void *ws, size_t ws_bytes, void *stream);

/* Static description of a status code. */
const char *fq_status_string(fq_status s);

/* Message of the last error on the calling thread ("" if none). */
const char *fq_last_error(void);

/* Library version, e.g. "0.1.0". */
const char *fq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FQ_H */
