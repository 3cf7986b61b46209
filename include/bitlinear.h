/*
 * bitlinear.h — C ABI of the MI355X (gfx950) BitLinear library.
 *
 * The library computes the BitNet b1.58 BitLinear forward pass in five steps:
 * absmean ternarisation of a weight matrix, packing of the codes, per-token
 * symmetric absmax INT8 activation quantisation, an integer product of INT8
 * activations against {-1, 0, +1} codes with INT32 accumulation, and the
 * gamma * scale / 127 dequant epilogue. Sources, cited by page title and
 * section:
 *   [QAT-en] "QAT and BitNet: A Deep Dive into 1-bit and 1.58-bit
 *            Quantization-Aware Training" (kongchang.com)
 *   [QAT-zh] "QAT与BitNet：1-bit及1.58-bit量化训练解析" (kongchang.com)
 *   [b158]   "BitNet b1.58深度解析：三值权重如何重塑大模型推理" (0539edu.com)
 *
 * Conventions for every call:
 *  - Shapes: W is [N, K] row-major (out_features x in_features), x is [M, K]
 *    row-major (M tokens), y is [M, N] row-major: y = x W^T ([b158] §4.2,
 *    y_i = sum_j w_ij x_j).
 *  - Every array argument is a DEVICE pointer, owned and allocated by the
 *    caller, 16-byte aligned, except the weight scales (gamma, gammas), which
 *    need only 4-byte alignment so that a stack of matrices can keep its
 *    scales in consecutive floats. The library never allocates, frees or
 *    synchronises: each call only enqueues kernels on `stream` (a hipStream_t
 *    passed as void*, NULL = the default stream) and returns.
 *  - Argument errors are detected before any HIP call; the call then returns
 *    BL_ERR_INVALID_ARG with no side effect. Bad arguments are: a NULL
 *    required pointer, a misaligned pointer, a negative size, K < 1,
 *    K > 16909320 (127*K must fit in INT32), an unknown dtype / layout /
 *    scheme, a too-small workspace. M = 0 or N = 0 is an empty problem and
 *    returns BL_OK without launching anything (pack_weights needs N >= 1).
 *  - If the current device is not a gfx950 GPU, or a launch fails, the call
 *    returns BL_ERR_DEVICE (the HIP error is consumed). Kernels that fault
 *    later surface at the caller's next synchronisation.
 *  - Non-finite inputs (NaN, Inf) are outside the contract.
 *  - Calls may come from several host threads and streams. The library's
 *    only process-wide state is per-device and set once: the result of the
 *    architecture check, the compute-unit count and the raised LDS limit of
 *    kernels that use more than 64 KiB, all kept in atomics. Concurrent calls
 *    that write the same output buffers race like any other GPU work.
 */
#ifndef BITLINEAR_H
#define BITLINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    BL_OK = 0,
    BL_ERR_INVALID_ARG = 1,
    BL_ERR_UNSUPPORTED = 2,
    BL_ERR_DEVICE = 3
} bl_status;

/* Element types of floating-point inputs and outputs. bf16 values are
 * widened exactly to fp32 before any arithmetic. */
typedef enum { BL_F32 = 0, BL_BF16 = 1 } bl_dtype;

/* Packed weight layouts ([b158] §2.3 and §6.3: two bits per weight with the
 * patterns 00, 01, 10, four weights per byte; or five ternary values per
 * byte since 3^5 = 243 <= 256, 1.6 bits per weight).
 *
 * BL_PACK_2BIT: the stored field is u = c + 1 (00 = -1, 01 = 0, 10 = +1; 11
 *   is never written). A row takes row_bytes = roundup(ceil(K/4), 16) bytes.
 *   Codes are grouped by 16 into one little-endian 32-bit word; code k of a
 *   row sits in byte 4*(k/16) + (k%4) at bits 2*((k%16)/4)..+1, so that
 *   (word >> 2j) & 0x03030303 holds codes 4j..4j+3 of the group in its four
 *   bytes. Padding codes (k >= K) are 0.
 * BL_PACK_BASE3: byte j of a row holds codes 5j..5j+4 as the base-3 number
 *   t0 + 3 t1 + 9 t2 + 27 t3 + 81 t4 with t = c + 1 (first code in the least
 *   significant trit; values 0..242). row_bytes = roundup(ceil(K/5), 16);
 *   padding trits are t = 1 (code 0).
 * BL_PACK_1BIT: binary codes only (BL_BINARY), one bit per weight as in the
 *   1-bit BitLinear ([QAT-en] "What Does BitLinear Change?": +-1 weights at
 *   1 bit each). Bit 1 = +1, bit 0 = -1. Codes are grouped by 32 into one
 *   little-endian 32-bit word; code k of a row sits in byte 4*(k/32) + (k%4)
 *   at bit (k%32)/4, so that (word >> j) & 0x01010101 holds codes 4j..4j+3 in
 *   its four bytes. row_bytes = roundup(ceil(K/8), 16); padding bits are 0
 *   (the products never read them). Every bit pattern is a valid matrix. */
typedef enum { BL_PACK_2BIT = 0, BL_PACK_BASE3 = 1, BL_PACK_1BIT = 2 } bl_layout;

/* Weight quantisers.
 * BL_TERNARY (b1.58): gamma = mean|W|; c = clamp(round(W / (gamma + eps)),
 *   -1, 1), round half to even ([QAT-en] "The Ternary Weight Recipe" and its
 *   ternary_weights code; [b158] §3.1).
 * BL_BINARY (1-bit BitNet): alpha = mean(W); c = +1 where W > alpha, else -1;
 *   the weight scale is beta = mean|W| ([QAT-en] "The BitLinear Recipe",
 *   steps 2 and 4). */
typedef enum { BL_TERNARY = 0, BL_BINARY = 1 } bl_scheme;

/* Bytes one packed row of K codes occupies in `layout`; -1 for K < 1 or an
 * unknown layout. Host-only, pure. */
int64_t bitlinear_packed_row_bytes(int64_t K, int layout);

/* Device workspace (bytes) bitlinear_pack_weights needs for an N x K matrix:
 * it holds the per-block partial sums of the two-pass mean reduction. 0 for
 * N < 1, K < 1 or an N * K past the int64 range (shapes the pack refuses). */
size_t bitlinear_pack_workspace_bytes(int64_t N, int64_t K);

/* Quantise and pack a latent weight matrix ([QAT-en] "The Ternary Weight
 * Recipe"; [b158] §3.1 and §6.3; [QAT-en] "The BitLinear Recipe" for
 * BL_BINARY).
 *   W         [N, K] w_dtype (BL_F32 or BL_BF16), read only.
 *   eps       added to gamma before the division (1e-5 in the pages' code);
 *             ignored by BL_BINARY. Must be finite and >= 0.
 *   packed    out: [N, bitlinear_packed_row_bytes(K, layout)] uint8.
 *   gamma     out: 1 float, the weight scale the epilogue multiplies by
 *             (gamma = mean|W| for BL_TERNARY; beta = mean|W| for BL_BINARY).
 *             It stays on the device; no host synchronisation happens.
 *   workspace device scratch of at least bitlinear_pack_workspace_bytes(N, K)
 *             bytes; its contents are overwritten.
 * The mean is accumulated in fp64 and rounded once to fp32. Layout
 * BL_PACK_1BIT holds binary codes only: BL_TERNARY with it returns
 * BL_ERR_INVALID_ARG. */
bl_status bitlinear_pack_weights(const void *W, int w_dtype, int64_t N, int64_t K,
                                 int scheme, int layout, float eps,
                                 uint8_t *packed, float *gamma,
                                 void *workspace, size_t workspace_bytes,
                                 void *stream);

/* Allocation-free variant of bitlinear_pack_weights, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): the same quantisation and packing, with
 * the same arguments and results, but the mean's partial sums live in the
 * library's own scratch array of bitlinear_pack_noalloc_max_scratch_bytes()
 * bytes (16 KiB), held by every GPU the library runs on until the process
 * ends, instead of in a caller workspace. Nothing is allocated or freed, by
 * the library or by any routine it calls. Every call on one GPU shares that
 * GPU's scratch: calls that overlap on one GPU (concurrent streams, threads
 * or graph replays) race and may produce wrong scales; serialise them. Each
 * call rewrites every partial it reads, so nothing needs clearing between
 * calls. Shapes whose partial sums would not fit return BL_ERR_INVALID_ARG
 * (the mean uses at most 1024 partials, so every accepted shape fits); a
 * failed look-up of the scratch's device address returns BL_ERR_DEVICE. */
bl_status bitlinear_pack_weights_noalloc(const void *W, int w_dtype, int64_t N, int64_t K,
                                         int scheme, int layout, float eps,
                                         uint8_t *packed, float *gamma, void *stream);

/* Bytes of the allocation-free pack's scratch array (per GPU). Host-only. */
size_t bitlinear_pack_noalloc_max_scratch_bytes(void);

/* Per-token symmetric absmax INT8 quantisation ([b158] §3.2 and §5.2):
 * s_m = max(max_k |x[m,k]|, 1e-6); xq = clamp(round(x / s_m * 127), -127, 127)
 * with fp32 division, then * 127, then round half to even.
 *   x      [M, K] x_dtype (BL_F32 or BL_BF16), read only.
 *   xq     out: [M, K] int8 codes (never -128).
 *   scale  out: [M] float, the s_m above. */
bl_status bitlinear_quant_acts(const void *x, int x_dtype, int64_t M, int64_t K,
                               int8_t *xq, float *scale, void *stream);

/* Integer product and dequant epilogue ([b158] §4.2: +1 adds, -1 subtracts,
 * 0 skips; §3.3: INT32 accumulator; §5.2-5.3: x_q / 127 * scale and
 * out * gamma):
 *   acc[m,n] = sum_k xq[m,k] * c[n,k]             (exact INT32)
 *   y[m,n]   = acc[m,n] * gamma * scale[m] / 127  (fp32, then y_dtype)
 *   xq, scale  from bitlinear_quant_acts ([M, K] int8, [M] float).
 *   packed     [N, row_bytes] in `layout`; gamma: 1 float (device).
 *   y          out: [M, N], y_dtype BL_F32 or BL_BF16 (round to nearest even).
 *   acc        optional out: [M, N] int32 accumulators, or NULL.
 * Dispatch on M: small batches (M <= 16) stream the packed weights once;
 * medium batches stream them once per 16-token chunk (all chunks in one
 * launch) while that is measured faster, i.e. for a few chunks and moderate
 * N; larger M runs the tiled INT8 matrix-core product. Results do not depend
 * on the path (the INT32 sums are exact). */
bl_status bitlinear_forward(const int8_t *xq, const float *scale,
                            const uint8_t *packed, int layout, const float *gamma,
                            int64_t M, int64_t N, int64_t K,
                            void *y, int y_dtype, int32_t *acc, void *stream);

/* Fused decode step: per-token INT8 quantisation of x (exactly as
 * bitlinear_quant_acts) and the product with its epilogue (exactly as
 * bitlinear_forward) in one launch, for the latency-bound decode regime.
 *   x       [M, K] x_dtype (BL_F32 or BL_BF16), read only.
 *   packed  [N, row_bytes] in `layout`; gamma: 1 float (device).
 *   y       out: [M, N] y_dtype; acc: optional out [M, N] int32, or NULL.
 * Only 1 <= M <= 4 is supported: every workgroup re-derives the token scales
 * from x, which pays off only for a handful of tokens. Larger M returns
 * BL_ERR_UNSUPPORTED (use bitlinear_quant_acts + bitlinear_forward).
 * Sources as for bitlinear_quant_acts and bitlinear_forward. */
bl_status bitlinear_linear(const void *x, int x_dtype, const uint8_t *packed, int layout,
                           const float *gamma, int64_t M, int64_t N, int64_t K,
                           void *y, int y_dtype, int32_t *acc, void *stream);

/* Stacked matrices: several weight matrices that share an input (the Q, K and
 * V projections of an attention block) stored as consecutive row segments of
 * one packed matrix, each segment quantised on its own with its own gamma, so
 * one launch serves all of them (launch latency dominates the decode regime).
 * Per segment the result is exactly that of bitlinear_forward /
 * bitlinear_linear on the segment alone; y holds the segments' outputs side by
 * side along its columns.
 *   packed    [N, row_bytes] with N = sum(seg_rows): segment s occupies the
 *             seg_rows[s] rows after segments 0..s-1 (pack each segment with
 *             bitlinear_pack_weights into its row range, and its gamma into
 *             gammas + s).
 *   gammas    device array of nseg floats.
 *   seg_rows  HOST array of nseg row counts, each >= 1; 1 <= nseg <= 8.
 *   y, acc    [M, N].
 * Other arguments, limits and errors as for bitlinear_forward /
 * bitlinear_linear; a bad segment table returns BL_ERR_INVALID_ARG. */
bl_status bitlinear_forward_segmented(const int8_t *xq, const float *scale, const uint8_t *packed,
                                      int layout, const float *gammas, const int64_t *seg_rows,
                                      int nseg, int64_t M, int64_t K, void *y, int y_dtype,
                                      int32_t *acc, void *stream);
bl_status bitlinear_linear_segmented(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                     const float *gammas, const int64_t *seg_rows, int nseg,
                                     int64_t M, int64_t K, void *y, int y_dtype, int32_t *acc,
                                     void *stream);

/* Alternative decode scheme for the base-3 layout, one token: instead of
 * expanding each weight byte into five codes, the workgroup tabulates, for
 * every group of five activations, the partial sums of the first two and the
 * last three trits (9 + 27 entries) and reads two entries per weight byte
 * ([b158] §2.3 and §6.3: five weights per byte are unpacked by table lookup
 * or bit operations). Same arguments and result as bitlinear_forward (acc
 * bit-identical); kept to compare the lookup scheme with the in-register
 * decode. Only layout BL_PACK_BASE3 and M = 1 are supported (else
 * BL_ERR_UNSUPPORTED); M = 0 or N = 0 is a no-op. */
bl_status bitlinear_forward_lut(const int8_t *xq, const float *scale, const uint8_t *packed,
                                int layout, const float *gamma, int64_t M, int64_t N, int64_t K,
                                void *y, int y_dtype, int32_t *acc, void *stream);

/* Backward products of the straight-through estimator, for training with the
 * codes the forward pass used ([QAT-en] "How Gradients Flow: Fake Quantization
 * and STE": the backward pass treats rounding as the identity, so gradients
 * reach the latent weights; [b158] §5.3, the BitLinear layer with the
 * straight-through estimator). With y = x W_q^T and W_q = gamma * c:
 *   grad_x = grad_y W_q   and   grad_W = grad_y^T x.
 * Both run on the bf16 matrix cores with fp32 accumulation (fp32 operands
 * as exact bf16 pieces, below).
 *
 * bitlinear_backward_input: grad_x[m,k] = gamma * sum_n grad_y[m,n] * c[n,k].
 *   grad_y  [M, N], gy_dtype BL_BF16 or BL_F32. fp32 values are split exactly
 *           into three bf16 pieces (hi + mid + lo, 8 significant bits each) and
 *           the contraction runs over all three into one fp32 sum, so each
 *           product term is still exact (for |grad_y| >= 2^-110; smaller
 *           values may lose bits below 2^-133). Three times the matrix-core
 *           work of bf16 grad_y.
 *   packed  [N, row_bytes] codes in `layout` (BL_PACK_2BIT, BL_PACK_BASE3 or
 *           BL_PACK_1BIT: the forward's own matrix; no transposed copy is
 *           needed); gamma: 1 float (device).
 *   grad_x  out: [M, K] fp32.
 * Requires N % 8 == 0 (else BL_ERR_UNSUPPORTED).
 * Dimensions above 2^24 return BL_ERR_INVALID_ARG.
 * M = 0 is a no-op; N = 0 writes zeros. */
bl_status bitlinear_backward_input(const void *grad_y, int gy_dtype, const uint8_t *packed,
                                   int layout, const float *gamma, int64_t M, int64_t N,
                                   int64_t K, float *grad_x, void *stream);

/* bitlinear_backward_weight: grad_w[n,k] = sum_m grad_y[m,n] * x[m,k].
 *   grad_y  [M, N]; x [M, K] (the layer input); both of `dtype`: BL_BF16
 *           (products exact in fp32, fp32 sums), or BL_F32: each value is
 *           split exactly into three bf16 pieces, and the six piece products
 *           other than mid.lo, lo.mid and lo.lo are summed in fp32 (6M
 *           terms), so each product is exact to within 2^-20 of its
 *           magnitude (for values >= 2^-110; see backward_input). Six times
 *           the matrix-core work of bf16.
 *   grad_w  out: [N, K] fp32.
 * Requires N % 8 == 0 and K % 8 == 0 (else BL_ERR_UNSUPPORTED). N = 0 is a
 * no-op; M = 0 writes zeros. */
bl_status bitlinear_backward_weight(const void *grad_y, const void *x, int dtype, int64_t M,
                                    int64_t N, int64_t K, float *grad_w, void *stream);

/* ---- Products with bias, activation and residual in the epilogue ----------
 *
 *   z[m,n] = gamma * scale[m] / 127 * acc[m,n] + bias[n]
 *   y[m,n] = act(z[m,n]) + res_scale * residual[m,n]
 *
 * acc is the exact INT32 sum of bitlinear_forward; everything after it is fp32,
 * rounded once to y's type. Activations: BL_ACT_NONE z; BL_ACT_RELU max(z, 0);
 * BL_ACT_RELU2 max(z, 0)^2; BL_ACT_SILU z / (1 + e^-z); BL_ACT_GELU
 * z (1 + erf(z / sqrt 2)) / 2; BL_ACT_GELU_TANH z (1 + tanh(sqrt(2 / pi) (z +
 * 0.044715 z^3))) / 2. (The pages keep the block's nonlinear parts in high
 * precision, [b158] §3.3.) */
typedef enum {
    BL_ACT_NONE = 0,
    BL_ACT_RELU = 1,
    BL_ACT_RELU2 = 2,
    BL_ACT_SILU = 3,
    BL_ACT_GELU = 4,
    BL_ACT_GELU_TANH = 5
} bl_act;

/* bitlinear_forward_epilogue: the product of bitlinear_forward_segmented (one
 * segment for a plain matrix) with that epilogue.
 *   bias      [N] bias_dtype, or NULL.
 *   residual  [M, N] of y's type, or NULL; y itself may be passed, to add in
 *             place. res_scale (finite) is ignored without it.
 *   z         optional out: [M, N] of y's type, the pre-activation (what
 *             bitlinear_epilogue_backward reads), or NULL.
 * Other arguments, limits, dispatch and errors as for
 * bitlinear_forward_segmented. Apart from residual and y, no output may
 * overlap another argument. */
bl_status bitlinear_forward_epilogue(const int8_t *xq, const float *scale, const uint8_t *packed,
                                     int layout, const float *gammas, const int64_t *seg_rows,
                                     int nseg, int64_t M, int64_t K, const void *bias,
                                     int bias_dtype, int act, const void *residual,
                                     float res_scale, void *z, void *y, int y_dtype,
                                     void *stream);

/* bitlinear_linear_epilogue: the same from unquantised x, fused into one
 * launch as bitlinear_linear (1 <= M <= 4, else BL_ERR_UNSUPPORTED). */
bl_status bitlinear_linear_epilogue(const void *x, int x_dtype, const uint8_t *packed, int layout,
                                    const float *gammas, const int64_t *seg_rows, int nseg,
                                    int64_t M, int64_t K, const void *bias, int bias_dtype,
                                    int act, const void *residual, float res_scale, void *z,
                                    void *y, int y_dtype, void *stream);

/* Device workspace (bytes) of bitlinear_epilogue_backward; 0 for an empty or
 * refused shape. */
size_t bitlinear_epilogue_backward_workspace_bytes(int64_t M, int64_t N);

/* Backward of the epilogue:
 *   grad_z = grad_y * act'(z);  grad_bias[n] = sum_m grad_z[m,n];
 *   grad_residual = res_scale * grad_y.
 * grad_z is what bitlinear_backward_input and _weight take as their grad_y.
 *   grad_y   [M, N] gy_dtype.   z: [M, N] z_dtype; may be NULL for BL_ACT_NONE.
 *   grad_z   out [M, N] gz_dtype, or NULL.
 *   grad_bias out [N] fp32, or NULL: fp32 sums of the unrounded grad_z over at
 *            most 512 tokens at a time, added in fp64 in a fixed order. Needs the workspace.
 *   grad_residual out [M, N] gy_dtype, or NULL.
 * relu's slope at 0 is 0. At least one output is required; outputs may not
 * overlap inputs. M, N at most 2^24. M = 0 writes zeros to grad_bias. */
bl_status bitlinear_epilogue_backward(const void *grad_y, int gy_dtype, const void *z, int z_dtype,
                                      int act, float res_scale, int64_t M, int64_t N, void *grad_z,
                                      int gz_dtype, float *grad_bias, void *grad_residual,
                                      void *workspace, size_t workspace_bytes, void *stream);

/* ---- Norms before and after a block ----------------------------------------
 *
 * What stands between two blocks of a transformer layer, in one pass over the
 * residual stream h [M, K] and the block's output [M, K]:
 *   p  = norm_post(block)
 *   h' = res_scale * h + gate * p
 *   n  = norm_pre(h')
 * norm(x) = (x - mu) * weight / sqrt(var + eps) + bias over each row, with
 * mu = mean(x), var = mean((x - mu)^2) for BL_NORM_LAYER and mu = 0, var =
 * mean(x^2) for BL_NORM_RMS; BL_NORM_NONE leaves x as it is (no weight, no
 * bias). n is the input of the next BitLinear layer ([QAT-en] "The BitLinear
 * Recipe": activations are normalised, then quantised); it can leave as
 * values, as the INT8 codes and scale of bitlinear_quant_acts, or both. */
typedef enum { BL_NORM_NONE = 0, BL_NORM_RMS = 1, BL_NORM_LAYER = 2 } bl_norm;
/* BL_GATE_CHANNEL: [K] of p_dtype, shared by the tokens. BL_GATE_TOKEN:
 * [M, K] of x_dtype, a row for each token. */
typedef enum { BL_GATE_NONE = 0, BL_GATE_CHANNEL = 1, BL_GATE_TOKEN = 2 } bl_gate;

/* bitlinear_block_norm.
 *   h        [M, K] h_dtype.
 *   block    [M, K] x_dtype, or NULL: then h' = h, h_out must be NULL, and
 *            there is no gate and no norm_post.
 *   gate     as gate_kind says (NULL for BL_GATE_NONE).
 *   *_weight, *_bias  [K] p_dtype, or NULL for 1 and 0. eps: finite, > 0.
 *   h_out    out [M, K] h_dtype: h'; may be h itself (update in place).
 *   n        out [M, K] x_dtype, or NULL.
 *   xq, scale  out [M, K] int8 and [M] float, or both NULL: the codes that
 *            bitlinear_quant_acts gives for n in fp32 (before n's rounding).
 *   stats    out [M, 4] float, or NULL: post mean, post 1 / deviation, pre
 *            mean, pre 1 / deviation (0 and 1 without the norm), for the
 *            backward pass.
 * norm_pre takes h' before it is rounded to h_dtype. With norm_pre at least
 * one of n and xq is required; without, both must be NULL. M = 0 is a no-op.
 * Apart from h and h_out, no output may overlap another argument. */
bl_status bitlinear_block_norm(const void *h, int h_dtype, const void *block, int x_dtype,
                               float res_scale, const void *gate, int gate_kind, int post_kind,
                               const void *post_weight, const void *post_bias, float post_eps,
                               int pre_kind, const void *pre_weight, const void *pre_bias,
                               float pre_eps, int p_dtype, int64_t M, int64_t K, void *h_out,
                               void *n, int8_t *xq, float *scale, float *stats, void *stream);

/* Device workspace (bytes) of bitlinear_block_norm_backward; 0 for an empty or
 * refused shape. */
size_t bitlinear_block_norm_backward_workspace_bytes(int64_t M, int64_t K);

/* bitlinear_block_norm_backward: gradients of the pass above. (Codes have the
 * straight-through estimator's gradient: hand the gradient of the quantised
 * input in as grad_n.)
 *   grad_h_out [M, K] h_dtype, or NULL (zero): the gradient of h' from its
 *            other uses (the residual path).
 *   grad_n   [M, K] gn_dtype; NULL exactly when pre_kind is BL_NORM_NONE.
 *   h_out    [M, K] h_dtype: h' as the forward pass stored it (h itself
 *            without a block). block, gate, weights, biases: as in the forward
 *            pass. stats: its [M, 4].
 *   grad_h   out [M, K] h_dtype.
 *   grad_block out [M, K] x_dtype, or NULL (must be NULL without a block).
 *   grad_gate  out [K] float (channel) or [M, K] x_dtype (token), or NULL.
 *   grad_*_weight, grad_*_bias  out [K] float, or NULL; each needs its norm.
 * Row sums are held in fp32 or fp64; column sums are fp32 over at most 512
 * tokens at a time, added in fp64 in a fixed order, so that results do not
 * change from run to run. The workspace is always needed (it holds the
 * column partials and per-row sums). No output may overlap an input. M, K at
 * most 2^24. M = 0 writes zeros to the [K] outputs. */
bl_status bitlinear_block_norm_backward(
    const void *grad_h_out, const void *grad_n, int gn_dtype, const void *h_out, int h_dtype,
    const void *block, int x_dtype, const float *stats, float res_scale, const void *gate,
    int gate_kind, int post_kind, const void *post_weight, const void *post_bias, int pre_kind,
    const void *pre_weight, int p_dtype, int64_t M, int64_t K, void *grad_h, void *grad_block,
    void *grad_gate, float *grad_post_weight, float *grad_post_bias, float *grad_pre_weight,
    float *grad_pre_bias, void *workspace, size_t workspace_bytes, void *stream);

/* Dry run of the product dispatch: describes, without launching anything or
 * touching device memory, the kernel launches bitlinear_forward (fused = 0)
 * or bitlinear_linear with bf16 x (fused = 1) would enqueue for an M x N x K
 * product in `layout` with output type y_dtype. The stacked (segmented)
 * variants dispatch exactly as the plain calls with N = sum of the segments.
 * One line per launch: the kernel instantiation as the profiler names it,
 * then "grid=GXxGY block=THREADS lds=BYTES". Writes at most len - 1
 * characters and a terminating NUL into buf (buf may be NULL when len is 0).
 * Returns the number of launches (0 for M = 0 or N = 0), or -1 for arguments
 * the call itself would refuse. Launch shapes that depend on the device's
 * compute-unit count use the current device's, and assume none without a GPU.
 * For tests and profiling: it lets a caller check which kernel configuration
 * serves a shape. Host-only; safe to call from several threads. */
int bitlinear_forward_plan(int64_t M, int64_t N, int64_t K, int layout, int y_dtype, int fused,
                           char *buf, size_t len);

/* Human-readable name of a status code (static string). */
const char *bitlinear_status_string(int status);

/* Library version, (major << 16) | minor. */
int bitlinear_version(void);

/* Digest of the source files the library was built from (32 hex digits; a
 * static string), so that a binding can refuse a library built from other
 * sources than the ones beside it. "unknown" if the build did not set it. */
const char *bitlinear_source_hash(void);

#ifdef __cplusplus
}
#endif

#endif /* BITLINEAR_H */
