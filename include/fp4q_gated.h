/*
 * fp4q_gated.h -- C ABI of the library's operators for gated feed-forward layers: what a
 * tensor-parallel rank computes between the norm's 8-bit output (fp4q_rmsnorm) and its second
 * projection (fp4q_gemm8), forward and backward, and the products of a few rows with weights
 * that are held in 4 bits, for single tokens.
 *
 *   fp4q_gated8            y = act(x gate^T) * (x up^T) of 8-bit operands
 *   fp4q_gated8_backward   the gradients of both products, as 8-bit codes
 *   fp4q_gemv4             a few rows times a weight held as an FP4 payload
 *   fp4q_gated4            fp4q_gated8's form for a few rows and such weights
 *
 * 8-bit operands, codes and scales are those of fp4q_linear.h, FP4 payloads those of fp4q.h,
 * and so are the conventions: device pointers that the caller owns, asynchronous on `stream`,
 * no allocation, no state, arguments validated on the host before any HIP call (shape, then
 * flags, formats, types and activation, then NULL, alignment, workspace size (FP4Q_ERR_SHAPE)
 * and overlap of an output with an input or another output (FP4Q_ERR_ARG)), FP4Q_ERR_LAUNCH
 * for a failed launch.  Tensors, codes, micro-scales and workspaces are aligned to 16 bytes,
 * scales to 4.  A size that would need more than 2^32 - 1 threads returns FP4Q_ERR_SHAPE.
 * Results do not depend on timing: no atomics, every sum in a fixed order.
 *
 * Joined halves.  The weights of the gate and the up projection, N rows each, are one operand
 * of R = P + N rows, where P = N rounded up to a multiple of 128: the gate's rows, rows of
 * zeros from N to P, the up projection's rows.  So each half begins a block of scales, and
 * one product serves both halves: with the joined gradients [M x R] of fp4q_gated8_backward
 * (columns N to P are zeros) the input gradient is one fp4q_gemm8 over K = R with the joined
 * weight's transposed codes, and the joined weight's gradient is one over K = M.
 *
 * Activations (g the gate's product):
 *   FP4Q_ACT_SILU       g / (1 + exp(-g))
 *   FP4Q_ACT_GELU       g (1 + erf(g / sqrt 2)) / 2
 *   FP4Q_ACT_GELU_TANH  g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2
 *   FP4Q_ACT_RELU       max(g, 0), with derivative 0 at 0
 * At an infinite g they and their derivatives take their limits.  A factor 1 / (1 + exp(-g)) (or
 * its like) that lies below 2^-126 may count as 0.
 */
#ifndef FP4Q_GATED_H
#define FP4Q_GATED_H

#include <stddef.h>
#include <stdint.h>

#include "fp4q_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FP4Q_ACT_SILU = 0, FP4Q_ACT_GELU = 1, FP4Q_ACT_GELU_TANH = 2, FP4Q_ACT_RELU = 3 };

/* y[m][n] = act(g) * u, with g = sum over k of a[m][k] w[n][k] and u = sum over k of
 * a[m][k] w[P + n][k], of the operands' values.
 *   a, a_scales   [M x K] codes with rows of 128
 *   w, w_scales   [R x K] codes of the joined weight with tiles of 128 x 128
 *                 (fp4q_quantize8 with FP4Q_FLAG_TILES): scales [ceil(K/128) x ceil(R/128)]
 *   y             [M x N] bf16
 *   gate, up      [M x N] bf16, g and u for the backward pass; both NULL for none
 *   workspace     fp4q_gated8_workspace bytes of scratch memory (NULL if 0)
 * The sums are fp4q_gemm8's with bf16 output (the 8-bit matrix core's, held and scaled in
 * fp32, with the same bound); the activation and the product are of the fp32 sums, and each
 * output is rounded once.  0 <= M, N, K < 2^27, pitches < 2^23. */
int fp4q_gated8_workspace(int64_t M, int64_t N, int64_t K, size_t *bytes);
int fp4q_gated8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
                const uint8_t *w, int64_t w_pitch, int w_format, const float *w_scales, int64_t M,
                int64_t N, int64_t K, int act, void *y, void *gate, void *up, void *workspace,
                size_t workspace_bytes, void *stream);

/* Gradients of fp4q_gated8, in fp32 of the stored gate and up, each rounded once to 8 bits:
 *   dgate = dy * up * act'(gate),  dup = dy * act(gate)
 *   dy, gate, up         [rows x cols] of `dtype` (FP4Q_OUT_F32 or FP4Q_OUT_BF16)
 *   codes, scales        the joined [dgate | 0 | dup], [rows x R] codes of `format` with rows
 *                        of 128, pitch code_pitch, and scales [ceil(R/128) x rows]
 *   codes_t, scales_t    the same transposed, [R x rows] codes (rows of 128 of a column of the
 *                        joined tensor), pitch code_t_pitch, and scales [ceil(rows/128) x R]
 *   y_codes_t, y_scales_t  y = act(gate) * up transposed, [cols x rows] E4M3 codes, pitch
 *                        y_t_pitch, and scales [ceil(rows/128) x cols]: the operand of the
 *                        second projection's weight gradient
 * Each is what fp4q_quantize8 makes of the fp32 tensor.  Each pair may be NULL, not all
 * three.  The products are taken from left to right, and one that leaves fp32's range on the way
 * is infinite: it, and a gate of +infinity in dup and y, give their blocks NaN scales.
 * rows >= 0, 1 <= cols; rows, cols < 2^23, pitches < 2^25. */
int fp4q_gated8_backward(const void *dy, const void *gate, const void *up, int64_t rows, int64_t cols,
                         int dtype, int act, int format, uint8_t *codes, int64_t code_pitch,
                         float *scales, uint8_t *codes_t, int64_t code_t_pitch, float *scales_t,
                         uint8_t *y_codes_t, int64_t y_t_pitch, float *y_scales_t, void *stream);

/* out[m][n] = sum over k of x[m][k] W[n][k], where W [N x K] is a payload: what
 * fp4q_decompress makes of it in exact arithmetic.  Made for few rows of x: its time is that
 * of reading the payload, once for all of up to 16 columns (rows of x times their parts, below),
 * else once for every 32.  Any number is taken.
 *   x           [M x K] of `dtype`
 *   codes, micro_scales, block_scales   W as fp4q_compress_ex makes it; K % 256 == 0
 *   flags       FP4Q_FLAG_NO_FWHT for a payload made with that flag.  Otherwise W is
 *               H Q / 16 in each block of 256, and x is transformed instead: H is symmetric,
 *               so x W^T = (x H / 16) Q^T.
 *   out         [M x N] of out_dtype
 *   workspace   fp4q_gemv4_workspace bytes of scratch memory (NULL if 0)
 * The codes times their micro-scales are exact in fp16.  x becomes fp16 under a power of two
 * (2^98 at most) for each row and block of 256: bf16 x exactly, but for values 2^-28 below
 * the block's largest; fp32 or transformed x in two parts, to 2^-22 of each value (and
 * 2^-39 of the block's largest), but for transformed bf16 x with bf16 out, which takes one
 * part, to 2^-11 (x itself has 8 bits, and so has out; fp32 out takes two).  Products are exact and
 * added in fp32 by the matrix core, a block's sum times its scale in fp32.  As for fp4q_compress, x must be finite with
 * |x| < 2^118, which is not checked (a row of x that is not gives a row of out that is not);
 * of x what lies below 2^-112, and of a block's sum what lies below 2^-126 before its scale
 * (times 2^17), may be dropped.
 * 0 <= M < 2^19, 0 <= N < 2^27, 0 < K < 2^24. */
int fp4q_gemv4_workspace(int64_t M, int64_t K, int dtype, uint32_t flags, size_t *bytes);
int fp4q_gemv4(const void *x, int dtype, int64_t M, const uint8_t *codes, const uint8_t *micro_scales,
               const float *block_scales, int64_t N, int64_t K, void *out, int out_dtype,
               uint32_t flags, void *workspace, size_t workspace_bytes, void *stream);

/* out[m][n] = act(g) * u of two such products, g with the gate's payload and u with the up
 * projection's (each [N x K]), computed in fp32 and rounded once.  The workspace is
 * fp4q_gemv4_workspace's. */
int fp4q_gated4(const void *x, int dtype, int64_t M, const uint8_t *gate_codes, const uint8_t *gate_micro,
                const float *gate_block, const uint8_t *up_codes, const uint8_t *up_micro,
                const float *up_block, int64_t N, int64_t K, int act, void *out, int out_dtype,
                uint32_t flags, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4Q_GATED_H */
