/*
 * fp4q_linear.h -- C ABI of the library's 8-bit linear-layer operators: what a
 * tensor-parallel rank runs between the receiver's sum of one AllReduce
 * (fp4q_decompress_accumulate) and the sender of the next (fp4q_compress).
 *
 *   fp4q_rmsnorm            residual addition, root-mean-square norm, 8-bit output
 *   fp4q_rmsnorm_backward   its gradients
 *   fp4q_quantize8          a tensor to 8-bit codes with a scale per 128 values
 *   fp4q_gemm8              the product of two such operands
 *
 * 8-bit operands.  Codes are OCP E4M3FN or E5M2 bytes, row-major [rows x cols]
 * with a pitch (bytes from one row to the next) that is a multiple of 16; the
 * bytes between cols and the pitch are never used as values, but every row, the
 * last one too, must be readable up to cols rounded up to a multiple of 16.
 * A scale is one fp32 value for a block of codes; the value of a code is
 * code * scale.  Blocks are either
 *   rows of 128   128 neighbours in a row (the last block of a row may be
 *                 shorter); scales [ceil(cols/128) x rows], or
 *   tiles         128 x 128 (ragged at both ends); scales
 *                 [ceil(cols/128) x ceil(rows/128)],
 * row-major and without padding: the 128-group of the columns comes first, so
 * that the scales of one step of a product lie together.
 *
 * Quantising a block with largest magnitude A: scale = max(A, 2^-100) / fmax
 * rounded to fp32, where fmax is 448 (E4M3) or 57344 (E5M2); code = the 8-bit
 * value nearest to v / scale (the quotient rounded to fp32 first; ties to
 * even; zeros are stored as +0).  A block that holds an infinity or a NaN gets
 * a NaN scale and NaN codes.  Quotients of values below 2^-99 may be off by one
 * unit of fp32.
 *
 * Conventions are those of fp4q.h: device pointers that the caller owns,
 * asynchronous on `stream`, no allocation, no state, arguments validated on the
 * host before any HIP call (shape, then flags, formats and types, then NULL,
 * alignment, workspace size (FP4Q_ERR_SHAPE) and overlap of an output with an
 * input or another output (FP4Q_ERR_ARG)), FP4Q_ERR_LAUNCH for a failed launch.
 * Tensors, codes and workspaces are aligned to 16 bytes, scales, rstd, dweight
 * to 4.  A size that would need more than 2^32 - 1 threads returns FP4Q_ERR_SHAPE.
 * Results do not depend on timing: no atomics, every sum in a fixed order.
 * Element types are FP4Q_OUT_F32 and FP4Q_OUT_BF16.
 */
#ifndef FP4Q_LINEAR_H
#define FP4Q_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#include "fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { FP4Q_GROUP8 = 128 };
enum { FP4Q_E4M3 = 0, FP4Q_E5M2 = 1 };
/* fp4q_quantize8: one scale per 128 x 128 tile; fp4q_gemm8: b's scales are tiles. */
enum { FP4Q_FLAG_TILES = 1u << 1 };
/* fp4q_gemm8: add the product to fp32 `out` instead of overwriting it. */
enum { FP4Q_FLAG_ACCUMULATE = 1u << 2 };

/* h = x + residual (rounded to the type; h = x without a residual),
 * r = 1 / sqrt(mean(h^2) + eps) per row, y = h * r * weight, in fp32.
 *   x, residual  [rows x cols] of `dtype`; residual may be NULL
 *   weight       [cols] of `dtype`
 *   eps          finite and > 0
 *   h            [rows x cols] of `dtype`, the sum; required with a residual
 *                (and may then be the residual itself: updated in place), NULL
 *                without one
 *   y            [rows x cols] of `dtype`, or NULL
 *   codes        E4M3 codes of the fp32 y (not of the rounded y), rows of 128,
 *                pitch code_pitch, with scales [ceil(cols/128) x rows]; both NULL
 *                for none
 *   rstd         [rows] fp32, r; or NULL
 * At least one of y and codes.  rows >= 0, 1 <= cols < 2^28.  The squares of a
 * row must sum to a finite fp32 value. */
int fp4q_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int64_t rows,
                 int64_t cols, int dtype, void *h, void *y, uint8_t *codes, int64_t code_pitch,
                 float *scales, float *rstd, void *stream);

/* Gradients of fp4q_rmsnorm.  With g = dy * weight and xhat = h * rstd:
 *   dx      = rstd * (g - xhat * mean(g * xhat)) + dh    [rows x cols] of `dtype`
 *             (the gradient of x and of the residual alike)
 *   dweight = sum over the rows of dy * xhat             [cols] fp32
 *   h       what the norm was taken of (the forward's h, or x without a residual)
 *   dh      the gradient that reaches h by other paths (the residual stream's), or NULL
 *   workspace  fp4q_rmsnorm_backward_workspace bytes of scratch memory
 * With no rows, dweight is set to zero. */
int fp4q_rmsnorm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes);
int fp4q_rmsnorm_backward(const void *dy, const void *h, const void *weight, const float *rstd,
                          const void *dh, int64_t rows, int64_t cols, int dtype, void *dx,
                          float *dweight, void *workspace, size_t workspace_bytes, void *stream);

/* 8-bit codes and scales of x [rows x cols] of `dtype`.
 *   codes, scales      rows of 128 of x, or with FP4Q_FLAG_TILES its tiles
 *   codes_t, scales_t  the same of x transposed (codes_t is [cols x rows] with
 *                      pitch code_t_pitch): its blocks are 128 neighbours in a
 *                      column of x; with FP4Q_FLAG_TILES the same tiles, so
 *                      that codes_t holds the same codes
 * Either pair may be NULL, not both.  rows >= 0, 1 <= cols; rows, cols < 2^28,
 * fewer than 2^31 tiles of 128 x 128. */
int fp4q_quantize8(const void *x, int64_t rows, int64_t cols, int dtype, int format, uint8_t *codes,
                   int64_t code_pitch, float *scales, uint8_t *codes_t, int64_t code_t_pitch,
                   float *scales_t, uint32_t flags, void *stream);

/* out[m][n] = sum over k of a[m][k] b[n][k], of the operands' values: a [M x K]
 * with rows of 128, b [N x K] with rows of 128 or (FP4Q_FLAG_TILES) tiles.
 * The sum over a block of 128 comes from the matrix cores; it is multiplied by b's
 * scale, then by a's, and added in fp32.  In every block the products of a's codes
 * with b's values must sum to a finite fp32 value; the product of the two scales
 * need not be one.  With fp32 output the matrix core works on the codes' values in
 * bf16 (exact products, fp32 sums).  With bf16 output it works on the codes
 * themselves, twice as fast, and drops what lies below 2^-13 of the largest of 8
 * neighbouring products (k = 8 i .. 8 i + 7): of each 8 at most 7 * 2^-13 of the
 * largest one.  Over normally distributed values that is about 2e-5 of the result, a
 * hundredth of bf16's rounding; where large products cancel, it can be most of the
 * result.  Such sums (outliers of both signs) want fp32 output.
 *   forward        a = activations, b = weight [out x in]
 *   input gradient a = output gradient, b = the transposed weight (codes_t)
 *   weight gradient a = the transposed output gradient, b = the transposed
 *                  activations (codes_t, rows of 128), K = tokens
 *   out         [M x N] of out_dtype, overwritten (zero for K = 0), or with
 *               FP4Q_FLAG_ACCUMULATE (fp32 only) added to
 *   workspace   fp4q_gemm8_workspace bytes of scratch memory (NULL if 0)
 * 0 <= M, N, K < 2^28, pitches < 2^23. */
int fp4q_gemm8_workspace(int64_t M, int64_t N, int64_t K, int out_dtype, uint32_t flags, size_t *bytes);
int fp4q_gemm8(const uint8_t *a, int64_t a_pitch, int a_format, const float *a_scales,
               const uint8_t *b, int64_t b_pitch, int b_format, const float *b_scales, int64_t M,
               int64_t N, int64_t K, void *out, int out_dtype, uint32_t flags, void *workspace,
               size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4Q_LINEAR_H */
