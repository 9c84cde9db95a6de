/*
 * cp_ops.h - the dense operators on either side of a CP table (gfx950).
 *
 * A row table is trained uncompressed before its rows are coded
 * (cp_table_encode, cp.h), and the rows a lookup decodes feed a readout:
 *   - cp_embed_lookup, cp_embed_plan, cp_embed_grad: the lookup into an
 *     uncompressed table and its gradient, summed per row in token order;
 *   - cp_rms_norm, cp_rms_norm_grad: root-mean-square norm with the
 *     residual's addition and an 8-bit output;
 *   - cp_quantize_fp8: the 8-bit form of a matrix, also transposed;
 *   - cp_gemm_fp8: the product of two 8-bit matrices.
 *
 * 8-bit values are e4m3 (OCP: largest finite value 448, no infinities) with
 * e8m0 scales: byte b stands for 2^(b - 127). A group of 128 values whose
 * largest finite magnitude is A has the least scale 2^e with A / 2^e <= 448
 * (e >= -127; 1 when A is 0), and each value x becomes x / 2^e rounded to
 * nearest even. Values that are not finite become e4m3's NaN and take no
 * part in A.
 *
 * Types: a cp_dtype names the element type of an array of 16- or 32-bit
 * floating point; arithmetic runs in 32 bits and rounds once, to nearest
 * even, where a result is stored.
 *
 * Conventions as in cp.h: a cp_status from every call, argument checks on
 * the host before any launch, work asynchronous on `stream`, on the current
 * device, nothing allocated; kernels only (a call can be captured in a HIP
 * graph). Strides are in elements; the rows of an input may overlap (a stride
 * of 0 repeats one row), those of an output may not. Arrays are aligned to
 * their element type unless a call says otherwise. Results do not depend on how the GPU
 * schedules the work: the same call gives the same bits.
 */
#ifndef CP_OPS_H
#define CP_OPS_H

#include <stdint.h>

#include "cp.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CP_DTYPE_F32 = 0,
    CP_DTYPE_BF16 = 1,
    CP_DTYPE_F16 = 2,
    /* not a type: makes every nonnegative 32-bit value a valid cp_dtype */
    CP_DTYPE_MAX_ENUM = 0x7FFFFFFF
} cp_dtype;

/* ------------------------------------------------------------------------
 * Embedding: the uncompressed row table
 * --------------------------------------------------------------------- */

/* out[j][0..d) = scale * table[ids[j]][0..d) for 0 <= ids[j] < rows. A
 * negative id is padding: a zero row. An id >= rows gives a zero row too and
 * sets *bad_id (device int32, may be NULL) to 1; it is never cleared here.
 *   table - device, rows x d of table_dtype, row_stride elements apart.
 *   ids   - device int64[n]. out - device n x d of out_dtype, contiguous.
 * Errors: INVALID_ARGUMENT (NULL or misaligned pointers with n > 0 and d > 0,
 * unknown dtype, n or d above 2^31 - 1, rows above 2^62), HIP. */
cp_status cp_embed_lookup(const void *table, cp_dtype table_dtype, uint64_t rows, uint64_t d, uint64_t row_stride,
                          const int64_t *ids, uint64_t n, float scale, void *out, cp_dtype out_dtype, int32_t *bad_id,
                          void *stream);

/* Device workspace bytes of cp_embed_plan for n ids into `rows` rows. */
uint64_t cp_embed_plan_workspace_bytes(uint64_t n, uint64_t rows);

/* Groups a batch's ids by row, for the gradient: a stable sort of the ids in
 * [0, rows) (others take no part).
 *   order  - device int32[n] (written: the first starts[*count]): positions
 *            in the batch, by row, then by position.
 *   slot   - device int32[n]: slot[i] = the distinct row that order[i] looked
 *            up, as its index in unique; -1 from starts[*count] on.
 *   unique - device int64[n]: the distinct rows, ascending.
 *   starts - device int32[n + 1]: row unique[u]'s lookups are
 *            order[starts[u] .. starts[u + 1]).
 *   count  - device int64: the number of distinct rows.
 *   workspace - device, 256-byte aligned, >= cp_embed_plan_workspace_bytes.
 * Errors: INVALID_ARGUMENT (NULL or misaligned pointers, n above 2^31 - 4096,
 * rows above 2^62, workspace too small), HIP. */
cp_status cp_embed_plan(const int64_t *ids, uint64_t n, uint64_t rows, int32_t *order, int32_t *slot, int64_t *unique,
                        int32_t *starts, int64_t *count, void *workspace, uint64_t workspace_bytes, void *stream);

/* Device workspace bytes of cp_embed_grad for n lookups of d values. */
uint64_t cp_embed_grad_workspace_bytes(uint64_t n, uint64_t d);

/* The lookup's gradient in 32 bits from a plan of the same n ids: row u is
 * scale * (the sum of dout[order[i]][0..d) over row unique[u]'s lookups).
 *   rows == 0: grad is float[n][d]; row u of it belongs to row unique[u] of
 *              the table (the first *count rows are written).
 *   rows  > 0: grad is float[rows][d], the whole table's gradient (rows as
 *              given to the plan): rows not looked up are zero.
 *   dout      - device, n x d of dtype, dout_stride elements apart.
 *   workspace - device, 256-byte aligned, >= cp_embed_grad_workspace_bytes.
 * Errors: INVALID_ARGUMENT (NULL or misaligned pointers, unknown dtype,
 * n or d above 2^31 - 4096, workspace too small), UNSUPPORTED (d above 2^21),
 * HIP. */
cp_status cp_embed_grad(const int32_t *order, const int32_t *slot, const int64_t *unique, const int32_t *starts,
                        const int64_t *count, uint64_t n, uint64_t rows, const void *dout, cp_dtype dtype, uint64_t d,
                        uint64_t dout_stride, float scale, float *grad, void *workspace, uint64_t workspace_bytes,
                        void *stream);

/* ------------------------------------------------------------------------
 * Root-mean-square norm
 * --------------------------------------------------------------------- */

/* Per row of n: h = x + residual (residual may be NULL), rstd =
 * 1 / sqrt(mean(h^2) + eps), y = h * rstd * weight, with h and y in 32 bits.
 * Outputs, each NULL when not wanted:
 *   h_out - h rounded to dtype, contiguous (needs a residual);
 *   y_out - y rounded to dtype, contiguous;
 *   q     - y in e4m3 with a scale for each 128 values of a row, rows
 *           q_stride bytes apart (a multiple of 16, >= d), 16-byte aligned;
 *   q_scale - (with q) the e8m0 scales, ceil(d / 128) per row, rows
 *           scale_stride bytes apart;
 *   rstd  - float[n].
 * x and residual have dtype, rows x_stride and residual_stride elements
 * apart; weight[d] has dtype.
 * Errors: INVALID_ARGUMENT, HIP. */
cp_status cp_rms_norm(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                      const void *weight, cp_dtype dtype, uint64_t n, uint64_t d, float eps, void *h_out, void *y_out,
                      uint8_t *q, uint64_t q_stride, uint8_t *q_scale, uint64_t scale_stride, float *rstd,
                      void *stream);

/* Device workspace bytes of cp_rms_norm_grad. */
uint64_t cp_rms_norm_grad_workspace_bytes(uint64_t n, uint64_t d);

/* The norm's gradient. x is the norm's input (h_out, where there was a
 * residual: rounded, while the forward pass took y and rstd from the unrounded
 * h) and rstd what the forward pass stored:
 *   xhat = x * rstd, g = dy * weight,
 *   dx = rstd * (g - xhat * mean(g * xhat)) + dres (dres may be NULL),
 *   dw[c] = sum over rows of dy * xhat, in 32 bits (float[d]).
 * dy, x, dres have dtype and row strides of their own; dx is contiguous.
 * dw may be NULL. workspace - device, 256-byte aligned.
 * Errors: INVALID_ARGUMENT, HIP. */
cp_status cp_rms_norm_grad(const void *dy, uint64_t dy_stride, const void *x, uint64_t x_stride, const float *rstd,
                           const void *weight, const void *dres, uint64_t dres_stride, cp_dtype dtype, uint64_t n,
                           uint64_t d, void *dx, float *dw, void *workspace, uint64_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * 8 bits
 * --------------------------------------------------------------------- */

/* The 8-bit form of x (n x d of dtype, rows x_stride elements apart).
 *   blocks == 0: a scale for each 128 values of a row. q is n x d, scale is
 *     n x ceil(d / 128); qt (may be NULL) is the 8-bit form of x transposed,
 *     d x n, with groups of 128 along n: scale_t is d x ceil(n / 128).
 *   blocks == 1: a scale for each 128 x 128 block: scale is ceil(n / 128) x
 *     ceil(d / 128); qt (may be NULL) is q transposed and scale_t (ceil(d /
 *     128) x ceil(n / 128)) scale transposed.
 * Strides in bytes: q_stride >= d and qt_stride >= n are multiples of 16 and
 * q, qt 16-byte aligned; scale_stride and scale_t_stride cover their rows.
 * Errors: INVALID_ARGUMENT, HIP. */
cp_status cp_quantize_fp8(const void *x, cp_dtype dtype, uint64_t n, uint64_t d, uint64_t x_stride, int blocks,
                          uint8_t *q, uint64_t q_stride, uint8_t *scale, uint64_t scale_stride, uint8_t *qt,
                          uint64_t qt_stride, uint8_t *scale_t, uint64_t scale_t_stride, void *stream);

/* Device workspace bytes of cp_gemm_fp8. */
uint64_t cp_gemm_fp8_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype out_dtype);

/* out[i][j] = sum over l of A[i][l] B[j][l], accumulated in 32 bits:
 *   A - m x k of e4m3, rows a_stride bytes apart, with a scale for each 128
 *       values of a row: a_scale is m x ceil(k / 128), a_scale_stride apart;
 *   B - n x k of e4m3, with scales like A's (b_blocks == 0) or one for each
 *       128 x 128 block: b_scale is ceil(n / 128) x ceil(k / 128);
 *   out - m x n of out_dtype, rows out_stride elements apart.
 * a and b are 16-byte aligned, their strides multiples of 16 and at least k;
 * a_scale and b_scale 4-byte aligned, their strides multiples of 4; every
 * row is readable up to its stride rounded down to the next multiple of 16
 * (4 for scales) past its values, which need not be initialised.
 * A scale byte of 255 is NaN. A 16-bit output comes from the 8-bit matrix
 * instruction, which cuts products before it adds them: of the 8 at l = 8 g to
 * 8 g + 7, each loses what lies below 2^(E - 13), E being the largest sum of
 * the exponents of the two e4m3 factors among the products that are not zero
 * (a factor below 2^-6 counts with -6). With factors of 2^-6 and more that is
 * less than 2^-13 of the largest of the 8 products for each of the others. The
 * sums of 8 are added in 32 bits. A 32-bit output is summed without that cut,
 * from each operand's scaled values, which have to lie within the range of
 * 32-bit floating point (those below 2^-124 may lose bits).
 * workspace - device, 256-byte aligned.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (a stride above 2^22, m or n above
 * 2^25, or an output of 2^24 tiles of 256 x 128 or more), HIP. */
cp_status cp_gemm_fp8(const uint8_t *a, uint64_t a_stride, const uint8_t *a_scale, uint64_t a_scale_stride,
                      const uint8_t *b, uint64_t b_stride, const uint8_t *b_scale, uint64_t b_scale_stride,
                      int b_blocks, uint64_t m, uint64_t n, uint64_t k, void *out, uint64_t out_stride,
                      cp_dtype out_dtype, void *workspace, uint64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CP_OPS_H */
