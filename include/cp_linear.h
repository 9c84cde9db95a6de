/*
 * cp_linear.h - the readout's product in 16 and 32 bits, its gradients, and
 * dropout (gfx950).
 *
 * Decoded rows of a memory layer (cp.h) go through a product with a bias and
 * an activation and join the residual stream:
 *   - cp_linear: the product with all of that in its epilogue;
 *   - cp_linear_act_grad: the gradient back through the epilogue;
 *   - cp_linear_dx, cp_linear_dw: the two products of the backward pass;
 *   - cp_dropout: the mask on its own, for looked-up rows.
 *
 * Dropout keeps no mask. Whether the value in row i and column j of a matrix
 * is kept follows from the two 64-bit numbers rng[0] (seed) and rng[1]
 * (offset), which lie on the device, so that a captured graph can move on by
 * itself: Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random
 * numbers: as easy as 1, 2, 3", 2011) with the seed as its key (low word
 * first) and the counter (j / 8, i, low word of the offset, high word) gives
 * four words, whose halves of 16 bits (low half first) belong to columns 8 (j
 * / 8) to 8 (j / 8) + 7. A value is kept where its half is at least t =
 * round(65536 p), and what is kept is multiplied by 65536 / (65536 - t): p
 * counts in steps of 2^-16, and the mean is kept exactly. What is dropped is
 * 0, whatever it was. The same numbers, rows and columns give the same mask in
 * each of the calls below; two masks of one step need two offsets.
 *
 * Activations, with z in 32 bits (at an infinity each has its limit):
 *   relu max(z, 0) (slope 0 at 0), gelu z Phi(z), Phi the normal distribution,
 *   gelu_tanh z / (1 + exp(-2 u)) with u = sqrt(2 / pi) (z + 0.044715 z^3),
 *   silu z / (1 + exp(-z)).
 * Each but relu is z share(z), its slope share + z share'. However far below 0 z
 * lies, the value is within 18 x 2^-24 of its size (2^-15 of it for a dtype of 16
 * bits) and the slope within 48 x 2^-24 of its two terms' magnitudes, before
 * they are rounded; an exponential below 2^-126 may count as 0. At NaN relu's
 * slope is 0, the others' NaN.
 *
 * Conventions as in cp_ops.h: types, statuses, strides in elements, inputs
 * whose rows may overlap, 32-bit arithmetic with one rounding where a result
 * is stored, equal calls give equal bits. An output must not overlap an input
 * or another output, except where a call says so; rows of one may lie between
 * rows of another, equally far apart.
 */
#ifndef CP_LINEAR_H
#define CP_LINEAR_H

#include <stdint.h>

#include "cp_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CP_ACT_NONE = 0,
    CP_ACT_RELU = 1,
    CP_ACT_GELU = 2,
    CP_ACT_GELU_TANH = 3,
    CP_ACT_SILU = 4,
    /* not an activation: makes every nonnegative 32-bit value a valid cp_act */
    CP_ACT_MAX_ENUM = 0x7FFFFFFF
} cp_act;

/* Device workspace bytes of cp_linear with these sizes. */
uint64_t cp_linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype);

/* z[i][j] = sum over l of x[i][l] w[j][l] + bias[j], a = act(z), y = drop(a) +
 * residual, all of dtype:
 *   x - m x k, w - n x k, bias - n or NULL, residual - m x n or NULL (may be y
 *   itself, with y's stride);
 *   y - m x n, rows y_stride apart; z_out - m x n, contiguous, or NULL: z
 *   rounded, which cp_linear_act_grad reads (y comes from the unrounded z);
 *   p - 0 (rng may be NULL) up to 1 - 2^-16; rng - device uint64[2].
 * workspace - device, 256-byte aligned.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (a stride of x or w above 2^22, k above
 * 2^22, m or n above 2^25, or an output of 2^24 tiles of 64 x 64 or more),
 * HIP. */
cp_status cp_linear(const void *x, uint64_t x_stride, const void *w, uint64_t w_stride, const void *bias,
                    const void *residual, uint64_t residual_stride, cp_dtype dtype, uint64_t m, uint64_t n, uint64_t k,
                    cp_act act, double p, const uint64_t *rng, void *y, uint64_t y_stride, void *z_out,
                    void *workspace, uint64_t workspace_bytes, void *stream);

/* Device workspace bytes of cp_linear_act_grad with a db, also where m is 0 (0
 * without one, and for n = 0). */
uint64_t cp_linear_act_grad_workspace_bytes(uint64_t m, uint64_t n);

/* Back through cp_linear's epilogue: dz = drop(dy) act'(z), db[j] = the sum of
 * dz over rows, in 32 bits from the unrounded dz (float[n], may be NULL; zeros
 * where m is 0). z is what cp_linear stored (rounded: the slope is taken at
 * slightly another point than z); not read, and may be NULL, with CP_ACT_NONE.
 * dy and z have dtype and row strides of their own; dz is contiguous and may be
 * dy, z or both themselves, where those are contiguous. The gradient of the
 * residual is dy.
 * Errors: INVALID_ARGUMENT, HIP. */
cp_status cp_linear_act_grad(const void *dy, uint64_t dy_stride, const void *z, uint64_t z_stride, cp_dtype dtype,
                             uint64_t m, uint64_t n, cp_act act, double p, const uint64_t *rng, void *dz, float *db,
                             void *workspace, uint64_t workspace_bytes, void *stream);

/* Device workspace bytes of cp_linear_dx and cp_linear_dw with these sizes. */
uint64_t cp_linear_dx_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype);
uint64_t cp_linear_dw_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype);

/* dx[i][l] = sum over j of dz[i][j] w[j][l] + dres[i][l], all of dtype: dz - m x
 * n, w - n x k, dres - m x k or NULL (may be dx itself), dx - m x k, contiguous.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (a stride above 2^22, a size above
 * 2^22 for the row length and 2^25 for the rows, or an output of 2^24 tiles of
 * 64 x 64 or more), HIP. */
cp_status cp_linear_dx(const void *dz, uint64_t dz_stride, const void *w, uint64_t w_stride, const void *dres,
                       uint64_t dres_stride, cp_dtype dtype, uint64_t m, uint64_t n, uint64_t k, void *dx,
                       void *workspace, uint64_t workspace_bytes, void *stream);

/* dw[j][l] = sum over i of dz[i][j] x[i][l], in 32 bits (float, n x k, rows
 * dw_stride apart). add - 0, or 1: that is added to what dw holds. dz - m x n
 * and x - m x k have dtype.
 * Errors: as cp_linear_dx. */
cp_status cp_linear_dw(const void *dz, uint64_t dz_stride, const void *x, uint64_t x_stride, cp_dtype dtype,
                       uint64_t m, uint64_t n, uint64_t k, int add, float *dw, uint64_t dw_stride, void *workspace,
                       uint64_t workspace_bytes, void *stream);

/* y = drop(x) + residual (may be NULL): n x d of dtype. y is contiguous and may
 * be x or residual itself, where those are contiguous. drop's gradient is the
 * same call on the gradient, without a residual.
 * Errors: INVALID_ARGUMENT, HIP. */
cp_status cp_dropout(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride, cp_dtype dtype,
                     uint64_t n, uint64_t d, double p, const uint64_t *rng, void *y, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CP_LINEAR_H */
