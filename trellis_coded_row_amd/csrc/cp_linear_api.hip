// cp_linear_api.hip - the C ABI of the readout's product, its gradients and
// dropout (declared in include/cp_linear.h): argument checks on the host, then
// the launch.
#include <math.h>

#include "../../include/cp_linear.h"
#include "cp_linear_internal.h"
#include "cp_status.h"

static constexpr uint64_t kMaxCount = 0x7FFFFFFFull;   // lengths that kernels hold in 32 bits
static constexpr uint64_t kMaxStride = 1ull << 22;     // a tile's rows then lie within 2^31 bytes
static constexpr uint64_t kMaxRows = 1ull << 25;
static constexpr uint64_t kMaxTiles = 1ull << 24;      // workgroups of 256 threads: a launch has fewer than 2^32

static bool dtype_ok(cp_dtype t) { return t == CP_DTYPE_F32 || t == CP_DTYPE_BF16 || t == CP_DTYPE_F16; }

static bool act_ok(cp_act a)
{
    return a == CP_ACT_NONE || a == CP_ACT_RELU || a == CP_ACT_GELU || a == CP_ACT_GELU_TANH || a == CP_ACT_SILU;
}

// A pointer to use: not NULL, aligned to `bytes` (a power of two).
static bool good(const void *p, uint64_t bytes) { return p && ((uintptr_t)p & (bytes - 1)) == 0; }

static bool good_or_null(const void *p, uint64_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Byte ranges of n rows, `stride` elements apart, stay below 2^62.
static bool spans(uint64_t n, uint64_t stride) { return n == 0 || stride <= (1ull << 60) / n; }

// The bytes of n rows of d elements, `stride` apart; nowhere without values.
struct Range {
    uintptr_t begin, end;
    uint64_t row, pitch;  // bytes of a row, and from one to the next (0: a single one)
};

static Range range_of(const void *p, uint64_t n, uint64_t d, uint64_t stride, uint64_t es)
{
    const uintptr_t at = (uintptr_t)p;
    if (!p || n == 0 || d == 0) return {0, 0, 0, 0};
    return {at, at + ((n - 1) * stride + d) * es, d * es, n > 1 ? stride * es : 0};
}

// Whether a's rows and b's lie between each other all the way: rows equally far
// apart, b's behind a's and before the next of them.
static bool between(Range a, Range b)
{
    const uint64_t pitch = a.pitch ? a.pitch : b.pitch;
    if (pitch == 0 || (b.pitch && b.pitch != pitch)) return false;
    const uint64_t behind = b.begin >= a.begin ? (b.begin - a.begin) % pitch : (pitch - (a.begin - b.begin) % pitch) % pitch;
    return behind >= a.row && behind + b.row <= pitch;
}

static bool overlap(Range a, Range b) { return a.begin < b.end && b.begin < a.end && !between(a, b); }

// The mask's threshold from the share that is dropped, and whether that is one.
static bool drop_of(double p, const uint64_t *rng, cpk::Drop *out)
{
    if (!(p >= 0.0 && p < 1.0)) return false;  // (NaN too)
    const uint32_t t = (uint32_t)nearbyint(65536.0 * p);
    if (t > 65535 || (t > 0 && !good(rng, 8))) return false;
    out->threshold = t;
    out->scale = (float)(65536.0 / (65536.0 - t));
    out->rng = t ? rng : nullptr;
    return true;
}

static bool workspace_ok(const void *p, uint64_t bytes, uint64_t need)
{
    return need == 0 || (good(p, 256) && bytes >= need);
}

// A product of m x n outputs within what a launch holds.
static bool too_large(uint64_t m, uint64_t n)
{
    return m > kMaxRows || n > kMaxRows || cpk::div_up(m, 64) * cpk::div_up(n, 64) >= kMaxTiles;
}

// The launches read their status with hipGetLastError: an earlier failure of
// an unrelated call must not be taken for theirs.
static void forget_earlier_error() { (void)hipGetLastError(); }

extern "C" {

uint64_t cp_linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype)
{
    if (!dtype_ok(dtype) || m == 0 || n == 0 || k == 0 || k > kMaxStride || too_large(m, n)) return 0;
    return cpk::linear_workspace_bytes(m, n, k, dtype);
}

cp_status cp_linear(const void *x, uint64_t x_stride, const void *w, uint64_t w_stride, const void *bias,
                    const void *residual, uint64_t residual_stride, cp_dtype dtype, uint64_t m, uint64_t n, uint64_t k,
                    cp_act act, double p, const uint64_t *rng, void *y, uint64_t y_stride, void *z_out,
                    void *workspace, uint64_t workspace_bytes, void *stream)
{
    cpk::LinearArgs a{};
    if (!dtype_ok(dtype) || !act_ok(act) || !drop_of(p, rng, &a.e.drop)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (k > kMaxStride || too_large(m, n) || (m > 1 && x_stride > kMaxStride) || (n > 1 && w_stride > kMaxStride))
        return CP_ERR_UNSUPPORTED;
    if ((m > 1 && y_stride < n) || !spans(m, y_stride) || (residual && !spans(m, residual_stride)))
        return CP_ERR_INVALID_ARGUMENT;
    if (!good_or_null(bias, es) || !good_or_null(residual, es) || !good_or_null(z_out, es))
        return CP_ERR_INVALID_ARGUMENT;
    if (m == 0 || n == 0) return CP_OK;
    if (!good(y, es)) return CP_ERR_INVALID_ARGUMENT;
    if (k > 0) {
        if (!good(x, es) || !good(w, es)) return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::linear_workspace_bytes(m, n, k, dtype)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    const Range out[2] = {range_of(y, m, n, y_stride, es), range_of(z_out, m, n, n, es)};
    const Range in[4] = {range_of(x, k ? m : 0, k, x_stride, es), range_of(w, k ? n : 0, k, w_stride, es),
                         range_of(bias, 1, n, n, es), range_of(a.e.drop.rng, 1, 2, 2, 8)};
    for (const Range &i : in)
        if (overlap(out[0], i) || overlap(out[1], i)) return CP_ERR_INVALID_ARGUMENT;
    const Range r = range_of(residual, m, n, residual_stride, es);
    const bool in_place = residual == y && (m == 1 || residual_stride == y_stride);
    if (overlap(out[0], out[1]) || overlap(out[1], r) || (!in_place && overlap(out[0], r)))
        return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    a.a = x;
    a.b = w;
    a.a_stride = m > 1 ? x_stride : k;
    a.b_stride = n > 1 ? w_stride : k;
    a.dtype = dtype;
    a.m = m;
    a.n = n;
    a.k = k;
    a.e.bias = bias;
    a.e.residual = residual;
    a.e.residual_stride = residual_stride;
    a.e.y = y;
    a.e.y_stride = y_stride;
    a.e.z = z_out;
    a.e.act = act;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::linear_rows_by_rows(a));
}

uint64_t cp_linear_act_grad_workspace_bytes(uint64_t m, uint64_t n)
{
    if (n == 0 || m > kMaxCount || n > kMaxCount) return 0;
    return cpk::act_grad_workspace_bytes(m, n);
}

cp_status cp_linear_act_grad(const void *dy, uint64_t dy_stride, const void *z, uint64_t z_stride, cp_dtype dtype,
                             uint64_t m, uint64_t n, cp_act act, double p, const uint64_t *rng, void *dz, float *db,
                             void *workspace, uint64_t workspace_bytes, void *stream)
{
    cpk::ActGradArgs a{};
    if (!dtype_ok(dtype) || !act_ok(act) || !drop_of(p, rng, &a.drop)) return CP_ERR_INVALID_ARGUMENT;
    if (m > kMaxCount || n > kMaxCount || !spans(m, dy_stride) || !spans(m, n)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (!good_or_null(db, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (n == 0) return CP_OK;
    // (without rows db becomes zeros, by the same launches)
    const Range sums = range_of(db, 1, n, n, 4), numbers = range_of(a.drop.rng, 1, 2, 2, 8);
    if (db && !workspace_ok(workspace, workspace_bytes, cpk::act_grad_workspace_bytes(m, n)))
        return CP_ERR_INVALID_ARGUMENT;
    if (overlap(sums, numbers)) return CP_ERR_INVALID_ARGUMENT;
    if (m > 0) {
        if (!good(dy, es) || !good(dz, es)) return CP_ERR_INVALID_ARGUMENT;
        if (act != CP_ACT_NONE && (!good(z, es) || !spans(m, z_stride))) return CP_ERR_INVALID_ARGUMENT;
        const Range out = range_of(dz, m, n, n, es);
        const Range in[2] = {range_of(dy, m, n, dy_stride, es),
                             range_of(act == CP_ACT_NONE ? nullptr : z, m, n, z_stride, es)};
        const bool itself[2] = {dy == dz && (m == 1 || dy_stride == n), z == dz && (m == 1 || z_stride == n)};
        for (int q = 0; q < 2; ++q)
            if (overlap(sums, in[q]) || (!itself[q] && overlap(out, in[q]))) return CP_ERR_INVALID_ARGUMENT;
        if (overlap(out, sums) || overlap(out, numbers)) return CP_ERR_INVALID_ARGUMENT;
    }
    if (m == 0 && !db) return CP_OK;
    forget_earlier_error();
    a.dy = dy;
    a.z = z;
    a.dy_stride = dy_stride;
    a.z_stride = z_stride;
    a.dtype = dtype;
    a.m = m;
    a.n = n;
    a.act = act;
    a.dz = dz;
    a.db = db;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::act_grad(a));
}

// (the products of the backward pass reduce over n and over m)
uint64_t cp_linear_dx_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype)
{
    if (!dtype_ok(dtype) || m == 0 || n == 0 || k == 0 || n > kMaxStride || k > kMaxStride || too_large(m, k)) return 0;
    return cpk::linear_tile_workspace_bytes(m, k, n, dtype);
}

cp_status cp_linear_dx(const void *dz, uint64_t dz_stride, const void *w, uint64_t w_stride, const void *dres,
                       uint64_t dres_stride, cp_dtype dtype, uint64_t m, uint64_t n, uint64_t k, void *dx,
                       void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (n > kMaxStride || k > kMaxStride || too_large(m, k) || (m > 1 && dz_stride > kMaxStride) ||
        (n > 1 && w_stride > kMaxStride))
        return CP_ERR_UNSUPPORTED;
    if (!good_or_null(dres, es) || (dres && !spans(m, dres_stride))) return CP_ERR_INVALID_ARGUMENT;
    if (m == 0 || k == 0) return CP_OK;
    if (!good(dx, es)) return CP_ERR_INVALID_ARGUMENT;
    if (n > 0) {
        if (!good(dz, es) || !good(w, es)) return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::linear_tile_workspace_bytes(m, k, n, dtype)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    const Range out = range_of(dx, m, k, k, es);
    if (overlap(out, range_of(dz, m, n, dz_stride, es)) || overlap(out, range_of(w, n, k, w_stride, es)))
        return CP_ERR_INVALID_ARGUMENT;
    const bool in_place = dres == dx && (m == 1 || dres_stride == k);
    if (!in_place && overlap(out, range_of(dres, m, k, dres_stride, es))) return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    cpk::LinearArgs a{};
    a.a = dz;
    a.b = w;
    a.a_stride = m > 1 ? dz_stride : n;
    a.b_stride = n > 1 ? w_stride : k;
    a.dtype = dtype;
    a.m = m;
    a.n = k;
    a.k = n;
    a.e.residual = dres;
    a.e.residual_stride = dres_stride;
    a.e.y = dx;
    a.e.y_stride = k;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::linear_rows_by_columns(a));
}

uint64_t cp_linear_dw_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype dtype)
{
    if (!dtype_ok(dtype) || m == 0 || n == 0 || k == 0 || m > kMaxRows || n > kMaxStride || k > kMaxStride ||
        too_large(n, k))
        return 0;
    return cpk::linear_tile_workspace_bytes(n, k, m, dtype);
}

cp_status cp_linear_dw(const void *dz, uint64_t dz_stride, const void *x, uint64_t x_stride, cp_dtype dtype,
                       uint64_t m, uint64_t n, uint64_t k, int add, float *dw, uint64_t dw_stride, void *workspace,
                       uint64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || (add != 0 && add != 1)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (m > kMaxRows || n > kMaxStride || k > kMaxStride || too_large(n, k) || (m > 1 && dz_stride > kMaxStride) ||
        (m > 1 && x_stride > kMaxStride))
        return CP_ERR_UNSUPPORTED;
    if ((n > 1 && dw_stride < k) || !spans(n, dw_stride)) return CP_ERR_INVALID_ARGUMENT;
    if (n == 0 || k == 0) return CP_OK;
    if (!good(dw, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (m > 0) {
        if (!good(dz, es) || !good(x, es)) return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::linear_tile_workspace_bytes(n, k, m, dtype)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    const Range out = range_of(dw, n, k, dw_stride, 4);
    if (overlap(out, range_of(dz, m, n, dz_stride, es)) || overlap(out, range_of(x, m, k, x_stride, es)))
        return CP_ERR_INVALID_ARGUMENT;
    if (m == 0 && add) return CP_OK;
    forget_earlier_error();
    cpk::LinearArgs a{};
    a.a = dz;
    a.b = x;
    a.a_stride = m > 1 ? dz_stride : n;
    a.b_stride = m > 1 ? x_stride : k;
    a.dtype = dtype;
    a.m = n;
    a.n = k;
    a.k = m;
    a.e.residual = add ? dw : nullptr;
    a.e.residual_stride = dw_stride;
    a.e.y = dw;
    a.e.y_stride = dw_stride;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::linear_columns_by_columns(a));
}

cp_status cp_dropout(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride, cp_dtype dtype,
                     uint64_t n, uint64_t d, double p, const uint64_t *rng, void *y, void *stream)
{
    cpk::DropoutArgs a{};
    if (!dtype_ok(dtype) || !drop_of(p, rng, &a.drop)) return CP_ERR_INVALID_ARGUMENT;
    if (n > kMaxCount || d > kMaxCount || !spans(n, x_stride) || !spans(n, d)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (residual && (!good(residual, es) || !spans(n, residual_stride))) return CP_ERR_INVALID_ARGUMENT;
    if (n == 0 || d == 0) return CP_OK;
    if (!good(x, es) || !good(y, es)) return CP_ERR_INVALID_ARGUMENT;
    const Range out = range_of(y, n, d, d, es);
    if (!(x == y && (n == 1 || x_stride == d)) && overlap(out, range_of(x, n, d, x_stride, es)))
        return CP_ERR_INVALID_ARGUMENT;
    if (!(residual == y && (n == 1 || residual_stride == d)) &&
        overlap(out, range_of(residual, n, d, residual_stride, es)))
        return CP_ERR_INVALID_ARGUMENT;
    if (overlap(out, range_of(a.drop.rng, 1, 2, 2, 8))) return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    a.x = x;
    a.residual = residual;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.dtype = dtype;
    a.n = n;
    a.d = d;
    a.y = y;
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::dropout(a));
}

}  // extern "C"
