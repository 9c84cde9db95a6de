// cp_ops_api.hip - the C ABI of the dense operators (declared in
// include/cp_ops.h): argument checks on the host, then the launch.
#include "../../include/cp_ops.h"
#include "cp_ops_internal.h"
#include "cp_status.h"

static constexpr uint64_t kMaxCount = 0x7FFFFFFFull;           // lengths that kernels hold in 32 bits
static constexpr uint64_t kMaxSorted = 0x7FFFFFFFull - 4095;   // ids of one plan
static constexpr uint64_t kMaxGradColumns = 1ull << 21;        // a launch has fewer than 2^16 workgroups along y
static constexpr uint64_t kMaxGemmStride = 1ull << 22;         // a tile's rows then lie within 2^31 bytes
static constexpr uint64_t kMaxGemmRows = 1ull << 25;           // a launch for few rows of A then has fewer than 2^32 threads
static constexpr uint64_t kMaxGemmTiles = 1ull << 24;          // as one of tiles, of 256 threads each, then has

static bool dtype_ok(cp_dtype t) { return t == CP_DTYPE_F32 || t == CP_DTYPE_BF16 || t == CP_DTYPE_F16; }

// A pointer to use: not NULL, aligned to `bytes` (a power of two).
static bool good(const void *p, uint64_t bytes) { return p && ((uintptr_t)p & (bytes - 1)) == 0; }

static bool good_or_null(const void *p, uint64_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }

// Byte ranges of n rows, `stride` elements apart, stay below 2^62.
static bool spans(uint64_t n, uint64_t stride, uint64_t bytes)
{
    return n == 0 || stride <= (1ull << 62) / bytes / n;
}

// A product whose largest tiles (256 x 128, or twice that) are too many for a launch.
static bool too_many_tiles(uint64_t m, uint64_t n)
{
    return cpk::div_up(m, 256) * cpk::div_up(n, 128) >= kMaxGemmTiles;
}

static bool workspace_ok(const void *p, uint64_t bytes, uint64_t need)
{
    return need == 0 || (good(p, 256) && bytes >= need);
}

// The launches read their status with hipGetLastError: an earlier failure of
// an unrelated call must not be taken for theirs.
static void forget_earlier_error() { (void)hipGetLastError(); }

extern "C" {

cp_status cp_embed_lookup(const void *table, cp_dtype table_dtype, uint64_t rows, uint64_t d, uint64_t row_stride,
                          const int64_t *ids, uint64_t n, float scale, void *out, cp_dtype out_dtype, int32_t *bad_id,
                          void *stream)
{
    if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype)) return CP_ERR_INVALID_ARGUMENT;
    if (n > kMaxCount || d > kMaxCount) return CP_ERR_INVALID_ARGUMENT;
    if (rows > (1ull << 62) || !spans(rows, row_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (!good_or_null(bad_id, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (n == 0 || d == 0) return CP_OK;
    if (rows > 0 && !good(table, cpk::dtype_bytes(table_dtype))) return CP_ERR_INVALID_ARGUMENT;
    if (!good(ids, 8) || !good(out, cpk::dtype_bytes(out_dtype))) return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    cpk::EmbedLookupArgs a{};
    a.table = table;
    a.table_dtype = table_dtype;
    a.rows = rows;
    a.d = d;
    a.row_stride = row_stride;
    a.ids = ids;
    a.n = n;
    a.scale = scale;
    a.out = out;
    a.out_dtype = out_dtype;
    a.bad_id = bad_id;
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::embed_lookup(a));
}

uint64_t cp_embed_plan_workspace_bytes(uint64_t n, uint64_t rows)
{
    if (n > kMaxSorted || rows > (1ull << 62)) return 0;
    return cpk::embed_plan_workspace_bytes(n, rows);
}

cp_status cp_embed_plan(const int64_t *ids, uint64_t n, uint64_t rows, int32_t *order, int32_t *slot, int64_t *unique,
                        int32_t *starts, int64_t *count, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (n > kMaxSorted || rows > (1ull << 62)) return CP_ERR_INVALID_ARGUMENT;
    if (!good(starts, 4) || !good(count, 8)) return CP_ERR_INVALID_ARGUMENT;
    if (n > 0) {
        if (!good(ids, 8) || !good(order, 4) || !good(slot, 4) || !good(unique, 8)) return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::embed_plan_workspace_bytes(n, rows)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    forget_earlier_error();
    cpk::EmbedPlanArgs a{};
    a.ids = ids;
    a.n = n;
    a.rows = rows;
    a.order = order;
    a.slot = slot;
    a.unique = unique;
    a.starts = starts;
    a.count = count;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::embed_plan(a));
}

uint64_t cp_embed_grad_workspace_bytes(uint64_t n, uint64_t d)
{
    if (n > kMaxSorted || d > kMaxGradColumns) return 0;
    return cpk::embed_grad_workspace_bytes(n, d);
}

cp_status cp_embed_grad(const int32_t *order, const int32_t *slot, const int64_t *unique, const int32_t *starts,
                        const int64_t *count, uint64_t n, uint64_t rows, const void *dout, cp_dtype dtype, uint64_t d,
                        uint64_t dout_stride, float scale, float *grad, void *workspace, uint64_t workspace_bytes,
                        void *stream)
{
    if (!dtype_ok(dtype) || n > kMaxSorted || d > kMaxSorted) return CP_ERR_INVALID_ARGUMENT;
    if (d > kMaxGradColumns) return CP_ERR_UNSUPPORTED;
    if (rows > (1ull << 62) || !spans(rows, d, 4) || !spans(n, dout_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (d == 0 || (n == 0 && rows == 0)) return CP_OK;
    if (!good(starts, 4) || !good(count, 8) || !good(grad, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (n > 0) {
        if (!good(order, 4) || !good(slot, 4) || !good(unique, 8) || !good(dout, cpk::dtype_bytes(dtype)))
            return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::embed_grad_workspace_bytes(n, d)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    forget_earlier_error();
    cpk::EmbedGradArgs a{};
    a.order = order;
    a.slot = slot;
    a.unique = unique;
    a.starts = starts;
    a.count = count;
    a.n = n;
    a.rows = rows;
    a.dout = dout;
    a.dtype = dtype;
    a.d = d;
    a.stride = dout_stride;
    a.scale = scale;
    a.grad = grad;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::embed_grad(a));
}

cp_status cp_rms_norm(const void *x, uint64_t x_stride, const void *residual, uint64_t residual_stride,
                      const void *weight, cp_dtype dtype, uint64_t n, uint64_t d, float eps, void *h_out, void *y_out,
                      uint8_t *q, uint64_t q_stride, uint8_t *q_scale, uint64_t scale_stride, float *rstd,
                      void *stream)
{
    if (!dtype_ok(dtype) || n > kMaxCount || d > kMaxCount || d == 0) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (!spans(n, x_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (residual && !spans(n, residual_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (h_out && !residual) return CP_ERR_INVALID_ARGUMENT;  // h is x itself
    if ((q != nullptr) != (q_scale != nullptr)) return CP_ERR_INVALID_ARGUMENT;
    if (q && (!good(q, 16) || q_stride < d || q_stride % 16 || scale_stride < cpk::div_up(d, 128) ||
              !spans(n, q_stride, 1) || !spans(n, scale_stride, 1)))
        return CP_ERR_INVALID_ARGUMENT;
    if (!good_or_null(residual, es) || !good_or_null(h_out, es) || !good_or_null(y_out, es) || !good_or_null(rstd, 4))
        return CP_ERR_INVALID_ARGUMENT;
    if (n == 0) return CP_OK;
    if (!good(x, es) || !good(weight, es)) return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    cpk::NormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.x_stride = x_stride;
    a.residual_stride = residual_stride;
    a.dtype = dtype;
    a.n = n;
    a.d = d;
    a.eps = eps;
    a.h = h_out;
    a.y = y_out;
    a.q = q;
    a.q_scale = q_scale;
    a.q_stride = q_stride;
    a.scale_stride = scale_stride;
    a.rstd = rstd;
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::rms_norm(a));
}

uint64_t cp_rms_norm_grad_workspace_bytes(uint64_t n, uint64_t d)
{
    if (n > kMaxCount || d > kMaxCount) return 0;
    return cpk::rms_norm_grad_workspace_bytes(n, d);
}

cp_status cp_rms_norm_grad(const void *dy, uint64_t dy_stride, const void *x, uint64_t x_stride, const float *rstd,
                           const void *weight, const void *dres, uint64_t dres_stride, cp_dtype dtype, uint64_t n,
                           uint64_t d, void *dx, float *dw, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(dtype) || n > kMaxCount || d > kMaxCount || d == 0) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t es = cpk::dtype_bytes(dtype);
    if (!spans(n, dy_stride, 4) || !spans(n, x_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (dres && !spans(n, dres_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (!good_or_null(dres, es) || !good_or_null(dw, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (n > 0) {
        if (!good(dy, es) || !good(x, es) || !good(rstd, 4) || !good(weight, es) || !good(dx, es))
            return CP_ERR_INVALID_ARGUMENT;
        if (dw && !workspace_ok(workspace, workspace_bytes, cpk::rms_norm_grad_workspace_bytes(n, d)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    forget_earlier_error();
    cpk::NormGradArgs a{};
    a.dy = dy;
    a.x = x;
    a.weight = weight;
    a.dres = dres;
    a.dy_stride = dy_stride;
    a.x_stride = x_stride;
    a.dres_stride = dres_stride;
    a.rstd = rstd;
    a.dtype = dtype;
    a.n = n;
    a.d = d;
    a.dx = dx;
    a.dw = dw;
    a.workspace = static_cast<uint8_t *>(workspace);
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::rms_norm_grad(a));
}

cp_status cp_quantize_fp8(const void *x, cp_dtype dtype, uint64_t n, uint64_t d, uint64_t x_stride, int blocks,
                          uint8_t *q, uint64_t q_stride, uint8_t *scale, uint64_t scale_stride, uint8_t *qt,
                          uint64_t qt_stride, uint8_t *scale_t, uint64_t scale_t_stride, void *stream)
{
    if (!dtype_ok(dtype) || n > kMaxCount || d > kMaxCount || (blocks != 0 && blocks != 1))
        return CP_ERR_INVALID_ARGUMENT;
    if (!spans(n, x_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t gd = cpk::div_up(d, 128), gn = cpk::div_up(n, 128);
    if (q_stride < d || q_stride % 16 || scale_stride < gd || !spans(n, q_stride, 1) || !spans(n, scale_stride, 1))
        return CP_ERR_INVALID_ARGUMENT;
    if ((qt != nullptr) != (scale_t != nullptr)) return CP_ERR_INVALID_ARGUMENT;
    if (qt && (!good(qt, 16) || qt_stride < n || qt_stride % 16 || scale_t_stride < gn || !spans(d, qt_stride, 1) ||
               !spans(d, scale_t_stride, 1)))
        return CP_ERR_INVALID_ARGUMENT;
    if (n == 0 || d == 0) return CP_OK;
    if (!good(x, cpk::dtype_bytes(dtype)) || !good(q, 16) || !scale) return CP_ERR_INVALID_ARGUMENT;
    forget_earlier_error();
    cpk::QuantArgs a{};
    a.x = x;
    a.dtype = dtype;
    a.n = n;
    a.d = d;
    a.x_stride = x_stride;
    a.blocks = blocks != 0;
    a.q = q;
    a.scale = scale;
    a.qt = qt;
    a.scale_t = scale_t;
    a.q_stride = q_stride;
    a.scale_stride = scale_stride;
    a.qt_stride = qt_stride;
    a.scale_t_stride = scale_t_stride;
    a.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::quantize_fp8(a));
}

uint64_t cp_gemm_fp8_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, cp_dtype out_dtype)
{
    if (!dtype_ok(out_dtype) || m == 0 || n == 0 || k == 0 || m > kMaxGemmRows || n > kMaxGemmRows ||
        k > kMaxGemmStride || too_many_tiles(m, n))
        return 0;
    return cpk::gemm_fp8_workspace_bytes(m, n, k, out_dtype);
}

cp_status cp_gemm_fp8(const uint8_t *a, uint64_t a_stride, const uint8_t *a_scale, uint64_t a_scale_stride,
                      const uint8_t *b, uint64_t b_stride, const uint8_t *b_scale, uint64_t b_scale_stride,
                      int b_blocks, uint64_t m, uint64_t n, uint64_t k, void *out, uint64_t out_stride,
                      cp_dtype out_dtype, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (!dtype_ok(out_dtype) || (b_blocks != 0 && b_blocks != 1)) return CP_ERR_INVALID_ARGUMENT;
    const uint64_t groups = cpk::div_up(k, 128);
    if (a_stride < k || b_stride < k || a_stride % 16 || b_stride % 16 || a_scale_stride < groups ||
        b_scale_stride < groups || a_scale_stride % 4 || b_scale_stride % 4 || out_stride < n)
        return CP_ERR_INVALID_ARGUMENT;
    if (m > kMaxGemmRows || n > kMaxGemmRows || a_stride > kMaxGemmStride || b_stride > kMaxGemmStride ||
        a_scale_stride > kMaxGemmStride || b_scale_stride > kMaxGemmStride || too_many_tiles(m, n))
        return CP_ERR_UNSUPPORTED;
    if (!spans(m, out_stride, 4)) return CP_ERR_INVALID_ARGUMENT;
    if (m == 0 || n == 0) return CP_OK;
    if (!good(out, cpk::dtype_bytes(out_dtype))) return CP_ERR_INVALID_ARGUMENT;
    if (k > 0) {
        if (!good(a, 16) || !good(b, 16) || !good(a_scale, 4) || !good(b_scale, 4)) return CP_ERR_INVALID_ARGUMENT;
        if (!workspace_ok(workspace, workspace_bytes, cpk::gemm_fp8_workspace_bytes(m, n, k, out_dtype)))
            return CP_ERR_INVALID_ARGUMENT;
    }
    forget_earlier_error();
    cpk::GemmArgs g{};
    g.a = a;
    g.a_scale = a_scale;
    g.b = b;
    g.b_scale = b_scale;
    g.a_stride = a_stride;
    g.a_scale_stride = a_scale_stride;
    g.b_stride = b_stride;
    g.b_scale_stride = b_scale_stride;
    g.b_blocks = b_blocks != 0;
    g.m = m;
    g.n = n;
    g.k = k;
    g.out = out;
    g.out_stride = out_stride;
    g.out_dtype = out_dtype;
    g.workspace = static_cast<uint8_t *>(workspace);
    g.stream = (hipStream_t)stream;
    return cpk::status_of(cpk::gemm_fp8(g));
}

}  // extern "C"
