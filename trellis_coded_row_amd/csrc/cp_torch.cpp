// cp_torch.cpp - the dense operators' torch functions (trellis_coded_row_amd/
// ops.py): checks of the tensors, outputs, workspaces, and the C call
// (include/cp_ops.h), one Python call each.
//
// A call for a single token's step ends before its caller does: what the
// host spends is what the step costs. The same in Python took 7.3 us for a
// lookup and 13.5 us for a norm with four outputs, of which the kernel's
// launch is 2.7 us.
//
// Arguments come by position, as ops.py passes them. `stream` is None
// (torch's current stream), an object with a cuda_stream, or a whole number.
#include "cp_torch.h"

using namespace cpt;

namespace {

// What this was built for and from, as build.py looks for it in the file.
[[gnu::used]] const char marks[] = CP_TORCH_MARKS;

// (table, ids, scale, dtype, out, bad_id, stream) -> out
PyObject *embed_lookup(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 7);
    const at::Tensor &table = tensor(arg[0], "table"), &ids = tensor(arg[1], "ids");
    const int64_t stride = matrix(table, "table"), n = ids_of(ids), rows = table.size(0), d = table.size(1);
    const c10::Device device = table.device();
    same_device(ids, "ids", device);
    const Stream stream(arg[6], device);
    at::Tensor out;
    if (arg[4] == Py_None) {
        out = empty({n, d}, arg[3] == Py_None ? table.scalar_type() : type_of(arg[3], "dtype"), device);
        stream.keep(out);
    } else {
        out = tensor(arg[4], "out");
        TORCH_CHECK_VALUE(out.is_cuda() && code_of(out.scalar_type()) >= 0 && out.dim() == 2 && out.size(0) == n &&
                              out.size(1) == d && out.is_contiguous() &&
                              (arg[3] == Py_None || type_of(arg[3], "dtype") == out.scalar_type()),
                          "out must be a contiguous device tensor of shape (", n, ", ", d, ")");
        same_device(out, "out", device);
    }
    int32_t *bad = nullptr;
    if (arg[5] != Py_None) {
        const at::Tensor &b = tensor(arg[5], "bad_id");
        vector(b, "bad_id", at::ScalarType::Int, 1, device);
        bad = ptr<int32_t>(b);
    }
    const float scale = (float)number(arg[2]);
    call("cp_embed_lookup", device, cp_embed_lookup, ptr(table), (cp_dtype)code_of(table.scalar_type()), rows, d,
         stride, ptr<int64_t>(ids), n, scale, ptr(out), (cp_dtype)code_of(out.scalar_type()), bad, stream.handle());
    if (arg[4] != Py_None) written(out);
    if (bad) written(tensor(arg[5], "bad_id"));
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

// (ids, rows, stream) -> (order, slot, unique, starts, count)
PyObject *embed_plan(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 3);
    const at::Tensor &ids = tensor(arg[0], "ids");
    const int64_t n = ids_of(ids), rows = whole(arg[1]);
    TORCH_CHECK_VALUE(rows >= 0, "rows must not be negative");
    const c10::Device device = ids.device();
    const Stream stream(arg[2], device);
    const at::Tensor order = empty({n}, at::ScalarType::Int, device), slot = empty({n}, at::ScalarType::Int, device),
                     unique = empty({n}, at::ScalarType::Long, device),
                     starts = empty({n + 1}, at::ScalarType::Int, device),
                     number = empty({}, at::ScalarType::Long, device);
    for (const at::Tensor &t : {order, slot, unique, starts, number}) stream.keep(t);
    const uint64_t need = cp_embed_plan_workspace_bytes(n, rows);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_embed_plan", device, cp_embed_plan, ptr<int64_t>(ids), n, rows, ptr<int32_t>(order), ptr<int32_t>(slot),
         ptr<int64_t>(unique), ptr<int32_t>(starts), ptr<int64_t>(number), ptr(ws), need, stream.handle());
    return tuple({order, slot, unique, starts, number});
    END_HANDLE_TH_ERRORS
}

// (n, rows, order, slot, unique, starts, count, dout, scale, whole, stream) -> grad
PyObject *embed_grad(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 11);
    const int64_t planned = whole(arg[0]), table_rows = whole(arg[1]);
    const at::Tensor &order = tensor(arg[2], "order"), &slot = tensor(arg[3], "slot"),
                     &unique = tensor(arg[4], "unique"), &starts = tensor(arg[5], "starts"),
                     &number_of = tensor(arg[6], "count"), &dout = tensor(arg[7], "dout");
    const int64_t stride = matrix(dout, "dout"), n = dout.size(0), d = dout.size(1);
    const c10::Device device = dout.device();
    TORCH_CHECK_VALUE(n == planned, "dout has ", n, " rows, the plan ", planned, " lookups");
    vector(order, "the plan's order", at::ScalarType::Int, n, device);
    vector(slot, "the plan's slot", at::ScalarType::Int, n, device);
    vector(unique, "the plan's unique", at::ScalarType::Long, n, device);
    vector(starts, "the plan's starts", at::ScalarType::Int, n + 1, device);
    TORCH_CHECK_VALUE(number_of.scalar_type() == at::ScalarType::Long && number_of.numel() == 1,
                      "the plan's count must be one int64");
    same_device(number_of, "the plan's count", device);
    const bool all = truth(arg[9]);
    const float scale = (float)number(arg[8]);
    const Stream stream(arg[10], device);
    const at::Tensor grad = empty({all ? table_rows : n, d}, at::ScalarType::Float, device);
    if (grad.numel() == 0) return wrapped(grad);
    stream.keep(grad);
    const uint64_t need = cp_embed_grad_workspace_bytes(n, d);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_embed_grad", device, cp_embed_grad, ptr<int32_t>(order), ptr<int32_t>(slot), ptr<int64_t>(unique),
         ptr<int32_t>(starts), ptr<int64_t>(number_of), n, all ? table_rows : 0, ptr(dout),
         (cp_dtype)code_of(dout.scalar_type()), d, stride, scale, ptr<float>(grad), ptr(ws), need, stream.handle());
    return wrapped(grad);
    END_HANDLE_TH_ERRORS
}

// (x, weight, residual, eps, y, fp8, rstd, stream) -> (h, y, q, scale, rstd), None where not made
PyObject *rms_norm(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 8);
    const at::Tensor &x = tensor(arg[0], "x"), &weight = tensor(arg[1], "weight");
    const int64_t stride = matrix(x, "x"), n = x.size(0), d = x.size(1);
    TORCH_CHECK_VALUE(d > 0, "x has no columns");
    const c10::Device device = x.device();
    const auto type = x.scalar_type();
    vector(weight, "weight", type, d, device);
    const float eps = (float)number(arg[3]);
    const bool eight = truth(arg[5]);
    const Stream stream(arg[7], device);
    at::Tensor residual, h, y, q, scale, rstd;
    int64_t residual_stride = 0;
    if (arg[2] != Py_None) {
        residual = tensor(arg[2], "residual");
        residual_stride = matrix_like(residual, "residual", x);
        h = empty({n, d}, type, device);
        stream.keep(h);
    }
    if (truth(arg[4])) y = empty({n, d}, type, device);
    if (eight) {
        EightBits t = empty_eight_bits(n, d, n, groups_of(d), device);
        q = std::move(t.q);
        scale = std::move(t.scale);
    }
    if (truth(arg[6])) rstd = empty({n}, at::ScalarType::Float, device);
    for (const at::Tensor &t : {y, q, scale, rstd}) stream.keep(t);
    if (n)
        call("cp_rms_norm", device, cp_rms_norm, ptr(x), stride, ptr(residual), residual_stride, ptr(weight),
             (cp_dtype)code_of(type), n, d, eps, ptr(h), ptr(y), ptr<uint8_t>(q), eight ? q.stride(0) : 0,
             ptr<uint8_t>(scale), eight ? scale.stride(0) : 0, ptr<float>(rstd), stream.handle());
    return tuple({residual.defined() ? h : x, y, q, scale, rstd});
    END_HANDLE_TH_ERRORS
}

// (dy, x, rstd, weight, dres, stream) -> (dx, dw)
PyObject *rms_norm_grad(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 6);
    const at::Tensor &dy = tensor(arg[0], "dy"), &x = tensor(arg[1], "x"), &rstd = tensor(arg[2], "rstd"),
                     &weight = tensor(arg[3], "weight");
    const int64_t stride = matrix(x, "x"), n = x.size(0), d = x.size(1);
    TORCH_CHECK_VALUE(d > 0, "x has no columns");
    const c10::Device device = x.device();
    const auto type = x.scalar_type();
    const int64_t dy_stride = matrix_like(dy, "dy", x);
    vector(rstd, "rstd", at::ScalarType::Float, n, device);
    vector(weight, "weight", type, d, device);
    at::Tensor dres;
    int64_t dres_stride = 0;
    if (arg[4] != Py_None) {
        dres = tensor(arg[4], "dres");
        dres_stride = matrix_like(dres, "dres", x);
    }
    const Stream stream(arg[5], device);
    const at::Tensor dx = empty({n, d}, type, device), dw = empty({d}, at::ScalarType::Float, device);
    stream.keep(dx);
    stream.keep(dw);
    const uint64_t need = cp_rms_norm_grad_workspace_bytes(n, d);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_rms_norm_grad", device, cp_rms_norm_grad, ptr(dy), dy_stride, ptr(x), stride, ptr<float>(rstd),
         ptr(weight), ptr(dres), dres_stride, (cp_dtype)code_of(type), n, d, ptr(dx), ptr<float>(dw), ptr(ws), need,
         stream.handle());
    return tuple({dx, dw});
    END_HANDLE_TH_ERRORS
}

// (x, blocks, transposed, stream) -> (q, scale, qt, scale_t), None where not made
PyObject *quantize_fp8(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 4);
    const at::Tensor &x = tensor(arg[0], "x");
    const int64_t stride = matrix(x, "x"), n = x.size(0), d = x.size(1), gn = groups_of(n), gd = groups_of(d);
    const c10::Device device = x.device();
    const bool blocks = truth(arg[1]), both = truth(arg[2]);
    const Stream stream(arg[3], device);
    const EightBits t = empty_eight_bits(n, d, blocks ? gn : n, gd, device);
    const at::Tensor &q = t.q, &scale = t.scale;
    at::Tensor qt, scale_t;
    if (both) {
        EightBits other = empty_eight_bits(d, n, blocks ? gd : d, gn, device);
        qt = std::move(other.q);
        scale_t = std::move(other.scale);
    }
    for (const at::Tensor &t : {q, scale, qt, scale_t}) stream.keep(t);
    if (n && d)
        call("cp_quantize_fp8", device, cp_quantize_fp8, ptr(x), (cp_dtype)code_of(x.scalar_type()), n, d, stride,
             blocks, ptr<uint8_t>(q), q.stride(0), ptr<uint8_t>(scale), scale.stride(0), ptr<uint8_t>(qt),
             both ? qt.stride(0) : 0, ptr<uint8_t>(scale_t), both ? scale_t.stride(0) : 0, stream.handle());
    return tuple({q, scale, qt, scale_t});
    END_HANDLE_TH_ERRORS
}

// Row stride of an 8-bit matrix whose rows start on `unit` bytes and can be
// read up to the next multiple of it.
int64_t operand(const at::Tensor &t, const char *name, at::ScalarType type, int64_t unit, c10::Device device)
{
    TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type);
    int64_t stride = rows_of(t, name);
    same_device(t, name, device);
    const int64_t rows = t.size(0), cols = t.size(1), wide = up(cols, unit);
    if (rows <= 1 || cols == 0) stride = wide;  // nothing goes by it
    if (rows && cols) {
        TORCH_CHECK_VALUE(stride % unit == 0 && stride >= wide && (uintptr_t)t.data_ptr() % unit == 0, "the rows of ",
                          name, " must start on ", unit, " bytes");
        TORCH_CHECK_VALUE(wide == cols || (int64_t)t.storage().nbytes() >= t.storage_offset() + (rows - 1) * stride + wide,
                          "the last row of ", name, " must be readable up to a multiple of ", unit, " bytes");
    }
    return stride;
}

// (a, a_scale, b, b_scale, dtype, out, stream) -> out
PyObject *gemm_fp8(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 7);
    const at::Tensor &a = tensor(arg[0], "a"), &a_scale = tensor(arg[1], "a_scale"), &b = tensor(arg[2], "b"),
                     &b_scale = tensor(arg[3], "b_scale");
    const c10::Device device = a.device();
    const int64_t a_stride = operand(a, "a", kE4m3, 16, device), b_stride = operand(b, "b", kE4m3, 16, device),
                  as_stride = operand(a_scale, "a_scale", kE8m0, 4, device),
                  bs_stride = operand(b_scale, "b_scale", kE8m0, 4, device);
    const int64_t m = a.size(0), k = a.size(1), n = b.size(0), groups = groups_of(k);
    TORCH_CHECK_VALUE(b.size(1) == k, "a has ", k, " columns, b ", b.size(1));
    TORCH_CHECK_VALUE(a_scale.size(0) == m && a_scale.size(1) == groups, "a_scale must have shape (", m, ", ", groups, ")");
    const bool by_row = b_scale.size(0) == n && b_scale.size(1) == groups;
    TORCH_CHECK_VALUE(by_row || (b_scale.size(0) == groups_of(n) && b_scale.size(1) == groups),
                      "b_scale must have shape (", n, ", ", groups, ") or (", groups_of(n), ", ", groups, ")");
    const Stream stream(arg[6], device);
    const auto type = type_of(arg[4], "dtype");
    at::Tensor out;
    int64_t out_stride = n;
    if (arg[5] == Py_None) {
        out = empty({m, n}, type, device);
        stream.keep(out);
    } else {
        out = tensor(arg[5], "out");
        TORCH_CHECK_VALUE(out.scalar_type() == type, "out must have dtype ", type);
        const int64_t s = rows_of(out, "out");
        TORCH_CHECK_VALUE(out.size(0) == m && out.size(1) == n, "out must have shape (", m, ", ", n, ")");
        TORCH_CHECK_VALUE(m <= 1 || s >= n, "the rows of out must not overlap");
        same_device(out, "out", device);
        if (m > 1) out_stride = s;
    }
    const uint64_t need = cp_gemm_fp8_workspace_bytes(m, n, k, (cp_dtype)code_of(type));
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_gemm_fp8", device, cp_gemm_fp8, ptr<uint8_t>(a), a_stride, ptr<uint8_t>(a_scale), as_stride,
         ptr<uint8_t>(b), b_stride, ptr<uint8_t>(b_scale), bs_stride, !by_row, m, n, k, ptr(out), out_stride,
         (cp_dtype)code_of(type), ptr(ws), need, stream.handle());
    if (arg[5] != Py_None) written(out);
    return wrapped(out);
    END_HANDLE_TH_ERRORS
}

// (CPError): see cp_error.
PyObject *setup(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 1);
    Py_INCREF(arg[0]);
    Py_XDECREF(cp_error);
    cp_error = arg[0];
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

#define FUNCTION(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef functions[] = {
    FUNCTION(embed_lookup), FUNCTION(embed_plan),   FUNCTION(embed_grad), FUNCTION(rms_norm), FUNCTION(rms_norm_grad),
    FUNCTION(quantize_fp8), FUNCTION(gemm_fp8), FUNCTION(setup),      {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cp_torch", "The dense operators on torch tensors.", -1, functions,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern PyMethodDef linear_functions[];  // cp_torch_linear.cpp

PyMODINIT_FUNC PyInit__cp_torch()
{
    PyObject *const m = PyModule_Create(&module);
    if (m && PyModule_AddFunctions(m, linear_functions) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
