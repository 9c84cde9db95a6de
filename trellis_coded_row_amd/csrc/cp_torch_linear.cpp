// cp_torch_linear.cpp - the torch functions of the readout's product, its
// gradients and dropout (trellis_coded_row_amd/readout.py): checks of the
// tensors, outputs, workspaces, and the C call (include/cp_linear.h), one
// Python call each. Arguments come by position, as readout.py passes them.
#include "../../include/cp_linear.h"
#include "cp_torch.h"

using namespace cpt;

namespace {

cp_act act_of(PyObject *o)
{
    if (o == Py_None) return CP_ACT_NONE;
    static const struct {
        const char *name;
        cp_act act;
    } known[] = {{"relu", CP_ACT_RELU}, {"gelu", CP_ACT_GELU}, {"gelu_tanh", CP_ACT_GELU_TANH}, {"silu", CP_ACT_SILU}};
    if (PyUnicode_Check(o))
        for (const auto &k : known)
            if (PyUnicode_CompareWithASCIIString(o, k.name) == 0) return k.act;
    TORCH_CHECK_VALUE(false, "act must be None, 'relu', 'gelu', 'gelu_tanh' or 'silu'");
}

// The share that is dropped and the generator's numbers.
struct Dropped {
    double p;
    const uint64_t *rng;
};

Dropped dropped(PyObject *p, PyObject *rng, c10::Device device)
{
    Dropped d{number(p), nullptr};
    TORCH_CHECK_VALUE(d.p >= 0.0 && d.p <= 1.0 - 1.0 / 65536, "p must be at least 0 and at most 1 - 2^-16");
    if (rng == Py_None) {
        TORCH_CHECK_VALUE(d.p == 0.0, "dropout needs rng, a device tensor of (seed, offset)");
        return d;
    }
    const at::Tensor &t = tensor(rng, "rng");
    vector(t, "rng", at::ScalarType::Long, 2, device);
    d.rng = reinterpret_cast<const uint64_t *>(ptr<int64_t>(t));
    return d;
}

// A matrix of another's type and device; its row stride.
int64_t matrix_of(const at::Tensor &t, const char *name, const at::Tensor &x, int64_t rows, int64_t cols)
{
    TORCH_CHECK_VALUE(t.scalar_type() == x.scalar_type(), name, " must be ", x.scalar_type());
    const int64_t stride = rows_of(t, name);
    TORCH_CHECK_VALUE(t.size(0) == rows && t.size(1) == cols, name, " must have shape (", rows, ", ", cols, "), not ",
                      t.sizes());
    same_device(t, name, x.device());
    return stride;
}

// (x, weight, bias, residual, act, p, rng, z, stream) -> (y, z), None where not made
PyObject *linear(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 9);
    const at::Tensor &x = tensor(arg[0], "x"), &w = tensor(arg[1], "weight");
    const int64_t stride = matrix(x, "x"), m = x.size(0), k = x.size(1);
    TORCH_CHECK_VALUE(w.dim() == 2 && w.size(1) == k, "weight must have ", k, " columns, as x has");
    const int64_t n = w.size(0), w_stride = matrix_of(w, "weight", x, n, k);
    const c10::Device device = x.device();
    const auto type = x.scalar_type();
    at::Tensor bias, residual, z;
    int64_t residual_stride = 0;
    if (arg[2] != Py_None) {
        bias = tensor(arg[2], "bias");
        vector(bias, "bias", type, n, device);
    }
    if (arg[3] != Py_None) {
        residual = tensor(arg[3], "residual");
        residual_stride = matrix_of(residual, "residual", x, m, n);
    }
    const cp_act act = act_of(arg[4]);
    const Dropped drop = dropped(arg[5], arg[6], device);
    const Stream stream(arg[8], device);
    const at::Tensor y = empty({m, n}, type, device);
    stream.keep(y);
    if (truth(arg[7])) {
        z = empty({m, n}, type, device);
        stream.keep(z);
    }
    const cp_dtype code = (cp_dtype)code_of(type);
    const uint64_t need = cp_linear_workspace_bytes(m, n, k, code);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_linear", device, cp_linear, ptr(x), stride, ptr(w), w_stride, ptr(bias), ptr(residual), residual_stride,
         code, m, n, k, act, drop.p, drop.rng, ptr(y), n, ptr(z), ptr(ws), need, stream.handle());
    return tuple({y, z});
    END_HANDLE_TH_ERRORS
}

// (dy, z, act, p, rng, db, stream) -> (dz, db), None where not made
PyObject *linear_act_grad(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 7);
    const at::Tensor &dy = tensor(arg[0], "dy");
    const int64_t stride = matrix(dy, "dy"), m = dy.size(0), n = dy.size(1);
    const c10::Device device = dy.device();
    const cp_act act = act_of(arg[2]);
    at::Tensor z, db;
    int64_t z_stride = 0;
    if (arg[1] != Py_None) {
        z = tensor(arg[1], "z");
        z_stride = matrix_of(z, "z", dy, m, n);
    }
    TORCH_CHECK_VALUE(z.defined() || act == CP_ACT_NONE, "an activation's gradient needs z");
    const Dropped drop = dropped(arg[3], arg[4], device);
    const bool sums = truth(arg[5]);
    const Stream stream(arg[6], device);
    const at::Tensor dz = empty({m, n}, dy.scalar_type(), device);
    stream.keep(dz);
    if (sums) {
        db = empty({n}, at::ScalarType::Float, device);
        stream.keep(db);
    }
    const uint64_t need = sums ? cp_linear_act_grad_workspace_bytes(m, n) : 0;
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_linear_act_grad", device, cp_linear_act_grad, ptr(dy), stride, ptr(z), z_stride,
         (cp_dtype)code_of(dy.scalar_type()), m, n, act, drop.p, drop.rng, ptr(dz), ptr<float>(db), ptr(ws), need,
         stream.handle());
    return tuple({dz, db});
    END_HANDLE_TH_ERRORS
}

// (dz, weight, dres, stream) -> dx
PyObject *linear_dx(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 4);
    const at::Tensor &dz = tensor(arg[0], "dz"), &w = tensor(arg[1], "weight");
    const int64_t stride = matrix(dz, "dz"), m = dz.size(0), n = dz.size(1);
    TORCH_CHECK_VALUE(w.dim() == 2 && w.size(0) == n, "weight must have ", n, " rows, as dz has columns");
    const int64_t k = w.size(1), w_stride = matrix_of(w, "weight", dz, n, k);
    const c10::Device device = dz.device();
    at::Tensor dres;
    int64_t dres_stride = 0;
    if (arg[2] != Py_None) {
        dres = tensor(arg[2], "dres");
        dres_stride = matrix_of(dres, "dres", dz, m, k);
    }
    const Stream stream(arg[3], device);
    const at::Tensor dx = empty({m, k}, dz.scalar_type(), device);
    stream.keep(dx);
    const cp_dtype code = (cp_dtype)code_of(dz.scalar_type());
    const uint64_t need = cp_linear_dx_workspace_bytes(m, n, k, code);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_linear_dx", device, cp_linear_dx, ptr(dz), stride, ptr(w), w_stride, ptr(dres), dres_stride, code, m, n, k,
         ptr(dx), ptr(ws), need, stream.handle());
    return wrapped(dx);
    END_HANDLE_TH_ERRORS
}

// (dz, x, into, stream) -> dw
PyObject *linear_dw(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 4);
    const at::Tensor &dz = tensor(arg[0], "dz"), &x = tensor(arg[1], "x");
    const int64_t stride = matrix(dz, "dz"), m = dz.size(0), n = dz.size(1);
    TORCH_CHECK_VALUE(x.dim() == 2 && x.size(0) == m, "x must have ", m, " rows, as dz has");
    const int64_t k = x.size(1), x_stride = matrix_of(x, "x", dz, m, k);
    const c10::Device device = dz.device();
    const Stream stream(arg[3], device);
    const bool add = arg[2] != Py_None;
    at::Tensor dw;
    int64_t dw_stride = k;
    if (add) {
        dw = tensor(arg[2], "into");
        TORCH_CHECK_VALUE(dw.scalar_type() == at::ScalarType::Float, "into must be float32");
        const int64_t s = rows_of(dw, "into");
        TORCH_CHECK_VALUE(dw.size(0) == n && dw.size(1) == k, "into must have shape (", n, ", ", k, ")");
        TORCH_CHECK_VALUE(n <= 1 || s >= k, "the rows of into must not overlap");
        same_device(dw, "into", device);
        if (n > 1) dw_stride = s;
    } else {
        dw = empty({n, k}, at::ScalarType::Float, device);
        stream.keep(dw);
    }
    const cp_dtype code = (cp_dtype)code_of(dz.scalar_type());
    const uint64_t need = cp_linear_dw_workspace_bytes(m, n, k, code);
    const at::Tensor ws = stream.workspace(need, device);
    call("cp_linear_dw", device, cp_linear_dw, ptr(dz), stride, ptr(x), x_stride, code, m, n, k, (int)add,
         ptr<float>(dw), dw_stride, ptr(ws), need, stream.handle());
    if (add) written(dw);
    return wrapped(dw);
    END_HANDLE_TH_ERRORS
}

// (x, p, rng, residual, out, stream) -> y
PyObject *dropout(PyObject *, PyObject *const *arg, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    arguments(count, 6);
    const at::Tensor &x = tensor(arg[0], "x");
    const int64_t stride = matrix(x, "x"), n = x.size(0), d = x.size(1);
    const c10::Device device = x.device();
    const Dropped drop = dropped(arg[1], arg[2], device);
    at::Tensor residual;
    int64_t residual_stride = 0;
    if (arg[3] != Py_None) {
        residual = tensor(arg[3], "residual");
        residual_stride = matrix_of(residual, "residual", x, n, d);
    }
    const Stream stream(arg[5], device);
    at::Tensor y;
    if (arg[4] == Py_None) {
        y = empty({n, d}, x.scalar_type(), device);
        stream.keep(y);
    } else {
        y = tensor(arg[4], "out");
        matrix_of(y, "out", x, n, d);
        TORCH_CHECK_VALUE(y.is_contiguous(), "out must be contiguous");
    }
    call("cp_dropout", device, cp_dropout, ptr(x), stride, ptr(residual), residual_stride,
         (cp_dtype)code_of(x.scalar_type()), n, d, drop.p, drop.rng, ptr(y), stream.handle());
    if (arg[4] != Py_None) written(y);
    return wrapped(y);
    END_HANDLE_TH_ERRORS
}

}  // namespace

#define FUNCTION(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
extern PyMethodDef linear_functions[];
PyMethodDef linear_functions[] = {FUNCTION(linear),    FUNCTION(linear_act_grad), FUNCTION(linear_dx),
                                  FUNCTION(linear_dw), FUNCTION(dropout),         {nullptr, nullptr, 0, nullptr}};
