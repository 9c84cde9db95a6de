// cp_torch.h - what the torch functions of cp_torch.cpp and
// cp_torch_linear.cpp share: checks of tensors, the stream of a call, the C call.
#pragma once

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/GradMode.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/cp_ops.h"

namespace cpt {

constexpr int64_t kGroup = 128;  // values that share a scale
constexpr auto kE4m3 = at::ScalarType::Float8_e4m3fn, kE8m0 = at::ScalarType::Float8_e8m0fnu;

inline PyObject *cp_error = nullptr;  // CPError(status, name)

inline int64_t up(int64_t v, int64_t unit) { return (v + unit - 1) / unit * unit; }

inline int64_t groups_of(int64_t v) { return (v + kGroup - 1) / kGroup; }

inline int code_of(at::ScalarType t)
{
    return t == at::ScalarType::Float      ? CP_DTYPE_F32
           : t == at::ScalarType::BFloat16 ? CP_DTYPE_BF16
           : t == at::ScalarType::Half     ? CP_DTYPE_F16
                                           : -1;
}

// Whether memory holds the tensor's values: that of a wrapper (a transform's,
// a subclass's), a sparse matrix or a lazy negative does not.
inline bool in_memory(const at::Tensor &t)
{
    if (!t.has_storage() || t.layout() != at::kStrided || t.is_neg()) return false;
    try {
        return t.numel() == 0 || t.const_data_ptr();
    } catch (const c10::Error &) {
        return false;
    }
}

inline const at::Tensor &tensor(PyObject *o, const char *name)
{
    TORCH_CHECK_VALUE(THPVariable_Check(o), name, " must be a tensor");
    const at::Tensor &t = THPVariable_Unpack(o);
    TORCH_CHECK_VALUE(in_memory(t), name, " must be a plain dense tensor with memory of its own");
    // a result without its gradient's graph would end the caller's backward pass there, silently
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, which this function does not record: pass a detached tensor, or call it "
                      "under torch.no_grad() (a gradient's function is a call of its own)");
    return t;
}

inline void same_device(const at::Tensor &t, const char *name, c10::Device device)
{
    TORCH_CHECK_VALUE(t.device() == device, name, " is on ", t.device(), ", not on ", device);
}

// A 2-D device tensor whose rows are contiguous; its row stride.
inline int64_t rows_of(const at::Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(t.is_cuda() && t.dim() == 2, name, " must be a 2-D device tensor");
    TORCH_CHECK_VALUE(t.size(1) <= 1 || t.stride(1) == 1, name, " must have contiguous rows");
    return t.stride(0);
}

// The same of a type that the operators compute in.
inline int64_t matrix(const at::Tensor &t, const char *name)
{
    TORCH_CHECK_VALUE(code_of(t.scalar_type()) >= 0, name, " must be float32, bfloat16 or float16");
    return rows_of(t, name);
}

// The same, like another matrix.
inline int64_t matrix_like(const at::Tensor &t, const char *name, const at::Tensor &x)
{
    TORCH_CHECK_VALUE(t.scalar_type() == x.scalar_type(), name, " must be ", x.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == x.sizes(), name, " must have shape ", x.sizes(), ", not ", t.sizes());
    same_device(t, name, x.device());
    return rows_of(t, name);
}

inline void vector(const at::Tensor &t, const char *name, at::ScalarType type, int64_t length, c10::Device device)
{
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == type && t.dim() == 1 && t.size(0) == length && t.is_contiguous(),
                      name, " must be a contiguous ", type, " device tensor of ", length, " values");
    same_device(t, name, device);
}

inline int64_t ids_of(const at::Tensor &t)
{
    TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == at::ScalarType::Long && t.dim() == 1 && t.is_contiguous(),
                      "ids must be a contiguous 1-D int64 device tensor");
    return t.size(0);
}

inline at::Tensor empty(c10::IntArrayRef sizes, at::ScalarType type, c10::Device device)
{
    return at::Tensor(at::detail::empty_cuda(sizes, type, device, std::nullopt));
}

// An 8-bit matrix and its scales: rows x cols of e4m3 whose rows start on 16
// bytes and srows x scols of e8m0 whose rows start on 4, each row readable up
// to there. They are used and dropped together, so they share an allocation
// (one takes about 0.9 us of a call of 7).
struct EightBits {
    at::Tensor q, scale;
};

inline EightBits empty_eight_bits(int64_t rows, int64_t cols, int64_t srows, int64_t scols, c10::Device device)
{
    const int64_t wide = up(cols, 16), swide = up(scols, 4), first = up(rows * wide, 256);
    EightBits t;
    t.q = empty({first + srows * swide}, kE4m3, device);
    t.scale = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(t.q.storage()), t.q.key_set(),
                                                       c10::scalarTypeToTypeMeta(kE8m0));
    t.scale.unsafeGetTensorImpl()->set_storage_offset(first);
    t.scale.unsafeGetTensorImpl()->set_sizes_and_strides(c10::IntArrayRef{srows, scols}, c10::IntArrayRef{swide, 1});
    t.q.unsafeGetTensorImpl()->set_sizes_and_strides(c10::IntArrayRef{rows, cols}, c10::IntArrayRef{wide, 1});
    return t;
}

// A caller's tensor was written: autograd then refuses to use it as a value saved before.
inline void written(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

inline void *ptr(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

template <typename T>
T *ptr(const at::Tensor &t)
{
    return static_cast<T *>(ptr(t));
}

// The stream of a call, torch's current one while this lives: what is made for
// the call comes from that stream's memory. A block that the caller's own
// current stream gave back may still be read there by work that the call's
// stream does not wait for. An output that the call returns is also made known
// to the allocator as used by the caller's stream (keep), so that dropping it
// there does not hand its memory to the call's stream too early.
class Stream {
  public:
    Stream(PyObject *o, c10::Device device) : before_(c10::hip::getCurrentHIPStream(device.index()))
    {
        handle_ = o == Py_None ? before_.stream() : static_cast<hipStream_t>(handle_of(o));
        other_ = handle_ != before_.stream();
        if (other_)
            c10::hip::setCurrentHIPStream(handle_ ? c10::hip::getStreamFromExternal(handle_, device.index())
                                                  : c10::hip::getDefaultHIPStream(device.index()));
    }

    ~Stream()
    {
        if (other_) c10::hip::setCurrentHIPStream(before_);
    }

    Stream(const Stream &) = delete;
    Stream &operator=(const Stream &) = delete;

    void *handle() const { return handle_; }

    void keep(const at::Tensor &t) const
    {
        // (torch names this device type cuda on tensors, hip in its HIPStream)
        if (other_ && t.defined()) t.record_stream(c10::Stream(c10::Stream::UNSAFE, t.device(), before_.id()));
    }

    at::Tensor workspace(uint64_t bytes, c10::Device device) const
    {
        return bytes ? empty({(int64_t)bytes}, at::ScalarType::Byte, device) : at::Tensor();
    }

  private:
    static void *handle_of(PyObject *o)
    {
        PyObject *const of = PyObject_GetAttrString(o, "cuda_stream");
        if (!of) {
            if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw python_error();
            PyErr_Clear();
        }
        PyObject *const number = PyNumber_Long(of ? of : o);
        Py_XDECREF(of);
        if (!number) throw python_error();
        void *const handle = PyLong_AsVoidPtr(number);
        Py_DECREF(number);
        if (!handle && PyErr_Occurred()) throw python_error();
        return handle;
    }

    c10::hip::HIPStream before_;
    hipStream_t handle_ = nullptr;
    bool other_ = false;
};

// Python's lock, given up while this lives.
class Unlocked {
  public:
    Unlocked() : python_(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(python_); }
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;

  private:
    PyThreadState *python_;
};

// A C call with `device` current; CPError for a status other than CP_OK. Its
// arguments, tensors' pointers among them, are made before Python's lock is
// given up: to make them can fail.
template <typename F, typename... Args>
inline void call(const char *name, c10::Device device, F f, Args... args)
{
    cp_status st;
    {
        const c10::DeviceGuard guard(device);
        const Unlocked unlocked;  // (a launch may wait for room in its queue)
        st = f(args...);
    }
    if (st == CP_OK) return;
    PyObject *const e = PyObject_CallFunction(cp_error, "is", (int)st, name);
    if (e) {
        PyErr_SetObject(cp_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// None for a tensor that was not made.
inline PyObject *wrapped(const at::Tensor &t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

inline PyObject *tuple(std::initializer_list<at::Tensor> list)
{
    PyObject *const out = PyTuple_New((Py_ssize_t)list.size());
    if (!out) throw python_error();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : list) {
        PyObject *const w = wrapped(t);
        if (!w) {
            Py_DECREF(out);
            throw python_error();
        }
        PyTuple_SET_ITEM(out, i++, w);
    }
    return out;
}

inline bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

inline double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

inline int64_t whole(PyObject *o)
{
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

inline at::ScalarType type_of(PyObject *o, const char *name)
{
    TORCH_CHECK_VALUE(THPDtype_Check(o) && code_of(reinterpret_cast<THPDtype *>(o)->scalar_type) >= 0, name,
                      " must be float32, bfloat16 or float16");
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

inline void arguments(Py_ssize_t got, Py_ssize_t want)
{
    TORCH_CHECK_TYPE(got == want, "expected ", want, " arguments, got ", got);
}

}  // namespace cpt
