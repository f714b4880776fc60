// The tensor-level calls of the linear layers and the norm, as a CPython extension: argument checks,
// allocation of the outputs from PyTorch's caching allocator on the current stream, and one call of the
// C ABI (include/attn.h).  Nothing is computed here.  The same through Python and ctypes took 13 to 16
// us a call on the GB300's host, several times what the smallest kernels take on the GPU; this takes
// about 4.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "attn.h"

namespace {

constexpr auto kBf16 = at::kBFloat16, kF32 = at::kFloat, kE4m3 = at::kFloat8_e4m3fn;

PyObject *g_fail = nullptr;   // raises AttnError(code, where)

struct Refused {};   // a Python exception is set

[[noreturn]] void refuse(const std::string &why)
{
    PyErr_SetString(PyExc_ValueError, why.c_str());
    throw Refused{};
}

std::string describe(c10::IntArrayRef shape)
{
    std::string s = "[";
    for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + "]";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

// An operand: a contiguous tensor of this type and shape on this device.
void *operand(PyObject *o, const char *name, c10::ScalarType type, c10::IntArrayRef shape, c10::Device dev)
{
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || t.sizes() != shape || t.device() != dev || !t.is_contiguous())
        refuse(std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor of shape " +
               describe(shape) + " on " + dev.str() + ", got " + c10::toString(t.scalar_type()) + " " +
               describe(t.sizes()) + " on " + t.device().str() + (t.is_contiguous() ? "" : ", not contiguous"));
    return t.data_ptr();
}

void *operand_or_null(PyObject *o, const char *name, c10::ScalarType type, c10::IntArrayRef shape, c10::Device dev)
{
    return o == Py_None ? nullptr : operand(o, name, type, shape, dev);
}

// One fp32 number a row.  A slice of rows starts on any element, the C ABI takes pointers to 16 bytes: those
// numbers are copied first (on the current stream; call it with the device's guard set).
const float *aligned(void *p, PyObject *o, at::Tensor &copy)
{
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) return static_cast<const float *>(p);
    copy = THPVariable_Unpack(o).detach().clone();
    return static_cast<const float *>(copy.data_ptr());
}

// Rows [..., width] of a contiguous CUDA tensor.
struct Rows {
    const at::Tensor &t;
    c10::Device dev;
    int64_t M, width;
    Rows(PyObject *o, const char *name, c10::ScalarType type) : t(tensor(o, name)), dev(t.device())
    {
        if (!t.is_cuda() || t.scalar_type() != type || t.dim() < 1 || !t.is_contiguous())
            refuse(std::string(name) + ": expected a contiguous " + c10::toString(type) + " CUDA tensor [..., width]");
        width = t.size(-1);
        M = width ? t.numel() / width : 0;
    }
    c10::DimVector lead() const { return c10::DimVector(t.sizes().begin(), t.sizes().end() - 1); }
    c10::DimVector with(int64_t last) const
    {
        c10::DimVector s = lead();
        s.push_back(last);
        return s;
    }
};

// The C ABI counts in ints; what does not fit becomes a size it refuses.
int count(int64_t n) { return n > 0x7fffffff ? -1 : (int)n; }

int64_t matrix_columns(PyObject *o, const char *name)
{
    const at::Tensor &t = tensor(o, name);
    if (t.dim() != 2) refuse(std::string(name) + ": expected a matrix");
    return t.size(1);
}

at::Tensor empty(c10::IntArrayRef shape, c10::ScalarType type, c10::Device dev)
{
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

void *at_or_null(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

cudaStream_t stream(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

// Allocation and launch run without the interpreter's lock: either may wait for the GPU.
class Unlocked {
    PyThreadState *state = PyEval_SaveThread();

public:
    ~Unlocked() { PyEval_RestoreThread(state); }
};

void check(int code, const char *where)
{
    if (code == ATTN_OK) return;
    PyObject *r = PyObject_CallFunction(g_fail, "is", code, where);   // raises
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
    throw Refused{};
}

PyObject *wrap(const at::Tensor &t)
{
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

template <class... T>
PyObject *tuple(const T &...t)
{
    PyObject *r = PyTuple_New(sizeof...(T));
    if (!r) return nullptr;
    Py_ssize_t i = 0;
    ((void)PyTuple_SetItem(r, i++, wrap(t)), ...);
    if (PyErr_Occurred()) {
        Py_DECREF(r);
        return nullptr;
    }
    return r;
}

using Args = PyObject *const *;

// An entry of the module: the number of arguments, and C++ exceptions turned into Python's.
template <int N, PyObject *(*F)(Args)>
PyObject *entry(PyObject *, Args a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    try {
        return F(a);
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

bool flag(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v == 1;
}

int integer(PyObject *o)
{
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return (int)v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

// x, w, bias, residual, act, keep_z -> y or (y, z)
PyObject *linear_forward(Args a)
{
    const Rows x(a[0], "x", kBf16);
    const int64_t N = matrix_columns(a[1], "w");
    const c10::DimVector shape = x.with(N);
    const void *w = operand(a[1], "w", kBf16, {x.width, N}, x.dev);
    const auto *bias = static_cast<const float *>(operand_or_null(a[2], "bias", kF32, {N}, x.dev));
    const void *res = operand_or_null(a[3], "residual", kBf16, shape, x.dev);
    const auto act = static_cast<attn_activation>(integer(a[4]));
    const bool keep = flag(a[5]);
    at::Tensor y, z;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        y = empty(shape, kBf16, x.dev);
        if (keep) z = empty(shape, kBf16, x.dev);
        code = attn_linear(x.t.data_ptr(), w, bias, res, y.data_ptr(), at_or_null(z), count(x.M), count(x.width),
                           count(N), act, stream(x.dev));
    }
    check(code, "attn_linear");
    return keep ? tuple(y, z) : wrap(y);
}

// x, w, dy, z, act, bias, need_dx, need_dw -> (dx, dw, dbias)
PyObject *linear_backward(Args a)
{
    const Rows x(a[0], "x", kBf16);
    const int64_t N = matrix_columns(a[1], "w");
    const c10::DimVector shape = x.with(N);
    const void *w = operand(a[1], "w", kBf16, {x.width, N}, x.dev), *dy = operand(a[2], "dy", kBf16, shape, x.dev);
    const auto act = static_cast<attn_activation>(integer(a[4]));
    const void *z = act == ATTN_ACT_NONE ? nullptr : operand_or_null(a[3], "z", kBf16, shape, x.dev);
    if (act != ATTN_ACT_NONE && a[3] == Py_None)
        refuse("linear_backward needs the pre-activation z that linear_forward(keep_z=True) returns");
    const bool bias = flag(a[5]), need_dx = flag(a[6]), need_dw = flag(a[7]);
    at::Tensor dx, dw, db;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        if (need_dx) dx = empty(x.t.sizes(), kBf16, x.dev);
        if (need_dw) dw = empty({x.width, N}, kBf16, x.dev);
        if (bias) db = empty({N}, kF32, x.dev);
        const size_t bytes = attn_linear_bwd_workspace_size(count(x.M), count(x.width), count(N), act);
        const at::Tensor ws = empty({(int64_t)(bytes ? bytes : 1)}, at::kByte, x.dev);
        code = attn_linear_bwd(x.t.data_ptr(), w, dy, z, at_or_null(dx), at_or_null(dw),
                               static_cast<float *>(at_or_null(db)), ws.data_ptr(), bytes, count(x.M), count(x.width),
                               count(N), act, stream(x.dev));
    }
    check(code, "attn_linear_bwd");
    return tuple(dx, dw, db);
}

// Attention's [B, H, N, d_k].
struct Heads {
    const at::Tensor &t;
    c10::Device dev;
    int64_t B, H, N, d;
    explicit Heads(PyObject *o) : t(tensor(o, "o")), dev(t.device())
    {
        if (t.dim() != 4 || !t.is_cuda() || t.scalar_type() != kBf16 || !t.is_contiguous())
            refuse("o: expected a contiguous bf16 CUDA tensor [B, H, N, d_k]");
        B = t.size(0);
        H = t.size(1);
        N = t.size(2);
        d = t.size(3);
    }
};

// o, w, bias, residual -> y
PyObject *out_proj_forward(Args a)
{
    const Heads o(a[0]);
    const int64_t N = matrix_columns(a[1], "w");
    const void *w = operand(a[1], "w", kBf16, {o.H * o.d, N}, o.dev);
    const auto *bias = static_cast<const float *>(operand_or_null(a[2], "bias", kF32, {N}, o.dev));
    const void *res = operand_or_null(a[3], "residual", kBf16, {o.B, o.N, N}, o.dev);
    at::Tensor y;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(o.dev);
        y = empty({o.B, o.N, N}, kBf16, o.dev);
        code = attn_out_proj(o.t.data_ptr(), w, bias, res, y.data_ptr(), count(o.B), count(o.H), count(o.N), count(o.d),
                             count(N), stream(o.dev));
    }
    check(code, "attn_out_proj");
    return wrap(y);
}

// o, w, dy, bias, need_do, need_dw -> (do, dw, dbias)
PyObject *out_proj_backward(Args a)
{
    const Heads o(a[0]);
    const int64_t N = matrix_columns(a[1], "w");
    const void *w = operand(a[1], "w", kBf16, {o.H * o.d, N}, o.dev),
               *dy = operand(a[2], "dy", kBf16, {o.B, o.N, N}, o.dev);
    const bool bias = flag(a[3]), need_do = flag(a[4]), need_dw = flag(a[5]);
    at::Tensor d_o, dw, db;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(o.dev);
        if (need_do) d_o = empty(o.t.sizes(), kBf16, o.dev);
        if (need_dw) dw = empty({o.H * o.d, N}, kBf16, o.dev);
        if (bias) db = empty({N}, kF32, o.dev);
        const size_t bytes =
            attn_out_proj_bwd_workspace_size(count(o.B), count(o.H), count(o.N), count(o.d), count(N));
        const at::Tensor ws = empty({(int64_t)(bytes ? bytes : 1)}, at::kByte, o.dev);
        code = attn_out_proj_bwd(o.t.data_ptr(), w, dy, at_or_null(d_o), at_or_null(dw),
                                 static_cast<float *>(at_or_null(db)), ws.data_ptr(), bytes, count(o.B), count(o.H),
                                 count(o.N), count(o.d), count(N), stream(o.dev));
    }
    check(code, "attn_out_proj_bwd");
    return tuple(d_o, dw, db);
}

// xq, x_scale, wq, w_scale, bias, residual, act -> y
PyObject *linear_q8(Args a)
{
    const Rows x(a[0], "xq", kE4m3);
    matrix_columns(a[2], "wq");
    const int64_t N = THPVariable_Unpack(a[2]).size(0);
    const c10::DimVector shape = x.with(N);
    void *xs = operand(a[1], "x_scale", kF32, x.lead(), x.dev);
    const void *w = operand(a[2], "wq", kE4m3, {N, x.width}, x.dev);
    const auto *ws = static_cast<const float *>(operand(a[3], "w_scale", kF32, {N}, x.dev));
    const auto *bias = static_cast<const float *>(operand_or_null(a[4], "bias", kF32, {N}, x.dev));
    const void *res = operand_or_null(a[5], "residual", kBf16, shape, x.dev);
    const auto act = static_cast<attn_activation>(integer(a[6]));
    at::Tensor y, copy;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        y = empty(shape, kBf16, x.dev);
        code = attn_linear_q8(x.t.data_ptr(), aligned(xs, a[1], copy), w, ws, bias, res, y.data_ptr(), count(x.M), count(x.width), count(N),
                              act, stream(x.dev));
    }
    check(code, "attn_linear_q8");
    return wrap(y);
}

// x, weight, residual, eps -> (y, h or None, rstd)
PyObject *rms_norm_forward(Args a)
{
    const Rows x(a[0], "x", kBf16);
    const auto *weight = static_cast<const float *>(operand(a[1], "weight", kF32, {x.width}, x.dev));
    const void *res = operand_or_null(a[2], "residual", kBf16, x.t.sizes(), x.dev);
    const auto eps = (float)number(a[3]);
    at::Tensor y, h, rstd;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        y = empty(x.t.sizes(), kBf16, x.dev);
        if (res || a[2] != Py_None) h = empty(x.t.sizes(), kBf16, x.dev);
        rstd = empty(x.lead(), kF32, x.dev);
        code = attn_rms_norm(x.t.data_ptr(), res, weight, y.data_ptr(), at_or_null(h),
                             static_cast<float *>(rstd.data_ptr()), count(x.M), count(x.width), eps, stream(x.dev));
    }
    check(code, "attn_rms_norm");
    return tuple(y, h, rstd);
}

// dy, h, weight, rstd, dh -> (dx, dweight)
PyObject *rms_norm_backward(Args a)
{
    const Rows h(a[1], "h", kBf16);
    const void *dy = operand(a[0], "dy", kBf16, h.t.sizes(), h.dev);
    const auto *weight = static_cast<const float *>(operand(a[2], "weight", kF32, {h.width}, h.dev));
    void *rstd = operand(a[3], "rstd", kF32, h.lead(), h.dev);
    const void *dh = operand_or_null(a[4], "dh", kBf16, h.t.sizes(), h.dev);
    at::Tensor dx, dweight, copy;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(h.dev);
        dx = empty(h.t.sizes(), kBf16, h.dev);
        dweight = empty({h.width}, kF32, h.dev);
        const size_t bytes = attn_rms_norm_bwd_workspace_size(count(h.M), count(h.width));
        const at::Tensor ws = empty({(int64_t)(bytes ? bytes : 1)}, at::kByte, h.dev);
        code = attn_rms_norm_bwd(dy, h.t.data_ptr(), weight, aligned(rstd, a[3], copy), dh, dx.data_ptr(),
                                 static_cast<float *>(dweight.data_ptr()), ws.data_ptr(), bytes, count(h.M),
                                 count(h.width), stream(h.dev));
    }
    check(code, "attn_rms_norm_bwd");
    return tuple(dx, dweight);
}

// x, weight, residual, eps -> (yq, scale, h or None)
PyObject *rms_norm_q8(Args a)
{
    const Rows x(a[0], "x", kBf16);
    const auto *weight = static_cast<const float *>(operand(a[1], "weight", kF32, {x.width}, x.dev));
    const void *res = operand_or_null(a[2], "residual", kBf16, x.t.sizes(), x.dev);
    const auto eps = (float)number(a[3]);
    at::Tensor yq, scale, h;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        yq = empty(x.t.sizes(), kE4m3, x.dev);
        scale = empty(x.lead(), kF32, x.dev);
        if (res || a[2] != Py_None) h = empty(x.t.sizes(), kBf16, x.dev);
        code = attn_rms_norm_q8(x.t.data_ptr(), res, weight, yq.data_ptr(), static_cast<float *>(scale.data_ptr()),
                                at_or_null(h), count(x.M), count(x.width), eps, stream(x.dev));
    }
    check(code, "attn_rms_norm_q8");
    return tuple(yq, scale, h);
}

// x -> (xq, scale)
PyObject *quantize_q8(Args a)
{
    const Rows x(a[0], "x", kBf16);
    at::Tensor xq, scale;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        xq = empty(x.t.sizes(), kE4m3, x.dev);
        scale = empty(x.lead(), kF32, x.dev);
        code = attn_quantize_q8(x.t.data_ptr(), xq.data_ptr(), static_cast<float *>(scale.data_ptr()), count(x.M),
                                count(x.width), stream(x.dev));
    }
    check(code, "attn_quantize_q8");
    return tuple(xq, scale);
}

// A callable that raises AttnError(code, where).
PyObject *set_error(PyObject *, PyObject *callable)
{
    Py_XDECREF(g_fail);
    Py_INCREF(callable);
    g_fail = callable;
    Py_RETURN_NONE;
}

#define ENTRY(name, n) {#name, (PyCFunction)(void *)entry<n, name>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(linear_forward, 6),
                         ENTRY(linear_backward, 8),
                         ENTRY(out_proj_forward, 4),
                         ENTRY(out_proj_backward, 6),
                         ENTRY(linear_q8, 7),
                         ENTRY(rms_norm_forward, 4),
                         ENTRY(rms_norm_backward, 5),
                         ENTRY(rms_norm_q8, 4),
                         ENTRY(quantize_q8, 1),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() { return PyModule_Create(&module); }
