// The tensor-level calls of the linear layers, the norm, positions and the cache, as a CPython extension: argument checks,
// allocation of the outputs from PyTorch's caching allocator on the current stream, and one call of the
// C ABI (include/attn.h).  Nothing is computed here.  The same through Python and ctypes took 13 to 16
// us a call on the GB300's host, several times what the smallest kernels take on the GPU; this takes
// about 4.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
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
    return v != (int)v ? -1 : (int)v;
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

// [B, H, N, d_k] heads under a name.
struct HeadsOf {
    const at::Tensor &t;
    c10::Device dev;
    int64_t B, H, N, d;
    HeadsOf(PyObject *o, const char *name) : t(tensor(o, name)), dev(t.device())
    {
        if (t.dim() != 4 || !t.is_cuda() || t.scalar_type() != kBf16 || !t.is_contiguous())
            refuse(std::string(name) + ": expected a contiguous bf16 CUDA tensor [B, H, N, d_k]");
        B = t.size(0);
        H = t.size(1);
        N = t.size(2);
        d = t.size(3);
    }
};

constexpr auto kI32 = at::kInt, kI64 = at::kLong;

// The cache's calls have no backward: an operand that a graph is being recorded for is refused, not cut off from it.
void refuse_graph(std::initializer_list<PyObject *> operands, const char *what)
{
    if (!at::GradMode::is_enabled()) return;
    for (PyObject *o : operands)
        if (THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad())
            refuse(std::string(what) + " has no backward: run it under torch.no_grad(), or on detached tensors");
}

// What a call wrote in place: a recorded graph that saved such a tensor refuses its backward, as after PyTorch's own
// in-place operators.
void written(std::initializer_list<PyObject *> outputs)
{
    for (PyObject *o : outputs) {
        if (!THPVariable_Check(o)) continue;
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
}

// Turns a position of the pairs, [rotated / 2] int64 (the bits of the C ABI's uint64).
const uint64_t *turns_of(PyObject *o, c10::Device dev, int64_t &rotated)
{
    const at::Tensor &t = tensor(o, "turns");
    if (t.dim() != 1) refuse("turns: expected a vector, as rotary_turns() makes it");
    rotated = 2 * t.size(0);
    return static_cast<const uint64_t *>(operand(o, "turns", kI64, t.sizes(), dev));
}

// x, turns, positions or None, interleaved, amplitude, backward -> y
PyObject *rotary(Args a)
{
    const HeadsOf x(a[0], "x");
    int64_t rotated;
    const uint64_t *turns = turns_of(a[1], x.dev, rotated);
    const int *positions = nullptr;
    int64_t stride = 0;
    if (a[2] != Py_None) {
        const bool each = tensor(a[2], "positions").dim() == 2;
        const c10::DimVector shape = each ? c10::DimVector{x.B, x.N} : c10::DimVector{x.N};
        positions = static_cast<const int *>(operand(a[2], "positions", kI32, shape, x.dev));
        stride = each ? x.N : 0;
    }
    const int interleaved = flag(a[3]);
    const auto amplitude = (float)number(a[4]);
    const bool backward = flag(a[5]);
    at::Tensor y;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(x.dev);
        y = empty(x.t.sizes(), kBf16, x.dev);
        code = (backward ? attn_rotary_bwd : attn_rotary)(x.t.data_ptr(), y.data_ptr(), positions, stride, turns,
                                                          count(x.B), count(x.H), count(x.N), count(x.d),
                                                          count(rotated), interleaved, amplitude, stream(x.dev));
    }
    check(code, backward ? "attn_rotary_bwd" : "attn_rotary");
    return wrap(y);
}

// k, v, cache_k, cache_v, lengths, turns, positions, interleaved, amplitude, rows, q, weights, slot_positions
// -> q turned, or None
PyObject *cache_append(Args a)
{
    const HeadsOf k(a[0], "k"), ck(a[2], "cache_k");
    refuse_graph({a[0], a[1], a[2], a[3], a[10], a[11]}, "cache_append");
    const void *v = operand(a[1], "v", kBf16, k.t.sizes(), k.dev);
    if (ck.dev != k.dev || ck.B != k.B || ck.H != k.H || ck.d != k.d)
        refuse("cache_k: expected [" + std::to_string(k.B) + ", " + std::to_string(k.H) + ", C, " +
               std::to_string(k.d) + "] on " + k.dev.str());
    void *cv = operand(a[3], "cache_v", kBf16, ck.t.sizes(), k.dev);
    const auto *lengths = static_cast<const int *>(operand(a[4], "lengths", kI32, {k.B}, k.dev));
    int64_t rotated = 0, n = k.N, Hq = 0;
    const uint64_t *turns = a[5] == Py_None ? nullptr : turns_of(a[5], k.dev, rotated);
    const auto *positions = static_cast<const int *>(operand_or_null(a[6], "positions", kI32, {k.B, k.N}, k.dev));
    const int interleaved = flag(a[7]);
    const auto amplitude = (float)number(a[8]);
    const int *rows = nullptr;
    if (a[9] != Py_None) {
        n = matrix_columns(a[9], "rows");
        rows = static_cast<const int *>(operand(a[9], "rows", kI32, {k.B, n}, k.dev));
    }
    const void *q = nullptr;
    at::Tensor q_out;
    if (a[10] != Py_None) {
        const HeadsOf heads(a[10], "q");
        Hq = heads.H;
        q = operand(a[10], "q", kBf16, {k.B, Hq, k.N, k.d}, k.dev);
        if (rows) refuse("q: the queries of all tokens are turned, `rows` takes some of them");
    }
    auto *weights = static_cast<float *>(operand_or_null(a[11], "weights", kF32, {k.B, k.H, ck.N}, k.dev));
    auto *slots = static_cast<int *>(operand_or_null(a[12], "slot_positions", kI32, {k.B, k.H, ck.N}, k.dev));
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(k.dev);
        if (a[10] != Py_None) q_out = empty({k.B, Hq, k.N, k.d}, kBf16, k.dev);
        code = attn_cache_append(k.t.data_ptr(), v, ck.t.data_ptr(), cv, lengths, turns, positions, rows, q,
                                 at_or_null(q_out), weights, slots, count(k.B), count(k.H), count(Hq), count(k.N),
                                 count(n), count(k.d), count(ck.N), count(rotated), interleaved, amplitude,
                                 stream(k.dev));
    }
    check(code, "attn_cache_append");
    written({a[2], a[3], a[11], a[12]});
    return wrap(q_out);
}

// q, cache_k, cache_v, lengths, tree, weights, counted, weights_out, scale or None -> (o, lse), and weights_out with weights
PyObject *cache_attention(Args a)
{
    const HeadsOf q(a[0], "q"), k(a[1], "cache_k");
    refuse_graph({a[0], a[1], a[2], a[5], a[7]}, "cache_attention");
    if (k.dev != q.dev || k.B != q.B || k.d != q.d || k.H < 1 || q.H % k.H)
        refuse("cache_k: expected [" + std::to_string(q.B) + ", H, C, " + std::to_string(q.d) + "] on " + q.dev.str() +
               ", H a divisor of q's " + std::to_string(q.H) + " heads, got " + describe(k.t.sizes()) + " on " +
               k.dev.str());
    const void *v = operand(a[2], "cache_v", kBf16, k.t.sizes(), q.dev);
    const auto *lengths = static_cast<const int *>(operand(a[3], "lengths", kI32, {q.B}, q.dev));
    const auto *tree = static_cast<const uint64_t *>(operand_or_null(a[4], "tree", kI64, {q.B, q.N}, q.dev));
    const auto *weights = static_cast<const float *>(operand_or_null(a[5], "weights", kF32, {k.B, k.H, k.N}, q.dev));
    const auto *counted = static_cast<const uint64_t *>(operand_or_null(a[6], "counted", kI64, {q.B}, q.dev));
    auto *given = static_cast<float *>(operand_or_null(a[7], "weights_out", kF32, {k.B, k.H, k.N}, q.dev));
    if (a[5] == Py_None && a[7] != Py_None) refuse("weights_out goes with weights");
    const auto scale = (float)(a[8] == Py_None ? 1.0 / std::sqrt((double)q.d) : number(a[8]));
    const bool fresh = a[5] != Py_None && a[7] == Py_None;
    at::Tensor o, lse, out;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(q.dev);
        o = empty(q.t.sizes(), kBf16, q.dev);
        lse = empty({q.B, q.H, q.N}, kF32, q.dev);
        if (fresh) out = empty({k.B, k.H, k.N}, kF32, q.dev);
        const int G = count(q.H / k.H);
        const size_t bytes =
            attn_cache_attention_workspace_size(count(q.B), count(k.H), G, count(q.N), count(k.N), count(q.d), weights != nullptr);
        at::Tensor ws;
        if (bytes) ws = empty({(int64_t)bytes}, at::kByte, q.dev);
        code = attn_cache_attention(q.t.data_ptr(), k.t.data_ptr(), v, lengths, tree, counted, weights,
                                    fresh ? static_cast<float *>(out.data_ptr()) : given, o.data_ptr(),
                                    static_cast<float *>(lse.data_ptr()), at_or_null(ws), bytes, count(q.B),
                                    count(k.H), G, count(q.N), count(k.N), count(q.d), scale, stream(q.dev));
    }
    check(code, "attn_cache_attention");
    written({a[7]});
    if (a[5] == Py_None) return tuple(o, lse);
    if (a[7] == Py_None) return tuple(o, lse, out);
    return tuple(o, lse, THPVariable_Unpack(a[7]));
}

// cache_k, cache_v, weights, slot_positions, lengths, keep, recent, weights_out, positions_out
// -> (weights_out, positions_out, lengths_out)
PyObject *cache_evict(Args a)
{
    const HeadsOf k(a[0], "cache_k");
    refuse_graph({a[0], a[1], a[2], a[7]}, "cache_evict");
    void *v = operand(a[1], "cache_v", kBf16, k.t.sizes(), k.dev);
    const c10::DimVector slots{k.B, k.H, k.N};
    const auto *weights = static_cast<const float *>(operand(a[2], "weights", kF32, slots, k.dev));
    const auto *positions = static_cast<const int *>(operand(a[3], "slot_positions", kI32, slots, k.dev));
    const auto *lengths = static_cast<const int *>(operand(a[4], "lengths", kI32, {k.B}, k.dev));
    const int keep = integer(a[5]), recent = integer(a[6]);
    auto *w_given = static_cast<float *>(operand_or_null(a[7], "weights_out", kF32, slots, k.dev));
    auto *p_given = static_cast<int *>(operand_or_null(a[8], "positions_out", kI32, slots, k.dev));
    at::Tensor w, p, n;
    int code;
    {
        Unlocked u;
        const c10::cuda::CUDAGuard guard(k.dev);
        if (a[7] == Py_None) w = empty(slots, kF32, k.dev);
        if (a[8] == Py_None) p = empty(slots, kI32, k.dev);
        n = empty({k.B}, kI32, k.dev);
        const size_t bytes = attn_cache_evict_workspace_size(count(k.B), count(k.H), count(k.N), count(k.d), keep);
        at::Tensor ws;
        if (bytes) ws = empty({(int64_t)bytes}, at::kByte, k.dev);
        code = attn_cache_evict(k.t.data_ptr(), v, weights, positions, lengths,
                                w_given || !w.defined() ? w_given : static_cast<float *>(w.data_ptr()),
                                p_given || !p.defined() ? p_given : static_cast<int *>(p.data_ptr()),
                                static_cast<int *>(n.data_ptr()), at_or_null(ws), bytes, count(k.B), count(k.H),
                                count(k.N), count(k.d), keep, recent, stream(k.dev));
    }
    check(code, "attn_cache_evict");
    written({a[0], a[1], a[7], a[8]});
    return tuple(a[7] == Py_None ? w : THPVariable_Unpack(a[7]), a[8] == Py_None ? p : THPVariable_Unpack(a[8]), n);
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
                         ENTRY(rotary, 6),
                         ENTRY(cache_append, 13),
                         ENTRY(cache_attention, 9),
                         ENTRY(cache_evict, 9),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
#undef ENTRY

PyModuleDef module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_attn_binding() { return PyModule_Create(&module); }
