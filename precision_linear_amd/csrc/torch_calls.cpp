// The binding's short calls: a Python extension that takes the ordinary call of
// an operator (outputs allocated here, automatic plan, no workspace given) from torch tensors to the C ABI in one step.
//
// A small call's time is the host's, and what binding.py does for it, attribute
// by attribute, costs 5 to 7 us beside the 4 us of a launch.  Host time of a
// call, there and here (MI355X's host, one row of 64 columns): linear 9.2 and
// 4.3 us, layer norm with its statistics 10.0 and 5.2, its gradient 11.6 and 5.4,
// linear's gradient (three launches) 20.1 and 13.0.  What is left beside the
// launches is the tensors of outputs and scratch memory, some 0.5 us each.
//
// Each function returns the outputs as a tuple, the library's status where it
// refuses the call, or None where an argument is not the ordinary one: wrong
// ones and the less usual forms are binding.py's to refuse or to run.  Nothing
// is enqueued before that is known.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/ops/empty_cuda_dispatch.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstring>
#include <vector>

#include "../../include/adamw.h"
#include "../../include/fp8_cross_entropy.h"
#include "../../include/fp8_layer_norm.h"
#include "../../include/fp8_linear.h"
#include "../../include/fp8_quantize_weight.h"

namespace {

// The library's entry points (binding.py gives their addresses once it has
// loaded the library).
struct Library {
    decltype(&fp8_layer_norm) norm;
    decltype(&fp8_layer_norm_backward) norm_backward;
    decltype(&fp8_layer_norm_backward_workspace_size) norm_backward_workspace;
    decltype(&fp8_linear) linear;
    decltype(&fp8_scaled_mm_workspace_size) mm_workspace;
    decltype(&fp8_linear_backward) linear_backward;
    decltype(&fp8_linear_backward_workspace_size) linear_backward_workspace;
    decltype(&fp8_linear_cross_entropy) cross_entropy;
    decltype(&fp8_linear_cross_entropy_workspace_size) cross_entropy_workspace;
    decltype(&fp8_linear_cross_entropy_backward) cross_entropy_backward;
    decltype(&fp8_linear_cross_entropy_backward_workspace_size) cross_entropy_backward_workspace;
    decltype(&fp8_quantize_weight) quantize_weight;
    decltype(&fp8_quantize_weight_workspace_size) quantize_weight_workspace;
    decltype(&adamw_step) adamw;
};
Library g_lib{};
PyObject* g_workspace = nullptr;   // binding._workspace(device, stream, bytes, kind)

// A tensor argument as it must be; null: `None`.
struct Arg {
    const at::Tensor* t = nullptr;
    bool given = false, ok = true;
    explicit Arg(PyObject* o) {
        if (o == Py_None) return;
        given = true;
        ok = THPVariable_CheckExact(o);
        if (ok) t = &THPVariable_Unpack(o);
    }
    // On GPU `dev`, contiguous.
    bool on(int dev) const { return ok && given && t->is_cuda() && t->get_device() == dev && t->is_contiguous(); }
    bool matrix(int dev, at::ScalarType type, int64_t rows, int64_t cols) const {
        return on(dev) && t->scalar_type() == type && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols;
    }
    bool vector(int dev, at::ScalarType type, int64_t n) const {
        return on(dev) && t->scalar_type() == type && t->numel() == n;
    }
    void* ptr() const { return t ? t->data_ptr() : nullptr; }
};
// `None`, or as the check says.
#define OPTIONAL_ARG(a, check) (!(a).given || (a).check)

// The stored format of an operand's codes, or -1.
int code_format(const at::Tensor& t) {
    switch (t.scalar_type()) {
        case at::kFloat8_e4m3fn:
        case at::kByte: return FP8MM_E4M3FN;
        case at::kFloat8_e5m2: return FP8MM_E5M2;
        default: return -1;
    }
}

// The GPU of a call's first tensor, if it is the current one (the library
// launches there), or -1.
int device_of(const Arg& a) {
    if (!a.ok || !a.given || !a.t->is_cuda()) return -1;
    const int dev = a.t->get_device();
    return c10::hip::current_device() == dev ? dev : -1;
}

at::Tensor allocate(const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
    return at::cuda::empty(shape, type, {}, like.device(), {}, {});
}

PyObject* pass(const at::Tensor& t) {
    if (t.defined()) return THPVariable_Wrap(t);
    Py_RETURN_NONE;
}

template <size_t N>
PyObject* tuple_of(const at::Tensor (&t)[N]) {
    PyObject* out = PyTuple_New(N);
    if (!out) return nullptr;
    for (size_t i = 0; i < N; ++i) {
        PyObject* o = pass(t[i]);
        if (!o) {
            Py_DECREF(out);
            return nullptr;
        }
        PyTuple_SET_ITEM(out, i, o);
    }
    return out;
}

// Workspaces that binding.py has handed out, by GPU, stream and kind.  They are
// its own (it never frees one); the reference here only keeps the address valid.
// While a graph is captured, binding.py is asked each time: a capture has its own.
enum Kind { kMm, kNorm };
const char* const kKindNames[] = {"mm", "layer_norm"};
struct Workspace {
    int dev;
    hipStream_t stream;
    Kind kind;
    at::Tensor t;
};

// False: a Python error is set.
bool workspace(int dev, hipStream_t stream, Kind kind, int64_t bytes, const at::Tensor& like, void** out) {
    static std::vector<Workspace>* held = new std::vector<Workspace>;   // (not destroyed after the interpreter)
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    const bool eager = hipStreamIsCapturing(stream, &capture) != hipSuccess || capture == hipStreamCaptureStatusNone;
    for (Workspace& w : *held)
        if (eager && w.dev == dev && w.stream == stream && w.kind == kind) {
            if (w.t.numel() >= bytes) {
                *out = w.t.data_ptr();
                return true;
            }
            w = held->back();
            held->pop_back();
            break;
        }
    PyObject* device = THPDevice_New(like.device());
    if (!device) return false;
    PyObject* r = PyObject_CallFunction(g_workspace, "NKLs", device, (unsigned long long)(uintptr_t)stream,
                                        (long long)bytes, kKindNames[kind]);
    if (!r) return false;
    *out = THPVariable_Unpack(r).data_ptr();
    if (eager) held->push_back(Workspace{dev, stream, kind, THPVariable_Unpack(r)});
    Py_DECREF(r);
    return true;
}

bool is_flag(PyObject* o, bool* v) {
    *v = o == Py_True;
    return o == Py_True || o == Py_False;
}

// None for w or b, or a vector of them: the ABI's type in *type.
bool norm_param(const Arg& a, int dev, int64_t cols, int* type) {
    if (!a.given) return true;
    if (!a.on(dev) || a.t->numel() != cols) return false;
    const at::ScalarType s = a.t->scalar_type();
    if (s != at::kFloat && s != at::kBFloat16) return false;
    const int code = s == at::kFloat ? FP8LN_FP32 : FP8LN_BF16;
    const bool agrees = *type < 0 || *type == code;
    *type = code;
    return agrees;
}

// (x, w, b, eps, y, format or -1, stats) -> (y, q, scale, mean, rstd)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7 || !g_lib.norm) Py_RETURN_NONE;
    const Arg x(a[0]), w(a[1]), b(a[2]);
    bool want_y, stats;
    const int dev = device_of(x);
    if (dev < 0 || !PyFloat_CheckExact(a[3]) || !is_flag(a[4], &want_y) || !PyLong_CheckExact(a[5]) ||
        !is_flag(a[6], &stats))
        Py_RETURN_NONE;
    const double eps = PyFloat_AS_DOUBLE(a[3]);
    const long format = PyLong_AsLong(a[5]);
    const at::ScalarType type = x.t->scalar_type();
    if (!(eps >= 0.0) || std::isinf(eps) || format < -1 || format > 1 || (!want_y && format < 0) ||
        (type != at::kBFloat16 && type != at::kFloat) || x.t->dim() != 2 || !x.t->is_contiguous())
        Py_RETURN_NONE;
    const int64_t rows = x.t->size(0), cols = x.t->size(1);
    int param = -1;
    if (rows == 0 || cols == 0 || (format >= 0 && cols % 16 != 0) || !norm_param(w, dev, cols, &param) ||
        !norm_param(b, dev, cols, &param))
        Py_RETURN_NONE;
    at::Tensor out[5];
    if (want_y) out[0] = allocate(*x.t, {rows, cols}, type);
    if (format >= 0) {
        out[1] = allocate(*x.t, {rows, cols}, at::kByte);
        out[2] = allocate(*x.t, {rows}, at::kFloat);
    }
    if (stats) {
        out[3] = allocate(*x.t, {rows}, at::kFloat);
        out[4] = allocate(*x.t, {rows}, at::kFloat);
    }
    auto f32 = [](const at::Tensor& t) { return t.defined() ? t.data_ptr<float>() : nullptr; };
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.norm(x.ptr(), type == at::kFloat ? FP8LN_FP32 : FP8LN_BF16, w.ptr(), b.ptr(),
                        param < 0 ? FP8LN_FP32 : param, (float)eps, out[0].defined() ? out[0].data_ptr() : nullptr,
                        out[1].defined() ? out[1].data_ptr() : nullptr, format < 0 ? 0 : (int)format, f32(out[2]),
                        f32(out[3]), f32(out[4]), rows, cols, reinterpret_cast<ihipStream_t*>(stream));
    }
    if (st != FP8LN_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (dy, x, mean, rstd, w, residual_grad) -> (dx, dw, db)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6 || !g_lib.norm) Py_RETURN_NONE;
    const Arg dy(a[0]), x(a[1]), mean(a[2]), rstd(a[3]), w(a[4]), res(a[5]);
    const int dev = device_of(x);
    if (dev < 0) Py_RETURN_NONE;
    const at::ScalarType type = x.t->scalar_type();
    if ((type != at::kBFloat16 && type != at::kFloat) || x.t->dim() != 2 || !x.t->is_contiguous()) Py_RETURN_NONE;
    const int64_t rows = x.t->size(0), cols = x.t->size(1);
    int param = -1;
    if (rows == 0 || cols == 0 || !dy.matrix(dev, type, rows, cols) || !mean.vector(dev, at::kFloat, rows) ||
        !rstd.vector(dev, at::kFloat, rows) || !norm_param(w, dev, cols, &param) ||
        !OPTIONAL_ARG(res, matrix(dev, type, rows, cols)))
        Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const int64_t need = g_lib.norm_backward_workspace(rows, cols);
    void* ws = nullptr;
    if (need > 0 && !workspace(dev, stream, kNorm, need, *x.t, &ws)) return nullptr;
    at::Tensor out[3];
    out[0] = allocate(*x.t, {rows, cols}, type);
    out[1] = allocate(*x.t, {cols}, at::kFloat);
    out[2] = allocate(*x.t, {cols}, at::kFloat);
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.norm_backward(dy.ptr(), x.ptr(), type == at::kFloat ? FP8LN_FP32 : FP8LN_BF16,
                                 static_cast<const float*>(mean.ptr()), static_cast<const float*>(rstd.ptr()),
                                 w.ptr(), param < 0 ? FP8LN_FP32 : param, res.ptr(), out[0].data_ptr(),
                                 out[1].data_ptr<float>(), out[2].data_ptr<float>(), rows, cols, ws, need,
                                 reinterpret_cast<ihipStream_t*>(stream));
    }
    if (st != FP8LN_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (a, b, scale_a, scale_b, bias, residual, activation, preact, mode) -> (out,)
PyObject* linear(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 9 || !g_lib.norm) Py_RETURN_NONE;
    const Arg a(arg[0]), b(arg[1]), sa(arg[2]), sb(arg[3]), bias(arg[4]), res(arg[5]), pre(arg[7]);
    const int dev = device_of(a);
    if (dev < 0 || !PyLong_CheckExact(arg[6]) || !PyLong_CheckExact(arg[8])) Py_RETURN_NONE;
    const int act = (int)PyLong_AsLong(arg[6]), mode = (int)PyLong_AsLong(arg[8]);
    if (!a.on(dev) || !b.on(dev) || a.t->dim() != 2 || b.t->dim() != 2) Py_RETURN_NONE;
    const int64_t M = a.t->size(0), K = a.t->size(1), N = b.t->size(0);
    const int fa = code_format(*a.t), fb = code_format(*b.t);
    const bool rowwise = mode == FP8MM_ROWWISE;
    if (M == 0 || N == 0 || b.t->size(1) != K || fa < 0 || fb < 0 || (!rowwise && mode != FP8MM_PER_TENSOR) ||
        !sa.vector(dev, at::kFloat, rowwise ? M : 1) || !sb.vector(dev, at::kFloat, rowwise ? N : 1) ||
        !OPTIONAL_ARG(bias, vector(dev, at::kBFloat16, N)) ||
        !OPTIONAL_ARG(res, matrix(dev, at::kBFloat16, M, N)) || !OPTIONAL_ARG(pre, matrix(dev, at::kBFloat16, M, N)))
        Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const int64_t need = g_lib.mm_workspace(M, N, K, mode, bias.given, -1, 0);
    void* ws = nullptr;
    if (need > 0 && !workspace(dev, stream, kMm, need, *a.t, &ws)) return nullptr;
    at::Tensor out[1];
    out[0] = allocate(*a.t, {M, N}, at::kBFloat16);
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.linear(a.ptr(), fa, b.ptr(), fb, static_cast<const float*>(sa.ptr()),
                          static_cast<const float*>(sb.ptr()), bias.ptr(), res.ptr(), act, pre.ptr(),
                          out[0].data_ptr(), M, N, K, mode, reinterpret_cast<ihipStream_t*>(stream), -1, 0, ws,
                          need > 0 ? need : 0);
    }
    if (st != FP8MM_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (dy, x, wt, wt_scale, z, activation) -> (dx, dw, dbias)
PyObject* linear_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 6 || !g_lib.norm) Py_RETURN_NONE;
    const Arg dy(a[0]), x(a[1]), wt(a[2]), swt(a[3]), z(a[4]);
    const int dev = device_of(dy);
    if (dev < 0 || !PyLong_CheckExact(a[5])) Py_RETURN_NONE;
    const int act = (int)PyLong_AsLong(a[5]);
    if (!x.on(dev) || !wt.on(dev) || dy.t->dim() != 2 || x.t->dim() != 2) Py_RETURN_NONE;
    const int64_t M = dy.t->size(0), N = dy.t->size(1), K = x.t->size(1);
    const int fw = code_format(*wt.t);
    if (M == 0 || N < 16 || N % 16 != 0 || K < 16 || K % 16 != 0 || fw < 0 || wt.t->dim() != 2 ||
        wt.t->size(0) != K || wt.t->size(1) != N || !dy.matrix(dev, at::kBFloat16, M, N) ||
        !x.matrix(dev, at::kBFloat16, M, K) || !swt.vector(dev, at::kFloat, K) ||
        !OPTIONAL_ARG(z, matrix(dev, at::kBFloat16, M, N)) || (act != FP8MM_ACT_NONE && !z.given))
        Py_RETURN_NONE;
    const int64_t need = g_lib.linear_backward_workspace(M, N, K, 1, 1);
    if (need < 0) Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const at::Tensor ws = allocate(*dy.t, {need}, at::kByte);
    at::Tensor out[3];
    out[0] = allocate(*dy.t, {M, K}, at::kBFloat16);
    out[1] = allocate(*dy.t, {N, K}, at::kBFloat16);
    out[2] = allocate(*dy.t, {N}, at::kFloat);
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.linear_backward(dy.ptr(), x.ptr(), wt.ptr(), fw, static_cast<const float*>(swt.ptr()), z.ptr(),
                                   act, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr<float>(), M, N, K,
                                   reinterpret_cast<ihipStream_t*>(stream), ws.data_ptr(), need);
    }
    if (st != FP8MM_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (a, b, scale_a, scale_b, target, ignore_index, mode) -> (loss, lse)
PyObject* cross_entropy(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 7 || !g_lib.norm) Py_RETURN_NONE;
    const Arg a(arg[0]), b(arg[1]), sa(arg[2]), sb(arg[3]), target(arg[4]);
    const int dev = device_of(a);
    if (dev < 0 || !PyLong_CheckExact(arg[5]) || !PyLong_CheckExact(arg[6])) Py_RETURN_NONE;
    int overflow = 0;
    const int64_t ignore = PyLong_AsLongLongAndOverflow(arg[5], &overflow);
    const int mode = (int)PyLong_AsLong(arg[6]);
    if (overflow || !a.on(dev) || !b.on(dev) || a.t->dim() != 2 || b.t->dim() != 2) Py_RETURN_NONE;
    const int64_t M = a.t->size(0), K = a.t->size(1), V = b.t->size(0);
    const int fa = code_format(*a.t), fb = code_format(*b.t);
    const bool rowwise = mode == FP8MM_ROWWISE;
    if (M == 0 || b.t->size(1) != K || fa < 0 || fb < 0 || (!rowwise && mode != FP8MM_PER_TENSOR) ||
        !sa.vector(dev, at::kFloat, rowwise ? M : 1) || !sb.vector(dev, at::kFloat, rowwise ? V : 1) ||
        !target.vector(dev, at::kLong, M) || target.t->dim() != 1)
        Py_RETURN_NONE;
    const int64_t need = g_lib.cross_entropy_workspace(M, V, K);
    if (need < 0) Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const at::Tensor ws = allocate(*a.t, {need}, at::kByte);
    at::Tensor out[2];
    for (at::Tensor& t : out) t = allocate(*a.t, {M}, at::kFloat);
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.cross_entropy(a.ptr(), fa, b.ptr(), fb, static_cast<const float*>(sa.ptr()),
                                 static_cast<const float*>(sb.ptr()), static_cast<const int64_t*>(target.ptr()), ignore,
                                 out[0].data_ptr<float>(), out[1].data_ptr<float>(), M, V, K, mode,
                                 reinterpret_cast<ihipStream_t*>(stream), ws.data_ptr(), need);
    }
    if (st != FP8MM_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (dloss, a, b, scale_a, scale_b, target, loss, lse, x, wt, wt_scale, ignore_index,
// mode) -> (dx, dw)
PyObject* cross_entropy_backward(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 13 || !g_lib.norm) Py_RETURN_NONE;
    const Arg dl(arg[0]), a(arg[1]), b(arg[2]), sa(arg[3]), sb(arg[4]), target(arg[5]), loss(arg[6]), lse(arg[7]);
    const Arg x(arg[8]), wt(arg[9]), swt(arg[10]);
    const int dev = device_of(a);
    if (dev < 0 || !PyLong_CheckExact(arg[11]) || !PyLong_CheckExact(arg[12])) Py_RETURN_NONE;
    int overflow = 0;
    const int64_t ignore = PyLong_AsLongLongAndOverflow(arg[11], &overflow);
    const int mode = (int)PyLong_AsLong(arg[12]);
    if (overflow || !a.on(dev) || !b.on(dev) || a.t->dim() != 2 || b.t->dim() != 2 || !wt.on(dev)) Py_RETURN_NONE;
    const int64_t M = a.t->size(0), K = a.t->size(1), V = b.t->size(0), Vp = (V + 15) / 16 * 16;
    const int fa = code_format(*a.t), fb = code_format(*b.t), fw = code_format(*wt.t);
    const bool rowwise = mode == FP8MM_ROWWISE;
    if (M == 0 || V == 0 || b.t->size(1) != K || fa < 0 || fb < 0 || fw < 0 ||
        (!rowwise && mode != FP8MM_PER_TENSOR) || !sa.vector(dev, at::kFloat, rowwise ? M : 1) ||
        !sb.vector(dev, at::kFloat, rowwise ? V : 1) || !target.vector(dev, at::kLong, M) || target.t->dim() != 1 ||
        !dl.vector(dev, at::kFloat, M) || dl.t->dim() != 1 || !loss.vector(dev, at::kFloat, M) ||
        !lse.vector(dev, at::kFloat, M) || !x.matrix(dev, at::kBFloat16, M, K) || wt.t->dim() != 2 ||
        wt.t->size(0) != K || wt.t->size(1) != Vp || !swt.vector(dev, at::kFloat, K))
        Py_RETURN_NONE;
    const int64_t need = g_lib.cross_entropy_backward_workspace(M, V, K, 1, 1);
    if (need < 0) Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const at::Tensor ws = allocate(*a.t, {need}, at::kByte);
    at::Tensor out[2];
    out[0] = allocate(*a.t, {M, K}, at::kBFloat16);
    out[1] = allocate(*a.t, {V, K}, at::kBFloat16);
    auto f32 = [](const Arg& t) { return static_cast<const float*>(t.ptr()); };
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.cross_entropy_backward(f32(dl), 1, a.ptr(), fa, b.ptr(), fb, f32(sa), f32(sb),
                                          static_cast<const int64_t*>(target.ptr()), ignore, f32(loss), f32(lse),
                                          x.ptr(), wt.ptr(), fw, f32(swt), out[0].data_ptr(), out[1].data_ptr(), M, V,
                                          K, mode, reinterpret_cast<ihipStream_t*>(stream), ws.data_ptr(), need);
    }
    if (st != FP8MM_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// (w, format) -> (q, scale, qt, scale_t)
PyObject* quantize_weight(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 2 || !g_lib.norm) Py_RETURN_NONE;
    const Arg w(arg[0]);
    const int dev = device_of(w);
    if (dev < 0 || !PyLong_CheckExact(arg[1]) || !w.on(dev) || w.t->dim() != 2) Py_RETURN_NONE;
    const at::ScalarType type = w.t->scalar_type();
    const int64_t N = w.t->size(0), K = w.t->size(1);
    if ((type != at::kBFloat16 && type != at::kFloat) || N == 0) Py_RETURN_NONE;
    const int64_t need = g_lib.quantize_weight_workspace(N, K);
    if (need < 0) Py_RETURN_NONE;
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    const at::Tensor ws = allocate(*w.t, {need}, at::kByte);
    at::Tensor out[4];
    out[0] = allocate(*w.t, {N, K}, at::kByte);
    out[1] = allocate(*w.t, {N}, at::kFloat);
    out[2] = allocate(*w.t, {K, (N + 15) / 16 * 16}, at::kByte);
    out[3] = allocate(*w.t, {K}, at::kFloat);
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.quantize_weight(w.ptr(), type == at::kFloat ? FP8W_FP32 : FP8W_BF16, (int)PyLong_AsLong(arg[1]),
                                   out[0].data_ptr(), out[1].data_ptr<float>(), out[2].data_ptr(),
                                   out[3].data_ptr<float>(), N, K, reinterpret_cast<ihipStream_t*>(stream),
                                   ws.data_ptr(), need);
    }
    if (st != FP8MM_OK) return PyLong_FromLong(st);
    return tuple_of(out);
    END_HANDLE_TH_ERRORS
}

// A list of tensors as adamw_step's must be: one for each parameter, of one type.  It is
// held as a tuple, whose tensors stay while the interpreter is free.
struct List {
    PyObject* held = nullptr;
    PyObject* const* items = nullptr;
    Py_ssize_t size = 0;
    bool given = false, ok = true;
    explicit List(PyObject* o) {
        if (o == Py_None) return;
        given = true;
        ok = PyList_CheckExact(o) || PyTuple_CheckExact(o);
        if (!ok) return;
        held = PySequence_Tuple(o);
        if (!held) {
            PyErr_Clear();
            ok = false;
            return;
        }
        items = PySequence_Fast_ITEMS(held);
        size = PyTuple_GET_SIZE(held);
    }
    List(const List&) = delete;
    ~List() { Py_XDECREF(held); }
    // Their contents have changed: what torch's graphs saved of them before is no longer there.
    void written() const {
        for (Py_ssize_t i = 0; i < size; ++i) {
            c10::TensorImpl* t = THPVariable_Unpack(items[i]).unsafeGetTensorImpl();
            if (!t->is_inference()) t->bump_version();   // (those have no version)
        }
    }
    // Tensor i if it is on GPU `dev`, contiguous and of `type`, else null.
    const at::Tensor* get(Py_ssize_t i, int dev, at::ScalarType type) const {
        if (!THPVariable_CheckExact(items[i]) && !THPVariable_Check(items[i])) return nullptr;
        const at::Tensor& t = THPVariable_Unpack(items[i]);
        return t.is_cuda() && t.get_device() == dev && t.is_contiguous() && t.scalar_type() == type ? &t : nullptr;
    }
    at::ScalarType type() const {
        return size > 0 && THPVariable_Check(items[0]) ? THPVariable_Unpack(items[0]).scalar_type() : at::kDouble;
    }
};

// A number, or a tensor of one element on the GPU.
bool number(PyObject* o, int dev, at::ScalarType type, double* value, const void** ptr) {
    if (PyFloat_CheckExact(o)) *value = PyFloat_AS_DOUBLE(o);
    else if (PyLong_CheckExact(o)) {
        *value = PyLong_AsDouble(o);
        if (PyErr_Occurred()) {
            PyErr_Clear();
            return false;
        }
    } else {
        const Arg t(o);
        if (!t.vector(dev, type, 1)) return false;
        *ptr = t.ptr();
    }
    return true;
}

// (params, grads, exp_avg, exp_avg_sq, master, exp_avg_scale, exp_avg_sq_scale, step,
// lr, betas, eps, weight_decay, grad_scale, seed) -> status
PyObject* adamw(PyObject*, PyObject* const* arg, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 14 || !g_lib.norm) Py_RETURN_NONE;
    const List p(arg[0]), g(arg[1]), m(arg[2]), v(arg[3]), w(arg[4]), ms(arg[5]), vs(arg[6]);
    const Py_ssize_t count = p.size;
    if (!p.ok || count == 0 || !THPVariable_Check(p.items[0])) Py_RETURN_NONE;
    for (const List* l : {&g, &m, &v, &w, &ms, &vs})
        if (!l->ok || (l->given && l->size != count)) Py_RETURN_NONE;
    const at::Tensor& first = THPVariable_Unpack(p.items[0]);
    if (!first.is_cuda() || c10::hip::current_device() != first.get_device()) Py_RETURN_NONE;
    const int dev = first.get_device();
    const at::ScalarType pt = p.type(), gt = g.type(), mt = m.type(), vt = v.type();
    auto wide = [](at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; };
    auto codes = [](at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; };
    const bool eight = codes(mt);
    if (!g.given || !m.given || !v.given || !wide(pt) || !wide(gt) || (eight ? !codes(vt) : mt != at::kFloat || vt != at::kFloat) ||
        ms.given != eight || vs.given != eight || (w.given && pt != at::kBFloat16))
        Py_RETURN_NONE;
    adamw_numbers num{};
    double step = 1, seed = 0, grad_scale = 0;
    const void *lr_ptr = nullptr, *step_ptr = nullptr, *seed_ptr = nullptr, *scale_ptr = nullptr;
    if (!PyTuple_CheckExact(arg[9]) || PyTuple_GET_SIZE(arg[9]) != 2 || !PyFloat_Check(PyTuple_GET_ITEM(arg[9], 0)) ||
        !PyFloat_Check(PyTuple_GET_ITEM(arg[9], 1)) || !PyFloat_Check(arg[10]) || !PyFloat_Check(arg[11]) ||
        PyFloat_CheckExact(arg[7]) || PyFloat_CheckExact(arg[13]) ||
        !number(arg[7], dev, at::kFloat, &step, &step_ptr) || !number(arg[8], dev, at::kFloat, &num.lr, &lr_ptr) ||
        (arg[12] != Py_None && (!number(arg[12], dev, at::kFloat, &grad_scale, &scale_ptr) || !scale_ptr)))
        Py_RETURN_NONE;
    if (PyLong_CheckExact(arg[13])) num.seed = (uint32_t)PyLong_AsUnsignedLongLongMask(arg[13]);
    else if (!number(arg[13], dev, at::kLong, &seed, &seed_ptr)) Py_RETURN_NONE;
    if (!(step >= 1 && step < 9e15)) Py_RETURN_NONE;
    num.step = (int64_t)step;
    num.beta1 = PyFloat_AS_DOUBLE(PyTuple_GET_ITEM(arg[9], 0));
    num.beta2 = PyFloat_AS_DOUBLE(PyTuple_GET_ITEM(arg[9], 1));
    num.eps = PyFloat_AS_DOUBLE(arg[10]);
    num.weight_decay = PyFloat_AS_DOUBLE(arg[11]);
    num.lr_ptr = static_cast<const float*>(lr_ptr);
    num.step_ptr = static_cast<const float*>(step_ptr);
    num.seed_ptr = static_cast<const int64_t*>(seed_ptr);
    num.grad_scale_ptr = static_cast<const float*>(scale_ptr);
    std::vector<adamw_tensor> list((size_t)count);
    for (Py_ssize_t i = 0; i < count; ++i) {
        const at::Tensor *tp = p.get(i, dev, pt), *tg = g.get(i, dev, gt), *tm = m.get(i, dev, mt), *tv = v.get(i, dev, vt);
        if (!tp || !tg || !tm || !tv || tg->sizes() != tp->sizes() || tm->sizes() != tp->sizes() ||
            tv->sizes() != tp->sizes())
            Py_RETURN_NONE;
        adamw_tensor& t = list[(size_t)i];
        t = adamw_tensor{tp->data_ptr(), tg->data_ptr(), tm->data_ptr(), tv->data_ptr(), nullptr, nullptr, nullptr,
                         tp->numel()};
        if (w.given) {
            const at::Tensor* tw = w.get(i, dev, at::kFloat);
            if (!tw || tw->sizes() != tp->sizes()) Py_RETURN_NONE;
            t.master = tw->data_ptr<float>();
        }
        if (eight) {
            const at::Tensor *a = ms.get(i, dev, at::kFloat), *b = vs.get(i, dev, at::kFloat);
            const int64_t blocks = (t.numel + 255) / 256;
            if (!a || !b || a->dim() != 1 || b->dim() != 1 || a->numel() != blocks || b->numel() != blocks) Py_RETURN_NONE;
            t.exp_avg_scale = a->data_ptr<float>();
            t.exp_avg_sq_scale = b->data_ptr<float>();
        }
    }
    const hipStream_t stream = c10::hip::getCurrentHIPStream(dev).stream();
    int st;
    {
        pybind11::gil_scoped_release free_interpreter;
        st = g_lib.adamw(list.data(), count, pt == at::kFloat ? ADAMW_FP32 : ADAMW_BF16,
                         gt == at::kFloat ? ADAMW_FP32 : ADAMW_BF16, eight ? 8 : 32, &num,
                         reinterpret_cast<ihipStream_t*>(stream));
    }
    if (st == ADAMW_OK)
        for (const List* l : {&p, &m, &v, &w, &ms, &vs}) l->written();
    return PyLong_FromLong(st);
    END_HANDLE_TH_ERRORS
}

// (addresses of the entry points in Library's order, workspace function)
PyObject* use_library(PyObject*, PyObject* args) {
    constexpr int kEntries = sizeof(Library) / sizeof(void*);
    PyObject *addresses, *ws;
    if (!PyArg_ParseTuple(args, "O!O", &PyTuple_Type, &addresses, &ws)) return nullptr;
    if (PyTuple_GET_SIZE(addresses) != kEntries) {
        PyErr_SetString(PyExc_ValueError, "use_library: wrong number of entry points");
        return nullptr;
    }
    void* p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(addresses, i));
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "use_library: null entry point");
            return nullptr;
        }
    }
    static_assert(sizeof(p) == sizeof(g_lib), "one address for each entry");
    memcpy(&g_lib, p, sizeof(p));
    Py_INCREF(ws);
    Py_XSETREF(g_workspace, ws);
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
constexpr PyMethodDef fast(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    fast<layer_norm>("layer_norm"), fast<layer_norm_backward>("layer_norm_backward"), fast<linear>("linear"),
    fast<linear_backward>("linear_backward"), fast<cross_entropy>("cross_entropy"), fast<cross_entropy_backward>("cross_entropy_backward"),
    fast<quantize_weight>("quantize_weight"), fast<adamw>("adamw_step"),
    {"use_library", use_library, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&g_module); }
