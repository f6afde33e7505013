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

#include "../../include/fp8_layer_norm.h"
#include "../../include/fp8_linear.h"

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
    fast<linear_backward>("linear_backward"), {"use_library", use_library, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&g_module); }
