// The usual case of the binding's feed-forward calls, compiled: checks of the tensor arguments, outputs
// and workspace from torch's allocator, the current stream, and the one C-ABI call.  A decode step's
// calls are as short as their launch, and the same steps in Python cost more than the kernel (M = 1,
// K = 11008, N = 4096: 9 us of GPU time, 14 us a call).
//
// Every function returns NotImplemented for whatever is not the usual case (a wrong type, shape,
// device or layout, another current device): the caller's Python then takes the call and raises the
// error or switches the device.  A status other than W4_OK is returned as an int.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cstring>

#include "w4a16.h"

namespace {

struct Abi {
    decltype(&w4_gemm_fused) fused;
    decltype(&w4_gemm_gated) gated;
    decltype(&w4_gemm_dx) dx;
    decltype(&w4_gemm_dx_gated) dx_gated;
    decltype(&w4_act_backward) act_backward;
    decltype(&w4_gemm_fused_workspace_size) fused_ws;
    decltype(&w4_gemm_gated_workspace_size) gated_ws;
    decltype(&w4_gemm_dx_workspace_size) dx_ws;
    decltype(&w4_act_backward_workspace_size) act_ws;
} abi;

// Argument reader: `ok` falls to false at the first argument that is not the usual case.
struct Args {
    PyObject* const* a;
    bool ok = true;
    c10::Device dev{c10::DeviceType::CPU};

    bool none(int i) const { return a[i] == Py_None; }
    int64_t integer(int i) {
        if (PyBool_Check(a[i])) return a[i] == Py_True;
        int overflow = 0;
        const long long v = PyLong_CheckExact(a[i]) ? PyLong_AsLongLongAndOverflow(a[i], &overflow) : LLONG_MAX;
        if (overflow || v < INT_MIN || v > INT_MAX) ok = false;  // the C calls take an int
        return ok ? v : 0;
    }
    const at::Tensor* tensor(PyObject* o) {
        if (ok && THPVariable_CheckExact(o)) return &THPVariable_Unpack(o);
        ok = false;
        return nullptr;
    }
    // The first matrix: its device is the call's, and must be the current one.
    const at::Tensor* first(int i, int64_t& rows, int64_t& cols) {
        const at::Tensor* t = tensor(a[i]);
        if (!t || t->dim() != 2 || !t->is_cuda() || t->device().index() != c10::cuda::current_device()) {
            ok = false;
            return nullptr;
        }
        dev = t->device();
        rows = t->size(0);
        cols = t->size(1);
        return half(t, rows, cols) ? t : nullptr;
    }
    bool fits(const at::Tensor* t, c10::ScalarType type, int64_t rows, int64_t cols) {
        ok = ok && t && t->scalar_type() == type && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols &&
             t->device() == dev && t->is_contiguous();
        return ok;
    }
    bool half(const at::Tensor* t, int64_t rows, int64_t cols) { return fits(t, at::kHalf, rows, cols); }
    uint16_t* matrix(PyObject* o, int64_t rows, int64_t cols) {
        const at::Tensor* t = tensor(o);
        return half(t, rows, cols) ? static_cast<uint16_t*>(t->data_ptr()) : nullptr;
    }
    uint16_t* optional(int i, int64_t rows, int64_t cols) { return none(i) ? nullptr : matrix(a[i], rows, cols); }
    uint16_t* vector(int i, int64_t n) {
        if (none(i)) return nullptr;
        const at::Tensor* t = tensor(a[i]);
        ok = ok && t && t->scalar_type() == at::kHalf && t->dim() == 1 && t->size(0) == n && t->device() == dev &&
             t->is_contiguous();
        return ok ? static_cast<uint16_t*>(t->data_ptr()) : nullptr;
    }
};

struct Layer {
    const uint32_t* packed = nullptr;
    const uint16_t* scales = nullptr;
    const uint8_t* zeros = nullptr;
};
Layer layer(Args& x, PyObject* p, PyObject* s, PyObject* z, int64_t N, int64_t K) {
    Layer l;
    const at::Tensor *tp = x.tensor(p), *ts = x.tensor(s), *tz = x.tensor(z);
    if (K % 128 == 0 && x.fits(tp, at::kInt, N, K / 8) && x.fits(ts, at::kHalf, N, K / 128) &&
        x.fits(tz, at::kByte, N, K / 128)) {
        l.packed = static_cast<const uint32_t*>(tp->data_ptr());
        l.scales = static_cast<const uint16_t*>(ts->data_ptr());
        l.zeros = static_cast<const uint8_t*>(tz->data_ptr());
    } else {
        x.ok = false;
    }
    return l;
}
Layer layer(Args& x, PyObject* triple, int64_t N, int64_t K) {
    PyObject* o[3];
    if (PyTuple_CheckExact(triple) && PyTuple_GET_SIZE(triple) == 3)
        for (int i = 0; i < 3; ++i) o[i] = PyTuple_GET_ITEM(triple, i);
    else {
        x.ok = false;
        return {};
    }
    return layer(x, o[0], o[1], o[2], N, K);
}

int64_t rows_of(Args& x, PyObject* o, int dim) {  // a size of a matrix argument, -1 where it is none
    const at::Tensor* t = x.tensor(o);
    if (!t || t->dim() != 2) {
        x.ok = false;
        return -1;
    }
    return t->size(dim);
}

at::Tensor empty(const Args& x, int64_t rows, int64_t cols) {
    return at::empty({rows, cols}, at::TensorOptions().dtype(at::kHalf).device(x.dev));
}

// The caller's workspace where it is large enough, else a new one, held by `keep`.
struct Workspace {
    void* p = nullptr;
    size_t bytes = 0;
    at::Tensor keep;
    bool take(Args& x, PyObject* given, size_t need) {
        if (given != Py_None) {
            const at::Tensor* t = x.tensor(given);
            if (!t || t->device() != x.dev || !t->is_contiguous()) return x.ok = false;
            if (t->nbytes() >= need) {
                p = t->data_ptr();
                bytes = t->nbytes();
                return true;
            }
        }
        if (need) {
            keep = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(x.dev));
            p = keep.data_ptr();
            bytes = need;
        }
        return true;
    }
};

void* stream_of(const Args& x) { return c10::cuda::getCurrentCUDAStream(x.dev.index()).stream(); }
uint16_t* h(at::Tensor& t) { return static_cast<uint16_t*>(t.data_ptr()); }

PyObject* not_usual() {
    if (PyErr_Occurred()) PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
template <typename... T>
PyObject* wrap_tuple(const T&... t) {
    PyObject* r = PyTuple_New(sizeof...(T));
    int i = 0;
    if (r) (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
    return r;
}

// An output: the caller's tensor (checked) or a new one.
struct Out {
    at::Tensor t;
    bool take(Args& x, PyObject* given, int64_t rows, int64_t cols) {
        if (given == Py_None) {
            if (x.ok) t = empty(x, rows, cols);
            return x.ok;
        }
        const at::Tensor* g = x.tensor(given);
        if (x.half(g, rows, cols)) t = *g;
        return x.ok;
    }
};

template <typename F>
PyObject* guarded(F&& f) {  // no C++ exception leaves for Python: torch's own become Python's
    HANDLE_TH_ERRORS
    return f();
    END_HANDLE_TH_ERRORS
}

// X, packed, scales, zeros, bias, activation, residual, save_pre, group, out, workspace, flags
PyObject* fused(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 12) return not_usual();
        Args x{a};
        int64_t M, K;
        const at::Tensor* X = x.first(0, M, K);
        if (!X) return not_usual();
        const int64_t N = rows_of(x, a[1], 0);
        const Layer w = layer(x, a[1], a[2], a[3], N, K);
        const uint16_t *bias = x.vector(4, N), *residual = x.optional(6, M, N);
        const int64_t act = x.integer(5), pre = x.integer(7), group = x.integer(8), flags = x.integer(11);
        size_t need = 0;
        if (!x.ok || abi.fused_ws(M, N, K, (int)group, &need) != W4_OK) return not_usual();
        Workspace ws;
        Out Y, Z;
        if (!ws.take(x, a[10], need) || !Y.take(x, a[9], M, N) || (pre && !Z.take(x, Py_None, M, N))) return not_usual();
        const w4_status st = abi.fused(static_cast<const uint16_t*>(X->data_ptr()), M, N, K, w.packed, w.scales, w.zeros,
                                       (int)group, bias, (int)act, residual, h(Y.t), pre ? h(Z.t) : nullptr, ws.p, ws.bytes,
                                       (int)flags, stream_of(x));
        if (st != W4_OK) return PyLong_FromLong(st);
        return pre ? wrap_tuple(Y.t, Z.t) : wrap(Y.t);
    });
}

// X, gate, up, activation, save_pre, group, out, workspace, flags
PyObject* gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 9) return not_usual();
        Args x{a};
        int64_t M, K;
        const at::Tensor* X = x.first(0, M, K);
        if (!X || !PyTuple_CheckExact(a[1]) || PyTuple_GET_SIZE(a[1]) != 3) return not_usual();
        const int64_t N = rows_of(x, PyTuple_GET_ITEM(a[1], 0), 0);
        const Layer g = layer(x, a[1], N, K), u = layer(x, a[2], N, K);
        const int64_t act = x.integer(3), pre = x.integer(4), group = x.integer(5), flags = x.integer(8);
        size_t need = 0;
        if (!x.ok || abi.gated_ws(M, N, K, (int)group, &need) != W4_OK) return not_usual();
        Workspace ws;
        Out H, G, U;
        if (!ws.take(x, a[7], need) || !H.take(x, a[6], M, N) ||
            (pre && !(G.take(x, Py_None, M, N) && U.take(x, Py_None, M, N))))
            return not_usual();
        const w4_status st = abi.gated(static_cast<const uint16_t*>(X->data_ptr()), M, N, K, g.packed, g.scales, g.zeros,
                                       u.packed, u.scales, u.zeros, (int)group, (int)act, h(H.t), pre ? h(G.t) : nullptr,
                                       pre ? h(U.t) : nullptr, ws.p, ws.bytes, (int)flags, stream_of(x));
        if (st != W4_OK) return PyLong_FromLong(st);
        return pre ? wrap_tuple(H.t, G.t, U.t) : wrap(H.t);
    });
}

// dY, packed, scales, zeros, dY2, weights2, group, out, workspace
PyObject* dx(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 9) return not_usual();
        Args x{a};
        int64_t M, N;
        const at::Tensor* dY = x.first(0, M, N);
        if (!dY || x.none(4) != x.none(5)) return not_usual();
        const int64_t K = rows_of(x, a[1], 1) * 8;
        const Layer w = layer(x, a[1], a[2], a[3], N, K);
        const bool two = !x.none(4);
        const uint16_t* dY2 = x.optional(4, M, N);
        const Layer w2 = two ? layer(x, a[5], N, K) : Layer{};
        const int64_t group = x.integer(6);
        size_t need = 0;
        if (!x.ok || abi.dx_ws(M, N, K, two ? 2 : 1, (int)group, &need) != W4_OK) return not_usual();
        Workspace ws;
        Out dX;
        if (!ws.take(x, a[8], need) || !dX.take(x, a[7], M, K)) return not_usual();
        const w4_status st = abi.dx(static_cast<const uint16_t*>(dY->data_ptr()), M, N, K, w.packed, w.scales, w.zeros, dY2,
                                    w2.packed, w2.scales, w2.zeros, (int)group, h(dX.t), ws.p, ws.bytes, stream_of(x));
        return st != W4_OK ? PyLong_FromLong(st) : wrap(dX.t);
    });
}

// dY, packed, scales, zeros, G, U, activation, group, out[0], out[1], workspace
PyObject* dx_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 11) return not_usual();
        Args x{a};
        int64_t M, N;
        const at::Tensor* dY = x.first(0, M, N);
        if (!dY) return not_usual();
        const int64_t K = rows_of(x, a[1], 1) * 8;
        const Layer w = layer(x, a[1], a[2], a[3], N, K);
        const uint16_t *G = x.matrix(a[4], M, K), *U = x.matrix(a[5], M, K);
        const int64_t act = x.integer(6), group = x.integer(7);
        size_t need = 0;
        if (!x.ok || abi.dx_ws(M, N, K, 1, (int)group, &need) != W4_OK) return not_usual();
        Workspace ws;
        Out dG, dU;
        if (!ws.take(x, a[10], need) || !dG.take(x, a[8], M, K) || !dU.take(x, a[9], M, K)) return not_usual();
        const w4_status st = abi.dx_gated(static_cast<const uint16_t*>(dY->data_ptr()), M, N, K, w.packed, w.scales, w.zeros,
                                          (int)group, G, U, (int)act, h(dG.t), h(dU.t), ws.p, ws.bytes, stream_of(x));
        return st != W4_OK ? PyLong_FromLong(st) : wrap_tuple(dG.t, dU.t);
    });
}

// dY, Z, U, activation, bias_grad, out[0], out[1], workspace
PyObject* act_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 8) return not_usual();
        Args x{a};
        int64_t M, N;
        const at::Tensor* dY = x.first(0, M, N);
        if (!dY) return not_usual();
        const uint16_t *Z = x.optional(1, M, N), *U = x.optional(2, M, N);
        const bool gated = !x.none(2);  // by the argument: an empty tensor has no address
        const int64_t act = x.integer(3), bias = x.integer(4);
        if (x.ok && gated && bias) return PyLong_FromLong(W4_ERR_UNSUPPORTED);
        size_t need = 0;
        if (!x.ok || (bias && abi.act_ws(M, N, &need) != W4_OK)) return not_usual();
        Workspace ws;
        Out dZ, dU;
        at::Tensor db;
        if ((bias && !ws.take(x, a[7], need)) || !dZ.take(x, a[5], M, N) || (gated && !dU.take(x, a[6], M, N)))
            return not_usual();
        if (bias) db = at::empty({N}, at::TensorOptions().dtype(at::kFloat).device(x.dev));
        const w4_status st = abi.act_backward(static_cast<const uint16_t*>(dY->data_ptr()), Z, U, M, N, (int)act, h(dZ.t),
                                              gated ? h(dU.t) : nullptr, bias ? static_cast<float*>(db.data_ptr()) : nullptr, ws.p,
                                              ws.bytes, stream_of(x));
        if (st != W4_OK) return PyLong_FromLong(st);
        if (gated) return wrap_tuple(dZ.t, dU.t);
        return bias ? wrap_tuple(dZ.t, db) : wrap(dZ.t);
    });
}

// Addresses of the loaded library's entry points, in Abi's order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    constexpr Py_ssize_t kEntries = sizeof(Abi) / sizeof(void*);
    if (n != kEntries) {
        PyErr_SetString(PyExc_ValueError, "bind: one address per entry point");
        return nullptr;
    }
    void* p[kEntries];
    for (Py_ssize_t i = 0; i < n; ++i)
        if (!(p[i] = PyLong_AsVoidPtr(a[i]))) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null address");
            return nullptr;
        }
    memcpy(&abi, p, sizeof(abi));
    Py_RETURN_NONE;
}

#define FAST(name) \
    { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {FAST(bind), FAST(fused), FAST(gated), FAST(dx), FAST(dx_gated), FAST(act_backward), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ffn_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ffn_call() { return PyModule_Create(&module); }
