// binding.cpp -- the short way of a decoding step's calls from Python into librmm.
//
// A step makes a handful of calls whose kernels take a few microseconds, so the
// marshalling counts: taken apart one attribute at a time in Python, the tensors of a
// call cost more than its launch.  Us per call in a row of them, through Python and
// ctypes and through this: q/k/v append of 64 tokens 12.2 and 7.0, probabilities of a
// row 6.4 and 4.4, verification of a chain 9.5 and 5.6, keeping one cache 10.4 and 3.5,
// sixteen 21 and 11 (where the kernels take as long).
//
// Each function checks everything that rmm.py checks -- dtypes, shapes, contiguity, one
// device, the current one -- and either makes the call and returns its status, or
// returns None where something is not as it expects; rmm.py then takes the tensors
// apart itself, names what is wrong, or serves the rarer layouts.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>
#include <vector>

#include "rmm.h"

namespace {

// The tensors of one call: `ok` turns false at the first that is not as asked.
struct Call {
    bool ok = true;
    int device = -1;

    const at::Tensor* tensor(PyObject* o) {
        if (!THPVariable_Check(o)) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(o);
    }
    bool here(const at::Tensor& t) {
        if (!t.is_cuda()) return false;
        if (device < 0) {
            device = t.get_device();
            return device == c10::cuda::current_device();
        }
        return t.get_device() == device;
    }
    // a contiguous tensor of this type and shape, on the call's device
    void* of(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = ok ? tensor(o) : nullptr;
        if (!t || t->scalar_type() != type || t->sizes() != at::IntArrayRef(shape) || !t->is_contiguous() || !here(*t)) {
            ok = false;
            return nullptr;
        }
        return t->data_ptr();
    }
    void* of_or_none(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) {
        return o == Py_None ? nullptr : of(o, type, shape);
    }
    // sizes of a tensor of `dims` dimensions, all within an int
    template <int dims>
    void sizes(PyObject* o, int64_t (&n)[dims]) {
        const at::Tensor* t = ok ? tensor(o) : nullptr;
        if (!t || t->dim() != dims) {
            ok = false;
            for (int64_t& x : n) x = 0;
            return;
        }
        for (int i = 0; i < dims; ++i) {
            n[i] = t->size(i);
            if (n[i] > INT_MAX) ok = false;
        }
    }
    long integer(PyObject* o) {
        const long v = PyLong_AsLong(o);
        if (v == -1 && PyErr_Occurred()) PyErr_Clear(), ok = false;
        if (v < INT_MIN || v > INT_MAX) ok = false;
        return v;
    }
    double number(PyObject* o) {
        const double v = PyFloat_AsDouble(o);
        if (v == -1.0 && PyErr_Occurred()) PyErr_Clear(), ok = false;
        return v;
    }
    rmm_stream_t stream(PyObject* o) {  // None: the current one; else its handle
        if (!ok || o == Py_None) return ok ? c10::cuda::getCurrentCUDAStream(device).stream() : nullptr;
        void* s = PyLong_AsVoidPtr(o);
        if (!s && PyErr_Occurred()) PyErr_Clear(), ok = false;
        return s;
    }
};

constexpr at::ScalarType kBf16 = at::kBFloat16, kF32 = at::kFloat, kI32 = at::kInt;

// The call's status, made without the interpreter's lock (a launch may have to wait for
// the GPU, and the GPU for a callback that takes the lock); None where `c` is not ok.
template <typename F>
PyObject* make(const Call& c, F call) {
    if (!c.ok) Py_RETURN_NONE;
    rmm_status rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = call();
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// A Python function of `want` positional arguments; C++ exceptions end here.
template <int want, typename Body>
PyObject* guarded(Py_ssize_t n, Body body) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "takes %d arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return body();
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// Yq, Yk, Yv, Q, Kt, V, lens, L0, parents, q_norm, k_norm, eps, inv_freq, interleaved, stream
PyObject* qkv_rope(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded<15>(nargs, [&]() -> PyObject* {
        Call c;
        int64_t q[4], k[4], f[1] = {0};
        c.sizes(a[3], q);
        c.sizes(a[4], k);
        const int64_t B = q[0], Hq = q[1], T = q[2], d = q[3], Hkv = k[1], ldL = k[3];
        void* Q = c.of(a[3], kBf16, {B, Hq, T, d});
        void* Kt = c.of(a[4], kBf16, {B, Hkv, d, ldL});
        void* V = c.of(a[5], kBf16, {B, Hkv, ldL, d});
        void* Yq = c.of(a[0], kBf16, {B * T, Hq * d});
        void* Yk = c.of(a[1], kBf16, {B * T, Hkv * d});
        void* Yv = c.of(a[2], kBf16, {B * T, Hkv * d});
        void* lens = c.of_or_none(a[6], kI32, {B});
        const long L0 = c.integer(a[7]);
        void* parents = c.of_or_none(a[8], kI32, {B, T});
        void* qn = c.of_or_none(a[9], kBf16, {d});
        void* kn = c.of_or_none(a[10], kBf16, {d});
        const double eps = c.number(a[11]);
        void* freq = nullptr;
        if (a[12] != Py_None) {
            c.sizes(a[12], f);
            freq = c.of(a[12], kF32, {f[0]});
            if (f[0] > INT_MAX / 2) c.ok = false;
        }
        const int interleaved = PyObject_IsTrue(a[13]);
        if (interleaved < 0) PyErr_Clear(), c.ok = false;
        const rmm_stream_t s = c.stream(a[14]);
        return make(c, [&] {
            return rmm_qkv_rope(Yq, Yk, Yv, (int)B, (int)T, (int)Hq, (int)Hkv, (int)d, qn, kn, (float)eps,
                static_cast<const float*>(freq), (int)(2 * f[0]), interleaved,
                static_cast<const int32_t*>(lens), (int)L0, static_cast<const int32_t*>(parents), Q, Kt, V,
                (int)ldL, s);
        });
    });
}

// Q, Kt, V, lens, r, parents, scale, O, idx_out, workspace, stream
PyObject* attn_tree(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded<11>(nargs, [&]() -> PyObject* {
        Call c;
        int64_t q[4], k[4], w[1];
        c.sizes(a[0], q);
        c.sizes(a[1], k);
        const int64_t B = q[0], Hq = q[1], T = q[2], d = q[3], Hkv = k[1], ldL = k[3];
        void* Q = c.of(a[0], kBf16, {B, Hq, T, d});
        void* Kt = c.of(a[1], kBf16, {B, Hkv, d, ldL});
        void* V = c.of(a[2], kBf16, {B, Hkv, ldL, d});
        void* lens = c.of(a[3], kI32, {B});
        const double r = c.number(a[4]);
        void* parents = c.of_or_none(a[5], kI32, {B, T});
        const double scale = c.number(a[6]);
        void* O = c.of(a[7], kBf16, {B, Hq, T, d});
        void* idx = nullptr;
        if (a[8] != Py_None) {  // any shape with room for the kept sets
            const at::Tensor* t = c.tensor(a[8]);
            const int kept = rmm_k_for((int)d, r);
            if (!t || t->scalar_type() != kI32 || !t->is_contiguous() || !c.here(*t) ||
                t->numel() < B * Hkv * (kept > 0 ? kept : 0))
                c.ok = false;
            else
                idx = t->data_ptr();
        }
        c.sizes(a[9], w);
        void* ws = c.of(a[9], at::kByte, {w[0]});
        const rmm_stream_t s = c.stream(a[10]);
        return make(c, [&] {
            return rmm_attn_tree(Q, Kt, V, static_cast<const int32_t*>(lens), static_cast<const int32_t*>(parents), (int)B,
                (int)Hq, (int)Hkv, (int)T, (int)ldL, (int)d, r, (float)scale, O, static_cast<int32_t*>(idx),
                ws, (size_t)w[0], s, nullptr);
        });
    });
}

// X, temperature, Y, stream
PyObject* softmax(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded<4>(nargs, [&]() -> PyObject* {
        Call c;
        int64_t x[2];
        c.sizes(a[0], x);
        void* X = c.of(a[0], kBf16, {x[0], x[1]});
        const double t = c.number(a[1]);
        void* Y = c.of(a[2], kF32, {x[0], x[1]});
        const rmm_stream_t s = c.stream(a[3]);
        return make(c, [&] {
            return rmm_softmax(X, (int)x[0], (int)x[1], x[1], (float)t, static_cast<float*>(Y), x[1], s);
        });
    });
}

// P, tokens, parents, u, Qd, path, emitted, count, stream; P and Qd [B, T, V] or [B*T, V]
PyObject* tree_verify(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded<9>(nargs, [&]() -> PyObject* {
        Call c;
        int64_t n[2];
        c.sizes(a[1], n);
        const int64_t B = n[0], T = n[1];
        const at::Tensor* p = c.tensor(a[0]);
        const int64_t V = p && p->dim() > 0 ? p->size(-1) : 0;
        if (V > INT_MAX) c.ok = false;
        auto rows = [&](PyObject* o) -> const float* {
            const at::Tensor* t = c.ok ? c.tensor(o) : nullptr;
            if (!t) return nullptr;
            return static_cast<const float*>(t->dim() == 3 ? c.of(o, kF32, {B, T, V}) : c.of(o, kF32, {B * T, V}));
        };
        const float* P = rows(a[0]);
        void* tokens = c.of(a[1], kI32, {B, T});
        void* parents = c.of(a[2], kI32, {B, T});
        void* u = c.of(a[3], kF32, {B, T});
        const float* Qd = a[4] == Py_None ? nullptr : rows(a[4]);
        void* path = c.of(a[5], kI32, {B, T});
        void* emitted = c.of(a[6], kI32, {B, T});
        void* count = c.of(a[7], kI32, {B});
        const rmm_stream_t s = c.stream(a[8]);
        return make(c, [&] {
            return rmm_tree_verify(P, V, Qd, Qd ? V : 0, (int)B, (int)T, (int)V, static_cast<const int32_t*>(tokens),
                static_cast<const int32_t*>(parents), static_cast<const float*>(u),
                static_cast<int32_t*>(path), static_cast<int32_t*>(emitted), static_cast<int32_t*>(count),
                s);
        });
    });
}

// caches (a list of tuples (Kt, V)), lens, path, count, lens_out, stream
PyObject* cache_keep(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
    return guarded<6>(nargs, [&]() -> PyObject* {
        Call c;
        int64_t n[2], k[4];
        c.sizes(a[2], n);
        const int64_t B = n[0], T = n[1];
        if (!PyList_Check(a[0]) || PyList_GET_SIZE(a[0]) < 1) Py_RETURN_NONE;
        const Py_ssize_t layers = PyList_GET_SIZE(a[0]);
        std::vector<void*> Kt((size_t)layers), V((size_t)layers);
        for (Py_ssize_t i = 0; i < layers && c.ok; ++i) {
            PyObject* pair = PyList_GET_ITEM(a[0], i);
            if (!PyTuple_Check(pair) || PyTuple_GET_SIZE(pair) != 2) Py_RETURN_NONE;
            if (i == 0) c.sizes(PyTuple_GET_ITEM(pair, 0), k);
            Kt[(size_t)i] = c.of(PyTuple_GET_ITEM(pair, 0), kBf16, {B, k[1], k[2], k[3]});
            V[(size_t)i] = c.of(PyTuple_GET_ITEM(pair, 1), kBf16, {B, k[1], k[3], k[2]});
        }
        void* lens = c.of(a[1], kI32, {B});
        void* path = c.of(a[2], kI32, {B, T});
        void* count = c.of(a[3], kI32, {B});
        void* lens_out = c.of(a[4], kI32, {B});
        const rmm_stream_t s = c.stream(a[5]);
        return make(c, [&] {
            return rmm_cache_keep((int)layers, Kt.data(), V.data(), (int)B, (int)k[1], (int)k[2], (int)k[3],
                static_cast<const int32_t*>(lens), static_cast<const int32_t*>(path),
                static_cast<const int32_t*>(count), (int)T, static_cast<int32_t*>(lens_out), s);
        });
    });
}

template <PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<qkv_rope>("qkv_rope"),       method<attn_tree>("attn_tree"),
                         method<softmax>("softmax"),         method<tree_verify>("tree_verify"),
                         method<cache_keep>("cache_keep"),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
