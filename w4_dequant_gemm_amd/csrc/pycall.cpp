// The Python binding's short way for its smallest calls: checks of a call's
// tensors, its results and workspace, and the call of the C entry point, in one
// step.  In Python they take longer than the kernels of one token (a
// mixture-of-experts call took 15 us of host time and takes 8 here, 7 of which are
// its two launches; a product 8.5 and 4.5; a routing 9.5 and 5.4).
//
// Each function takes what the Python function of its name was given and returns
// its result, or None where anything is not as the usual call has it (a tensor
// elsewhere, of another type or shape, not contiguous, a status other than
// W4_OK): the binding then goes its own way, which raises the errors.  So nothing
// is checked here that is not checked there, and nothing is computed here.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "../../include/w4.h"

namespace {

// the library's entry points, by address (bind())
decltype(&w4a16_linear) f_a16_linear;
decltype(&w4a8_linear) f_a8_linear;
decltype(&w4_gemm_workspace_bytes) f_gemm_ws;
decltype(&w4a8_gemm_workspace_bytes) f_a8_ws;
decltype(&w4_route) f_route;
decltype(&w4_route_workspace_bytes) f_route_ws;
decltype(&w4a16_moe) f_moe;
decltype(&w4a16_moe_workspace_bytes) f_moe_ws;
decltype(&w4_adjust_logits) f_adjust;

struct No {};   // not the usual call

PyObject* none() {
    PyErr_Clear();
    Py_RETURN_NONE;
}

// A call's arguments in order.  The first two are the GPU's index and the stream.
struct Args {
    PyObject* const* a;
    Py_ssize_t n, at = 0;
    int gpu;
    hipStream_t stream;
    Args(PyObject* const* a_, Py_ssize_t n_) : a(a_), n(n_) {
        gpu = static_cast<int>(number());
        stream = reinterpret_cast<hipStream_t>(static_cast<uintptr_t>(number()));
    }
    PyObject* next() {
        if (at >= n) throw No{};
        return a[at++];
    }
    int64_t number() {
        const int64_t v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw No{};
        return v;
    }
    float real() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw No{};
        return static_cast<float>(v);
    }
    const at::Tensor& any() {
        PyObject* const o = next();
        if (!THPVariable_Check(o)) throw No{};
        return THPVariable_Unpack(o);
    }
    const at::Tensor& tensor(at::ScalarType type) {
        const at::Tensor& t = any();
        usual(t, type);
        return t;
    }
    void usual(const at::Tensor& t, at::ScalarType type) const {
        if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != gpu || !t.is_contiguous()) throw No{};
    }
    // whether the next argument is not None; None is passed over
    bool given() {
        if (at >= n) throw No{};
        if (a[at] != Py_None) return true;
        ++at;
        return false;
    }
    // `count` elements of `type`, or null for None
    void* vector(at::ScalarType type, int64_t count) {
        if (!given()) return nullptr;
        const at::Tensor& t = tensor(type);
        if (t.numel() != count) throw No{};
        return t.data_ptr();
    }
};

void need(bool ok) {
    if (!ok) throw No{};
}

// other Python threads run during the call, as they do during a call by ctypes
struct Unlocked {
    PyThreadState* const state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F, typename... A>
void call(F* f, A... a) {
    int rc;
    {
        Unlocked u;
        rc = f(a...);
    }
    need(rc == W4_OK);
}

at::Tensor make(at::IntArrayRef size, at::ScalarType type, const at::Tensor& like) {
    return at::empty(size, like.options().dtype(type));
}

// the status' result: a tuple of tensors, one alone as itself
template <typename... T>
PyObject* result(const T&... t) {
    if constexpr (sizeof...(T) == 1) {
        return THPVariable_Wrap(t...);
    } else {
        PyObject* const tuple = PyTuple_New(sizeof...(T));
        if (!tuple) return nullptr;
        Py_ssize_t i = 0;
        (PyTuple_SET_ITEM(tuple, i++, THPVariable_Wrap(t)), ...);
        return tuple;
    }
}

// any C++ exception ends here, as "not the usual call"
template <typename F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (...) {
        return none();
    }
}

// (gpu, stream, X, wq, sz, G, bias, act, residual, a8)
PyObject* linear(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n);
        const at::Tensor &x = a.tensor(at::kBFloat16), &wq = a.tensor(at::kInt), &sz = a.tensor(at::kInt);
        const int64_t G = a.number();
        need(x.dim() == 2 && x.numel() > 0 && wq.dim() == 2 && G > 0 && G <= 0x7FFFFFFF);
        const int64_t M = x.size(0), K = x.size(1), N = wq.size(0);
        need(K > 0 && K % G == 0 && K % 8 == 0 && 8 * wq.numel() == N * K && sz.numel() == N * (K / G));
        const float* const bias = static_cast<const float*>(a.vector(at::kFloat, N));
        const int act = static_cast<int>(a.number());
        const uint16_t* residual = nullptr;
        if (a.given()) {
            const at::Tensor& r = a.tensor(at::kBFloat16);
            need(r.dim() == 2 && r.size(0) == M && r.size(1) == N);
            residual = static_cast<const uint16_t*>(r.data_ptr());
        }
        const bool a8 = a.number() != 0;
        const size_t bytes = a8 ? f_a8_ws(M, K, N) : f_gemm_ws(M, K, N);
        at::Tensor y = make({M, N}, at::kBFloat16, x), ws;
        if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, x);
        void* const w = bytes ? ws.data_ptr() : nullptr;
        const auto X = static_cast<const uint16_t*>(x.data_ptr());
        const auto q = static_cast<const uint32_t*>(wq.data_ptr()), s = static_cast<const uint32_t*>(sz.data_ptr());
        const auto Y = static_cast<uint16_t*>(y.data_ptr());
        if (!a8) {
            call(f_a16_linear, X, M, K, q, s, N, static_cast<int>(G), bias, act, residual, Y, w, bytes, a.stream);
            return result(y);
        }
        at::Tensor xq = make({M, K}, at::kByte, x), xs = make({M}, at::kFloat, x);
        call(f_a8_linear, X, M, K, q, s, N, static_cast<int>(G), bias, act, residual, Y, static_cast<uint8_t*>(xq.data_ptr()),
                         static_cast<float*>(xs.data_ptr()), w, bytes, a.stream);
        return result(y, xq, xs);
    });
}

// (gpu, stream, X, router, top_k, score, bias, renormalize, scale)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n);
        const at::Tensor &x = a.tensor(at::kBFloat16), &r = a.tensor(at::kBFloat16);
        need(x.dim() == 2 && x.numel() > 0 && r.dim() == 2 && x.size(1) == r.size(1));
        const int64_t T = x.size(0), H = x.size(1), E = r.size(0), k = a.number();
        need(k > 0 && k <= E && k <= 0x7FFF);
        const int score = static_cast<int>(a.number());
        const float* const bias = static_cast<const float*>(a.vector(at::kFloat, E));
        const int renormalize = static_cast<int>(a.number());
        const float scale = a.real();
        const size_t bytes = f_route_ws(T, H, E);
        at::Tensor ids = make({T, k}, at::kInt, x), weights = make({T, k}, at::kFloat, x), ws;
        if (bytes) ws = make({static_cast<int64_t>(bytes)}, at::kByte, x);
        call(f_route, static_cast<const uint16_t*>(x.data_ptr()), T, H, static_cast<const uint16_t*>(r.data_ptr()), E,
                     static_cast<int>(k), score, bias, renormalize, scale, static_cast<int32_t*>(ids.data_ptr()),
                     static_cast<float*>(weights.data_ptr()), bytes ? ws.data_ptr() : nullptr, bytes, a.stream);
        return result(ids, weights);
    });
}

// (gpu, stream, X, ids, weights, gate wq, sz, up wq, sz, down wq, sz, G, act, residual)
PyObject* moe(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n);
        const at::Tensor &x = a.tensor(at::kBFloat16), &ids = a.tensor(at::kInt), &weights = a.tensor(at::kFloat);
        need(x.dim() == 2 && x.numel() > 0 && ids.dim() == 2 && ids.size(0) == x.size(0) && weights.sizes() == ids.sizes());
        const at::Tensor* w[6];
        for (const at::Tensor*& t : w) t = &a.tensor(at::kInt);
        need(w[0]->dim() == 3);
        const int64_t T = x.size(0), H = x.size(1), k = ids.size(1), E = w[0]->size(0), I = w[0]->size(1), G = a.number();
        need(G > 0 && G <= 128 && H % G == 0 && I % G == 0 && k <= 0x7FFF);
        for (int i = 0; i < 6; i += 2) need(8 * w[i]->numel() == E * I * H && w[i + 1]->numel() == E * I * (H / G) && w[i]->size(0) == E);
        const int act = static_cast<int>(a.number());
        const uint16_t* residual = nullptr;
        if (a.given()) {
            const at::Tensor& r = a.tensor(at::kBFloat16);
            need(r.sizes() == x.sizes());
            residual = static_cast<const uint16_t*>(r.data_ptr());
        }
        const size_t bytes = f_moe_ws(T, static_cast<int>(k), E, H, I, static_cast<int>(G));
        need(bytes > 0);
        at::Tensor y = make({T, H}, at::kBFloat16, x), ws = make({static_cast<int64_t>(bytes)}, at::kByte, x);
        const uint32_t* p[6];
        for (int i = 0; i < 6; ++i) p[i] = static_cast<const uint32_t*>(w[i]->data_ptr());
        call(f_moe, static_cast<const uint16_t*>(x.data_ptr()), T, H, static_cast<const int32_t*>(ids.data_ptr()),
                   static_cast<const float*>(weights.data_ptr()), static_cast<int>(k), p[0], p[1], p[2], p[3], p[4], p[5], E, I,
                   static_cast<int>(G), act, residual, static_cast<uint16_t*>(y.data_ptr()), ws.data_ptr(), bytes, a.stream);
        return result(y);
    });
}

// (gpu, stream, logits, history, history_start, prompt_len, repetition, presence, frequency, bias_start, bias_ids,
//  bias_values, mask)
PyObject* adjust(PyObject*, PyObject* const* args, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Args a(args, n);
        const at::Tensor& x = a.any();
        const bool f32 = x.scalar_type() == at::kFloat;
        a.usual(x, f32 ? at::kFloat : at::kBFloat16);
        need(x.dim() == 2);
        const int64_t B = x.size(0), V = x.size(1);
        need(V > 0);
        // a list of any length, -1 if none is given; it and the rows' starts in it come together
        auto list = [&](at::ScalarType type, int64_t& count) -> void* {
            count = -1;
            if (!a.given()) return nullptr;
            const at::Tensor& t = a.tensor(type);
            count = t.numel();
            return t.data_ptr();
        };
        int64_t history_len, bias_len, values;
        const auto history = static_cast<const int32_t*>(list(at::kInt, history_len));
        const auto history_start = static_cast<const int32_t*>(a.vector(at::kInt, B + 1));
        need((history_len >= 0) == (history_start != nullptr));
        const auto prompt = static_cast<const int32_t*>(a.vector(at::kInt, B));
        const float* penalty[3];
        for (const float*& p : penalty) p = static_cast<const float*>(a.vector(at::kFloat, B));
        const auto bias_start = static_cast<const int32_t*>(a.vector(at::kInt, B + 1));
        const auto bias_ids = static_cast<const int32_t*>(list(at::kInt, bias_len));
        const auto bias_values = static_cast<const float*>(list(at::kFloat, values));
        need((bias_len >= 0) == (bias_start != nullptr) && bias_len == values);
        const uint32_t* mask = nullptr;
        int64_t mask_stride = 0;
        if (a.given()) {
            const at::Tensor& m = a.tensor(at::kInt);
            need(m.dim() == 2 && m.size(1) == (V + 31) / 32 && (m.size(0) == 1 || m.size(0) == B));
            mask = static_cast<const uint32_t*>(m.data_ptr());
            mask_stride = m.size(0) > 1 ? m.size(1) : 0;
        }
        at::Tensor out = make({B, V}, x.scalar_type(), x);
        call(f_adjust, x.data_ptr(), f32 ? W4_LOGITS_F32 : W4_LOGITS_BF16, B, V, V, history, std::max<int64_t>(history_len, 0), history_start, prompt,
                      penalty[0], penalty[1], penalty[2], bias_start, bias_ids, bias_values, std::max<int64_t>(bias_len, 0), mask, mask_stride,
                      out.data_ptr(), V, a.stream);
        return result(out);
    });
}

// the addresses of the entry points, in the order below
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    void** const to[] = {reinterpret_cast<void**>(&f_a16_linear), reinterpret_cast<void**>(&f_a8_linear),
                         reinterpret_cast<void**>(&f_gemm_ws),    reinterpret_cast<void**>(&f_a8_ws),
                         reinterpret_cast<void**>(&f_route),      reinterpret_cast<void**>(&f_route_ws),
                         reinterpret_cast<void**>(&f_moe),        reinterpret_cast<void**>(&f_moe_ws),
                         reinterpret_cast<void**>(&f_adjust)};
    if (n != static_cast<Py_ssize_t>(sizeof(to) / sizeof(to[0]))) {
        PyErr_SetString(PyExc_TypeError, "an address for each entry point");
        return nullptr;
    }
    for (Py_ssize_t i = 0; i < n; ++i) {
        void* const p = PyLong_AsVoidPtr(args[i]);
        if (!p) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
            return nullptr;
        }
        *to[i] = p;
    }
    Py_RETURN_NONE;
}

#define W4_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {W4_METHOD(bind), W4_METHOD(linear), W4_METHOD(route), W4_METHOD(moe), W4_METHOD(adjust), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_w4call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__w4call() { return PyModule_Create(&module); }
