// The calls of one decoding step from Python, without ctypes: each function checks its
// tensors (type, shape, dense, on the current CUDA device), takes the current stream and
// calls the library.  It returns the library's status, or -1 where a tensor is not as it
// should be or the call has an argument it does not handle; abi.py then goes through its
// own checks, which name the fault, and its own call.  A small call's time would be the
// host's: enqueuing one through ctypes and the checks in Python takes 5.5 to 9.5 us, this
// way 2.5 to 4.7 (on the GPU they take 2.6 to 6).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <initializer_list>

#include "biv.h"

namespace {

constexpr auto kBF16 = c10::ScalarType::BFloat16;
constexpr auto kF32 = c10::ScalarType::Float;
constexpr auto kI32 = c10::ScalarType::Int;

// Entry points of the loaded library, in the order in which bind() takes them.
struct {
    decltype(&biv_rope_kv_write_paged) rope_kv_write_paged;
    decltype(&biv_decode_attn_paged) decode_attn_paged;
    decltype(&biv_gemm_bias_act) gemm_bias_act;
    decltype(&biv_softmax) softmax;
    decltype(&biv_verify_sample) verify_sample;
} g_lib;

// One call's arguments: every look at them may find that the call is not for this file.
struct Args {
    PyObject* const* a;
    c10::DeviceIndex dev = -1;
    bool ok = true;

    const at::Tensor* tensor(int i) {
        if (!THPVariable_Check(a[i])) ok = false;
        if (!ok) return nullptr;
        const at::Tensor* t = &THPVariable_Unpack(a[i]);
        if (!t->is_cuda()) {
            ok = false;
            return nullptr;
        }
        if (dev < 0) dev = c10::cuda::current_device();
        if (t->get_device() != dev) ok = false;
        return t;
    }
    const at::Tensor* tensor(int i, c10::ScalarType type, int dims) {
        const at::Tensor* t = tensor(i);
        if (ok && (t->scalar_type() != type || t->dim() != dims || !t->is_contiguous())) ok = false;
        return t;
    }
    void* data(int i, c10::ScalarType type, std::initializer_list<int64_t> shape) {
        const at::Tensor* t = tensor(i, type, static_cast<int>(shape.size()));
        if (ok && t->sizes() != c10::IntArrayRef(shape.begin(), shape.size())) ok = false;
        return ok ? t->data_ptr() : nullptr;
    }
    void* data_or_none(int i, c10::ScalarType type, std::initializer_list<int64_t> shape) {
        return a[i] == Py_None ? nullptr : data(i, type, shape);
    }
    int64_t size(const at::Tensor* t, int d) {
        const int64_t n = ok ? t->size(d) : 0;
        if (n > INT_MAX) ok = false;
        return n;
    }
    int integer(int i) {
        int over = 0;
        const long x = PyLong_Check(a[i]) ? PyLong_AsLongAndOverflow(a[i], &over) : (ok = false, 0);
        if (over || x > INT_MAX || x < INT_MIN) ok = false;
        return static_cast<int>(x);
    }
    float number(int i) {
        if (!PyFloat_Check(a[i])) ok = false;
        return ok ? static_cast<float>(PyFloat_AS_DOUBLE(a[i])) : 0.0f;
    }
    biv_stream_t stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
};

template <typename F>
PyObject* answer(PyObject* const* a, Py_ssize_t n, Py_ssize_t want, F&& call) {
    long status = -1;
    if (n == want) {
        try {
            Args args{a};
            status = call(args);
        } catch (...) {                                    // a tensor without memory, sizes that are symbols, ...
            status = -1;
        }
    }
    if (PyErr_Occurred()) return nullptr;
    return PyLong_FromLong(status);
}

// The library's call without the interpreter's lock (a launch waits where the queue is
// full).  Nothing in it may throw: every pointer is taken before.
template <typename F>
long unlocked(F&& f) noexcept {
    PyThreadState* state = PyEval_SaveThread();
    const long status = f();
    PyEval_RestoreThread(state);
    return status;
}

// qkv, q_out, k_pages, v_pages, page_table, row_slot, row_pos, theta, K
PyObject* rope_kv_write_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(a, n, 9, [](Args& x) -> long {
        const at::Tensor *q = x.tensor(1, kBF16, 3), *k = x.tensor(2, kBF16, 4), *table = x.tensor(4, kI32, 2);
        if (!x.ok) return -1;
        const int64_t W = x.size(q, 0), Hq = x.size(q, 1), hd = x.size(q, 2);
        const int64_t n_pages = x.size(k, 0), Hkv = x.size(k, 1), page = x.size(k, 2);
        const int64_t n_slots = x.size(table, 0), max_pages = x.size(table, 1);
        if (k->size(3) != hd) return -1;
        void *qkv = x.data(0, kBF16, {W, (Hq + 2 * Hkv) * hd}), *v = x.data(3, kBF16, {n_pages, Hkv, page, hd});
        void *slot = x.data(5, kI32, {W}), *pos = x.data(6, kI32, {W});
        const float theta = x.number(7);
        const int K = x.integer(8);
        if (!x.ok) return -1;
        const biv_stream_t s = x.stream();
        void *q_at = q->data_ptr(), *k_at = k->data_ptr(), *table_at = table->data_ptr();
        return unlocked([&] {
            return g_lib.rope_kv_write_paged(qkv, q_at, k_at, v, static_cast<int32_t*>(table_at), static_cast<int32_t*>(slot), static_cast<int32_t*>(pos), nullptr, W, K, Hq, Hkv, hd,
                                             n_slots, max_pages, n_pages, page, theta, s);
        });
    });
}

// q, k_pages, v_pages, page_table, row_slot, row_pos, o, rows_per_group, workspace
PyObject* decode_attn_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(a, n, 9, [](Args& x) -> long {
        const at::Tensor *q = x.tensor(0, kBF16, 3), *k = x.tensor(1, kBF16, 4), *table = x.tensor(3, kI32, 2), *ws = x.tensor(8);
        if (!x.ok || !ws->is_contiguous()) return -1;
        const int64_t W = x.size(q, 0), Hq = x.size(q, 1), hd = x.size(q, 2);
        const int64_t n_pages = x.size(k, 0), Hkv = x.size(k, 1), page = x.size(k, 2);
        const int64_t n_slots = x.size(table, 0), max_pages = x.size(table, 1);
        if (k->size(3) != hd) return -1;
        void *v = x.data(2, kBF16, {n_pages, Hkv, page, hd}), *o = x.data(6, kBF16, {W, Hq, hd});
        void *slot = x.data(4, kI32, {W}), *pos = x.data(5, kI32, {W});
        const int rpg = x.integer(7);
        if (!x.ok) return -1;
        const biv_stream_t s = x.stream();
        void *q_at = q->data_ptr(), *k_at = k->data_ptr(), *table_at = table->data_ptr(), *ws_at = ws->data_ptr();
        const size_t ws_bytes = ws->nbytes();
        return unlocked([&] {
            return g_lib.decode_attn_paged(q_at, k_at, v, static_cast<int32_t*>(table_at), static_cast<int32_t*>(slot), static_cast<int32_t*>(pos), o, W, rpg, Hq, Hkv, hd, n_slots,
                                           max_pages, n_pages, page, ws_at, ws_bytes, s);
        });
    });
}

// A, B, C, bias, residual, act (its number)
PyObject* gemm_bias_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(a, n, 6, [](Args& x) -> long {
        const at::Tensor *A = x.tensor(0, kBF16, 2), *B = x.tensor(1, kBF16, 2), *out = x.tensor(2);
        if (!x.ok) return -1;
        const int64_t M = x.size(A, 0), K = x.size(A, 1), N = x.size(B, 0);
        const c10::ScalarType type = out->scalar_type();
        if (B->size(1) != K || (type != kBF16 && type != kF32)) return -1;
        void* C = x.data(2, type, {M, N});
        void *bias = x.data_or_none(3, kBF16, {N}), *residual = x.data_or_none(4, kBF16, {M, N});
        const int act = x.integer(5);
        if (!x.ok) return -1;
        const biv_stream_t s = x.stream();
        void *A_at = A->data_ptr(), *B_at = B->data_ptr();
        return unlocked([&] {
            return g_lib.gemm_bias_act(A_at, B_at, bias, residual, C, type == kF32 ? BIV_F32 : BIV_BF16, act, M, N,
                                       K, s);
        });
    });
}

// logits, probs (dense, of one shape), temperature
PyObject* softmax(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(a, n, 3, [](Args& x) -> long {
        const at::Tensor* logits = x.tensor(0, kF32, 2);
        if (!x.ok) return -1;
        const int64_t R = x.size(logits, 0), V = x.size(logits, 1);
        void* probs = x.data(1, kF32, {R, V});
        const float T = x.number(2);
        if (!x.ok) return -1;
        const biv_stream_t s = x.stream();
        void* at = logits->data_ptr();
        return unlocked([&] {
            return g_lib.softmax(static_cast<float*>(at), R, V, V, T, static_cast<float*>(probs), V, s);
        });
    });
}

// target, draft_probs, draft, u_accept, u_sample, p0, tokens, accept_len, new_len
PyObject* verify_sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return answer(a, n, 9, [](Args& x) -> long {
        const at::Tensor *tokens = x.tensor(6, kI32, 2), *target = x.tensor(0, kF32, 2);
        if (!x.ok) return -1;
        const int64_t N = x.size(tokens, 0), K = x.size(tokens, 1) - 1, V = x.size(target, 1);
        if (K < 0 || target->size(0) != N * (K + 1)) return -1;
        void* q = x.data_or_none(1, kF32, {N * K, V});
        void *draft = x.data(2, kI32, {N, K}), *u_accept = x.data(3, kF32, {N, K}), *u_sample = x.data(4, kF32, {N});
        void *p0 = x.data(5, kI32, {N}), *accept_len = x.data(7, kI32, {N}), *new_len = x.data(8, kI32, {N});
        if (!x.ok) return -1;
        const biv_stream_t s = x.stream();
        void *target_at = target->data_ptr(), *tokens_at = tokens->data_ptr();
        return unlocked([&] {
            return g_lib.verify_sample(static_cast<float*>(target_at), static_cast<float*>(q), static_cast<int32_t*>(draft),
                                       static_cast<float*>(u_accept), static_cast<float*>(u_sample), static_cast<int32_t*>(p0), N, K, V,
                                       static_cast<int32_t*>(tokens_at), static_cast<int32_t*>(accept_len),
                                       static_cast<int32_t*>(new_len), s);
        });
    });
}

// Addresses of the five entry points of the library that abi.py has loaded.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    void* at[5];
    if (n != 5) return PyErr_Format(PyExc_TypeError, "five addresses");
    for (int i = 0; i < 5; ++i) {
        at[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    g_lib.rope_kv_write_paged = reinterpret_cast<decltype(&biv_rope_kv_write_paged)>(at[0]);
    g_lib.decode_attn_paged = reinterpret_cast<decltype(&biv_decode_attn_paged)>(at[1]);
    g_lib.gemm_bias_act = reinterpret_cast<decltype(&biv_gemm_bias_act)>(at[2]);
    g_lib.softmax = reinterpret_cast<decltype(&biv_softmax)>(at[3]);
    g_lib.verify_sample = reinterpret_cast<decltype(&biv_verify_sample)>(at[4]);
    Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FAST(rope_kv_write_paged), FAST(decode_attn_paged), FAST(gemm_bias_act), FAST(softmax), FAST(verify_sample),
                          FAST(bind), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_biv_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose tensors this code reads (build.py gives it).
PyMODINIT_FUNC PyInit__biv_torch() {
    PyObject* m = PyModule_Create(&kModule);
    if (m && PyModule_AddStringConstant(m, "torch_version", BIV_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
