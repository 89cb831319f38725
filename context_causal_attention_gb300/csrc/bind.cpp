// bind.cpp -- the Python side of the short calls of speculative decoding: reads shapes, strides and addresses from
// torch tensors, checks them and calls the C ABI (include/cpattn.h), as ops.py does through ctypes for the longer
// calls.  A CPython module of its own because those calls are as short as their marshalling: eleven lists
// checked and passed from Python cost 6 us, here 0.3, where the kernel takes 4.  No arithmetic, no allocation.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/cpattn.h"

namespace {

// What is wrong with an argument: raised as ValueError or TypeError.
struct Wrong {
    PyObject *kind;
    std::string text;
};
[[noreturn]] void wrong(const std::string &text) { throw Wrong{PyExc_ValueError, text}; }

// The arguments of one call, in their order.
struct Arguments {
    PyObject *const *at;
    PyObject *const *end;
    int device = -2;  // of the tensors so far (-2: none, -3: several)

    PyObject *next() { return at < end ? *at++ : throw Wrong{PyExc_TypeError, "missing arguments"}; }
    int64_t integer() {
        const long long v = PyLong_AsLongLong(next());
        if (v == -1 && PyErr_Occurred()) throw Wrong{nullptr, ""};
        return v;
    }
    double number() {
        const double v = PyFloat_AsDouble(next());
        if (v == -1.0 && PyErr_Occurred()) throw Wrong{nullptr, ""};
        return v;
    }
    // A tensor, or nullptr for None.
    const at::Tensor *tensor(const char *what, bool needed = true) {
        PyObject *o = next();
        if (o == Py_None && !needed) return nullptr;
        if (!THPVariable_Check(o)) throw Wrong{PyExc_TypeError, std::string(what) + " must be a tensor"};
        const at::Tensor &t = THPVariable_Unpack(o);
        const int d = t.is_cuda() ? t.get_device() : -1;
        device = device == -2 || device == d ? d : -3;
        return &t;
    }
    // n contiguous int32 values.  (A list that is missing is the library's to refuse.)
    int32_t *list(int64_t n, const char *what) {
        const at::Tensor *t = tensor(what, false);
        if (!t) return nullptr;
        if (t->scalar_type() != at::kInt || t->numel() != n || !t->is_contiguous())
            wrong(std::string(what) + " must be contiguous int32 of " + std::to_string(n) + " values");
        return static_cast<int32_t *>(t->data_ptr());
    }
    // [rows, columns] of the next argument, which stays the next.
    void sizes2(const char *what, int64_t *rows, int64_t *columns) {
        PyObject *o = at < end ? *at : Py_None;
        if (!THPVariable_Check(o) || THPVariable_Unpack(o).dim() != 2) wrong(std::string(what) + " must be of two dimensions");
        *rows = THPVariable_Unpack(o).size(0);
        *columns = THPVariable_Unpack(o).size(1);
    }
    int64_t count(const char *what) {
        PyObject *o = at < end ? *at : Py_None;
        if (!THPVariable_Check(o)) throw Wrong{PyExc_TypeError, std::string(what) + " must be a tensor"};
        return THPVariable_Unpack(o).numel();
    }
    // The call's stream: the last argument, None for the current one.  Behind all checks of shapes.
    cudaStream_t stream() {
        PyObject *o = next();
        if (device != c10::cuda::current_device()) wrong("tensor must be on the current CUDA device");
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
        void *s = PyLong_AsVoidPtr(o);
        if (!s && PyErr_Occurred()) throw Wrong{nullptr, ""};
        return static_cast<cudaStream_t>(s);
    }
};

cp_dtype dtype_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return CP_BF16;
    if (t.scalar_type() == at::kFloat) return CP_F32;
    throw Wrong{PyExc_TypeError, "unsupported dtype (bf16 or fp32)"};
}
void contiguous(const at::Tensor &t) {
    if (!t.is_contiguous()) wrong("tensor must be contiguous");
}

// Two caches [n_pages, page_size, Nkv, D], both alike.
struct Caches {
    void *k, *v;
    int64_t n_pages, page, Nkv, D;
    explicit Caches(Arguments &a) {
        const at::Tensor &x = *a.tensor("k_cache"), &y = *a.tensor("v_cache");
        if (x.dim() != 4 || y.sizes() != x.sizes()) wrong("the caches must be [n_pages, page_size, Nkv, D], both alike");
        if (x.scalar_type() != at::kBFloat16 || y.scalar_type() != at::kBFloat16)
            throw Wrong{PyExc_TypeError, "the caches must be bf16"};
        contiguous(x);
        contiguous(y);
        k = x.data_ptr(), v = y.data_ptr();
        n_pages = x.size(0), page = x.size(1), Nkv = x.size(2), D = x.size(3);
    }
};

// Elements between the tokens of rows [R, H, D] whose head rows are dense.
int64_t token_step(const at::Tensor &t) {
    if (t.dim() != 3) wrong("expected [R, heads, D]");
    const int64_t R = t.size(0), H = t.size(1), D = t.size(2);
    if ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)) wrong("the head rows of a token must be dense");
    if (R <= 1) return H * D;
    if (t.stride(0) == 0) wrong("tokens must lie at one distance from one another");
    return t.stride(0);
}

template <typename F>
PyObject *guarded(PyObject *const *args, Py_ssize_t n, F f) {
    Arguments a{args, args + n};
    try {
        return PyLong_FromLong(f(a));
    } catch (const Wrong &w) {
        if (w.kind) PyErr_SetString(w.kind, w.text.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

PyObject *cache_plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Arguments &a) -> int {
        int64_t B, most;
        a.sizes2("table", &B, &most);
        int32_t *table = a.list(B * most, "table");
        const int64_t n_pages = a.count("free_pages");
        int32_t *free_pages = a.list(n_pages, "free_pages");
        const int32_t *had = a.list(B, "kv_had"), *keep = a.list(B, "kv_keep"), *fresh = a.list(B, "n_new");
        const int32_t *n_free = a.list(a.count("n_free"), "n_free");
        const int64_t page = a.integer(), R = a.integer(), base = a.integer();
        int32_t *kv_len = a.list(B, "kv_len"), *cu = a.list(B + 1, "cu_new"), *slots = a.list(R, "slots");
        int32_t *pos = a.list(R, "pos"), *left = a.list(2, "n_free_out");
        return cp_cache_plan(had, keep, fresh, B, table, most, page, free_pages, n_pages, n_free, base, R, kv_len, cu, slots,
                             pos, left, a.stream());
    });
}

PyObject *tree_plan(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Arguments &a) -> int {
        const int64_t R = a.count("parent");
        const int32_t *parent = a.list(R, "parent");
        const int64_t B = a.count("kv_len");
        const int32_t *kv_len = a.list(B, "kv_len"), *cu = a.list(B + 1, "cu_new");
        const int64_t words = a.integer(), base = a.integer();
        int32_t *mask = a.list(R * words, "mask"), *pos = a.list(R, "pos");
        return cp_tree_plan(parent, cu, kv_len, B, R, words, base, mask, pos, a.stream());
    });
}

PyObject *cache_append_at(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Arguments &a) -> int {
        const at::Tensor &k = *a.tensor("k"), &v = *a.tensor("v");
        const Caches c(a);
        if (k.dim() != 3 || k.size(1) != c.Nkv || k.size(2) != c.D || v.sizes() != k.sizes() ||
            v.scalar_type() != k.scalar_type())
            wrong("k and v must be [R, Nkv, D] of the cache's heads, of one dtype");
        const int64_t R = k.size(0);
        const int32_t *slots = a.list(R, "slots"), *pos = a.list(R, "pos");
        const cp_rope *rope = reinterpret_cast<const cp_rope *>(static_cast<uintptr_t>(a.integer()));
        a.tensor("rope", false);  // (its frequencies)
        const at::Tensor *q = a.tensor("q", false), *out = a.tensor("q_out", false);
        const at::Tensor *wq = a.tensor("wq", false), *wk = a.tensor("wk", false);
        int64_t N = 0, step = 0;
        if (q) {
            if (q->dim() != 3 || q->size(0) != R || q->size(2) != c.D || q->scalar_type() != k.scalar_type())
                wrong("q must be [R, N, D] of k's tokens and dtype");
            N = q->size(1);
            step = token_step(*q);
            if (!out || out->sizes() != q->sizes() || out->scalar_type() != at::kBFloat16 || !out->is_contiguous())
                wrong("q_out must be contiguous bf16 [R, N, D]");
        } else if (out) {
            wrong("q_out without q");
        }
        cp_dtype wd = CP_F32;
        for (const at::Tensor *w : {wq, wk})
            if (w) {
                if (w->numel() != c.D || !w->is_contiguous()) wrong("norm weights must be contiguous [D]");
                wd = dtype_of(*w);
            }
        if (wq && wk && wq->scalar_type() != wk->scalar_type()) wrong("wq and wk must have the same dtype");
        const float eps = static_cast<float>(a.number());
        return cp_cache_append_at(q ? q->data_ptr() : nullptr, k.data_ptr(), v.data_ptr(), step, token_step(k), token_step(v),
                                  dtype_of(k), R, N, c.Nkv, c.D, wq ? wq->data_ptr() : nullptr,
                                  wk ? wk->data_ptr() : nullptr, wd, eps, rope, c.k, c.v, c.n_pages, c.page, slots, pos,
                                  out ? out->data_ptr() : nullptr, a.stream());
    });
}

PyObject *cache_keep(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Arguments &a) -> int {
        a.tensor("caches");  // (one of them: all lie on its device)
        void *const *caches = reinterpret_cast<void *const *>(static_cast<uintptr_t>(a.integer()));
        const int64_t count = a.integer(), n_pages = a.integer(), page = a.integer(), Nkv = a.integer(), D = a.integer();
        int64_t B, max_pages, rows, most;
        a.sizes2("table", &B, &max_pages);
        const int32_t *table = a.list(B * max_pages, "table"), *cu = a.list(B + 1, "cu_new"), *kv_len = a.list(B, "kv_len");
        const int64_t R = a.integer();
        a.sizes2("kept", &rows, &most);
        const int32_t *kept = a.list(B * most, "kept"), *n_kept = a.list(B, "n_kept");
        int32_t *kv_keep = a.list(B, "kv_keep");
        return cp_cache_keep(caches, count, n_pages, page, Nkv, D, table, B, max_pages, cu, kv_len, R, kept, most, n_kept,
                             kv_keep, a.stream());
    });
}

PyObject *tree_attn_fwd(PyObject *, PyObject *const *args, Py_ssize_t n) {
    return guarded(args, n, [](Arguments &a) -> int {
        const at::Tensor &q = *a.tensor("q");
        const Caches c(a);
        if (q.dim() != 3 || q.size(2) != c.D || q.scalar_type() != at::kBFloat16 || !q.is_contiguous())
            wrong("q must be contiguous bf16 [R, N, D]");
        const int64_t R = q.size(0), N = q.size(1);
        int64_t rows, words, B, max_pages;
        a.sizes2("mask", &rows, &words);
        const int32_t *mask = a.list(R * words, "mask");
        const at::Tensor *pre = a.tensor("prefix_pages", false);
        const int64_t prefix = a.integer();
        if (prefix && pre &&
            (pre->scalar_type() != at::kInt || !pre->is_contiguous() || pre->numel() * c.page < prefix))
            wrong("prefix_pages must be contiguous int32 and cover prefix_len tokens");
        a.sizes2("table", &B, &max_pages);
        const int32_t *table = a.list(B * max_pages, "table"), *cu = a.list(B + 1, "cu_new"), *kv_len = a.list(B, "kv_len");
        const int64_t max_new = a.integer();
        const float scale = static_cast<float>(a.number());
        const at::Tensor &o = *a.tensor("o"), &lse = *a.tensor("lse"), &ws = *a.tensor("workspace");
        if (o.sizes() != q.sizes() || !o.is_contiguous()) wrong("o must be contiguous [R, N, D]");
        if (lse.dim() != 2 || lse.size(0) != N || lse.size(1) != R || lse.scalar_type() != at::kFloat || !lse.is_contiguous())
            wrong("lse must be contiguous fp32 [N, R]");
        contiguous(ws);
        return cp_tree_attn_fwd(q.data_ptr(), c.k, c.v, c.n_pages, c.page,
                                pre ? static_cast<const int32_t *>(pre->data_ptr()) : nullptr, prefix, table, B, max_pages,
                                cu, kv_len, mask, words, max_new, R, N, c.Nkv, c.D, scale, o.data_ptr(), dtype_of(o),
                                static_cast<float *>(lse.data_ptr()), ws.data_ptr(), ws.nbytes(), a.stream());
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"cache_plan", fast(cache_plan), METH_FASTCALL, nullptr},
                         {"tree_plan", fast(tree_plan), METH_FASTCALL, nullptr},
                         {"cache_append_at", fast(cache_append_at), METH_FASTCALL, nullptr},
                         {"cache_keep", fast(cache_keep), METH_FASTCALL, nullptr},
                         {"tree_attn_fwd", fast(tree_attn_fwd), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cpbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cpbind() { return PyModule_Create(&module); }
