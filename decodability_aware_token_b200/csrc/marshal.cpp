// Host side of the chunk operators' binding: reads the tensors' pointers, strides and shapes in C++ and calls the C
// ABI, since eleven tensors inspected from Python cost more host time than a small chunk takes on the GPU.  Each
// function returns the status of the C call, or None when an argument is not what the call needs: the caller then
// takes the Python path, which makes the same checks and words the refusal.  (A plan of 32 single tokens: 8.7 us of host
// time by the Python path, 3.8 this way, against 2.4 us on the GPU.)
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <initializer_list>

#include "../../include/focus.h"

namespace {

struct Args {
    PyObject* const* v;
    int dev;  // device index every tensor has to be on
    bool ok = true;

    int64_t i(int k) {
        const long long x = PyLong_AsLongLong(v[k]);
        if (x == -1 && PyErr_Occurred()) ok = false;
        return x;
    }
    int32_t i32(int k) {
        const int64_t x = i(k);
        if (x < INT32_MIN || x > INT32_MAX) ok = false;
        return (int32_t)x;
    }
    double f(int k) {
        const double x = PyFloat_AsDouble(v[k]);
        if (x == -1.0 && PyErr_Occurred()) ok = false;
        return x;
    }
    void* p(int k) { return reinterpret_cast<void*>((uintptr_t)i(k)); }
    const at::Tensor* tensor(int k, at::ScalarType dt) {
        if (!THPVariable_Check(v[k])) return ok = false, nullptr;
        const at::Tensor& t = THPVariable_Unpack(v[k]);
        if (!t.defined() || t.scalar_type() != dt || !t.is_cuda() || t.get_device() != dev || t.layout() != at::kStrided)
            return ok = false, nullptr;
        return &t;
    }
    // a dense tensor of the given shape
    void* dense(int k, at::ScalarType dt, std::initializer_list<int64_t> shape, size_t align = 4) {
        const at::Tensor* t = tensor(k, dt);
        if (!t) return nullptr;
        if (!t->sizes().equals(c10::IntArrayRef(shape)) || !t->is_contiguous()) return ok = false, nullptr;
        void* x = t->data_ptr();
        if (reinterpret_cast<uintptr_t>(x) % align) ok = false;
        return x;
    }
    int32_t* ints(int k, std::initializer_list<int64_t> shape) { return static_cast<int32_t*>(dense(k, at::kInt, shape)); }
    int64_t len(int k) {  // rows of a tensor
        if (!THPVariable_Check(v[k])) return ok = false, 0;
        const at::Tensor& t = THPVariable_Unpack(v[k]);
        if (!t.defined() || t.dim() < 1) return ok = false, 0;
        return t.size(0);
    }
    // [rows, heads, d] with dense heads and 16-byte aligned rows
    void* heads(int k, at::ScalarType dt, int64_t rows, int64_t n, int64_t d, int64_t& stride) {
        const at::Tensor* t = tensor(k, dt);
        if (!t) return nullptr;
        if (t->dim() != 3 || t->size(0) != rows || t->size(1) != n || t->size(2) != d || t->stride(2) != 1 ||
            (n > 1 && t->stride(1) != d))
            return ok = false, nullptr;
        stride = rows <= 1 ? n * d : t->stride(0);
        void* x = t->data_ptr();
        if (stride < n * d || reinterpret_cast<uintptr_t>(x) % 16 || stride * t->element_size() % 16) ok = false;
        return x;
    }
    // [pages, L, 2, Hkv, S, d]
    void* pool(int k, at::ScalarType dt, int64_t L, int64_t hkv, int64_t d, int32_t& n_pages, int32_t& page_size) {
        const at::Tensor* t = tensor(k, dt);
        if (!t) return nullptr;
        if (t->dim() != 6 || t->size(1) != L || t->size(2) != 2 || t->size(3) != hkv || t->size(5) != d ||
            !t->is_contiguous() || t->size(0) > INT32_MAX || t->size(4) > INT32_MAX)
            return ok = false, nullptr;
        n_pages = (int32_t)t->size(0);
        page_size = (int32_t)t->size(4);
        void* x = t->data_ptr();
        if (reinterpret_cast<uintptr_t>(x) % 16) ok = false;
        return x;
    }
};

template <typename Body> PyObject* guarded(Body&& body) {
    try {
        const int64_t rc = body();
        if (rc != INT64_MIN && !PyErr_Occurred()) return PyLong_FromLongLong(rc);
    } catch (...) {  // (a tensor without storage, for instance: the Python path words it)
    }
    PyErr_Clear();
    Py_RETURN_NONE;
}

// (fn, ctx, stream, device, max_pages, page_size, n_pages, prefix_len, new_len, page_table, free_pages, free_head,
//  row_offsets, kv_len, row_req, row_pos, row_slot, free_next)
PyObject* plan(PyObject*, PyObject* const* v, Py_ssize_t n_args) {
    return guarded([&]() -> int64_t {
        if (n_args != 18) return INT64_MIN;
        Args a{v, 0};
        a.dev = a.i32(3);
        focus_chunk_plan p{};
        const int64_t n = a.len(7), rows = a.len(14), free_n = a.len(10), max_pages = a.i(4);
        p.page_size = a.i32(5);
        p.n_pages = a.i32(6);
        if (!a.ok || n > INT32_MAX || rows > INT32_MAX || free_n > INT32_MAX) return INT64_MIN;
        p.n_requests = (int32_t)n;
        p.max_rows = (int32_t)rows;
        p.n_free = (int32_t)free_n;
        p.prefix_len = a.ints(7, {n});
        p.new_len = a.ints(8, {n});
        p.page_table = a.ints(9, {n, max_pages});
        p.free_pages = a.ints(10, {free_n});
        p.free_head = a.ints(11, {1});
        p.row_offsets = a.ints(12, {n + 1});
        p.kv_len = a.ints(13, {n});
        p.row_req = a.ints(14, {rows});
        p.row_pos = a.ints(15, {rows});
        p.row_slot = a.ints(16, {rows});
        p.free_next = a.ints(17, {1});
        auto fn = reinterpret_cast<decltype(&focus_chunk_plan_rows)>(a.p(0));
        auto* ctx = static_cast<focus_chunk_ctx*>(a.p(1));
        void* stream = a.p(2);
        return a.ok ? fn(ctx, &p, stream) : INT64_MIN;
    });
}

// (fn, ctx, stream, device, bf16, Hq, Hkv, d, L, layer, eps, q, k, v, kv_pool, row_pos, row_slot, q_norm, k_norm, out)
PyObject* qk(PyObject*, PyObject* const* v, Py_ssize_t n_args) {
    return guarded([&]() -> int64_t {
        if (n_args != 20) return INT64_MIN;
        Args a{v, 0};
        a.dev = a.i32(3);
        const at::ScalarType dt = a.i(4) ? at::kBFloat16 : at::kFloat;
        const int64_t hq = a.i(5), hkv = a.i(6), d = a.i(7), L = a.i(8), rows = a.len(11);
        focus_chunk_qk p{};
        p.layer = a.i32(9);
        p.eps = (float)a.f(10);
        if (!a.ok || p.layer < 0 || p.layer >= L || rows > INT32_MAX) return INT64_MIN;
        p.rows = (int32_t)rows;
        p.q = a.heads(11, dt, rows, hq, d, p.q_stride);
        p.k = a.heads(12, dt, rows, hkv, d, p.k_stride);
        p.v = a.heads(13, dt, rows, hkv, d, p.v_stride);
        p.kv_pool = a.pool(14, dt, L, hkv, d, p.n_pages, p.page_size);
        p.row_pos = a.ints(15, {rows});
        p.row_slot = a.ints(16, {rows});
        p.q_norm = v[17] == Py_None ? nullptr : a.dense(17, dt, {d}, 16);
        p.k_norm = v[18] == Py_None ? nullptr : a.dense(18, dt, {d}, 16);
        p.q_out = a.heads(19, dt, rows, hq, d, p.out_stride);
        auto fn = reinterpret_cast<decltype(&focus_chunk_qk_norm_rope)>(a.p(0));
        auto* ctx = static_cast<focus_chunk_ctx*>(a.p(1));
        void* stream = a.p(2);
        return a.ok ? fn(ctx, &p, stream) : INT64_MIN;
    });
}

// (fn, ctx, stream, device, bf16, Hq, Hkv, d, L, max_pages, layer, max_new, mask_block, scale, q, kv_pool, row_offsets,
//  kv_len, page_table, out)
PyObject* attention(PyObject*, PyObject* const* v, Py_ssize_t n_args) {
    return guarded([&]() -> int64_t {
        if (n_args != 20) return INT64_MIN;
        Args a{v, 0};
        a.dev = a.i32(3);
        const at::ScalarType dt = a.i(4) ? at::kBFloat16 : at::kFloat;
        const int64_t hq = a.i(5), hkv = a.i(6), d = a.i(7), L = a.i(8), max_pages = a.i(9), rows = a.len(14), n = a.len(17);
        focus_chunk_attn p{};
        p.layer = a.i32(10);
        p.max_new = a.i32(11);
        p.mask_block = a.i32(12);
        p.scale = (float)a.f(13);
        if (!a.ok || p.layer < 0 || p.layer >= L || rows > INT32_MAX || n > INT32_MAX) return INT64_MIN;
        p.rows = (int32_t)rows;
        p.n_requests = (int32_t)n;
        p.q = a.heads(14, dt, rows, hq, d, p.q_stride);
        p.kv_pool = a.pool(15, dt, L, hkv, d, p.n_pages, p.page_size);
        p.row_offsets = a.ints(16, {n + 1});
        p.kv_len = a.ints(17, {n});
        p.page_table = a.ints(18, {n, max_pages});
        p.out = a.heads(19, dt, rows, hq, d, p.out_stride);
        auto fn = reinterpret_cast<decltype(&focus_chunk_attention)>(a.p(0));
        auto* ctx = static_cast<focus_chunk_ctx*>(a.p(1));
        void* stream = a.p(2);
        return a.ok ? fn(ctx, &p, stream) : INT64_MIN;
    });
}

PyMethodDef methods[] = {
    {"plan", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan)), METH_FASTCALL, nullptr},
    {"qk", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(qk)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", "argument marshalling of the chunk operators", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) Py_CLEAR(m);
    return m;
}
