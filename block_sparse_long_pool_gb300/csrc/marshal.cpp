/* marshal.cpp -- the paged cache's calls from Python: tensors checked and passed on.
 *
 * A decode step's page plan or append takes 4 to 6 us on the device.  Checked and passed from
 * Python code one call takes 9 us of the host's time, and 6.3 from C through the tensors' Python
 * attributes (a dozen tensors' type, shape, device, layout and address at 60 ns each); here
 * they are read from torch's own tensor objects, in 2.7 with the launch.  A function returns its status, or None where
 * an argument is not as it has to be: the caller then says which one.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include <ATen/core/TensorBase.h>
#include <torch/csrc/autograd/python_variable.h>

#include "sparse_pool.h"

namespace {

constexpr int64_t D = 128, BLK = 64;

decltype(&sparse_page_plan) f_plan;
decltype(&sparse_paged_append_f8) f_append;
decltype(&sparse_paged_decode_attn_f8) f_attn;
decltype(&sparse_paged_chunk_attn_f8) f_chunk;
decltype(&sparse_rope) f_rope;
decltype(&sparse_page_fork) f_fork;
decltype(&sparse_paged_copy_f8) f_copy;

// The arguments of one call: `ok` turns false at the first that is not as it has to be.
struct Args {
    PyObject *const *a;
    int64_t idx;
    bool ok = true;

    const at::TensorBase *get(int i)
    {
        if (!THPVariable_Check(a[i])) {
            ok = false;
            return nullptr;
        }
        return &THPVariable_Unpack(a[i]);
    }
    bool none(int i) const { return a[i] == Py_None; }

    // extent x of argument i, which has `dims` of them
    int64_t extent(int i, int dims, int x)
    {
        const at::TensorBase *t = get(i);
        if (t == nullptr || t->dim() != dims || t->sizes()[x] > INT32_MAX) {
            ok = false;
            return 0;
        }
        return t->sizes()[x];
    }

    // the address of a contiguous tensor of this type and shape on the device
    template <typename T>
    T *tensor(int i, at::ScalarType type, at::IntArrayRef shape)
    {
        const at::TensorBase *t = ok ? get(i) : nullptr;
        ok = t != nullptr && t->scalar_type() == type && t->sizes() == shape && t->is_cuda() && t->get_device() == idx &&
             t->is_contiguous();
        return ok ? static_cast<T *>(t->data_ptr()) : nullptr;
    }

    // rows [n_tok][H][128] bf16, a token's values contiguous: address and token stride
    uint16_t *rows(int i, int64_t n_tok, int64_t H, long long *step)
    {
        const at::TensorBase *t = ok ? get(i) : nullptr;
        ok = t != nullptr && t->scalar_type() == at::kBFloat16 && t->sizes() == at::IntArrayRef({n_tok, H, D}) && t->is_cuda() &&
             t->get_device() == idx && t->stride(2) == 1 && (t->stride(1) == D || H <= 1);
        if (!ok)
            return nullptr;
        *step = n_tok > 1 ? t->stride(0) : H * D;   // of one token the stride is not used
        return static_cast<uint16_t *>(t->data_ptr());
    }
};

// Calls `body` with the arguments after the device and the stream, which are the first two; a
// tensor that has no address or sizes to give (it throws) is one that is not as it has to be.
template <typename F>
PyObject *call(PyObject *const *a, Py_ssize_t n, Py_ssize_t want, F body)
{
    if (n != want)
        return PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, n);
    const long long idx = PyLong_AsLongLong(a[0]);
    void *stream = reinterpret_cast<void *>(static_cast<intptr_t>(PyLong_AsLongLong(a[1])));
    if (PyErr_Occurred())
        return nullptr;
    Args x{a + 2, idx};
    int rc = 0;
    try {
        body(x, stream, &rc);
    } catch (...) {
        x.ok = false;
    }
    if (PyErr_Occurred())
        return nullptr;
    if (!x.ok)
        Py_RETURN_NONE;
    return PyLong_FromLong(rc);
}

// seq_len n_new block_table free_pages n_free cu_new start seq_len_out n_free_out slot_map tok_req
// tok_pos status
PyObject *page_plan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 15, [](Args &x, void *stream, int *rc) {
        const int64_t B = x.extent(2, 2, 0), max_blocks = x.extent(2, 2, 1), n_pages = x.extent(3, 1, 0);
        const int64_t n_tok = x.extent(9, 1, 0);
        int *p[13] = {};
        auto take = [&](int i, at::IntArrayRef shape) { p[i] = x.tensor<int>(i, at::kInt, shape); };
        for (int i : {0, 1, 6, 7})
            take(i, {B});
        take(2, {B, max_blocks});
        take(3, {n_pages});
        take(4, {1});
        take(5, {B + 1});
        take(8, {1});
        for (int i : {9, 10, 11})
            take(i, {n_tok});
        if (!x.none(12))
            take(12, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_plan(p[0], p[1], static_cast<int>(B), p[2], static_cast<int>(max_blocks), p[3], static_cast<int>(n_pages), p[4],
                     p[5], p[6], p[7], p[8], p[9], p[10], p[11], static_cast<int>(n_tok), p[12], stream);
        Py_END_ALLOW_THREADS
    });
}

// kv_pages kv_scale k_new v_new slot_map ktil tok_req tok_pos status
PyObject *paged_append_f8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 11, [](Args &x, void *stream, int *rc) {
        const int64_t n_pages = x.extent(0, 5, 0), H = x.extent(0, 5, 1), n_tok = x.extent(4, 1, 0);
        int64_t B = 0, N_cap = 0;
        long long k_step = 0, v_step = 0;
        float *ktil = nullptr;
        const int *req = nullptr, *pos = nullptr;
        uint8_t *pages = x.tensor<uint8_t>(0, at::kFloat8_e4m3fn, {n_pages, H, 2, BLK, D});
        float *scale = x.tensor<float>(1, at::kFloat, {n_pages, H, 2});
        const uint16_t *k = x.rows(2, n_tok, H, &k_step), *v = x.rows(3, n_tok, H, &v_step);
        const int *slots = x.tensor<int>(4, at::kInt, {n_tok});
        if (!x.none(5)) {
            B = x.extent(5, 4, 0);
            N_cap = x.extent(5, 4, 2);
            ktil = x.tensor<float>(5, at::kFloat, {B, H, N_cap, D});
            req = x.tensor<int>(6, at::kInt, {n_tok});
            pos = x.tensor<int>(7, at::kInt, {n_tok});
        }
        int *status = x.none(8) ? nullptr : x.tensor<int>(8, at::kInt, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_append(pages, scale, static_cast<int>(n_pages), static_cast<int>(H), k, v, k_step, v_step, slots,
                       static_cast<int>(n_tok), ktil, static_cast<int>(B), static_cast<int>(N_cap), req, pos, status, stream);
        Py_END_ALLOW_THREADS
    });
}

// Q kv_pages kv_scale block_table seq_len O workspace blk_idx count lse scale status
PyObject *paged_decode_attn_f8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 14, [](Args &x, void *stream, int *rc) {
        const double factor = PyFloat_AsDouble(x.a[10]);
        if (PyErr_Occurred())
            return;
        const int64_t H_q = x.extent(0, 3, 1), n_pages = x.extent(1, 5, 0), H = x.extent(1, 5, 1);
        const int64_t B = x.extent(3, 2, 0), max_blocks = x.extent(3, 2, 1);
        int64_t k_tot = 0;
        const int *ids = nullptr, *count = nullptr;
        const uint16_t *q = x.tensor<uint16_t>(0, at::kBFloat16, {B, H_q, D});
        const uint8_t *pages = x.tensor<uint8_t>(1, at::kFloat8_e4m3fn, {n_pages, H, 2, BLK, D});
        const float *scale = x.tensor<float>(2, at::kFloat, {n_pages, H, 2});
        const int *table = x.tensor<int>(3, at::kInt, {B, max_blocks});
        const int *len = x.tensor<int>(4, at::kInt, {B});
        uint16_t *o = x.tensor<uint16_t>(5, at::kBFloat16, {B, H_q, D});
        const int64_t bytes = x.ok && x.get(6) != nullptr ? x.get(6)->numel() : 0;
        void *ws = x.tensor<uint8_t>(6, at::kByte, {bytes});
        if (!x.none(7)) {
            k_tot = x.extent(7, 3, 2);
            ids = x.tensor<int>(7, at::kInt, {B, H, k_tot});
            count = x.tensor<int>(8, at::kInt, {B, H});
        }
        float *lse = x.none(9) ? nullptr : x.tensor<float>(9, at::kFloat, {B, H_q});
        int *status = x.none(11) ? nullptr : x.tensor<int>(11, at::kInt, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_attn(q, pages, scale, static_cast<int>(n_pages), table, static_cast<int>(max_blocks), ids, count,
                     static_cast<int>(k_tot), len, static_cast<int>(B), static_cast<int>(H_q), static_cast<int>(H),
                     static_cast<float>(factor), o, lse, ws, static_cast<size_t>(bytes), status, stream);
        Py_END_ALLOW_THREADS
    });
}

// Q kv_pages kv_scale block_table cu_new start O workspace lse scale status
PyObject *paged_chunk_attn_f8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 13, [](Args &x, void *stream, int *rc) {
        const double factor = PyFloat_AsDouble(x.a[9]);
        if (PyErr_Occurred())
            return;
        const int64_t n_tok = x.extent(0, 3, 0), H_q = x.extent(0, 3, 1), n_pages = x.extent(1, 5, 0), H = x.extent(1, 5, 1);
        const int64_t B = x.extent(3, 2, 0), max_blocks = x.extent(3, 2, 1);
        long long step = 0;
        const uint16_t *q = x.rows(0, n_tok, H_q, &step);
        const uint8_t *pages = x.tensor<uint8_t>(1, at::kFloat8_e4m3fn, {n_pages, H, 2, BLK, D});
        const float *scale = x.tensor<float>(2, at::kFloat, {n_pages, H, 2});
        const int *table = x.tensor<int>(3, at::kInt, {B, max_blocks});
        const int *cu = x.tensor<int>(4, at::kInt, {B + 1});
        const int *start = x.tensor<int>(5, at::kInt, {B});
        uint16_t *o = x.tensor<uint16_t>(6, at::kBFloat16, {n_tok, H_q, D});
        const int64_t bytes = x.ok && x.get(7) != nullptr ? x.get(7)->numel() : 0;
        void *ws = x.tensor<uint8_t>(7, at::kByte, {bytes});
        float *lse = x.none(8) ? nullptr : x.tensor<float>(8, at::kFloat, {n_tok, H_q});
        int *status = x.none(10) ? nullptr : x.tensor<int>(10, at::kInt, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_chunk(q, step, pages, scale, static_cast<int>(n_pages), table, static_cast<int>(max_blocks), cu, start,
                      static_cast<int>(n_tok), static_cast<int>(B), static_cast<int>(H_q), static_cast<int>(H),
                      static_cast<float>(factor), o, lse, ws, static_cast<size_t>(bytes), status, stream);
        Py_END_ALLOW_THREADS
    });
}

// Q K pos inv_freq Q_out K_out interleaved factor
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 10, [](Args &x, void *stream, int *rc) {
        const double factor = PyFloat_AsDouble(x.a[7]);
        const int interleaved = PyObject_IsTrue(x.a[6]);
        if (PyErr_Occurred())
            return;
        const int64_t n_tok = x.extent(0, 3, 0), H_q = x.extent(0, 3, 1), half = x.extent(3, 1, 0);
        const int64_t H = x.none(1) ? 0 : x.extent(1, 3, 1);
        long long step[4] = {};
        uint16_t *k = nullptr, *k_out = nullptr;
        uint16_t *q = x.rows(0, n_tok, H_q, &step[0]), *q_out = x.rows(4, n_tok, H_q, &step[2]);
        if (!x.none(1)) {
            k = x.rows(1, n_tok, H, &step[1]);
            k_out = x.rows(5, n_tok, H, &step[3]);
        }
        const int *pos = x.tensor<int>(2, at::kInt, {n_tok});
        const double *freq = x.tensor<double>(3, at::kDouble, {half});
        if (!x.ok || half > INT32_MAX / 2) {
            x.ok = false;
            return;
        }
        Py_BEGIN_ALLOW_THREADS
        *rc = f_rope(q, step[0], static_cast<int>(H_q), k, step[1], static_cast<int>(H), pos, static_cast<int>(n_tok), freq,
                     static_cast<int>(2 * half), interleaved, static_cast<float>(factor), q_out, step[2], k_out, step[3], stream);
        Py_END_ALLOW_THREADS
    });
}

// src seq_len block_table page_extra free_pages n_free copy_src copy_dst workspace fork_len status
PyObject *page_fork(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 13, [](Args &x, void *stream, int *rc) {
        const int64_t B = x.extent(2, 2, 0), max_blocks = x.extent(2, 2, 1), n_pages = x.extent(4, 1, 0);
        int *p[8] = {};
        auto take = [&](int i, at::IntArrayRef shape) { p[i] = x.tensor<int>(i, at::kInt, shape); };
        for (int i : {0, 1, 6, 7})
            take(i, {B});
        take(2, {B, max_blocks});
        take(3, {n_pages});
        take(4, {n_pages});
        take(5, {1});
        const int64_t bytes = x.ok && x.get(8) != nullptr ? x.get(8)->numel() : 0;
        void *ws = x.tensor<uint8_t>(8, at::kByte, {bytes});
        const int *most = x.none(9) ? nullptr : x.tensor<int>(9, at::kInt, {B});
        int *status = x.none(10) ? nullptr : x.tensor<int>(10, at::kInt, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_fork(p[0], most, static_cast<int>(B), p[1], p[2], static_cast<int>(max_blocks), p[3], p[4], static_cast<int>(n_pages),
                     p[5], p[6], p[7], ws, static_cast<size_t>(bytes), status, stream);
        Py_END_ALLOW_THREADS
    });
}

// kv_pages kv_scale copy_src copy_dst ktil src seq_len status
PyObject *paged_copy_f8(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return call(a, n, 10, [](Args &x, void *stream, int *rc) {
        const int64_t n_pages = x.extent(0, 5, 0), H = x.extent(0, 5, 1), n_copy = x.extent(2, 1, 0);
        int64_t B = 0, N_cap = 0;
        float *ktil = nullptr;
        const int *src = nullptr, *len = nullptr;
        uint8_t *pages = x.tensor<uint8_t>(0, at::kFloat8_e4m3fn, {n_pages, H, 2, BLK, D});
        float *scale = x.tensor<float>(1, at::kFloat, {n_pages, H, 2});
        const int *from = x.tensor<int>(2, at::kInt, {n_copy}), *to = x.tensor<int>(3, at::kInt, {n_copy});
        if (!x.none(4)) {
            B = x.extent(4, 4, 0);
            N_cap = x.extent(4, 4, 2);
            ktil = x.tensor<float>(4, at::kFloat, {B, H, N_cap, D});
            src = x.tensor<int>(5, at::kInt, {B});
            len = x.tensor<int>(6, at::kInt, {B});
        }
        int *status = x.none(7) ? nullptr : x.tensor<int>(7, at::kInt, {1});
        if (!x.ok)
            return;
        Py_BEGIN_ALLOW_THREADS
        *rc = f_copy(pages, scale, static_cast<int>(n_pages), static_cast<int>(H), from, to, static_cast<int>(n_copy), ktil,
                     static_cast<int>(B), static_cast<int>(N_cap), src, len, status, stream);
        Py_END_ALLOW_THREADS
    });
}

// The entry points' addresses: page_plan, paged_append_f8, paged_decode_attn_f8,
// paged_chunk_attn_f8, rope, page_fork, paged_copy_f8.
PyObject *setup(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    intptr_t f[7];
    if (n != 7)
        return PyErr_Format(PyExc_TypeError, "setup takes 7 arguments");
    for (int i = 0; i < 7; ++i)
        f[i] = static_cast<intptr_t>(PyLong_AsLongLong(a[i]));
    if (PyErr_Occurred())
        return nullptr;
    f_plan = reinterpret_cast<decltype(f_plan)>(f[0]);
    f_append = reinterpret_cast<decltype(f_append)>(f[1]);
    f_attn = reinterpret_cast<decltype(f_attn)>(f[2]);
    f_chunk = reinterpret_cast<decltype(f_chunk)>(f[3]);
    f_rope = reinterpret_cast<decltype(f_rope)>(f[4]);
    f_fork = reinterpret_cast<decltype(f_fork)>(f[5]);
    f_copy = reinterpret_cast<decltype(f_copy)>(f[6]);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t))
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"setup", fast(setup), METH_FASTCALL, nullptr},
                         {"page_plan", fast(page_plan), METH_FASTCALL, nullptr},
                         {"paged_append_f8", fast(paged_append_f8), METH_FASTCALL, nullptr},
                         {"paged_decode_attn_f8", fast(paged_decode_attn_f8), METH_FASTCALL, nullptr},
                         {"paged_chunk_attn_f8", fast(paged_chunk_attn_f8), METH_FASTCALL, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"page_fork", fast(page_fork), METH_FASTCALL, nullptr},
                         {"paged_copy_f8", fast(paged_copy_f8), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal()
{
    return PyModule_Create(&module);
}
