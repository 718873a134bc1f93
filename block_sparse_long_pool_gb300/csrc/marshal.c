/* marshal.c -- the paged cache's calls from Python: tensors checked and passed on.
 *
 * A decode step's page plan or append takes 4 to 6 us on the device.  Checked and passed from
 * Python code one call takes 9 us of the host's time, from here about 5: a dozen tensors'
 * type, shape, device, layout and address, asked for through their own attributes (no header
 * but Python's is needed), then the C entry point.  A function returns its status, or None
 * where an argument is not as it has to be: the caller then says which one.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stddef.h>
#include <stdint.h>

#include "sparse_pool.h"

typedef int (*plan_fn)(const int *, const int *, int, int *, int, int *, int, const int *, int *, int *, int *, int *, int *,
                       int *, int *, int, int *, void *);
typedef int (*append_fn)(uint8_t *, float *, int, int, const uint16_t *, const uint16_t *, long long, long long, const int *, int,
                         float *, int, int, const int *, const int *, int *, void *);
typedef int (*attn_fn)(const uint16_t *, const uint8_t *, const float *, int, const int *, int, const int *, const int *, int,
                       const int *, int, int, int, float, uint16_t *, float *, void *, size_t, int *, void *);

static PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_stride, *s_numel;
static PyObject *t_int32, *t_float32, *t_bfloat16, *t_float8, *t_uint8;
static plan_fn f_plan;
static append_fn f_append;
static attn_fn f_attn;

#define MOST_DIMS 5
#define D 128
#define BLK 64

/* A whole number that a method or attribute gives; -1 and *ok = 0 on any failure. */
static long long number(PyObject *v, int *ok)
{
    long long n = -1;
    if (v == NULL) {
        PyErr_Clear();
        *ok = 0;
        return -1;
    }
    n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        *ok = 0;
    }
    return n;
}

/* A tensor's extents; their number, or -1. */
static int dims_of(PyObject *t, long long *dims)
{
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    Py_ssize_t n, i;
    if (shape == NULL || !PyTuple_Check(shape) || PyTuple_GET_SIZE(shape) > MOST_DIMS) {
        PyErr_Clear();
        Py_XDECREF(shape);
        return -1;
    }
    n = PyTuple_GET_SIZE(shape);
    for (i = 0; i < n; ++i)
        dims[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
    Py_DECREF(shape);
    if (PyErr_Occurred()) {
        PyErr_Clear();
        return -1;
    }
    return (int)n;
}

static int has_dtype(PyObject *t, PyObject *dtype)
{
    PyObject *have = PyObject_GetAttr(t, s_dtype);
    const int same = have == dtype;
    if (have == NULL)
        PyErr_Clear();
    Py_XDECREF(have);
    return same;
}

static int on_device(PyObject *t, long long idx)
{
    int ok = 1;
    return number(PyObject_CallMethodNoArgs(t, s_get_device), &ok) == idx && ok;
}

static void *address(PyObject *t, int *ok)
{
    return (void *)(intptr_t)number(PyObject_CallMethodNoArgs(t, s_data_ptr), ok);
}

/* The address of a contiguous tensor of this type and shape on device idx; *ok = 0 if it is not one. */
static void *tensor(PyObject *t, PyObject *dtype, long long idx, int n, long long d0, long long d1, long long d2, long long d3,
                    long long d4, int *ok)
{
    const long long want[MOST_DIMS] = {d0, d1, d2, d3, d4};
    long long have[MOST_DIMS];
    PyObject *c;
    int i;
    if (!*ok)
        return NULL;
    *ok = 0;
    if (!has_dtype(t, dtype) || dims_of(t, have) != n)
        return NULL;
    for (i = 0; i < n; ++i)
        if (have[i] != want[i])
            return NULL;
    if (!on_device(t, idx))
        return NULL;
    c = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (c == NULL)
        PyErr_Clear();
    Py_XDECREF(c);
    if (c != Py_True)
        return NULL;
    *ok = 1;
    return address(t, ok);
}

#define TENSOR1(t, dt, a) tensor(t, dt, idx, 1, a, 0, 0, 0, 0, &ok)
#define TENSOR2(t, dt, a, b) tensor(t, dt, idx, 2, a, b, 0, 0, 0, &ok)
#define TENSOR3(t, dt, a, b, c) tensor(t, dt, idx, 3, a, b, c, 0, 0, &ok)
#define TENSOR4(t, dt, a, b, c, d) tensor(t, dt, idx, 4, a, b, c, d, 0, &ok)
#define TENSOR5(t, dt, a, b, c, d, e) tensor(t, dt, idx, 5, a, b, c, d, e, &ok)
#define OPTIONAL(t, call) ((t) == Py_None ? NULL : (call))

/* The number of a tensor's elements, 0 if it has none to tell. */
static long long numel(PyObject *t)
{
    int ok = 1;
    const long long n = number(PyObject_CallMethodNoArgs(t, s_numel), &ok);
    return ok ? n : 0;
}

static int fits(long long n)
{
    return n >= 0 && n <= 0x7fffffff;
}

/* idx, stream: the device and its stream; the others as sparse_page_plan of the binding. */
static PyObject *page_plan(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    long long table[MOST_DIMS], idx, n_pages, n_tok, B;
    void *stream, *p[13];
    int ok = 1, rc, i;
    if (n != 15)
        return PyErr_Format(PyExc_TypeError, "page_plan takes 15 arguments");
    idx = PyLong_AsLongLong(a[0]);
    stream = (void *)(intptr_t)PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred())
        return NULL;
    a += 2;   /* seq_len n_new block_table free_pages n_free cu_new start seq_len_out n_free_out slot_map tok_req tok_pos status */
    if (dims_of(a[2], table) != 2)
        Py_RETURN_NONE;
    B = table[0];
    n_pages = numel(a[3]);
    n_tok = numel(a[9]);
    if (!fits(B) || !fits(table[1]) || !fits(n_pages) || !fits(n_tok))
        Py_RETURN_NONE;
    p[2] = TENSOR2(a[2], t_int32, B, table[1]);
    p[3] = TENSOR1(a[3], t_int32, n_pages);
    p[4] = TENSOR1(a[4], t_int32, 1);
    p[5] = TENSOR1(a[5], t_int32, B + 1);
    p[8] = TENSOR1(a[8], t_int32, 1);
    for (i = 0; i < 4; ++i) {
        static const int per_request[4] = {0, 1, 6, 7};
        p[per_request[i]] = TENSOR1(a[per_request[i]], t_int32, B);
    }
    for (i = 9; i < 12; ++i)
        p[i] = TENSOR1(a[i], t_int32, n_tok);
    p[12] = OPTIONAL(a[12], TENSOR1(a[12], t_int32, 1));
    if (!ok)
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = f_plan(p[0], p[1], (int)B, p[2], (int)table[1], p[3], (int)n_pages, p[4], p[5], p[6], p[7], p[8], p[9], p[10], p[11],
                (int)n_tok, p[12], stream);
    Py_END_ALLOW_THREADS
    (void)self;
    return PyLong_FromLong(rc);
}

/* New rows [n_tok][H_kv][128] bf16, a token's values contiguous: address and token stride. */
static void *new_rows(PyObject *t, long long idx, long long n_tok, long long H, long long *step, int *ok)
{
    long long have[MOST_DIMS], s[3];
    PyObject *strides;
    int i;
    if (!*ok)
        return NULL;
    *ok = 0;
    if (!has_dtype(t, t_bfloat16) || dims_of(t, have) != 3 || have[0] != n_tok || have[1] != H || have[2] != D ||
        !on_device(t, idx))
        return NULL;
    strides = PyObject_CallMethodNoArgs(t, s_stride);
    if (strides == NULL || !PyTuple_Check(strides) || PyTuple_GET_SIZE(strides) != 3) {
        PyErr_Clear();
        Py_XDECREF(strides);
        return NULL;
    }
    for (i = 0; i < 3; ++i)
        s[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(strides, i));
    Py_DECREF(strides);
    if (s[2] != 1 || (s[1] != D && H > 1))
        return NULL;
    *step = n_tok > 1 ? s[0] : H * D;   /* of one token the stride is not used */
    *ok = 1;
    return address(t, ok);
}

/* idx, stream, kv_pages, kv_scale, k_new, v_new, slot_map, ktil, tok_req, tok_pos, status */
static PyObject *paged_append_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    long long pages[MOST_DIMS], keys[MOST_DIMS] = {0}, idx, n_tok, ks = 0, vs = 0;
    void *stream, *kv, *sc, *k, *v, *slots, *kt = NULL, *req = NULL, *pos = NULL, *st;
    int ok = 1, rc;
    if (n != 11)
        return PyErr_Format(PyExc_TypeError, "paged_append_f8 takes 11 arguments");
    idx = PyLong_AsLongLong(a[0]);
    stream = (void *)(intptr_t)PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred())
        return NULL;
    a += 2;
    if (dims_of(a[0], pages) != 5)
        Py_RETURN_NONE;
    n_tok = numel(a[4]);
    if (!fits(pages[0]) || !fits(pages[1]) || !fits(n_tok))
        Py_RETURN_NONE;
    kv = TENSOR5(a[0], t_float8, pages[0], pages[1], 2, BLK, D);
    sc = TENSOR3(a[1], t_float32, pages[0], pages[1], 2);
    k = new_rows(a[2], idx, n_tok, pages[1], &ks, &ok);
    v = new_rows(a[3], idx, n_tok, pages[1], &vs, &ok);
    slots = TENSOR1(a[4], t_int32, n_tok);
    if (a[5] != Py_None) {
        if (dims_of(a[5], keys) != 4 || !fits(keys[0]) || !fits(keys[2]))
            Py_RETURN_NONE;
        kt = TENSOR4(a[5], t_float32, keys[0], pages[1], keys[2], D);
        req = TENSOR1(a[6], t_int32, n_tok);
        pos = TENSOR1(a[7], t_int32, n_tok);
    }
    st = OPTIONAL(a[8], TENSOR1(a[8], t_int32, 1));
    if (!ok)
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = f_append(kv, sc, (int)pages[0], (int)pages[1], k, v, ks, vs, slots, (int)n_tok, kt, (int)keys[0], (int)keys[2], req, pos,
                  st, stream);
    Py_END_ALLOW_THREADS
    (void)self;
    return PyLong_FromLong(rc);
}

/* idx, stream, Q, kv_pages, kv_scale, block_table, seq_len, O, workspace, blk_idx, count, lse, scale, status */
static PyObject *paged_decode_attn_f8(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    long long heads[MOST_DIMS], pages[MOST_DIMS], table[MOST_DIMS], list[MOST_DIMS] = {0}, idx, bytes;
    void *stream, *q, *kv, *sc, *tb, *len, *o, *ws, *ids = NULL, *cnt = NULL, *lse, *st;
    double scale;
    int ok = 1, rc;
    if (n != 14)
        return PyErr_Format(PyExc_TypeError, "paged_decode_attn_f8 takes 14 arguments");
    idx = PyLong_AsLongLong(a[0]);
    stream = (void *)(intptr_t)PyLong_AsLongLong(a[1]);
    scale = PyFloat_AsDouble(a[12]);
    if (PyErr_Occurred())
        return NULL;
    a += 2;
    if (dims_of(a[0], heads) != 3 || dims_of(a[1], pages) != 5 || dims_of(a[3], table) != 2)
        Py_RETURN_NONE;
    bytes = numel(a[6]);
    if (!fits(heads[1]) || !fits(pages[0]) || !fits(pages[1]) || !fits(table[0]) || !fits(table[1]))
        Py_RETURN_NONE;
    q = TENSOR3(a[0], t_bfloat16, table[0], heads[1], D);
    kv = TENSOR5(a[1], t_float8, pages[0], pages[1], 2, BLK, D);
    sc = TENSOR3(a[2], t_float32, pages[0], pages[1], 2);
    tb = TENSOR2(a[3], t_int32, table[0], table[1]);
    len = TENSOR1(a[4], t_int32, table[0]);
    o = TENSOR3(a[5], t_bfloat16, table[0], heads[1], D);
    ws = TENSOR1(a[6], t_uint8, bytes);
    if (a[7] != Py_None) {
        if (dims_of(a[7], list) != 3 || !fits(list[2]))
            Py_RETURN_NONE;
        ids = TENSOR3(a[7], t_int32, table[0], pages[1], list[2]);
        cnt = TENSOR2(a[8], t_int32, table[0], pages[1]);
    }
    lse = OPTIONAL(a[9], TENSOR2(a[9], t_float32, table[0], heads[1]));
    st = OPTIONAL(a[11], TENSOR1(a[11], t_int32, 1));
    if (!ok)
        Py_RETURN_NONE;
    Py_BEGIN_ALLOW_THREADS
    rc = f_attn(q, kv, sc, (int)pages[0], tb, (int)table[1], ids, cnt, (int)list[2], len, (int)table[0], (int)heads[1],
                (int)pages[1], (float)scale, o, lse, ws, (size_t)bytes, st, stream);
    Py_END_ALLOW_THREADS
    (void)self;
    return PyLong_FromLong(rc);
}

/* setup(int32, float32, bfloat16, float8_e4m3fn, uint8, page_plan, paged_append_f8, paged_decode_attn_f8):
 * torch's types, and the entry points' addresses. */
static PyObject *setup(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    PyObject **types[5] = {&t_int32, &t_float32, &t_bfloat16, &t_float8, &t_uint8};
    intptr_t f[3];
    int i;
    if (n != 8)
        return PyErr_Format(PyExc_TypeError, "setup takes 8 arguments");
    for (i = 0; i < 3; ++i)
        f[i] = (intptr_t)PyLong_AsLongLong(a[5 + i]);
    if (PyErr_Occurred())
        return NULL;
    for (i = 0; i < 5; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*types[i], a[i]);
    }
    f_plan = (plan_fn)f[0];
    f_append = (append_fn)f[1];
    f_attn = (attn_fn)f[2];
    (void)self;
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, NULL},
    {"page_plan", (PyCFunction)(void (*)(void))page_plan, METH_FASTCALL, NULL},
    {"paged_append_f8", (PyCFunction)(void (*)(void))paged_append_f8, METH_FASTCALL, NULL},
    {"paged_decode_attn_f8", (PyCFunction)(void (*)(void))paged_decode_attn_f8, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void)
{
    PyObject **names[7] = {&s_dtype, &s_shape, &s_get_device, &s_is_contiguous, &s_data_ptr, &s_stride, &s_numel};
    static const char *const text[7] = {"dtype", "shape", "get_device", "is_contiguous", "data_ptr", "stride", "numel"};
    int i;
    for (i = 0; i < 7; ++i)
        if ((*names[i] = PyUnicode_InternFromString(text[i])) == NULL)
            return NULL;
    return PyModule_Create(&module);
}
