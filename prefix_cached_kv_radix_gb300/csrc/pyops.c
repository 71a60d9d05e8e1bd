/* _rxops: the argument checks and marshalling of the row, page and prompt operators as a CPython
 * extension: what the binding's Python code does for kv_pool_write_rope, kv_pool_copy,
 * kv_pool_fork and prompt_attention, with the same checks and the same library calls, in a
 * fraction of the time (a decode step's rotary write takes a few microseconds on the GPU, and
 * its 20 arguments as many in the interpreter).  No arithmetic of the operators happens here.
 *
 *   bind({"int32": dtype, "int64", "float32", "bfloat16", "get_device": f() -> index,
 *         "raw_stream": f(index) -> stream, "kv_pool_write_rope": address, ... })
 *   kv_pool_write_rope(desc_addr, rope_addr, batch, ..., stream) -> rc        (and the others)
 *
 * Tensors are read through their dtype, shape, stride(), data_ptr() and get_device().  A wrong
 * argument raises ValueError.  stream: None (the current stream) or the stream's address.  The
 * GIL is released during the native call. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "radix_attn.h"

typedef int (*rope_fn)(const rx_attn_desc*, const rx_rope_desc*, int32_t, const int32_t*, const int64_t*, const int32_t*,
                       const int64_t*, const int32_t*, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                       void*, int64_t, void*, int64_t, void*, void*, int32_t*, int64_t, int64_t, int32_t*, void*);
typedef int (*copy_fn)(const rx_attn_desc*, int32_t, void* const*, int64_t, int64_t, const int32_t*, const int32_t*, int32_t*, void*);
typedef int (*fork_fn)(const rx_attn_desc*, int32_t, void* const*, int32_t, const int32_t*, const int32_t*, const int32_t*,
                       const int64_t*, const int32_t*, const int32_t*, int32_t, int64_t, int32_t*, int64_t, int64_t, int32_t*, void*);
typedef int (*prompt_fn)(const rx_attn_desc*, int32_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                         const int64_t*, void*, int64_t, float*, int64_t, int32_t*, void*);

static rope_fn g_rope;
static copy_fn g_copy;
static fork_fn g_fork;
static prompt_fn g_prompt;
static PyObject *g_i32, *g_i64, *g_f32, *g_bf16;      /* torch dtypes */
static PyObject *g_get_device, *g_raw_stream;         /* callables */
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device, *s_contig, *s_numel;

/* ------------------------------------------------------------------ plain values */
static int as_i64(PyObject* o, int64_t* out) {
    *out = PyLong_AsLongLong(o);
    return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int as_i32(PyObject* o, int32_t* out) {
    int64_t v;
    if (as_i64(o, &v)) return -1;
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_Format(PyExc_ValueError, "%lld does not fit 32 bits", (long long)v);
        return -1;
    }
    *out = (int32_t)v;
    return 0;
}

static int as_ptr(PyObject* o, void** out) {
    *out = PyLong_AsVoidPtr(o);
    return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

/* the result of a method without arguments as an integer */
static int call_i64(PyObject* o, PyObject* method, int64_t* out) {
    PyObject* r = PyObject_CallMethodNoArgs(o, method);
    if (!r) return -1;
    const int rc = as_i64(r, out);
    Py_DECREF(r);
    return rc;
}

static int data_ptr(PyObject* o, void** out) {
    PyObject* r = PyObject_CallMethodNoArgs(o, s_data_ptr);
    if (!r) return -1;
    const int rc = as_ptr(r, out);
    Py_DECREF(r);
    return rc;
}

/* ------------------------------------------------------------------ tensors */
static int here(const char* name, PyObject* t, int64_t dev) {
    int64_t d;
    if (call_i64(t, s_get_device, &d)) return -1;
    if (d != dev) {
        PyErr_Format(PyExc_ValueError, d < 0 ? "%s: not on a CUDA device" : "%s: on device %lld, but the current device is cuda:%lld",
                     name, (long long)d, (long long)dev);
        return -1;
    }
    return 0;
}

static int has_dtype(const char* name, PyObject* t, PyObject* want) {
    PyObject* dt = PyObject_GetAttr(t, s_dtype);
    if (!dt) return -1;
    const int same = dt == want;
    Py_DECREF(dt);
    if (!same) PyErr_Format(PyExc_ValueError, "%s: want %R", name, want);
    return same ? 0 : -1;
}

/* up to `n` entries of shape or strides; the number there are, -1 on an error */
static int extents(PyObject* tuple, int64_t* out, int n) {
    if (!tuple) return -1;
    int have = PyTuple_Check(tuple) ? (int)PyTuple_GET_SIZE(tuple) : -1;
    for (int i = 0; i < have && i < n; ++i)
        if (as_i64(PyTuple_GET_ITEM(tuple, i), out + i)) have = -1;
    Py_DECREF(tuple);
    return have;
}

static PyObject* dtype_of(const rx_attn_desc* d) { return d->dtype == RX_F32 ? g_f32 : g_bf16; }

/* rows [>= total, heads, head_dim] of the descriptor's type, the heads of a row contiguous */
static int rows(const char* name, PyObject* t, int32_t heads, const rx_attn_desc* d, int64_t total, int64_t dev, void** ptr,
                int64_t* stride) {
    *ptr = NULL;
    *stride = 0;
    if (t == Py_None) return 0;
    int64_t sh[3] = {0, 0, 0}, st[3] = {0, 0, 0};
    if (has_dtype(name, t, dtype_of(d)) || here(name, t, dev)) return -1;
    const int nd = extents(PyObject_GetAttr(t, s_shape), sh, 3);
    if (nd < 0 || extents(PyObject_CallMethodNoArgs(t, s_stride), st, 3) < 0) return -1;
    if (nd != 3 || sh[1] != heads || sh[2] != d->head_dim || sh[0] < total || st[2] != 1 || (heads > 1 && st[1] != d->head_dim)) {
        PyErr_Format(PyExc_ValueError, "%s: want [%lld, %d, %d] with contiguous heads", name, (long long)total, (int)heads,
                     (int)d->head_dim);
        return -1;
    }
    const int64_t row = (int64_t)heads * d->head_dim;
    *stride = sh[0] > 1 || st[0] > row ? st[0] : row;
    return data_ptr(t, ptr);
}

/* `count` or more contiguous elements of a type, or a device address as it is */
static int array(const char* name, PyObject* t, PyObject* dtype, int64_t count, int64_t dev, void** ptr) {
    *ptr = NULL;
    if (t == Py_None) return 0;
    if (PyLong_Check(t)) return as_ptr(t, ptr);
    if (has_dtype(name, t, dtype) || here(name, t, dev)) return -1;
    PyObject* c = PyObject_CallMethodNoArgs(t, s_contig);
    if (!c) return -1;
    const int contiguous = c == Py_True;
    Py_DECREF(c);
    int64_t n;
    if (call_i64(t, s_numel, &n)) return -1;
    if (!contiguous || n < count) {
        PyErr_Format(PyExc_ValueError, "%s: want %lld contiguous elements", name, (long long)count);
        return -1;
    }
    return data_ptr(t, ptr);
}

/* a KV pool: contiguous [num_slots, hkv, head_dim] */
static int pool(const char* name, PyObject* t, const rx_attn_desc* d, int64_t dev, void** ptr) {
    const int64_t n = d->num_slots * d->hkv * d->head_dim;
    int64_t have;
    if (t == Py_None || PyLong_Check(t)) {
        PyErr_Format(PyExc_ValueError, "%s: want a tensor", name);
        return -1;
    }
    if (array(name, t, dtype_of(d), n, dev, ptr) || call_i64(t, s_numel, &have)) return -1;
    if (have != n) {
        PyErr_Format(PyExc_ValueError, "%s: want [%lld, %d, %d]", name, (long long)d->num_slots, (int)d->hkv, (int)d->head_dim);
        return -1;
    }
    return 0;
}

/* a table [rows, stride] of slots, its shape too */
static int table(const char* name, PyObject* t, int64_t dev, void** ptr, int64_t* n_rows, int64_t* stride) {
    int64_t sh[2] = {0, 0};
    if (array(name, t, g_i32, 0, dev, ptr)) return -1;
    const int nd = extents(PyObject_GetAttr(t, s_shape), sh, 2);
    if (nd < 0) return -1;
    if (nd != 2) {
        PyErr_Format(PyExc_ValueError, "%s: want [rows, stride]", name);
        return -1;
    }
    *n_rows = sh[0];
    *stride = sh[1];
    return 0;
}

static int current(PyObject* stream, int64_t* dev, void** out) {
    PyObject* d = PyObject_CallNoArgs(g_get_device);
    if (!d) return -1;
    int rc = as_i64(d, dev);
    if (!rc && stream != Py_None) {
        rc = as_ptr(stream, out);
    } else if (!rc) {
        PyObject* s = PyObject_CallOneArg(g_raw_stream, d);
        rc = s ? as_ptr(s, out) : -1;
        Py_XDECREF(s);
    }
    Py_DECREF(d);
    return rc;
}

static int want_args(Py_ssize_t have, Py_ssize_t want, const void* bound) {
    if (have != want || !bound) {
        PyErr_Format(PyExc_TypeError, bound ? "%zd arguments, got %zd" : "not bound", want, have);
        return -1;
    }
    return 0;
}

/* ------------------------------------------------------------------ the operators */
static PyObject* py_rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (want_args(n, 20, (const void*)g_rope)) return NULL;
    const rx_attn_desc* d;
    const rx_rope_desc* r;
    int32_t batch;
    int64_t total, dev, qs, ks, vs, os, xs, rt_stride = 0, sh[2] = {0, 0}, unused;
    void *ps, *pi, *ns, *qi, *pos, *q, *k, *v, *o, *x, *kp = NULL, *vp = NULL, *rt, *st, *stream;
    if (as_ptr(a[0], (void**)&d) || as_ptr(a[1], (void**)&r) || as_i32(a[2], &batch) || as_i64(a[16], &total) ||
        current(a[19], &dev, &stream))
        return NULL;
    if (rows("q", a[8], d->hq, d, total, dev, &q, &qs) || rows("k_new", a[9], d->hkv, d, total, dev, &k, &ks) ||
        rows("v_new", a[10], d->hkv, d, total, dev, &v, &vs) || rows("q_out", a[11], d->hq, d, total, dev, &o, &os) ||
        rows("k_out", a[12], d->hkv, d, total, dev, &x, &xs))
        return NULL;
    if (extents(PyObject_GetAttr(a[7], s_shape), sh, 2) != 2 || sh[0] != r->n_axes || sh[1] < total) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "positions: want [%d, %lld]", (int)r->n_axes, (long long)total);
        return NULL;
    }
    if (a[5] != Py_None && (pool("k_pool", a[13], d, dev, &kp) || pool("v_pool", a[14], d, dev, &vp))) return NULL;
    if (a[18] != Py_None) {                   /* the table's stride, where it is given as an address */
        if (as_i64(a[18], &rt_stride)) return NULL;
    } else if (a[15] != Py_None && table("req_to_token", a[15], dev, &rt, &unused, &rt_stride)) {
        return NULL;
    }
    if (array("prefix_slots", a[3], g_i32, 0, dev, &ps) || array("prefix_indptr", a[4], g_i64, batch + 1ll, dev, &pi) ||
        array("new_slots", a[5], g_i32, total, dev, &ns) || array("qo_indptr", a[6], g_i64, batch + 1ll, dev, &qi) ||
        array("positions", a[7], g_i32, 0, dev, &pos) || array("req_to_token", a[15], g_i32, batch * rt_stride, dev, &rt) ||
        array("status", a[17], g_i32, 1, dev, &st))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = g_rope(d, r, batch, ps, pi, ns, qi, pos, sh[1], q, qs, k, ks, v, vs, o, os, x, xs, kp, vp, rt,
                                       rt_stride, total, st, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
}

/* the pools' addresses, in a block the caller frees with PyMem_Free; NULL on an error */
static void** pool_list(PyObject* seq, const rx_attn_desc* d, int64_t dev, int32_t* n) {
    PyObject* f = PySequence_Fast(seq, "pools: want a sequence of tensors");
    if (!f) return NULL;
    const Py_ssize_t m = PySequence_Fast_GET_SIZE(f);
    void** p = PyMem_Malloc(sizeof(void*) * (size_t)(m + 1));
    if (!p) PyErr_NoMemory();
    for (Py_ssize_t i = 0; p && i < m; ++i)
        if (pool("pools", PySequence_Fast_GET_ITEM(f, i), d, dev, p + i)) {
            PyMem_Free(p);
            p = NULL;
        }
    Py_DECREF(f);
    *n = (int32_t)m;
    return p;
}

static PyObject* py_copy(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (want_args(n, 7, (const void*)g_copy)) return NULL;
    const rx_attn_desc* d;
    int32_t np;
    int64_t page, dev, count, count2;
    void *src, *dst, *st, *stream, **list;
    if (as_ptr(a[0], (void**)&d) || as_i64(a[4], &page) || current(a[6], &dev, &stream)) return NULL;
    if (call_i64(a[2], s_numel, &count) || call_i64(a[3], s_numel, &count2)) return NULL;
    if (count != count2) {
        PyErr_SetString(PyExc_ValueError, "src, dst: one destination per source");
        return NULL;
    }
    if (array("src", a[2], g_i32, 0, dev, &src) || array("dst", a[3], g_i32, 0, dev, &dst) || array("status", a[5], g_i32, 1, dev, &st))
        return NULL;
    if (!(list = pool_list(a[1], d, dev, &np))) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = g_copy(d, np, list, page, count, src, dst, st, stream);
    Py_END_ALLOW_THREADS PyMem_Free(list);
    return PyLong_FromLong(rc);
}

static PyObject* py_fork(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (want_args(n, 12, (const void*)g_fork)) return NULL;
    const rx_attn_desc* d;
    int32_t np;
    int64_t total, dev, in_rows, in_stride, out_rows, out_stride;
    void *par, *keep, *len, *ti, *ts, *in, *out, *st, *stream, **list;
    if (as_ptr(a[0], (void**)&d) || as_i64(a[9], &total) || current(a[11], &dev, &stream)) return NULL;
    if (table("r2t_in", a[7], dev, &in, &in_rows, &in_stride) || table("r2t_out", a[8], dev, &out, &out_rows, &out_stride) ||
        array("parents", a[2], g_i32, out_rows, dev, &par) || array("keep_lens", a[3], g_i32, out_rows, dev, &keep) ||
        array("kv_lens", a[4], g_i32, out_rows, dev, &len) || array("tail_indptr", a[5], g_i64, out_rows + 1, dev, &ti) ||
        array("tail_slots", a[6], g_i32, total, dev, &ts) || array("status", a[10], g_i32, 1, dev, &st))
        return NULL;
    if (in_rows > INT32_MAX || out_rows > INT32_MAX) {
        PyErr_SetString(PyExc_ValueError, "tables: too many rows");
        return NULL;
    }
    if (!(list = pool_list(a[1], d, dev, &np))) return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = g_fork(d, np, list, (int32_t)out_rows, par, keep, len, ti, ts, in, (int32_t)in_rows, in_stride, out,
                                       out_stride, total, st, stream);
    Py_END_ALLOW_THREADS PyMem_Free(list);
    return PyLong_FromLong(rc);
}

static PyObject* py_prompt(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (want_args(n, 11, (const void*)g_prompt)) return NULL;
    const rx_attn_desc* d;
    int32_t batch;
    int64_t total, dev, qs, ks, vs, os;
    void *q, *k, *v, *o, *ip, *lse, *st, *stream;
    if (as_ptr(a[0], (void**)&d) || as_i32(a[1], &batch) || as_i64(a[8], &total) || current(a[10], &dev, &stream)) return NULL;
    if (rows("q", a[2], d->hq, d, total, dev, &q, &qs) || rows("k", a[3], d->hkv, d, total, dev, &k, &ks) ||
        rows("v", a[4], d->hkv, d, total, dev, &v, &vs) || rows("out", a[6], d->hq, d, total, dev, &o, &os) ||
        array("indptr", a[5], g_i64, batch + 1ll, dev, &ip) || array("lse", a[7], g_f32, total * d->hq, dev, &lse) ||
        array("status", a[9], g_i32, 1, dev, &st))
        return NULL;
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = g_prompt(d, batch, q, qs, k, ks, v, vs, ip, o, os, lse, total, st, stream);
    Py_END_ALLOW_THREADS return PyLong_FromLong(rc);
}

/* ------------------------------------------------------------------ module */
static PyObject* py_bind(PyObject* self, PyObject* m) {
    (void)self;
    const struct {
        const char* key;
        PyObject** to;
    } objs[] = {{"int32", &g_i32},       {"int64", &g_i64},           {"float32", &g_f32},
                {"bfloat16", &g_bf16}, {"get_device", &g_get_device}, {"raw_stream", &g_raw_stream}};
    for (size_t i = 0; i < sizeof(objs) / sizeof(objs[0]); ++i) {
        PyObject* o = PyMapping_GetItemString(m, objs[i].key);
        if (!o) return NULL;
        Py_XSETREF(*objs[i].to, o);
    }
    void* f[4];
    const char* names[4] = {"kv_pool_write_rope", "kv_pool_copy", "kv_pool_fork", "prompt_attention"};
    for (int i = 0; i < 4; ++i) {
        PyObject* o = PyMapping_GetItemString(m, names[i]);
        if (!o || as_ptr(o, &f[i])) {
            Py_XDECREF(o);
            return NULL;
        }
        Py_DECREF(o);
    }
    g_rope = (rope_fn)f[0];
    g_copy = (copy_fn)f[1];
    g_fork = (fork_fn)f[2];
    g_prompt = (prompt_fn)f[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", py_bind, METH_O, "Bind torch's types and the library's functions."},
                                {"kv_pool_write_rope", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, ""},
                                {"kv_pool_copy", (PyCFunction)(void (*)(void))py_copy, METH_FASTCALL, ""},
                                {"kv_pool_fork", (PyCFunction)(void (*)(void))py_fork, METH_FASTCALL, ""},
                                {"prompt_attention", (PyCFunction)(void (*)(void))py_prompt, METH_FASTCALL, ""},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rxops", "Marshalling of the row, page and prompt operators.", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__rxops(void) {
    s_dtype = PyUnicode_InternFromString("dtype");
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_contig = PyUnicode_InternFromString("is_contiguous");
    s_numel = PyUnicode_InternFromString("numel");
    if (!s_dtype || !s_shape || !s_stride || !s_data_ptr || !s_get_device || !s_contig || !s_numel) return NULL;
    return PyModule_Create(&module);
}
