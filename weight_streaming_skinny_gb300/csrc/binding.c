/*
 * Calls of the entry points around the linears from Python: reads the tensors'
 * types, devices, shapes and addresses through their Python attributes, checks
 * what the library cannot (that a pointer means what it should) and calls.
 *
 * A decode step makes these calls for every layer, and small ones take the GPU
 * less time than the host: marshalling by interpreted code and ctypes took 6 us of
 * a call's 14, this takes under 2.
 *
 * Each function returns the call's dl_status, or LOOK if some argument is not
 * what the plain case wants: the caller then says what is wrong with it.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <stdint.h>

#include "dl_linear.h"

enum { LOOK = -1, OTHER_DEVICE = -2 };

typedef int (*get_device_fn)(int*);
typedef dl_status (*append_fn)(const dl_kv_cache*, const void*, const void*, const void*, long long, long long,
                               long long, void*, const float*, const float*, int, int, const int*, const int*, int,
                               const int*, const int*, int, int, int, int, void*);
typedef dl_status (*attention_fn)(const dl_kv_cache*, const void*, long long, void*, float*, const int*, int,
                                  const int*, const int*, int, int, int, int, float, void*, size_t, void*);
typedef dl_status (*verify_fn)(const int*, const void*, const void*, int, const float*, const float*, const int*, int*,
                               int*, int, int, int, void*);

typedef dl_status (*norm_fn)(const dl_rows*, const dl_norm*, const dl_rows*, int, int, float, const dl_rows*, float,
                             const dl_norm*, const dl_rows*, const dl_rows*, int, int, void*);
typedef dl_status (*adapters_fn)(const dl_adapters*, const dl_rows*, const int*, const dl_rows*, const dl_rows*,
                                 const dl_rows*, int, void*, size_t, void*);
typedef dl_status (*free_fn)(const dl_kv_pages*, const int*, int, void*);
typedef dl_status (*list_fn)(const dl_kv_pages*, const int*, const int*, int*, int, void*, size_t, void*);
typedef dl_status (*compact_fn)(const dl_kv_pages*, int*, void*, size_t, void*);

static PyObject *g_tensor, *g_bf16, *g_i32, *g_f32, *g_raw_stream;
static get_device_fn g_get_device;
static append_fn g_append;
static attention_fn g_attention;
static verify_fn g_verify;
static norm_fn g_norm;
static adapters_fn g_adapters;
static free_fn g_free;
static list_fn g_reserve, g_fork;
static compact_fn g_compact;
static PyObject *s_dtype, *s_shape, *s_stride, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_cuda_stream;

/* Up to 4 integers of a tuple; -1 if it is none or has more. */
static int integers(PyObject* t, long long* v) {
    if (!t || !PyTuple_Check(t) || PyTuple_GET_SIZE(t) > 4) return -1;
    const int n = (int)PyTuple_GET_SIZE(t);
    for (int i = 0; i < n; ++i) {
        v[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (v[i] == -1 && PyErr_Occurred()) return -1;
    }
    return n;
}

typedef struct {
    void* ptr;
    int dims;
    long long shape[4], stride[4];
} view;

static int call_long(PyObject* t, PyObject* name, long long* out) {
    PyObject* r = PyObject_CallMethodNoArgs(t, name);
    if (!r) return 0;
    *out = PyLong_AsLongLong(r);
    Py_DECREF(r);
    return !(*out == -1 && PyErr_Occurred());
}

/* A tensor of `dtype` on device `dev`, dense unless `strided`; 0 if it is not that. */
static int look_at(PyObject* t, PyObject* dtype, long long dev, int strided, view* v) {
    long long x;
    if (!PyObject_TypeCheck(t, (PyTypeObject*)g_tensor)) return 0;
    PyObject* a = PyObject_GetAttr(t, s_dtype);
    if (!a) return 0;
    const int same = a == dtype;
    Py_DECREF(a);
    if (!same || !call_long(t, s_get_device, &x) || x != dev) return 0;
    a = PyObject_GetAttr(t, s_shape);
    v->dims = integers(a, v->shape);
    Py_XDECREF(a);
    if (v->dims < 0) return 0;
    if (strided) {
        a = PyObject_CallMethodNoArgs(t, s_stride);
        const int n = integers(a, v->stride);
        Py_XDECREF(a);
        if (n != v->dims) return 0;
    } else {
        a = PyObject_CallMethodNoArgs(t, s_is_contiguous);
        if (!a) return 0;
        const int dense = a == Py_True;
        Py_DECREF(a);
        if (!dense) return 0;
    }
    if (!call_long(t, s_data_ptr, &x)) return 0;
    v->ptr = (void*)(uintptr_t)x;
    return 1;
}

/* bf16 [tokens, heads, dim], a token's heads dense: elements from one token to the next. */
static int look_at_rows(PyObject* t, long long heads, long long dim, long long dev, view* v, long long* step) {
    if (!look_at(t, g_bf16, dev, 1, v) || v->dims != 3 || v->shape[2] != dim || (heads >= 0 && v->shape[1] != heads))
        return 0;
    if (v->shape[0] && v->shape[1] && (v->stride[2] != 1 || (v->shape[1] > 1 && v->stride[1] != dim))) return 0;
    *step = v->shape[0] > 1 ? v->stride[0] : v->shape[1] * dim;      /* one token has no next one */
    return 1;
}

static long long numel(const view* v) {
    long long n = 1;
    for (int i = 0; i < v->dims; ++i) n *= v->shape[i];
    return n;
}

/* The stream's address: None is the device's current one. */
static int stream_of(PyObject* s, long long dev, void** out) {
    long long x;
    PyObject* r;
    if (s == Py_None) {
        PyObject* d = PyLong_FromLongLong(dev);
        if (!d) return 0;
        r = PyObject_CallOneArg(g_raw_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(s)) {
        r = s;
        Py_INCREF(r);
    } else {
        r = PyObject_GetAttr(s, s_cuda_stream);
    }
    if (!r) return 0;
    x = PyLong_AsLongLong(r);
    Py_DECREF(r);
    if (x == -1 && PyErr_Occurred()) return 0;
    *out = (void*)(uintptr_t)x;
    return 1;
}

static int fits(long long x) { return x >= INT32_MIN && x <= INT32_MAX; }

/* block_table [batch, columns], seq_lens [batch], q_start [batch + 1] */
static int look_at_sequences(PyObject* table, PyObject* lens, PyObject* start, long long dev, view* t, view* l, view* s) {
    if (!look_at(table, g_i32, dev, 0, t) || !look_at(lens, g_i32, dev, 0, l) || !look_at(start, g_i32, dev, 0, s)) return 0;
    const long long batch = numel(l);
    return t->dims == 2 && t->shape[0] == batch && numel(s) == batch + 1 && fits(batch) && fits(t->shape[1]);
}

static int current(long long dev) {
    int now = -1;
    return g_get_device(&now) == 0 && now == dev;
}

/* The library's calls: other Python threads run meanwhile (a launch waits where the driver's queue is full). */
#define CALL(status, call)     \
    do {                       \
        Py_BEGIN_ALLOW_THREADS \
        status = (call);       \
        Py_END_ALLOW_THREADS \
    } while (0)

static PyObject* answer(long code) {
    if (code == LOOK) PyErr_Clear();
    return PyLong_FromLong(code);
}

/* attention(cache, device, kv_heads, dim, q, table, lens, start, max_q, scale, out, lse, workspace, bytes, stream) */
static PyObject* attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 15) return answer(LOOK);
    const uintptr_t cache = (uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    const long long dev = PyLong_AsLongLong(a[1]), heads = PyLong_AsLongLong(a[2]), dim = PyLong_AsLongLong(a[3]);
    const long long max_q = PyLong_AsLongLong(a[8]);
    const double scale = PyFloat_AsDouble(a[9]);
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[12]);
    const unsigned long long bytes = PyLong_AsUnsignedLongLong(a[13]);
    view q, t, l, s, o, e = {0};
    long long step;
    void* stream;
    if (PyErr_Occurred() || !fits(max_q) || !look_at_rows(a[4], -1, dim, dev, &q, &step) ||
        !look_at_sequences(a[5], a[6], a[7], dev, &t, &l, &s) || !look_at(a[10], g_bf16, dev, 0, &o) ||
        numel(&o) != numel(&q) || (a[11] != Py_None && (!look_at(a[11], g_f32, dev, 0, &e) || numel(&e) != q.shape[0] * q.shape[1])) ||
        !fits(q.shape[0]) || !fits(q.shape[1]) || !stream_of(a[14], dev, &stream))
        return answer(LOOK);
    (void)heads;
    if (!current(dev)) return answer(OTHER_DEVICE);
    dl_status status;
    CALL(status, g_attention((const dl_kv_cache*)cache, q.ptr, step, o.ptr, (float*)e.ptr, (const int*)t.ptr, (int)t.shape[1],
                             (const int*)l.ptr, (const int*)s.ptr, (int)t.shape[0], (int)q.shape[0], (int)q.shape[1],
                             (int)max_q, (float)scale, (void*)ws, (size_t)bytes, stream));
    return answer(status);
}

/* append(cache, device, kv_heads, dim, q, k, v, table, lens, start, max_q, cos, sin, positions, out, stream) */
static PyObject* append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 16) return answer(LOOK);
    const uintptr_t cache = (uintptr_t)PyLong_AsUnsignedLongLong(a[0]);
    const long long dev = PyLong_AsLongLong(a[1]), heads = PyLong_AsLongLong(a[2]), dim = PyLong_AsLongLong(a[3]);
    const long long max_q = PyLong_AsLongLong(a[10]);
    view q = {0}, k, v, t, l, s, c = {0}, i = {0}, p = {0}, o = {0};
    long long qs = 0, ks, vs, q_heads = 0, places = 0, rotary = 0;
    void* stream;
    if (PyErr_Occurred() || !fits(max_q) || !look_at_rows(a[5], heads, dim, dev, &k, &ks) ||
        !look_at_rows(a[6], heads, dim, dev, &v, &vs) || !look_at_sequences(a[7], a[8], a[9], dev, &t, &l, &s) ||
        v.shape[0] != k.shape[0] || !fits(k.shape[0]))
        return answer(LOOK);
    if (a[4] != Py_None) {
        if (!look_at_rows(a[4], -1, dim, dev, &q, &qs) || q.shape[0] != k.shape[0] || !look_at(a[14], g_bf16, dev, 0, &o) ||
            o.dims != 3 || o.shape[0] != q.shape[0] || o.shape[1] != q.shape[1] || o.shape[2] != dim || !fits(q.shape[1]))
            return answer(LOOK);
        q_heads = q.shape[1];
    } else if (a[14] != Py_None) {
        return answer(LOOK);
    }
    if (a[11] != Py_None || a[12] != Py_None) {
        if (!look_at(a[11], g_f32, dev, 0, &c) || !look_at(a[12], g_f32, dev, 0, &i) || c.dims != 2 || i.dims != 2 ||
            c.shape[0] != i.shape[0] || c.shape[1] != i.shape[1] || !fits(c.shape[0]) || !fits(2 * c.shape[1]))
            return answer(LOOK);
        places = c.shape[0];
        rotary = 2 * c.shape[1];
    }
    if ((a[13] != Py_None && (!look_at(a[13], g_i32, dev, 0, &p) || numel(&p) != k.shape[0])) ||
        !stream_of(a[15], dev, &stream))
        return answer(LOOK);
    if (!current(dev)) return answer(OTHER_DEVICE);
    dl_status status;
    CALL(status, g_append((const dl_kv_cache*)cache, q.ptr, k.ptr, v.ptr, qs, ks, vs, o.ptr, (const float*)c.ptr,
                          (const float*)i.ptr, (int)rotary, (int)places, (const int*)p.ptr, (const int*)t.ptr,
                          (int)t.shape[1], (const int*)l.ptr, (const int*)s.ptr, (int)t.shape[0], (int)k.shape[0],
                          (int)q_heads, (int)max_q, stream));
    return answer(status);
}

/* verify(device, drafts, target, u, u_next, draft_probs, draft_lens, tokens, count, stream) */
static PyObject* verify(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 10) return answer(LOOK);
    const long long dev = PyLong_AsLongLong(a[0]);
    view d, t, u, x, g = {0}, l = {0}, k, c;
    void* stream;
    if (PyErr_Occurred() || !look_at(a[1], g_i32, dev, 0, &d) || d.dims != 2) return answer(LOOK);
    const long long B = d.shape[0], S = d.shape[1];
    PyObject* kind = g_f32;
    if (!look_at(a[2], g_f32, dev, 0, &t)) {
        PyErr_Clear();
        kind = g_bf16;
        if (!look_at(a[2], g_bf16, dev, 0, &t)) return answer(LOOK);
    }
    if (t.dims != 3 || t.shape[0] != B || t.shape[1] != S + 1 || !look_at(a[3], g_f32, dev, 0, &u) || numel(&u) != B * S ||
        !look_at(a[4], g_f32, dev, 0, &x) || numel(&x) != B ||
        (a[5] != Py_None && (!look_at(a[5], kind, dev, 0, &g) || g.dims != 3 || g.shape[0] != B || g.shape[1] != S ||
                             g.shape[2] != t.shape[2])) ||
        (a[6] != Py_None && (!look_at(a[6], g_i32, dev, 0, &l) || numel(&l) != B)) ||
        !look_at(a[7], g_i32, dev, 0, &k) || numel(&k) != B * (S + 1) || !look_at(a[8], g_i32, dev, 0, &c) ||
        numel(&c) != B || !fits(B) || !fits(S) || !fits(t.shape[2]) || !stream_of(a[9], dev, &stream))
        return answer(LOOK);
    if (!current(dev)) return answer(OTHER_DEVICE);
    dl_status status;
    CALL(status, g_verify((const int*)d.ptr, g.ptr, t.ptr, kind == g_f32 ? DL_PROBS_F32 : DL_PROBS_BF16, (const float*)u.ptr,
                          (const float*)x.ptr, (const int*)l.ptr, (int*)k.ptr, (int*)c.ptr, (int)B, (int)S,
                          (int)t.shape[2], stream));
    return answer(status);
}

/* bf16 or fp32 rows [n, dim] of device `dev`, a row dense (None: none). */
static int look_at_matrix(PyObject* t, long long dev, view* v, dl_rows* r) {
    r->data = NULL;
    if (t == Py_None) return 1;
    if (!PyObject_TypeCheck(t, (PyTypeObject*)g_tensor)) return 0;
    PyObject* a = PyObject_GetAttr(t, s_dtype);
    if (!a) return 0;
    const int f32 = a == g_f32;
    Py_DECREF(a);
    if (!look_at(t, f32 ? g_f32 : g_bf16, dev, 1, v) || v->dims != 2 || !fits(v->shape[0]) || !fits(v->shape[1]) ||
        (v->shape[1] > 1 && v->shape[0] > 0 && v->stride[1] != 1))
        return 0;
    r->data = v->ptr;
    r->stride = v->shape[0] > 1 ? v->stride[0] : v->shape[1];
    r->dtype = f32 ? DL_ROWS_F32 : DL_ROWS_BF16;
    return 1;
}

/* The address of a dense tensor that the caller has just made. */
static int look_at_made(PyObject* t, dl_rows* r, long long stride, int dtype) {
    long long x;
    if (!call_long(t, s_data_ptr, &x)) return 0;
    r->data = (void*)(uintptr_t)x;
    r->stride = stride;
    r->dtype = dtype;
    return 1;
}

/* A norm's description (address, length of its weights or -1, their device or -1), or None. */
static int look_at_norm(PyObject* t, long long dim, long long dev, const dl_norm** out) {
    long long v[4];
    *out = NULL;
    if (t == Py_None) return 1;
    if (integers(t, v) != 3 || (v[1] >= 0 && (v[1] != dim || v[2] != dev))) return 0;
    *out = (const dl_norm*)(uintptr_t)v[0];
    return 1;
}

/* norm(device, y, post, gate, act, scale, h, h_scale, pre, out_h, out_x, stream, made); made: 1 out_h, 2 out_x was made
 * for this call, like h (or y), in bf16 */
static PyObject* norm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 13) return answer(LOOK);
    const long long dev = PyLong_AsLongLong(a[0]), act = PyLong_AsLongLong(a[4]), made = PyLong_AsLongLong(a[12]);
    const double scale = PyFloat_AsDouble(a[5]), h_scale = PyFloat_AsDouble(a[7]);
    view v[5];
    dl_rows y, h, gate = {0}, r, x;
    const dl_norm *post, *pre;
    void* stream;
    int kind = DL_GATE_NONE;
    if (PyErr_Occurred() || !look_at_matrix(a[1], dev, &v[0], &y) || !look_at_matrix(a[6], dev, &v[1], &h) ||
        (a[1] == Py_None && a[6] == Py_None))
        return answer(LOOK);
    const view* like = a[1] != Py_None ? &v[0] : &v[1];
    const long long rows = like->shape[0], dim = like->shape[1];
    if ((a[6] != Py_None && (v[1].shape[0] != rows || v[1].shape[1] != dim)) ||
        !(made & 1 ? look_at_made(a[9], &r, dim, a[6] != Py_None ? h.dtype : y.dtype)
                   : look_at_matrix(a[9], dev, &v[2], &r) && (a[9] == Py_None || (v[2].shape[0] == rows && v[2].shape[1] == dim))) ||
        !(made & 2 ? look_at_made(a[10], &x, dim, DL_ROWS_BF16)
                   : look_at_matrix(a[10], dev, &v[3], &x) && (a[10] == Py_None || (v[3].shape[0] == rows && v[3].shape[1] == dim))) ||
        !look_at_norm(a[2], dim, dev, &post) || !look_at_norm(a[8], dim, dev, &pre) || !stream_of(a[11], dev, &stream))
        return answer(LOOK);
    if (a[3] != Py_None) {
        if (look_at_matrix(a[3], dev, &v[4], &gate)) {
            if (v[4].shape[0] != rows || (v[4].shape[1] != 1 && v[4].shape[1] != dim)) return answer(LOOK);
            kind = v[4].shape[1] == dim ? DL_GATE_FULL : DL_GATE_ROW;
        } else {
            PyErr_Clear();
            gate.dtype = DL_ROWS_F32;
            if (!look_at(a[3], g_f32, dev, 0, &v[4])) {
                PyErr_Clear();
                gate.dtype = DL_ROWS_BF16;
                if (!look_at(a[3], g_bf16, dev, 0, &v[4])) return answer(LOOK);
            }
            if (v[4].dims != 1 || v[4].shape[0] != dim) return answer(LOOK);
            gate.data = v[4].ptr;
            gate.stride = dim;
            kind = DL_GATE_CHANNEL;
        }
    }
    if (!current(dev)) return answer(OTHER_DEVICE);
    dl_status status;
    CALL(status, g_norm(&y, post, &gate, kind, (int)act, (float)scale, &h, (float)h_scale, pre, &r, &x, (int)rows, (int)dim,
                        stream));
    return answer(status);
}

/* adapters((address, device, K, N), x, index, base, out, out_f32, workspace, bytes, stream, made); made: 1 out was made
 * for this call */
static PyObject* adapters(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    long long d[4];
    if (n != 10 || integers(a[0], d) != 4) return answer(LOOK);
    const long long dev = d[1], K = d[2], N = d[3], made = PyLong_AsLongLong(a[9]);
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[6]);
    const unsigned long long bytes = PyLong_AsUnsignedLongLong(a[7]);
    view v, i;
    dl_rows x, base, y, y32;
    void* stream;
    if (PyErr_Occurred() || a[1] == Py_None || !look_at_matrix(a[1], dev, &v, &x) || x.dtype != DL_ROWS_BF16 || v.shape[1] != K)
        return answer(LOOK);
    const long long T = v.shape[0];
    if (!look_at(a[2], g_i32, dev, 0, &i) || numel(&i) != T || !look_at_matrix(a[3], dev, &v, &base) ||
        (a[3] != Py_None && (v.shape[0] != T || v.shape[1] != N)) ||
        !(made ? look_at_made(a[4], &y, N, DL_ROWS_BF16)
               : a[4] != Py_None && look_at_matrix(a[4], dev, &v, &y) && y.dtype == DL_ROWS_BF16 && v.shape[0] == T && v.shape[1] == N) ||
        !look_at_matrix(a[5], dev, &v, &y32) ||
        (a[5] != Py_None && (y32.dtype != DL_ROWS_F32 || v.shape[0] != T || v.shape[1] != N)) ||
        !stream_of(a[8], dev, &stream))
        return answer(LOOK);
    if (!current(dev)) return answer(OTHER_DEVICE);
    dl_status status;
    CALL(status, g_adapters((const dl_adapters*)(uintptr_t)d[0], &x, (const int*)i.ptr, &base, &y, &y32, (int)T, (void*)ws,
                            (size_t)bytes, stream));
    return answer(status);
}

/* pages(what, (address, device), list, list or None, done or live or None, workspace, bytes, stream, made); what: 0 free,
 * 1 reserve, 2 fork, 3 compact (no lists); made: 1 done or live was made for this call */
static PyObject* pages(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    long long d[4];
    if (n != 9 || integers(a[1], d) != 2) return answer(LOOK);
    const long long what = PyLong_AsLongLong(a[0]), dev = d[1], made = PyLong_AsLongLong(a[8]);
    dl_rows out;
    const dl_kv_pages* pool = (const dl_kv_pages*)(uintptr_t)d[0];
    const uintptr_t ws = (uintptr_t)PyLong_AsUnsignedLongLong(a[5]);
    const unsigned long long bytes = PyLong_AsUnsignedLongLong(a[6]);
    view x = {0}, y = {0}, z = {0};
    void* stream;
    if (PyErr_Occurred() || what < 0 || what > 3 || !stream_of(a[7], dev, &stream)) return answer(LOOK);
    if (what < 3 && (!look_at(a[2], g_i32, dev, 0, &x) || x.dims != 1 || !fits(x.shape[0]))) return answer(LOOK);
    if ((what == 1 || what == 2) && (!look_at(a[3], g_i32, dev, 0, &y) || y.dims != 1 || y.shape[0] != x.shape[0]))
        return answer(LOOK);
    if (made) {
        if (!look_at_made(a[4], &out, 0, 0)) return answer(LOOK);
        z.ptr = out.data;
    } else if (what > 0 && (!look_at(a[4], g_i32, dev, 0, &z) || z.dims != 1 || z.shape[0] != (what == 3 ? 1 : x.shape[0])))
        return answer(LOOK);
    if (!current(dev)) return answer(OTHER_DEVICE);
    const int count = (int)x.shape[0];
    dl_status status;
    if (what == 0)
        CALL(status, g_free(pool, (const int*)x.ptr, count, stream));
    else if (what == 3)
        CALL(status, g_compact(pool, (int*)z.ptr, (void*)ws, (size_t)bytes, stream));
    else
        CALL(status, (what == 1 ? g_reserve : g_fork)(pool, (const int*)x.ptr, (const int*)y.ptr, (int*)z.ptr, count,
                                                      (void*)ws, (size_t)bytes, stream));
    return answer(status);
}

/* `n` addresses from Python integers. */
static int addresses(PyObject* const* a, uintptr_t* f, int n) {
    for (int i = 0; i < n; ++i) f[i] = (uintptr_t)PyLong_AsUnsignedLongLong(a[i]);
    return !PyErr_Occurred();
}

/* bind(Tensor, bfloat16, int32, float32, raw_stream, get_device, append, attention, verify): types, and addresses */
static PyObject* bind(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 9 || !PyType_Check(a[0])) {
        PyErr_SetString(PyExc_TypeError, "bind takes a type, four objects and four addresses");
        return NULL;
    }
    uintptr_t f[4];
    if (!addresses(a + 5, f, 4)) return NULL;
    PyObject** to[5] = {&g_tensor, &g_bf16, &g_i32, &g_f32, &g_raw_stream};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    g_get_device = (get_device_fn)f[0];
    g_append = (append_fn)f[1];
    g_attention = (attention_fn)f[2];
    g_verify = (verify_fn)f[3];
    Py_RETURN_NONE;
}

/* bind_more(norm, adapters, free, reserve, fork, compact): addresses */
static PyObject* bind_more(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    (void)self;
    if (n != 6) {
        PyErr_SetString(PyExc_TypeError, "bind_more takes six addresses");
        return NULL;
    }
    uintptr_t f[6];
    if (!addresses(a, f, 6)) return NULL;
    g_norm = (norm_fn)f[0];
    g_adapters = (adapters_fn)f[1];
    g_free = (free_fn)f[2];
    g_reserve = (list_fn)f[3];
    g_fork = (list_fn)f[4];
    g_compact = (compact_fn)f[5];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, NULL},
                                {"bind_more", (PyCFunction)(void (*)(void))bind_more, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
                                {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, NULL},
                                {"verify", (PyCFunction)(void (*)(void))verify, METH_FASTCALL, NULL},
                                {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, NULL},
                                {"adapters", (PyCFunction)(void (*)(void))adapters, METH_FASTCALL, NULL},
                                {"pages", (PyCFunction)(void (*)(void))pages, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    struct {
        PyObject** to;
        const char* name;
    } names[] = {{&s_dtype, "dtype"},           {&s_shape, "shape"},       {&s_stride, "stride"},
                 {&s_get_device, "get_device"}, {&s_is_contiguous, "is_contiguous"},
                 {&s_data_ptr, "data_ptr"},     {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof names / sizeof names[0]; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
