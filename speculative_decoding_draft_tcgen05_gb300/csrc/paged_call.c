/* Argument marshalling of the three entry points that a step calls once per
 * layer (include/dflash_paged.h), for the Python binding: checks the tensors,
 * takes their addresses and strides, finds the stream and makes the call, with
 * the interpreter's lock released. The tensors of a call, its handle and the
 * current device, which the launch goes to, have to be the same device. It does
 * nothing that the binding could not do through ctypes; it takes about half the
 * time, and the GPU's work on one block of a single sequence is shorter than
 * either. Knows tensors only by their Python attributes. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "dflash_paged.h"

typedef dflash_status (*norm_rope_fn)(const void *, int64_t, int64_t, void *, int64_t, int64_t, const void *, int64_t,
                                      int64_t, void *, int64_t, int64_t, int32_t, int32_t, int32_t, int32_t, int32_t,
                                      const dflash_qk_transform *, const int32_t *, void *);
typedef dflash_status (*append_fn)(dflash_paged_handle, const dflash_paged_cache *, const dflash_paged_batch *,
                                   const void *, int64_t, int64_t, const void *, int64_t, int64_t,
                                   const dflash_qk_transform *, const int32_t *, const void *, int64_t, int64_t, void *,
                                   int64_t, int64_t, void *);
typedef dflash_status (*attend_fn)(dflash_paged_handle, const dflash_paged_cache *, const dflash_paged_batch *,
                                   const void *, int64_t, int64_t, void *, int64_t, int64_t, float *, int32_t, int32_t,
                                   float, void *);

static norm_rope_fn call_norm_rope;
static append_fn call_append;
static attend_fn call_attend;
static int (*current_device)(void);
static PyObject *raw_stream;                 /* device index -> handle of its current stream */
static PyObject *t_int32, *t_float32;        /* torch dtypes */
static PyObject *t_bf16, *t_fp16;
static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_get_device, *s_spec,
    *s_cuda_stream;

typedef struct {
    void *p;
    int64_t token_stride, head_stride;
    int64_t n[3]; /* tokens, heads, head_dim */
} rows;

static int is_none(PyObject *o)
{
    return o == NULL || o == Py_None;
}

/* The call's device (-1: not known yet) is also that of `name`. */
static int same_device(long index, long *dev, const char *name)
{
    if (*dev < 0) *dev = index;
    if (*dev == index) return 0;
    PyErr_Format(PyExc_ValueError, "%s is on cuda:%ld, the call's other tensors or its handle on cuda:%ld", name, index, *dev);
    return -1;
}

static int has_dtype(PyObject *t, PyObject *dtype, const char *name)
{
    PyObject *o = PyObject_GetAttr(t, s_dtype);
    if (!o) return -1;
    const int same = o == dtype;
    if (!same) PyErr_Format(PyExc_TypeError, "%s must be %S, got %S", name, dtype, o);
    Py_DECREF(o);
    return same ? 0 : -1;
}

/* The sizes of a tensor of `dims` dimensions (want: those that it must have, -1 for any). */
static int sizes(PyObject *t, int dims, const int64_t *want, int64_t *n, const char *name)
{
    PyObject *o = PyObject_GetAttr(t, s_shape);
    if (!o) return -1;
    int bad = !PyTuple_Check(o) || PyTuple_GET_SIZE(o) != dims;
    for (int i = 0; !bad && i < dims; ++i) {
        n[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
        bad = want && want[i] >= 0 && n[i] != want[i];
    }
    if (bad && !PyErr_Occurred()) {
        PyObject *l = PyList_New(0);
        for (int i = 0; l && want && i < dims; ++i) {
            PyObject *v = want[i] >= 0 ? PyLong_FromLongLong(want[i]) : PyUnicode_FromString(":");
            if (v) PyList_Append(l, v);
            Py_XDECREF(v);
        }
        if (l) PyErr_Format(PyExc_ValueError, "%s must have %d dimensions %S, got %S", name, dims, l, o);
        Py_XDECREF(l);
    }
    Py_DECREF(o);
    return bad ? -1 : 0;
}

static int address(PyObject *t, long *dev, void **p, const char *name)
{
    PyObject *o = PyObject_CallMethodNoArgs(t, s_get_device);
    if (!o) return -1;
    const long index = PyLong_AsLong(o);
    Py_DECREF(o);
    if (index < 0) {
        if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
        return -1;
    }
    if (same_device(index, dev, name) < 0) return -1;
    o = PyObject_CallMethodNoArgs(t, s_data_ptr);
    if (!o) return -1;
    *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* Rows [tokens, heads, head_dim] with a contiguous last dimension. */
static int get_rows(PyObject *t, PyObject *dtype, const int64_t *want, long *dev, rows *r, const char *name)
{
    if (has_dtype(t, dtype, name) < 0 || sizes(t, 3, want, r->n, name) < 0 || address(t, dev, &r->p, name) < 0)
        return -1;
    PyObject *o = PyObject_CallMethodNoArgs(t, s_stride);
    if (!o) return -1;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) {
        Py_DECREF(o);
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        return -1;
    }
    /* a dimension of one row may carry any stride */
    r->token_stride = r->n[0] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0)) : 0;
    r->head_stride = r->n[1] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1)) : 0;
    const int64_t last = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 2));
    Py_DECREF(o);
    if (PyErr_Occurred()) return -1;
    if (last != 1) {
        PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
        return -1;
    }
    return 0;
}

/* A contiguous tensor of the given dtype and sizes, or NULL for None. */
static int get_plain(PyObject *t, PyObject *dtype, int dims, const int64_t *want, long *dev, void **p, const char *name)
{
    int64_t n[2];
    *p = NULL;
    if (is_none(t)) return 0;
    if (has_dtype(t, dtype, name) < 0 || sizes(t, dims, want, n, name) < 0 || address(t, dev, p, name) < 0) return -1;
    PyObject *o = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (!o) return -1;
    const int is = PyObject_IsTrue(o);
    Py_DECREF(o);
    if (is == 0) PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return is > 0 ? 0 : -1;
}

static int get_stream(PyObject *stream, long dev, void **s)
{
    PyObject *o;
    if (is_none(stream)) {
        PyObject *d = PyLong_FromLong(dev);
        if (!d) return -1;
        o = PyObject_CallOneArg(raw_stream, d);
        Py_DECREF(d);
    } else if (PyObject_HasAttr(stream, s_cuda_stream)) {
        o = PyObject_GetAttr(stream, s_cuda_stream);
    } else {
        o = PyNumber_Long(stream);
    }
    if (!o) return -1;
    *s = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return PyErr_Occurred() ? -1 : 0;
}

/* An object's `spec` tuple (the caller releases it). */
static PyObject *spec_of(PyObject *o, Py_ssize_t n, const char *name)
{
    PyObject *s = PyObject_GetAttr(o, s_spec);
    if (s && (!PyTuple_Check(s) || PyTuple_GET_SIZE(s) != n)) {
        Py_CLEAR(s);
        PyErr_Format(PyExc_TypeError, "%s has the wrong type", name);
    }
    return s;
}

/* QkTransform.spec: (address of the C structure, weights' dtype or None, weights' size, device or -1 without tensors). */
static int get_transform(PyObject *o, PyObject *dtype, int64_t head_dim, long *dev, const dflash_qk_transform **tr)
{
    *tr = NULL;
    if (is_none(o)) return 0;
    PyObject *s = spec_of(o, 4, "transform");
    if (!s) return -1;
    PyObject *wd = PyTuple_GET_ITEM(s, 1);
    int bad = 0;
    if (wd != Py_None && (wd != dtype || PyLong_AsLongLong(PyTuple_GET_ITEM(s, 2)) != head_dim)) {
        PyErr_Format(PyExc_TypeError, "norm weights must be %S [%lld], got %S [%S]", dtype, (long long)head_dim, wd,
                     PyTuple_GET_ITEM(s, 2));
        bad = 1;
    }
    const long index = PyLong_AsLong(PyTuple_GET_ITEM(s, 3));
    if (!bad && index >= 0) bad = same_device(index, dev, "transform") < 0;
    *tr = (const dflash_qk_transform *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(s, 0));
    Py_DECREF(s);
    return bad || PyErr_Occurred() ? -1 : 0;
}

/* A handle, cache and batch that fit together. handle.spec: (address, dtype, cache dtype, heads, kv_heads, head_dim,
 * cache shape, device); cache.spec: (address of the C structure, dtype, shape, device); batch.spec: (address of the C
 * structure, device). */
typedef struct {
    PyObject *dtype; /* borrowed from the handle */
    int64_t heads, kv_heads, head_dim;
    long dev; /* the handle's */
    dflash_paged_handle h;
    const dflash_paged_cache *cache;
    dflash_paged_batch *batch;
} call;

static int get_call(PyObject *handle, PyObject *cache, PyObject *batch, call *c)
{
    int ok = 0;
    PyObject *h = spec_of(handle, 8, "handle"), *k = NULL, *b = NULL;
    if (h) k = spec_of(cache, 4, "cache");
    if (k) b = spec_of(batch, 2, "batch");
    if (b) {
        c->h = (dflash_paged_handle)PyLong_AsVoidPtr(PyTuple_GET_ITEM(h, 0));
        c->dtype = PyTuple_GET_ITEM(h, 1); /* (kept alive by torch) */
        c->heads = PyLong_AsLongLong(PyTuple_GET_ITEM(h, 3));
        c->kv_heads = PyLong_AsLongLong(PyTuple_GET_ITEM(h, 4));
        c->head_dim = PyLong_AsLongLong(PyTuple_GET_ITEM(h, 5));
        c->cache = (const dflash_paged_cache *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(k, 0));
        c->batch = (dflash_paged_batch *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(b, 0));
        c->dev = PyLong_AsLong(PyTuple_GET_ITEM(h, 7));
        const long at[2] = {PyLong_AsLong(PyTuple_GET_ITEM(k, 3)), PyLong_AsLong(PyTuple_GET_ITEM(b, 1))};
        ok = !PyErr_Occurred() && same_device(at[0], &c->dev, "cache") == 0 && same_device(at[1], &c->dev, "batch") == 0;
        if (ok) {
            const int same = PyTuple_GET_ITEM(k, 1) == PyTuple_GET_ITEM(h, 2)
                                 ? PyObject_RichCompareBool(PyTuple_GET_ITEM(k, 2), PyTuple_GET_ITEM(h, 6), Py_EQ)
                                 : 0;
            if (same == 0)
                PyErr_Format(PyExc_ValueError, "the cache must be %S [pages, *%S], got %S [pages, *%S]",
                             PyTuple_GET_ITEM(h, 2), PyTuple_GET_ITEM(h, 6), PyTuple_GET_ITEM(k, 1), PyTuple_GET_ITEM(k, 2));
            ok = same > 0;
        }
    }
    Py_XDECREF(h);
    Py_XDECREF(k);
    Py_XDECREF(b);
    return ok ? 0 : -1;
}

/* Without a handle, whose device the library compares with the current one, that is done here. */
static int launch_device(long dev)
{
    const int now = current_device();
    if (now != dev) PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%ld, the current device is cuda:%d", dev, now);
    return now == dev ? 0 : -1;
}

/* norm_rope(q, k, q_out, k_out, transform, positions, stream) -> status */
static PyObject *norm_rope(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 7) return PyErr_Format(PyExc_TypeError, "norm_rope takes 7 arguments, got %zd", n);
    const int has_q = !is_none(a[0]), has_k = !is_none(a[1]);
    if (!has_q && !has_k) return PyErr_Format(PyExc_ValueError, "q or k must be given");
    PyObject *dt = PyObject_GetAttr(has_q ? a[0] : a[1], s_dtype);
    if (!dt) return NULL;
    rows q = {0}, qo = {0}, k = {0}, ko = {0};
    const dflash_qk_transform *tr = NULL;
    void *pos = NULL, *st = NULL;
    long dev = -1;
    int bad = 0;
    int64_t want[3] = {-1, -1, -1};
    if (has_q) bad = get_rows(a[0], dt, want, &dev, &q, "q") < 0 || get_rows(a[2], dt, q.n, &dev, &qo, "q_out") < 0;
    if (!bad && has_k) {
        if (has_q) want[0] = q.n[0], want[2] = q.n[2];
        bad = get_rows(a[1], dt, want, &dev, &k, "k") < 0 || get_rows(a[3], dt, k.n, &dev, &ko, "k_out") < 0;
    }
    const int64_t tokens = has_q ? q.n[0] : k.n[0], head_dim = has_q ? q.n[2] : k.n[2];
    bad = bad || get_transform(a[4], dt, head_dim, &dev, &tr) < 0 ||
          get_plain(a[5], t_int32, 1, &tokens, &dev, &pos, "positions") < 0 || launch_device(dev) < 0 ||
          get_stream(a[6], dev, &st) < 0;
    const int32_t code = dt == t_bf16 ? DFLASH_BF16 : (dt == t_fp16 ? DFLASH_FP16 : -1);
    Py_DECREF(dt);
    if (bad) return NULL;
    if (tokens > INT32_MAX || head_dim > INT32_MAX) return PyErr_Format(PyExc_ValueError, "too many tokens");
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_norm_rope(q.p, q.token_stride, q.head_stride, qo.p, qo.token_stride, qo.head_stride, k.p, k.token_stride,
                            k.head_stride, ko.p, ko.token_stride, ko.head_stride, (int32_t)tokens, (int32_t)q.n[1],
                            (int32_t)k.n[1], (int32_t)head_dim, code, tr, (const int32_t *)pos, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* append(handle, cache, batch, k, v, transform, q, q_out, positions, stream) -> status */
static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 10) return PyErr_Format(PyExc_TypeError, "append takes 10 arguments, got %zd", n);
    call c;
    if (get_call(a[0], a[1], a[2], &c) < 0) return NULL;
    rows k = {0}, v = {0}, q = {0}, qo = {0};
    const dflash_qk_transform *tr = NULL;
    void *pos = NULL, *st = NULL;
    int64_t want[3] = {-1, c.kv_heads, c.head_dim};
    if (get_rows(a[3], c.dtype, want, &c.dev, &k, "k") < 0 || get_rows(a[4], c.dtype, k.n, &c.dev, &v, "v") < 0 ||
        get_transform(a[5], c.dtype, c.head_dim, &c.dev, &tr) < 0)
        return NULL;
    if (!is_none(a[6])) {
        const int64_t as[3] = {k.n[0], c.heads, c.head_dim};
        if (get_rows(a[6], c.dtype, as, &c.dev, &q, "q") < 0 || get_rows(a[7], c.dtype, as, &c.dev, &qo, "q_out") < 0)
            return NULL;
    }
    if (get_plain(a[8], t_int32, 1, k.n, &c.dev, &pos, "positions") < 0 || get_stream(a[9], c.dev, &st) < 0) return NULL;
    if (k.n[0] > INT32_MAX) return PyErr_Format(PyExc_ValueError, "too many tokens");
    dflash_paged_batch b = *c.batch;
    b.tokens = (int32_t)k.n[0];
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_append(c.h, c.cache, &b, k.p, k.token_stride, k.head_stride, v.p, v.token_stride, v.head_stride, tr,
                         (const int32_t *)pos, q.p, q.token_stride, q.head_stride, qo.p, qo.token_stride, qo.head_stride, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* attend(handle, cache, batch, q, out, lse, causal, window, scale, stream) -> status; scale None: 1 / sqrt(head_dim) */
static PyObject *attend(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 10) return PyErr_Format(PyExc_TypeError, "attend takes 10 arguments, got %zd", n);
    call c;
    if (get_call(a[0], a[1], a[2], &c) < 0) return NULL;
    rows q = {0}, out = {0};
    void *lse = NULL, *st = NULL;
    const int64_t want[3] = {-1, c.heads, c.head_dim};
    if (get_rows(a[3], c.dtype, want, &c.dev, &q, "q") < 0 || get_rows(a[4], c.dtype, q.n, &c.dev, &out, "out") < 0 ||
        get_plain(a[5], t_float32, 2, q.n, &c.dev, &lse, "lse") < 0 || get_stream(a[9], c.dev, &st) < 0)
        return NULL;
    const int causal = PyObject_IsTrue(a[6]);
    const long long window = PyLong_AsLongLong(a[7]);
    const double scale = is_none(a[8]) ? (c.head_dim == 64 ? 0.125 : 0.08838834764831845) : PyFloat_AsDouble(a[8]);
    if (causal < 0 || PyErr_Occurred()) return NULL;
    if (q.n[0] > INT32_MAX) return PyErr_Format(PyExc_ValueError, "too many tokens");
    dflash_paged_batch b = *c.batch;
    b.tokens = (int32_t)q.n[0];
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_attend(c.h, c.cache, &b, q.p, q.token_stride, q.head_stride, out.p, out.token_stride, out.head_stride,
                         (float *)lse, causal, window > INT32_MAX ? INT32_MAX : (window < -1 ? -1 : (int32_t)window),
                         (float)scale, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* setup(norm_rope, append, attend, current_device: addresses; raw_stream; int32, float32, bfloat16, float16) */
static PyObject *setup(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *f[4], *o[5];
    if (!PyArg_ParseTuple(args, "OOOOOOOOO", &f[0], &f[1], &f[2], &f[3], &o[0], &o[1], &o[2], &o[3], &o[4])) return NULL;
    void *p[4];
    for (int i = 0; i < 4; ++i) p[i] = PyLong_AsVoidPtr(f[i]);
    if (PyErr_Occurred()) return NULL;
    call_norm_rope = (norm_rope_fn)p[0];
    call_append = (append_fn)p[1];
    call_attend = (attend_fn)p[2];
    current_device = (int (*)(void))p[3];
    PyObject **to[5] = {&raw_stream, &t_int32, &t_float32, &t_bf16, &t_fp16};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*to[i], o[i]);
    }
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"norm_rope", (PyCFunction)(void (*)(void))norm_rope, METH_FASTCALL, NULL},
                                {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, NULL},
                                {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, NULL},
                                {"setup", setup, METH_VARARGS, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__paged_call(void)
{
    struct {
        PyObject **to;
        const char *name;
    } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"},
                 {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"},
                 {&s_spec, "spec"}, {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return NULL;
    return PyModule_Create(&module);
}
