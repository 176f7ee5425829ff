/* Argument marshalling of the three entry points that a step calls once per
 * layer (include/dflash_paged.h), for the Python binding: checks the tensors,
 * takes their addresses and strides, finds the stream and makes the call, with
 * the interpreter's lock released. The tensors of a call, its handle and the
 * current device, which the launch goes to, have to be the same device. It does
 * nothing that the binding could not do through ctypes; it takes about half the
 * time, and the GPU's work on one block of a single sequence is shorter than
 * either. Knows tensors only by their Python attributes. */
#include "call.h"
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
    keep_objects(o);
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
    if (intern_names() < 0) return NULL;
    return PyModule_Create(&module);
}
