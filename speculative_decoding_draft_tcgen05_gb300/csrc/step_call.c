/* Argument marshalling of the calls that a step makes around its attention
 * (include/dflash_linear.h, dflash_logits.h, dflash_pages.h), for the Python
 * binding: as in paged_call.c, whose reasons hold here too. */
#include "call.h"
#include "dflash_linear.h"
#include "dflash_logits.h"
#include "dflash_pages.h"

typedef dflash_status (*linear_fn)(dflash_linear_handle, const void *, int64_t, int64_t, const void *, int64_t, void *, int64_t,
                                   void *);

typedef dflash_status (*logits_fn)(const void *, int64_t, int64_t, int32_t, int32_t, int64_t, int32_t,
                                   const dflash_logits_rules *, const int32_t *, int64_t, const int32_t *, int64_t, int64_t,
                                   void *, int64_t, int64_t, float *, int32_t *, void *);
typedef dflash_status (*extend_fn)(const dflash_page_pool *, const int32_t *, const int32_t *, int32_t, int32_t, int32_t *,
                                   int32_t *, int32_t *, int64_t, int32_t, int32_t *, int64_t *, int32_t *, void *);
typedef dflash_status (*trim_fn)(const dflash_page_pool *, const int32_t *, const int32_t *, int32_t, int32_t, void *);

static linear_fn call_linear;
static logits_fn call_logits;
static extend_fn call_extend;
static trim_fn call_trim;
static PyObject *t_int64;

typedef struct {
    void *p;
    int64_t stride;
    int64_t n[2];
} matrix;

/* Rows [rows, columns] with contiguous columns; one row may carry any stride. */
static int get_matrix(PyObject *t, PyObject *dtype, const int64_t *want, long *dev, matrix *m, const char *name)
{
    if (has_dtype(t, dtype, name) < 0 || sizes(t, 2, want, m->n, name) < 0 || address(t, dev, &m->p, name) < 0) return -1;
    PyObject *o = PyObject_CallMethodNoArgs(t, s_stride);
    if (!o) return -1;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) {
        Py_DECREF(o);
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        return -1;
    }
    m->stride = m->n[0] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0)) : m->n[1];
    const int64_t last = m->n[1] > 1 ? PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1)) : 1;
    Py_DECREF(o);
    if (PyErr_Occurred()) return -1;
    if (last != 1) {
        PyErr_Format(PyExc_ValueError, "%s's last dimension must be contiguous", name);
        return -1;
    }
    return 0;
}

/* linear(handle, x, out, residual, stream) -> status; handle.spec: (address, dtype, out dtype, n, k, device) */
static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 5) return PyErr_Format(PyExc_TypeError, "linear takes 5 arguments, got %zd", n);
    PyObject *h = spec_of(a[0], 6, "handle");
    if (!h) return NULL;
    dflash_linear_handle handle = (dflash_linear_handle)PyLong_AsVoidPtr(PyTuple_GET_ITEM(h, 0));
    long dev = PyLong_AsLong(PyTuple_GET_ITEM(h, 5));
    int64_t want[2] = {-1, PyLong_AsLongLong(PyTuple_GET_ITEM(h, 4))};
    matrix x, y, r = {0};
    int bad = PyErr_Occurred() || get_matrix(a[1], PyTuple_GET_ITEM(h, 1), want, &dev, &x, "x") < 0;
    if (!bad) {
        want[0] = x.n[0];
        want[1] = PyLong_AsLongLong(PyTuple_GET_ITEM(h, 3));
        bad = get_matrix(a[2], PyTuple_GET_ITEM(h, 2), want, &dev, &y, "out") < 0 ||
              (!is_none(a[3]) && get_matrix(a[3], PyTuple_GET_ITEM(h, 2), want, &dev, &r, "residual") < 0);
    }
    Py_DECREF(h);
    void *st = NULL;
    if (bad || get_stream(a[4], dev, &st) < 0) return NULL;
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_linear(handle, x.p, x.stride, x.n[0], r.p, r.stride, y.p, y.stride, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* logits(logits, rules, out, probs, argmax, draft, mask, stream) -> status; rules.spec: (address of the C structure,
 * batch or -1, device or -1) */
static PyObject *logits(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 8) return PyErr_Format(PyExc_TypeError, "logits takes 8 arguments, got %zd", n);
    PyObject *dt = PyObject_GetAttr(a[0], s_dtype);
    if (!dt) return NULL;
    const int32_t code = dt == t_bf16 ? DFLASH_BF16 : (dt == t_fp16 ? DFLASH_FP16 : (dt == t_float32 ? DFLASH_FP32 : -1));
    long dev = -1;
    rows x, y = {0}, q = {0}, m = {0};
    matrix d = {0};
    void *best = NULL, *st = NULL;
    const dflash_logits_rules *rules = NULL;
    const int64_t any[3] = {-1, -1, -1};
    int bad = get_rows(a[0], dt, any, &dev, &x, "logits") < 0 || (!is_none(a[2]) && get_rows(a[2], dt, x.n, &dev, &y, "out") < 0);
    Py_DECREF(dt);
    if (bad) return NULL;
    if (!is_none(a[3])) {
        if (get_rows(a[3], t_float32, x.n, &dev, &q, "probs") < 0) return NULL;
        if ((q.n[1] > 1 && q.head_stride != q.n[2]) || (q.n[0] > 1 && q.token_stride != q.n[1] * q.n[2]))
            return PyErr_Format(PyExc_ValueError, "probs must be contiguous");
    }
    if (get_plain(a[4], t_int32, 2, x.n, &dev, &best, "argmax") < 0) return NULL;
    if (!is_none(a[5])) {
        const int64_t want[2] = {x.n[0], x.n[1] > 0 ? x.n[1] - 1 : 0};
        if (get_matrix(a[5], t_int32, want, &dev, &d, "draft") < 0) return NULL;
    }
    if (!is_none(a[6])) {
        const int64_t want[3] = {x.n[0], x.n[1], x.n[2] / 32 + (x.n[2] % 32 != 0)};
        if (get_rows(a[6], t_int32, want, &dev, &m, "mask") < 0) return NULL;
    }
    if (!is_none(a[1])) {
        PyObject *s = spec_of(a[1], 3, "rules");
        if (!s) return NULL;
        rules = (const dflash_logits_rules *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(s, 0));
        const int64_t batch = PyLong_AsLongLong(PyTuple_GET_ITEM(s, 1));
        const long at = PyLong_AsLong(PyTuple_GET_ITEM(s, 2));
        Py_DECREF(s);
        if (PyErr_Occurred() || (at >= 0 && same_device(at, &dev, "rules") < 0)) return NULL;
        if (batch >= 0 && batch != x.n[0])
            return PyErr_Format(PyExc_ValueError, "the rules are for %lld sequences, the logits for %lld", (long long)batch, (long long)x.n[0]);
    }
    if (launch_device(dev) < 0 || get_stream(a[7], dev, &st) < 0) return NULL;
    if (x.n[0] > INT32_MAX || x.n[1] > INT32_MAX) return PyErr_Format(PyExc_ValueError, "too many positions");
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_logits(x.p, x.token_stride, x.head_stride, (int32_t)x.n[0], (int32_t)x.n[1], x.n[2], code, rules,
                         (const int32_t *)d.p, d.stride, (const int32_t *)m.p, m.token_stride, m.head_stride, y.p,
                         y.token_stride, y.head_stride, (float *)q.p, (int32_t *)best, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* PagePool.spec: (address of the C structure, requests, device) */
static const dflash_page_pool *get_pool(PyObject *o, long *dev)
{
    PyObject *s = spec_of(o, 3, "pool");
    if (!s) return NULL;
    const dflash_page_pool *p = (const dflash_page_pool *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(s, 0));
    *dev = PyLong_AsLong(PyTuple_GET_ITEM(s, 2));
    Py_DECREF(s);
    return PyErr_Occurred() ? NULL : p;
}

/* A contiguous vector of the given dtype and size (-1: any), or NULL for None (then *n is left as it was). */
static int get_vector(PyObject *t, PyObject *dtype, int64_t want, long *dev, void **p, int64_t *n, const char *name)
{
    *p = NULL;
    if (is_none(t)) return 0;
    if (get_plain(t, dtype, 1, &want, dev, p, name) < 0) return -1;
    int64_t size[2];
    if (sizes(t, 1, &want, size, name) < 0) return -1;
    if (n) *n = size[0];
    return 0;
}

/* extend(pool, batch, new_tokens, rows, positions, slots, granted, tokens, stream) -> status; batch.spec as in
 * paged_call.c, or None: only the others are wanted; tokens None: the size of positions and slots */
static PyObject *extend(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 9) return PyErr_Format(PyExc_TypeError, "extend takes 9 arguments, got %zd", n);
    long dev = -1;
    const dflash_page_pool *pool = get_pool(a[0], &dev);
    if (!pool) return NULL;
    if (is_none(a[2])) return PyErr_Format(PyExc_ValueError, "new_tokens must be given");
    void *add = NULL, *row = NULL, *pos = NULL, *slot = NULL, *ok = NULL, *st = NULL;
    int64_t count = -1, tokens = -1;
    if (get_vector(a[2], t_int32, -1, &dev, &add, &count, "new_tokens") < 0) return NULL;
    const dflash_paged_batch *b = NULL;
    if (!is_none(a[1])) {
        PyObject *s = spec_of(a[1], 2, "batch");
        if (!s) return NULL;
        b = (const dflash_paged_batch *)PyLong_AsVoidPtr(PyTuple_GET_ITEM(s, 0));
        const long at = PyLong_AsLong(PyTuple_GET_ITEM(s, 1));
        Py_DECREF(s);
        if (PyErr_Occurred() || (at >= 0 && same_device(at, &dev, "batch") < 0)) return NULL;
        if (b->batch != count)
            return PyErr_Format(PyExc_ValueError, "new_tokens must have the batch's %d entries, got %lld", b->batch, (long long)count);
    }
    if (!is_none(a[7])) {
        tokens = PyLong_AsLongLong(a[7]);
        if (PyErr_Occurred()) return NULL;
    }
    int64_t n_pos = -1, n_slot = -1;
    if (get_vector(a[3], t_int32, count, &dev, &row, NULL, "rows") < 0 ||
        get_vector(a[4], t_int32, -1, &dev, &pos, &n_pos, "positions") < 0 ||
        get_vector(a[5], t_int64, -1, &dev, &slot, &n_slot, "slots") < 0 ||
        get_vector(a[6], t_int32, count, &dev, &ok, NULL, "granted") < 0 || launch_device(dev) < 0 ||
        get_stream(a[8], dev, &st) < 0)
        return NULL;
    const int64_t least = n_pos >= 0 && (n_slot < 0 || n_pos < n_slot) ? n_pos : n_slot;
    if (tokens < 0 && is_none(a[7])) tokens = least >= 0 ? least : 1 << 30;
    if (least >= 0 && tokens > least)
        return PyErr_Format(PyExc_ValueError, "positions and slots must have room for tokens = %lld, got %lld", (long long)tokens, (long long)least);
    if (count > INT32_MAX || tokens > INT32_MAX || tokens < 0) return PyErr_Format(PyExc_ValueError, "tokens must be in [0, 2^31)");
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_extend(pool, (const int32_t *)row, (const int32_t *)add, (int32_t)count, (int32_t)tokens,
                         b ? (int32_t *)b->cu_tokens : NULL, b ? (int32_t *)b->lens : NULL, b ? (int32_t *)b->page_table : NULL,
                         b ? b->table_stride : 0, b ? b->table_cols : 0, (int32_t *)pos, (int64_t *)slot, (int32_t *)ok, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* trim(pool, counts, rows, base, batch, stream) -> status; counts None: everything of `batch` requests, or of `rows` */
static PyObject *trim(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    (void)self;
    if (n != 6) return PyErr_Format(PyExc_TypeError, "trim takes 6 arguments, got %zd", n);
    long dev = -1;
    const dflash_page_pool *pool = get_pool(a[0], &dev);
    if (!pool) return NULL;
    void *counts = NULL, *row = NULL, *st = NULL;
    int64_t count = -1;
    if (!is_none(a[4])) count = PyLong_AsLongLong(a[4]);
    const long long base = PyLong_AsLongLong(a[3]);
    if (PyErr_Occurred() || get_vector(a[1], t_int32, count, &dev, &counts, &count, "counts") < 0 ||
        get_vector(a[2], t_int32, count, &dev, &row, &count, "rows") < 0 || launch_device(dev) < 0 || get_stream(a[5], dev, &st) < 0)
        return NULL;
    if (count < 0) return PyErr_Format(PyExc_ValueError, "counts, rows or the batch must be given");
    if (count > INT32_MAX || base > INT32_MAX) return PyErr_Format(PyExc_ValueError, "out of range");
    int status;
    Py_BEGIN_ALLOW_THREADS;
    status = call_trim(pool, (const int32_t *)row, (const int32_t *)counts, base < 0 ? -1 : (int32_t)base, (int32_t)count, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(status);
}

/* setup(linear, logits, extend, trim, current_device: addresses; raw_stream; int32, float32, bfloat16, float16, int64) */
static PyObject *setup(PyObject *self, PyObject *args)
{
    (void)self;
    PyObject *f[5], *o[6];
    if (!PyArg_ParseTuple(args, "OOOOOOOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &o[0], &o[1], &o[2], &o[3], &o[4], &o[5]))
        return NULL;
    void *p[5];
    for (int i = 0; i < 5; ++i) p[i] = PyLong_AsVoidPtr(f[i]);
    if (PyErr_Occurred()) return NULL;
    call_linear = (linear_fn)p[0];
    call_logits = (logits_fn)p[1];
    call_extend = (extend_fn)p[2];
    call_trim = (trim_fn)p[3];
    current_device = (int (*)(void))p[4];
    keep_objects(o);
    Py_INCREF(o[5]);
    Py_XSETREF(t_int64, o[5]);
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, NULL},
                                {"logits", (PyCFunction)(void (*)(void))logits, METH_FASTCALL, NULL},
                                {"extend", (PyCFunction)(void (*)(void))extend, METH_FASTCALL, NULL},
                                {"trim", (PyCFunction)(void (*)(void))trim, METH_FASTCALL, NULL},
                                {"setup", setup, METH_VARARGS, NULL},
                                {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_call", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__step_call(void)
{
    if (intern_names() < 0) return NULL;
    return PyModule_Create(&module);
}
