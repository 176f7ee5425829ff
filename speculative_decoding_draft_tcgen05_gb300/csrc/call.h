/* What the modules that marshal calls for the Python binding share: reading
 * tensors (known only by their Python attributes), streams and the objects that
 * hold C structures. Included once per module; its state is the module's own. */
#ifndef DFLASH_CALL_H
#define DFLASH_CALL_H

#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

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

/* Without a handle, whose device the library compares with the current one, that is done here. */
static int launch_device(long dev)
{
    const int now = current_device();
    if (now != dev) PyErr_Format(PyExc_ValueError, "the tensors are on cuda:%ld, the current device is cuda:%d", dev, now);
    return now == dev ? 0 : -1;
}

/* Interns the attribute names; 0, or -1 with an exception. */
static int intern_names(void)
{
    struct {
        PyObject **to;
        const char *name;
    } names[] = {{&s_dtype, "dtype"}, {&s_shape, "shape"}, {&s_stride, "stride"},
                 {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"}, {&s_get_device, "get_device"},
                 {&s_spec, "spec"}, {&s_cuda_stream, "cuda_stream"}};
    for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
        if (!(*names[i].to = PyUnicode_InternFromString(names[i].name))) return -1;
    return 0;
}

/* Takes over setup()'s `raw_stream` and the four dtypes. */
static void keep_objects(PyObject *const *o)
{
    PyObject **to[5] = {&raw_stream, &t_int32, &t_float32, &t_bf16, &t_fp16};
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(o[i]);
        Py_XSETREF(*to[i], o[i]);
    }
}

#endif /* DFLASH_CALL_H */
