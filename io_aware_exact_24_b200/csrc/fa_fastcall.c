/*
 * fa_fastcall.c -- CPython module that marshals the calls of a decoding step.
 *
 * The 4-bit cache entry points take some 25 arguments, which ctypes converts in several
 * microseconds, as long as the kernels of a small step run.  The wrappers here take the same
 * arguments as those of binding.py and turn them into the same C calls: tensors (anything with
 * data_ptr()), integers and None become addresses, numbers become numbers.  They compute
 * nothing and link against nothing; init() hands them the entry points' addresses.  Of the
 * tensors, the dense ones must be contiguous, and they and the cache on the current device.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

typedef int (*rows_fn)(const void *, const void *, const void *, const void *, const void *, const void *, const void *,
                       const void *, const void *, int, int, int, int, int, int, int, void *);
typedef int (*fwd_fn)(const void *, const void *, const void *, const void *, const void *, const void *, const void *,
                      const void *, void *, void *, int, int, int, int, int, int, int, int, float, int, int, void *, size_t,
                      void *);

static rows_fn g_append, g_read;
static fwd_fn g_fwd;
static PyObject *g_data_ptr, *g_get_device, *g_is_contiguous;   /* names of a tensor's methods */
static PyObject *g_current;                                     /* returns the current device */

static int not_a_tensor(PyObject *x) {
    if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
        PyErr_Clear();
        PyErr_Format(PyExc_TypeError, "cannot take the address of %R", (PyObject *)Py_TYPE(x));
    }
    return 0;
}

/* Address of a tensor, an integer or None; -1 on success, else 0 with an exception set. */
static int address(PyObject *x, void **out) {
    if (x == Py_None) {
        *out = NULL;
        return -1;
    }
    if (PyLong_Check(x)) {
        *out = PyLong_AsVoidPtr(x);
        return *out != NULL || !PyErr_Occurred() ? -1 : 0;
    }
    PyObject *a = PyObject_CallMethodNoArgs(x, g_data_ptr);
    if (a == NULL) return not_a_tensor(x);
    *out = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return *out != NULL || !PyErr_Occurred() ? -1 : 0;
}

/* A tensor given here must lie on the current device, and, where asked, be contiguous: the
 * kernels would read other memory than it means, or fault.  Addresses are taken as they are. */
static int tensor_ok(PyObject *x, int contiguous) {
    if (x == Py_None || PyLong_Check(x)) return -1;
    PyObject *d = PyObject_CallMethodNoArgs(x, g_get_device);
    if (d == NULL) return not_a_tensor(x);
    const long dev = PyLong_AsLong(d);
    Py_DECREF(d);
    PyObject *c = PyObject_CallNoArgs(g_current);
    if (c == NULL) return 0;
    const long cur = PyLong_AsLong(c);
    Py_DECREF(c);
    if (PyErr_Occurred()) return 0;
    if (dev != cur) {
        PyErr_Format(PyExc_ValueError, "a tensor is on device %ld, the current device is %ld (-1: the CPU)", dev, cur);
        return 0;
    }
    if (contiguous) {
        PyObject *r = PyObject_CallMethodNoArgs(x, g_is_contiguous);
        if (r == NULL) return 0;
        const int yes = PyObject_IsTrue(r);
        Py_DECREF(r);
        if (yes < 0) return 0;
        if (!yes) {
            PyErr_SetString(PyExc_ValueError, "a tensor is not contiguous");
            return 0;
        }
    }
    return -1;
}

static int number(PyObject *x, int *out) {
    PyObject *i = PyNumber_Long(x);
    if (i == NULL) return 0;
    const long v = PyLong_AsLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) return 0;
    if (v < INT_MIN || v > INT_MAX) {
        PyErr_Format(PyExc_OverflowError, "%ld is not a C int", v);
        return 0;
    }
    *out = (int)v;
    return -1;
}

static int count_is(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return -1;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return 0;
}

/* 9 addresses, 7 numbers, the stream; a[dense] and a[dense + 1] are k and v, a[cache] a buffer of the cache */
static PyObject *rows_call(rows_fn fn, PyObject *const *a, Py_ssize_t n, int dense, int cache) {
    void *p[9], *stream;
    int v[7], i;
    if (!count_is(n, 17)) return NULL;
    if (!tensor_ok(a[dense], 1) || !tensor_ok(a[dense + 1], 1) || !tensor_ok(a[cache], 0)) return NULL;
    for (i = 0; i < 9; ++i)
        if (!address(a[i], &p[i])) return NULL;
    for (i = 0; i < 7; ++i)
        if (!number(a[9 + i], &v[i])) return NULL;
    if (!address(a[16], &stream)) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], v[0], v[1], v[2], v[3], v[4], v[5], v[6], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_append, a, n, 0, 2); }
static PyObject *read_back(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_read, a, n, 7, 0); }

/* 10 addresses, 8 numbers, scale, causal, window, workspace and its size, the stream */
static PyObject *fwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    void *p[10], *ws, *stream;
    int v[8], window, i;
    if (!count_is(n, 24)) return NULL;
    if (!tensor_ok(a[0], 1) || !tensor_ok(a[8], 1) || !tensor_ok(a[1], 0)) return NULL;   /* q, o, the cache */
    for (i = 0; i < 10; ++i)
        if (!address(a[i], &p[i])) return NULL;
    for (i = 0; i < 8; ++i)
        if (!number(a[10 + i], &v[i])) return NULL;
    const double scale = PyFloat_AsDouble(a[18]);
    if (scale == -1.0 && PyErr_Occurred()) return NULL;
    const int causal = PyObject_IsTrue(a[19]);
    if (causal < 0 || !number(a[20], &window) || !address(a[21], &ws)) return NULL;
    PyObject *size = PyNumber_Long(a[22]);
    if (size == NULL) return NULL;
    const size_t bytes = PyLong_AsSize_t(size);
    Py_DECREF(size);
    if (bytes == (size_t)-1 && PyErr_Occurred()) return NULL;
    if (!address(a[23], &stream)) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = g_fwd(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7],
               (float)scale, causal, window, ws, bytes, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *init(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    void *p[3];
    int i;
    if (!count_is(n, 4)) return NULL;
    Py_INCREF(a[3]);
    Py_XSETREF(g_current, a[3]);
    for (i = 0; i < 3; ++i)
        if (!address(a[i], &p[i])) return NULL;
    g_append = (rows_fn)p[0];
    g_read = (rows_fn)p[1];
    g_fwd = (fwd_fn)p[2];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, "init(fa_kv4_append, fa_kv4_read, fa_fwd_kv4, current_device): their addresses, and a function"},
    {"fa_kv4_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "status of fa_kv4_append"},
    {"fa_kv4_read", (PyCFunction)(void (*)(void))read_back, METH_FASTCALL, "status of fa_kv4_read"},
    {"fa_fwd_kv4", (PyCFunction)(void (*)(void))fwd, METH_FASTCALL, "status of fa_fwd_kv4"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "Argument marshalling for the 4-bit cache entry points.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    g_get_device = PyUnicode_InternFromString("get_device");
    g_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (g_data_ptr == NULL || g_get_device == NULL || g_is_contiguous == NULL) return NULL;
    return PyModule_Create(&module);
}
