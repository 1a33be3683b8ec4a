/*
 * fa_fastcall.c -- CPython module that marshals the calls of a decoding step.
 *
 * The 4-bit cache entry points take some 25 arguments, which ctypes converts in several
 * microseconds, as long as the kernels of a small step run.  The wrappers here take the same
 * arguments as those of binding.py and turn them into the same C calls: tensors (anything with
 * data_ptr()), integers and None become addresses, numbers become numbers.  They compute
 * nothing and link against nothing; init() hands them the entry points' addresses.
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
static PyObject *g_data_ptr;   /* "data_ptr" */

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
    if (a == NULL) {
        if (PyErr_ExceptionMatches(PyExc_AttributeError)) {
            PyErr_Clear();
            PyErr_Format(PyExc_TypeError, "cannot take the address of %R", (PyObject *)Py_TYPE(x));
        }
        return 0;
    }
    *out = PyLong_AsVoidPtr(a);
    Py_DECREF(a);
    return *out != NULL || !PyErr_Occurred() ? -1 : 0;
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

/* 9 addresses, 7 numbers, the stream */
static PyObject *rows_call(rows_fn fn, PyObject *const *a, Py_ssize_t n) {
    void *p[9], *stream;
    int v[7], i;
    if (!count_is(n, 17)) return NULL;
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

static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_append, a, n); }
static PyObject *read_back(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_read, a, n); }

/* 10 addresses, 8 numbers, scale, causal, window, workspace and its size, the stream */
static PyObject *fwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    void *p[10], *ws, *stream;
    int v[8], window, i;
    if (!count_is(n, 24)) return NULL;
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
    if (!count_is(n, 3)) return NULL;
    for (i = 0; i < 3; ++i)
        if (!address(a[i], &p[i])) return NULL;
    g_append = (rows_fn)p[0];
    g_read = (rows_fn)p[1];
    g_fwd = (fwd_fn)p[2];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, "init(fa_kv4_append, fa_kv4_read, fa_fwd_kv4): their addresses"},
    {"fa_kv4_append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, "status of fa_kv4_append"},
    {"fa_kv4_read", (PyCFunction)(void (*)(void))read_back, METH_FASTCALL, "status of fa_kv4_read"},
    {"fa_fwd_kv4", (PyCFunction)(void (*)(void))fwd, METH_FASTCALL, "status of fa_fwd_kv4"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", "Argument marshalling for the 4-bit cache entry points.", -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
    g_data_ptr = PyUnicode_InternFromString("data_ptr");
    return g_data_ptr == NULL ? NULL : PyModule_Create(&module);
}
