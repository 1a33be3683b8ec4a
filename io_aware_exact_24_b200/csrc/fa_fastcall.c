/*
 * fa_fastcall.c -- CPython module that marshals the calls of a decoding step.
 *
 * The 4-bit cache entry points take some 25 arguments, which ctypes converts in several
 * microseconds, as long as the kernels of a small step run.  The wrappers here take the same
 * arguments as those of binding.py and turn them into the same C calls: tensors (anything with
 * data_ptr()), integers and None become addresses, numbers become numbers.  They compute
 * nothing and link against nothing; init() hands them the entry points' addresses.  Tensors
 * must be contiguous, on the current device and of the argument's type: the kernels would read
 * other memory than they mean, or fault.  (Of a call that does nothing, B, heads or tokens 0,
 * only the dense ones and a buffer of the cache are looked at.)  Addresses are taken as they are.
 * That is 0.3 us of the 5.9 that an attention call takes the host, its launch included.
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
static PyObject *g_data_ptr, *g_get_device, *g_is_contiguous, *g_dtype;   /* names of a tensor's methods and its type's */
static PyObject *g_current;                                     /* returns the current device */
static PyObject *g_make_types;                                  /* returns a tuple of the types below */
static PyObject *g_types;                                       /* it, from the first tensor on */

enum type { BF16, F32, I32, U8, ANY };
struct arg {
    const char *name;
    enum type type;
};
static const struct arg append_args[9] = {{"k", BF16}, {"v", BF16}, {"k_codes", U8}, {"k_scales", BF16}, {"v_codes", U8},
                                          {"v_scales", BF16}, {"block_table", I32}, {"key_lens", I32}, {"new_lens", I32}};
static const struct arg read_args[9] = {{"k_codes", U8}, {"k_scales", BF16}, {"v_codes", U8}, {"v_scales", BF16},
                                        {"block_table", I32}, {"key_lens", I32}, {"first", I32}, {"k", BF16}, {"v", BF16}};
static const struct arg fwd_args[10] = {{"q", BF16}, {"k_codes", U8}, {"k_scales", BF16}, {"v_codes", U8}, {"v_scales", BF16},
                                        {"block_table", I32}, {"key_lens", I32}, {"q_lens", I32}, {"o", BF16}, {"lse", F32}};
static const struct arg workspace_arg = {"workspace", ANY};

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

static int current_device(long *dev) {
    PyObject *c = PyObject_CallNoArgs(g_current);
    if (c == NULL) return 0;
    *dev = PyLong_AsLong(c);
    Py_DECREF(c);
    return *dev != -1 || !PyErr_Occurred() ? -1 : 0;
}

static int tensor_on(PyObject *x, const struct arg *arg, long current) {
    if (x == Py_None || PyLong_Check(x)) return -1;
    PyObject *d = PyObject_CallMethodNoArgs(x, g_get_device);
    if (d == NULL) return not_a_tensor(x);
    const long dev = PyLong_AsLong(d);
    Py_DECREF(d);
    if (dev == -1 && PyErr_Occurred()) return 0;
    if (dev == current) return -1;
    PyErr_Format(PyExc_ValueError, "%s is on device %ld, the current device is %ld (-1: the CPU)", arg->name, dev, current);
    return 0;
}

static int tensor_contiguous(PyObject *x, const struct arg *arg) {
    if (x == Py_None || PyLong_Check(x)) return -1;
    PyObject *r = PyObject_CallMethodNoArgs(x, g_is_contiguous);
    if (r == NULL) return not_a_tensor(x);
    const int yes = PyObject_IsTrue(r);
    Py_DECREF(r);
    if (yes > 0) return -1;
    if (yes == 0) PyErr_Format(PyExc_ValueError, "%s is not contiguous", arg->name);
    return 0;
}

static int tensor_type(PyObject *x, const struct arg *arg) {
    if (x == Py_None || PyLong_Check(x) || arg->type == ANY) return -1;
    if (g_types == NULL) {
        g_types = PyObject_CallNoArgs(g_make_types);
        if (g_types == NULL) return 0;
        if (!PyTuple_Check(g_types) || PyTuple_GET_SIZE(g_types) != ANY) {
            Py_CLEAR(g_types);
            PyErr_SetString(PyExc_SystemError, "a tuple of types was expected");
            return 0;
        }
    }
    PyObject *want = PyTuple_GET_ITEM(g_types, arg->type), *t = PyObject_GetAttr(x, g_dtype);
    if (t == NULL) return not_a_tensor(x);
    const int same = t == want;                  /* (each type is one object) */
    if (!same) PyErr_Format(PyExc_ValueError, "%s is of type %R, %R expected", arg->name, t, want);
    Py_DECREF(t);
    return same ? -1 : 0;
}

static int tensor_ok(PyObject *x, const struct arg *arg, long current) {
    return tensor_on(x, arg, current) && tensor_contiguous(x, arg) && tensor_type(x, arg) ? -1 : 0;
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
static PyObject *rows_call(rows_fn fn, const struct arg *args, PyObject *const *a, Py_ssize_t n, int dense, int cache) {
    void *p[9], *stream;
    int v[7], i;
    long dev;
    if (!count_is(n, 17) || !current_device(&dev)) return NULL;
    for (i = 0; i < 7; ++i)
        if (!number(a[9 + i], &v[i])) return NULL;
    const int nothing = v[0] == 0 || v[1] == 0 || v[2] == 0;
    for (i = 0; i < 9; ++i) {
        const int is_dense = i == dense || i == dense + 1;
        if (nothing ? (is_dense || i == cache) && !tensor_on(a[i], &args[i], dev) : !tensor_ok(a[i], &args[i], dev)) return NULL;
        if (nothing && is_dense && !tensor_contiguous(a[i], &args[i])) return NULL;
        if (!address(a[i], &p[i])) return NULL;
    }
    if (!address(a[16], &stream)) return NULL;
    int st;
    Py_BEGIN_ALLOW_THREADS
    st = fn(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], v[0], v[1], v[2], v[3], v[4], v[5], v[6], stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

static PyObject *append(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_append, append_args, a, n, 0, 2); }
static PyObject *read_back(PyObject *self, PyObject *const *a, Py_ssize_t n) { return rows_call(g_read, read_args, a, n, 7, 0); }

/* 10 addresses, 8 numbers, scale, causal, window, workspace and its size, the stream */
static PyObject *fwd(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    void *p[10], *ws, *stream;
    int v[8], window, i;
    long dev;
    if (!count_is(n, 24) || !current_device(&dev)) return NULL;
    for (i = 0; i < 8; ++i)
        if (!number(a[10 + i], &v[i])) return NULL;
    const int nothing = v[0] == 0 || v[1] == 0 || v[2] == 0 || v[3] == 0;
    for (i = 0; i < 10; ++i) {
        const int is_dense = i == 0 || i == 8;   /* q and o */
        if (nothing ? (is_dense || i == 1) && !tensor_on(a[i], &fwd_args[i], dev) : !tensor_ok(a[i], &fwd_args[i], dev)) return NULL;
        if (nothing && is_dense && !tensor_contiguous(a[i], &fwd_args[i])) return NULL;
        if (!address(a[i], &p[i])) return NULL;
    }
    if (!nothing && !tensor_ok(a[21], &workspace_arg, dev)) return NULL;
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
    if (!count_is(n, 5)) return NULL;
    Py_INCREF(a[3]);
    Py_XSETREF(g_current, a[3]);
    Py_INCREF(a[4]);
    Py_XSETREF(g_make_types, a[4]);
    for (i = 0; i < 3; ++i)
        if (!address(a[i], &p[i])) return NULL;
    g_append = (rows_fn)p[0];
    g_read = (rows_fn)p[1];
    g_fwd = (fwd_fn)p[2];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, "init(fa_kv4_append, fa_kv4_read, fa_fwd_kv4, current_device, types): their addresses, and two functions"},
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
    g_dtype = PyUnicode_InternFromString("dtype");
    if (g_data_ptr == NULL || g_get_device == NULL || g_is_contiguous == NULL || g_dtype == NULL) return NULL;
    return PyModule_Create(&module);
}
