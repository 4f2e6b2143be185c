/* layer_py.c -- the Python side of the transformer-layer calls: checks of their
 * tensors, and the call into libbigemm.
 *
 * A call for a single token runs for 2 us on the GPU; reading and checking its
 * tensors' shapes, strides, types and addresses in Python took 6 us beside the
 * 2 us of the launch, so that is done here.  The library's functions come as
 * addresses (init), from the same libbigemm.so that the ctypes binding loaded.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/bigemm.h"

enum { DT_COUNT = 4, OTHER_DEVICE = -1 };

static PyObject *g_dtypes[DT_COUNT];                 /* torch dtypes of F32, F16, BF16, MXF8 */
static PyObject *g_scale_types[2];                   /* uint8, float8_e8m0fnu */
static PyObject *g_current_stream, *g_current_device, *g_workspace;
static PyObject *s_shape, *s_stride, *s_device, *s_ptr, *s_dtype, *s_numel, *s_contiguous;

static bigemm_status (*p_matmul)(int, int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const float *,
                                 int, int, bigemm_dtype, const void *, int64_t, bigemm_dtype, void *, int64_t, void *,
                                 uint64_t, void *);
static bigemm_status (*p_matmul_mx)(int, int, int, const void *, int64_t, const void *, const void *, int64_t,
                                    const void *, const float *, int, int, bigemm_dtype, const void *, int64_t,
                                    bigemm_dtype, void *, int64_t, void *, void *, uint64_t, void *);
static uint64_t (*p_workspace)(int, int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t);
static bigemm_status (*p_norm)(int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const float *, float,
                               void *, int64_t, bigemm_dtype, void *, int64_t, void *, void *);
static bigemm_status (*p_quantize)(int, int, bigemm_dtype, const void *, int64_t, void *, int64_t, void *, void *);

typedef struct {
    long long rows, cols, ld;
    void *ptr;
    int dtype;                       /* bigemm_dtype */
    long device;
} Matrix;

static int as_ll(PyObject *o, long long *v)          /* steals o */
{
    if (!o) return -1;
    *v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return *v == -1 && PyErr_Occurred() ? -1 : 0;
}

static int dtype_of(PyObject *t, const char *name, int *code)
{
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    Py_DECREF(d);                    /* torch's dtypes live for ever */
    for (int i = 0; i < DT_COUNT; ++i)
        if (d == g_dtypes[i]) {
            *code = i;
            return 0;
        }
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %R", name, d);
    return -1;
}

static int device_of(PyObject *t, long *dev)
{
    long long v;
    if (as_ll(PyObject_CallMethodNoArgs(t, s_device), &v) < 0) return -1;
    *dev = (long)v;
    return 0;
}

static int pointer_of(PyObject *t, void **p)
{
    PyObject *o = PyObject_CallMethodNoArgs(t, s_ptr);
    if (!o) return -1;
    *p = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return !*p && PyErr_Occurred() ? -1 : 0;
}

/* Two integers of a shape or a stride (steals o); 1 if there are not two. */
static int pair(PyObject *o, long long *a, long long *b)
{
    if (!o) return -1;
    int r = 1;
    if (PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 2) {
        *a = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 0));
        *b = PyLong_AsLongLong(PyTuple_GET_ITEM(o, 1));
        r = PyErr_Occurred() ? -1 : 0;
    }
    Py_DECREF(o);
    return r;
}

/* A 2-D CUDA tensor with a contiguous last axis.  like: its device, and rows and
 * cols where those are not negative, have to be these. */
static int matrix(PyObject *t, const char *name, Matrix *m, long device, long long rows, long long cols)
{
    long long one;
    int r = pair(PyObject_GetAttr(t, s_shape), &m->rows, &m->cols);
    if (r < 0 || device_of(t, &m->device) < 0) return -1;
    if (r || m->device < 0) {
        PyErr_Format(PyExc_ValueError, "%s: expected a 2-D CUDA tensor", name);
        return -1;
    }
    if ((rows >= 0 && m->rows != rows) || (cols >= 0 && m->cols != cols)) {
        PyErr_Format(PyExc_ValueError, "%s: expected %lld rows of %lld, got %lld of %lld", name, rows < 0 ? m->rows : rows,
                     cols < 0 ? m->cols : cols, m->rows, m->cols);
        return -1;
    }
    if (device >= 0 && m->device != device) {
        PyErr_Format(PyExc_ValueError, "%s: on cuda:%ld, expected cuda:%ld", name, m->device, device);
        return -1;
    }
    r = pair(PyObject_CallMethodNoArgs(t, s_stride), &m->ld, &one);
    if (r) {
        if (r > 0) PyErr_Format(PyExc_ValueError, "%s: no strides", name);
        return -1;
    }
    if (one != 1 && m->cols > 1) {
        PyErr_Format(PyExc_ValueError, "%s: the last axis must be contiguous", name);
        return -1;
    }
    if (m->ld < m->cols) {
        if (m->rows > 1) {
            PyErr_Format(PyExc_ValueError, "%s: rows overlap", name);
            return -1;
        }
        m->ld = m->cols;             /* a single row's stride may be anything */
    }
    if (m->rows > 0x7fffffffLL || m->cols > 0x7fffffffLL) {
        PyErr_Format(PyExc_ValueError, "%s: too large", name);
        return -1;
    }
    return dtype_of(t, name, &m->dtype) < 0 || pointer_of(t, &m->ptr) < 0 ? -1 : 0;
}

/* The address of a float32 vector of n elements, or null for None. */
static int vector(PyObject *t, const char *name, long long n, long device, void **p)
{
    *p = NULL;
    if (t == Py_None) return 0;
    long dev;
    int ok = 0;
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    Py_DECREF(d);
    if (device_of(t, &dev) < 0) return -1;
    PyObject *shape = PyObject_GetAttr(t, s_shape);
    if (!shape) return -1;
    if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 1) ok = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0)) == n;
    Py_DECREF(shape);
    PyObject *c = PyObject_CallMethodNoArgs(t, s_contiguous);
    if (!c) return -1;
    ok = ok && c == Py_True && d == g_dtypes[BIGEMM_F32] && dev == device;
    Py_DECREF(c);
    if (!ok) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous float32 vector of %lld elements on cuda:%ld", name, n,
                     device);
        return -1;
    }
    return pointer_of(t, p);
}

/* The address of the scales of a rows x cols MXFP8 matrix. */
static int scales(PyObject *t, const char *name, long long rows, long long cols, long device, void **p)
{
    long dev;
    long long n;
    const long long a = (rows + 127) / 128, b = (cols + 127) / 128;
    if (t == Py_None) {
        PyErr_Format(PyExc_ValueError, "%s: missing", name);
        return -1;
    }
    PyObject *d = PyObject_GetAttr(t, s_dtype);
    if (!d) return -1;
    Py_DECREF(d);
    if (device_of(t, &dev) < 0 || as_ll(PyObject_CallMethodNoArgs(t, s_numel), &n) < 0) return -1;
    PyObject *c = PyObject_CallMethodNoArgs(t, s_contiguous);
    if (!c) return -1;
    const int ok = c == Py_True && dev == device && n == a * b * 512 && (d == g_scale_types[0] || d == g_scale_types[1]);
    Py_DECREF(c);
    if (!ok) {
        PyErr_Format(PyExc_ValueError, "%s: expected contiguous scales of shape (%lld, %lld, 32, 4, 4) on cuda:%ld", name, a, b,
                     device);
        return -1;
    }
    return pointer_of(t, p);
}

/* The stream to use, as an address; 1 if another device than `device` is current. */
static int stream_on(PyObject *s, long device, void **stream)
{
    long long current;
    if (as_ll(PyObject_CallNoArgs(g_current_device), &current) < 0) return -1;
    if (current != device) return 1;
    PyObject *o;
    if (s == Py_None) {
        PyObject *d = PyLong_FromLong(device);
        if (!d) return -1;
        o = PyObject_CallOneArg(g_current_stream, d);
        Py_DECREF(d);
    } else if (PyLong_Check(s)) {
        o = Py_NewRef(s);
    } else {
        o = PyObject_GetAttrString(s, "cuda_stream");
    }
    if (!o) return -1;
    *stream = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return !*stream && PyErr_Occurred() ? -1 : 0;
}

static int arity(const char *name, Py_ssize_t got, Py_ssize_t want)
{
    if (got == want) return 0;
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, expected %zd", name, got, want);
    return -1;
}

/* product(x, x_scale, w, w_scale, bias, act, other, combine, out, out_scale, stream) -> status */
static PyObject *product(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix x, w, o = {0}, y;
    void *xs = NULL, *ws = NULL, *ys = NULL, *bias, *stream, *space = NULL;
    if (arity("product", n, 11) < 0 || matrix(a[0], "x", &x, -1, -1, -1) < 0 ||
        matrix(a[2], "w", &w, x.device, -1, x.cols) < 0)
        return NULL;
    if (w.dtype != x.dtype) return PyErr_Format(PyExc_TypeError, "w: of another dtype than x");
    const int mx = x.dtype == BIGEMM_MXF8;
    if (mx != (a[1] != Py_None))
        return PyErr_Format(PyExc_TypeError, "matmul_mx takes float8_e4m3fn matrices and their scales, matmul 16-bit ones");
    if (mx && (scales(a[1], "x_scale", x.rows, x.cols, x.device, &xs) < 0 ||
               scales(a[3], "w_scale", w.rows, w.cols, x.device, &ws) < 0))
        return NULL;
    if (vector(a[4], "bias", w.rows, x.device, &bias) < 0) return NULL;
    const int act = (int)PyLong_AsLong(a[5]), combine = (int)PyLong_AsLong(a[7]);
    if (PyErr_Occurred()) return NULL;
    if (combine != BIGEMM_COMBINE_NONE) {
        if (a[6] == Py_None) return PyErr_Format(PyExc_ValueError, "combine needs other");
        if (matrix(a[6], "other", &o, x.device, x.rows, w.rows) < 0) return NULL;
    }
    if (matrix(a[8], "out", &y, x.device, x.rows, w.rows) < 0) return NULL;
    if (y.dtype == BIGEMM_MXF8 && scales(a[9], "out_scale", y.rows, y.cols, x.device, &ys) < 0) return NULL;
    const int r = stream_on(a[10], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    PyObject *workspace = NULL;
    uint64_t bytes = 0;
    if (x.rows > 0)
        bytes = p_workspace((int)x.rows, (int)w.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, w.ptr, w.ld);
    if (bytes > 0) {
        /* torch's memory, the stream's until the call is done: it may be given out again after this returns */
        PyObject *b = PyLong_FromUnsignedLongLong(bytes);
        if (!b) return NULL;
        PyObject *const args[3] = {b, a[0], a[10]};
        workspace = PyObject_Vectorcall(g_workspace, args, 3, NULL);
        Py_DECREF(b);
        if (!workspace) return NULL;
        if (pointer_of(workspace, &space) < 0) {
            Py_DECREF(workspace);
            return NULL;
        }
    }
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    if (mx)
        st = p_matmul_mx((int)x.rows, (int)w.rows, (int)x.cols, x.ptr, x.ld, xs, w.ptr, w.ld, ws, bias, act, combine,
                         (bigemm_dtype)o.dtype, o.ptr, o.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, ys, space, bytes, stream);
    else
        st = p_matmul((int)x.rows, (int)w.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, w.ptr, w.ld, bias, act,
                      combine, (bigemm_dtype)o.dtype, o.ptr, o.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, space, bytes,
                      stream);
    Py_END_ALLOW_THREADS
    Py_XDECREF(workspace);
    return PyLong_FromLong(st);
}

/* norm(x, weight, residual, eps, sum_out, out, out_scale, stream) -> status */
static PyObject *norm(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix x, res = {0}, sum = {0}, y;
    void *weight, *ys = NULL, *stream;
    if (arity("norm", n, 8) < 0 || matrix(a[0], "x", &x, -1, -1, -1) < 0) return NULL;
    if (vector(a[1], "weight", x.cols, x.device, &weight) < 0) return NULL;
    if (a[2] != Py_None && matrix(a[2], "residual", &res, x.device, x.rows, x.cols) < 0) return NULL;
    const double eps = PyFloat_AsDouble(a[3]);
    if (PyErr_Occurred()) return NULL;
    if (a[4] != Py_None && matrix(a[4], "sum_out", &sum, x.device, x.rows, x.cols) < 0) return NULL;
    if ((res.ptr && res.dtype != x.dtype) || (sum.ptr && sum.dtype != x.dtype))
        return PyErr_Format(PyExc_TypeError, "residual and sum_out are of x's dtype");
    if (matrix(a[5], "out", &y, x.device, x.rows, x.cols) < 0) return NULL;
    if (y.dtype == BIGEMM_MXF8 && scales(a[6], "out_scale", y.rows, y.cols, x.device, &ys) < 0) return NULL;
    const int r = stream_on(a[7], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_norm((int)x.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, res.ptr, res.ld, weight, (float)eps, sum.ptr,
                sum.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, ys, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* quantize(x, out, scale, stream) -> status */
static PyObject *quantize(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix x, y;
    void *ys, *stream;
    if (arity("quantize", n, 4) < 0 || matrix(a[0], "x", &x, -1, -1, -1) < 0 ||
        matrix(a[1], "out", &y, x.device, x.rows, x.cols) < 0)
        return NULL;
    if (y.dtype != BIGEMM_MXF8) return PyErr_Format(PyExc_TypeError, "out: expected float8_e4m3fn");
    if (scales(a[2], "scale", x.rows, x.cols, x.device, &ys) < 0) return NULL;
    const int r = stream_on(a[3], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_quantize((int)x.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, y.ptr, y.ld, ys, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* init(dtypes, scale_types, current_stream, current_device, workspace, functions) */
static PyObject *init(PyObject *self, PyObject *args)
{
    PyObject *d, *st, *cs, *cd, *ws;
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "O!O!OOO(KKKKK)", &PyTuple_Type, &d, &PyTuple_Type, &st, &cs, &cd, &ws, &f[0], &f[1], &f[2], &f[3],
                          &f[4]))
        return NULL;
    if (PyTuple_GET_SIZE(d) != DT_COUNT || PyTuple_GET_SIZE(st) != 2)
        return PyErr_Format(PyExc_ValueError, "init: wrong number of dtypes");
    for (int i = 0; i < DT_COUNT; ++i) g_dtypes[i] = Py_NewRef(PyTuple_GET_ITEM(d, i));
    for (int i = 0; i < 2; ++i) g_scale_types[i] = Py_NewRef(PyTuple_GET_ITEM(st, i));
    g_current_stream = Py_NewRef(cs);
    g_current_device = Py_NewRef(cd);
    g_workspace = Py_NewRef(ws);
    p_matmul = (void *)(uintptr_t)f[0];
    p_matmul_mx = (void *)(uintptr_t)f[1];
    p_norm = (void *)(uintptr_t)f[2];
    p_quantize = (void *)(uintptr_t)f[3];
    p_workspace = (void *)(uintptr_t)f[4];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"product", (PyCFunction)(void (*)(void))product, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, NULL},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__layer(void)
{
    s_shape = PyUnicode_InternFromString("shape");
    s_stride = PyUnicode_InternFromString("stride");
    s_device = PyUnicode_InternFromString("get_device");
    s_ptr = PyUnicode_InternFromString("data_ptr");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_numel = PyUnicode_InternFromString("numel");
    s_contiguous = PyUnicode_InternFromString("is_contiguous");
    if (!s_shape || !s_stride || !s_device || !s_ptr || !s_dtype || !s_numel || !s_contiguous) return NULL;
    return PyModule_Create(&module);
}
