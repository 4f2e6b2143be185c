/* layer_py.c -- the Python side of the transformer-layer calls: checks of their
 * tensors (layer_tensor.cpp reads them), and the call into libbigemm.
 *
 * A call for a single token runs for 2 us on the GPU; reading and checking its
 * tensors' shapes, strides, types and addresses in Python took 6 us beside the
 * 2 us of the launch, so that is done here.  The library's functions come as
 * addresses (init), from the same libbigemm.so that the ctypes binding loaded.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/bigemm.h"
#include "layer_tensor.h"

enum { OTHER_DEVICE = -1 };

static PyObject *g_workspace, *g_alloc, *g_free;

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

static bigemm_status (*p_layernorm)(int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const float *,
                                    const float *, float, void *, int64_t, bigemm_dtype, void *, int64_t, void *, float *,
                                    float *, void *);
static bigemm_status (*p_layernorm_backward)(int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t,
                                             const float *, const float *, const float *, const void *, int64_t, void *,
                                             int64_t, float *, float *, void *, uint64_t, void *);
static bigemm_status (*p_rmsnorm_backward)(int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t,
                                           const float *, float, const void *, int64_t, void *, int64_t, float *, void *,
                                           uint64_t, void *);
static uint64_t (*p_norm_workspace)(int, int);
static bigemm_status (*p_gated)(int, int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const void *, int64_t,
                                const float *, const float *, int, void *, int64_t, void *, int64_t, void *, int64_t, void *,
                                uint64_t, void *);
static uint64_t (*p_gated_workspace)(int, int, int, const void *, int64_t, const void *, int64_t, const void *, int64_t);
static bigemm_status (*p_backward)(int, int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const void *,
                                   int64_t, void *, int64_t, void *, int64_t, float *, void *, uint64_t, void *);
static uint64_t (*p_backward_workspace)(int, int, int, const void *, int64_t, const void *, int64_t, const void *, int64_t);
static bigemm_status (*p_gated_backward)(int, int, int, bigemm_dtype, const void *, int64_t, const void *, int64_t, const void *,
                                         int64_t, const void *, int64_t, const void *, int64_t, const void *, int64_t, int,
                                         void *, int64_t, void *, int64_t, void *, int64_t, float *, float *, void *, uint64_t,
                                         void *);
static uint64_t (*p_gated_backward_workspace)(int, int, int, const void *, int64_t, const void *, int64_t, const void *, int64_t);

typedef struct {
    long long rows, cols, ld;
    void *ptr;
    int dtype;                       /* bigemm_dtype */
    long device;
} Matrix;

/* A 2-D CUDA tensor with a contiguous last axis.  like: its device, and rows and
 * cols where those are not negative, have to be these. */
static int matrix(PyObject *o, const char *name, Matrix *m, long device, long long rows, long long cols)
{
    LayerTensor t;
    if (layer_tensor(o, name, &t) < 0) return -1;
    m->rows = t.size[0], m->cols = t.size[1], m->ld = t.stride[0], m->device = t.device, m->ptr = t.ptr, m->dtype = t.type;
    if (t.dims != 2 || m->device < 0) {
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
    if (t.stride[1] != 1 && m->cols > 1) {
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
    if (m->dtype < BIGEMM_F32 || m->dtype > BIGEMM_MXF8) {
        PyObject *d = PyObject_GetAttrString(o, "dtype");
        if (d) PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %R", name, d);
        Py_XDECREF(d);
        return -1;
    }
    return 0;
}

/* The address of a float32 vector of n elements, or null for None. */
static int vector(PyObject *o, const char *name, long long n, long device, void **p)
{
    LayerTensor t;
    *p = NULL;
    if (o == Py_None) return 0;
    if (layer_tensor(o, name, &t) < 0) return -1;
    if (t.dims != 1 || t.size[0] != n || !t.contiguous || t.type != BIGEMM_F32 || t.device != device) {
        PyErr_Format(PyExc_ValueError, "%s: expected a contiguous float32 vector of %lld elements on cuda:%ld", name, n,
                     device);
        return -1;
    }
    *p = t.ptr;
    return 0;
}

/* The address of the scales of a rows x cols MXFP8 matrix. */
static int scales(PyObject *o, const char *name, long long rows, long long cols, long device, void **p)
{
    LayerTensor t;
    const long long a = (rows + 127) / 128, b = (cols + 127) / 128;
    if (o == Py_None) {
        PyErr_Format(PyExc_ValueError, "%s: missing", name);
        return -1;
    }
    if (layer_tensor(o, name, &t) < 0) return -1;
    if (!t.contiguous || t.device != device || t.numel != a * b * 512 || (t.type != TYPE_SCALE_U8 && t.type != TYPE_SCALE_E8M0)) {
        PyErr_Format(PyExc_ValueError, "%s: expected contiguous scales of shape (%lld, %lld, 32, 4, 4) on cuda:%ld", name, a, b,
                     device);
        return -1;
    }
    *p = t.ptr;
    return 0;
}

/* The stream to use, as an address; 1 if another device than `device` is current. */
static int stream_on(PyObject *s, long device, void **stream)
{
    long current;
    if (layer_current(device, &current, stream) < 0) return -1;
    if (current != device) return 1;
    if (s == Py_None) return 0;
    PyObject *o = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
    if (!o) return -1;
    *stream = PyLong_AsVoidPtr(o);
    Py_DECREF(o);
    return !*stream && PyErr_Occurred() ? -1 : 0;
}

/* A call's memory from torch, the stream's until the call is done: it may be given out again after this returns. */
typedef struct {
    PyObject *tensor, *address;      /* on a stream of its own, or on the current one */
    void *ptr;
} Space;

/* `bytes` of it (none for 0) beside t, for a call on `stream`, given as s.  On the current stream it comes as an address:
 * making a tensor takes 1.6 us by itself, and 7 between launches, whose code and data it drives out of the host's caches
 * (8 x 256 rmsnorm_backward: 4.8 us less). */
static int space_for(uint64_t bytes, PyObject *t, PyObject *s, void *stream, Space *space)
{
    space->tensor = space->address = NULL, space->ptr = NULL;
    if (bytes == 0) return 0;
    PyObject *b = PyLong_FromUnsignedLongLong(bytes);
    if (!b) return -1;
    if (s == Py_None) {
        PyObject *h = PyLong_FromVoidPtr(stream);
        if (h) {
            PyObject *const args[2] = {b, h};
            space->address = PyObject_Vectorcall(g_alloc, args, 2, NULL);
            Py_DECREF(h);
        }
        Py_DECREF(b);
        if (!space->address) return -1;
        space->ptr = PyLong_AsVoidPtr(space->address);
        return !space->ptr && PyErr_Occurred() ? -1 : 0;
    }
    PyObject *const args[3] = {b, t, s};
    space->tensor = PyObject_Vectorcall(g_workspace, args, 3, NULL);
    Py_DECREF(b);
    if (!space->tensor) return -1;
    LayerTensor made;
    if (layer_tensor(space->tensor, "workspace", &made) < 0) {
        Py_CLEAR(space->tensor);
        return -1;
    }
    space->ptr = made.ptr;
    return 0;
}

/* The call's answer, its memory given back. */
static PyObject *done(Space *space, bigemm_status st)
{
    Py_XDECREF(space->tensor);
    if (space->address) {
        PyObject *r = PyObject_CallOneArg(g_free, space->address);
        Py_DECREF(space->address);
        if (!r) return NULL;
        Py_DECREF(r);
    }
    return PyLong_FromLong(st);
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
    void *xs = NULL, *ws = NULL, *ys = NULL, *bias, *stream;
    Space space;
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
    uint64_t bytes = 0;
    if (x.rows > 0)
        bytes = p_workspace((int)x.rows, (int)w.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, w.ptr, w.ld);
    if (space_for(bytes, a[0], a[10], stream, &space) < 0) return NULL;
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    if (mx)
        st = p_matmul_mx((int)x.rows, (int)w.rows, (int)x.cols, x.ptr, x.ld, xs, w.ptr, w.ld, ws, bias, act, combine,
                         (bigemm_dtype)o.dtype, o.ptr, o.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, ys, space.ptr, bytes,
                         stream);
    else
        st = p_matmul((int)x.rows, (int)w.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, w.ptr, w.ld, bias, act,
                      combine, (bigemm_dtype)o.dtype, o.ptr, o.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, space.ptr, bytes,
                      stream);
    Py_END_ALLOW_THREADS
    return done(&space, st);
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

/* layernorm(x, weight, bias, residual, eps, sum_out, mean, rstd, out, out_scale, stream) -> status */
static PyObject *layernorm(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix x, res = {0}, sum = {0}, y;
    void *weight, *bias, *mean, *rstd, *ys = NULL, *stream;
    if (arity("layernorm", n, 11) < 0 || matrix(a[0], "x", &x, -1, -1, -1) < 0) return NULL;
    if (vector(a[1], "weight", x.cols, x.device, &weight) < 0 || vector(a[2], "bias", x.cols, x.device, &bias) < 0) return NULL;
    if (a[3] != Py_None && matrix(a[3], "residual", &res, x.device, x.rows, x.cols) < 0) return NULL;
    const double eps = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return NULL;
    if (a[5] != Py_None && matrix(a[5], "sum_out", &sum, x.device, x.rows, x.cols) < 0) return NULL;
    if ((a[3] != Py_None && res.dtype != x.dtype) || (a[5] != Py_None && sum.dtype != x.dtype))
        return PyErr_Format(PyExc_TypeError, "residual and sum_out are of x's dtype");
    if (vector(a[6], "mean_out", x.rows, x.device, &mean) < 0 || vector(a[7], "rstd_out", x.rows, x.device, &rstd) < 0)
        return NULL;
    if (matrix(a[8], "out", &y, x.device, x.rows, x.cols) < 0) return NULL;
    if (y.dtype == BIGEMM_MXF8 && scales(a[9], "out_scale", y.rows, y.cols, x.device, &ys) < 0) return NULL;
    const int r = stream_on(a[10], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_layernorm((int)x.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, res.ptr, res.ld, weight, bias, (float)eps,
                     sum.ptr, sum.ld, (bigemm_dtype)y.dtype, y.ptr, y.ld, ys, mean, rstd, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(st);
}

/* norm_backward(dout, x, mean, rstd, weight, eps, dsum, dx, dweight, dbias, stream) -> status; the root-mean-square
 * norm's where mean is None */
static PyObject *norm_backward(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix d, x, sum = {0}, dx;
    void *mean = NULL, *rstd = NULL, *weight, *dweight, *dbias = NULL, *stream;
    if (arity("norm_backward", n, 11) < 0 || matrix(a[1], "x", &x, -1, -1, -1) < 0 ||
        matrix(a[0], "dout", &d, x.device, x.rows, x.cols) < 0)
        return NULL;
    const int layer = a[9] != Py_None;
    if (layer) {
        if (a[2] == Py_None || a[3] == Py_None) return PyErr_Format(PyExc_ValueError, "mean and rstd: missing");
        if (vector(a[2], "mean", x.rows, x.device, &mean) < 0 || vector(a[3], "rstd", x.rows, x.device, &rstd) < 0) return NULL;
        if (vector(a[9], "dbias", x.cols, x.device, &dbias) < 0) return NULL;
    }
    if (vector(a[4], "weight", x.cols, x.device, &weight) < 0) return NULL;
    const double eps = PyFloat_AsDouble(a[5]);
    if (PyErr_Occurred()) return NULL;
    if (a[6] != Py_None && matrix(a[6], "dsum", &sum, x.device, x.rows, x.cols) < 0) return NULL;
    if (matrix(a[7], "dx", &dx, x.device, x.rows, x.cols) < 0) return NULL;
    if (d.dtype != x.dtype || dx.dtype != x.dtype || (a[6] != Py_None && sum.dtype != x.dtype))
        return PyErr_Format(PyExc_TypeError, "dout, dsum and dx are of x's dtype");
    if (vector(a[8], "dweight", x.cols, x.device, &dweight) < 0) return NULL;
    const int r = stream_on(a[10], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    const uint64_t bytes = p_norm_workspace((int)x.rows, (int)x.cols);
    Space space;
    if (space_for(bytes, a[1], a[10], stream, &space) < 0) return NULL;
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    if (layer)
        st = p_layernorm_backward((int)x.rows, (int)x.cols, (bigemm_dtype)x.dtype, d.ptr, d.ld, x.ptr, x.ld, mean, rstd, weight,
                                  sum.ptr, sum.ld, dx.ptr, dx.ld, dweight, dbias, space.ptr, bytes, stream);
    else
        st = p_rmsnorm_backward((int)x.rows, (int)x.cols, (bigemm_dtype)x.dtype, d.ptr, d.ld, x.ptr, x.ld, weight, (float)eps,
                                sum.ptr, sum.ld, dx.ptr, dx.ld, dweight, space.ptr, bytes, stream);
    Py_END_ALLOW_THREADS
    return done(&space, st);
}

/* A matrix of x's type, or nothing for None where `optional`. */
static int beside(PyObject *t, const char *name, Matrix *m, const Matrix *x, long long rows, long long cols, int optional)
{
    if (optional && t == Py_None) return 0;
    if (matrix(t, name, m, x->device, rows, cols) < 0) return -1;
    if (m->dtype == x->dtype) return 0;
    PyErr_Format(PyExc_TypeError, "%s: of another dtype than x", name);
    return -1;
}

/* gated(x, w_gate, w_up, bias_gate, bias_up, act, out, gate, up, stream) -> status */
static PyObject *gated(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix x, wg, wu, y, g = {0}, u = {0};
    void *bg, *bu, *stream;
    if (arity("gated", n, 10) < 0 || matrix(a[0], "x", &x, -1, -1, -1) < 0 || beside(a[1], "w_gate", &wg, &x, -1, x.cols, 0) < 0 ||
        beside(a[2], "w_up", &wu, &x, wg.rows, x.cols, 0) < 0 || vector(a[3], "bias_gate", wg.rows, x.device, &bg) < 0 ||
        vector(a[4], "bias_up", wg.rows, x.device, &bu) < 0)
        return NULL;
    const int act = (int)PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return NULL;
    if (beside(a[6], "out", &y, &x, x.rows, wg.rows, 0) < 0 || beside(a[7], "gate_out", &g, &x, x.rows, wg.rows, 1) < 0 ||
        beside(a[8], "up_out", &u, &x, x.rows, wg.rows, 1) < 0)
        return NULL;
    const int r = stream_on(a[9], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    const uint64_t bytes = p_gated_workspace((int)x.rows, (int)wg.rows, (int)x.cols, x.ptr, x.ld, wg.ptr, wg.ld, wu.ptr, wu.ld);
    Space space;
    if (space_for(bytes, a[0], a[9], stream, &space) < 0) return NULL;
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_gated((int)x.rows, (int)wg.rows, (int)x.cols, (bigemm_dtype)x.dtype, x.ptr, x.ld, wg.ptr, wg.ld, wu.ptr, wu.ld, bg, bu,
                 act, y.ptr, y.ld, g.ptr, g.ld, u.ptr, u.ld, space.ptr, bytes, stream);
    Py_END_ALLOW_THREADS
    return done(&space, st);
}

/* product_backward(dout, x, w, dx, dw, dbias, stream) -> status */
static PyObject *product_backward(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix d, x, w, dx, dw;
    void *dbias, *stream;
    if (arity("product_backward", n, 7) < 0 || matrix(a[1], "x", &x, -1, -1, -1) < 0 ||
        beside(a[2], "w", &w, &x, -1, x.cols, 0) < 0 || beside(a[0], "dout", &d, &x, x.rows, w.rows, 0) < 0 ||
        beside(a[3], "dx", &dx, &x, x.rows, x.cols, 0) < 0 || beside(a[4], "dw", &dw, &x, w.rows, x.cols, 0) < 0 ||
        vector(a[5], "dbias", w.rows, x.device, &dbias) < 0)
        return NULL;
    const int r = stream_on(a[6], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    const uint64_t bytes = p_backward_workspace((int)x.rows, (int)w.rows, (int)x.cols, d.ptr, d.ld, x.ptr, x.ld, w.ptr, w.ld);
    Space space;
    if (space_for(bytes, a[1], a[6], stream, &space) < 0) return NULL;
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_backward((int)x.rows, (int)w.rows, (int)x.cols, (bigemm_dtype)x.dtype, d.ptr, d.ld, x.ptr, x.ld, w.ptr, w.ld, dx.ptr,
                    dx.ld, dw.ptr, dw.ld, dbias, space.ptr, bytes, stream);
    Py_END_ALLOW_THREADS
    return done(&space, st);
}

/* gated_backward(dout, x, w_gate, w_up, gate, up, act, dx, dw_gate, dw_up, dbias_gate, dbias_up, stream) -> status */
static PyObject *gated_backward(PyObject *self, PyObject *const *a, Py_ssize_t n)
{
    Matrix d, x, wg, wu, g, u, dx, dwg, dwu;
    void *dbg, *dbu, *stream;
    if (arity("gated_backward", n, 13) < 0 || matrix(a[1], "x", &x, -1, -1, -1) < 0 ||
        beside(a[2], "w_gate", &wg, &x, -1, x.cols, 0) < 0 || beside(a[3], "w_up", &wu, &x, wg.rows, x.cols, 0) < 0 ||
        beside(a[0], "dout", &d, &x, x.rows, wg.rows, 0) < 0 || beside(a[4], "gate", &g, &x, x.rows, wg.rows, 0) < 0 ||
        beside(a[5], "up", &u, &x, x.rows, wg.rows, 0) < 0)
        return NULL;
    const int act = (int)PyLong_AsLong(a[6]);
    if (PyErr_Occurred()) return NULL;
    if (beside(a[7], "dx", &dx, &x, x.rows, x.cols, 0) < 0 || beside(a[8], "dw_gate", &dwg, &x, wg.rows, x.cols, 0) < 0 ||
        beside(a[9], "dw_up", &dwu, &x, wg.rows, x.cols, 0) < 0 || vector(a[10], "dbias_gate", wg.rows, x.device, &dbg) < 0 ||
        vector(a[11], "dbias_up", wg.rows, x.device, &dbu) < 0)
        return NULL;
    const int r = stream_on(a[12], x.device, &stream);
    if (r < 0) return NULL;
    if (r > 0) return PyLong_FromLong(OTHER_DEVICE);
    const uint64_t bytes = p_gated_backward_workspace((int)x.rows, (int)wg.rows, (int)x.cols, x.ptr, x.ld, wg.ptr, wg.ld, wu.ptr,
                                                      wu.ld);
    Space space;
    if (space_for(bytes, a[1], a[12], stream, &space) < 0) return NULL;
    bigemm_status st;
    Py_BEGIN_ALLOW_THREADS
    st = p_gated_backward((int)x.rows, (int)wg.rows, (int)x.cols, (bigemm_dtype)x.dtype, d.ptr, d.ld, x.ptr, x.ld, wg.ptr, wg.ld,
                          wu.ptr, wu.ld, g.ptr, g.ld, u.ptr, u.ld, act, dx.ptr, dx.ld, dwg.ptr, dwg.ld, dwu.ptr, dwu.ld, dbg,
                          dbu, space.ptr, bytes, stream);
    Py_END_ALLOW_THREADS
    return done(&space, st);
}

/* init(workspace, alloc, free, functions): workspace(bytes, tensor, stream) makes a tensor, alloc(bytes, stream) an
 * address for free */
static PyObject *init(PyObject *self, PyObject *args)
{
    PyObject *ws, *al, *fr, *functions;
    enum { COUNT = 15 };
    unsigned long long f[COUNT];
    if (!PyArg_ParseTuple(args, "OOOO!", &ws, &al, &fr, &PyTuple_Type, &functions)) return NULL;
    if (PyTuple_GET_SIZE(functions) != COUNT) return PyErr_Format(PyExc_ValueError, "init: wrong number of functions");
    for (int i = 0; i < COUNT; ++i) {
        f[i] = PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(functions, i));
        if (PyErr_Occurred()) return NULL;
    }
    g_workspace = Py_NewRef(ws);
    g_alloc = Py_NewRef(al);
    g_free = Py_NewRef(fr);
    p_matmul = (void *)(uintptr_t)f[0];
    p_matmul_mx = (void *)(uintptr_t)f[1];
    p_norm = (void *)(uintptr_t)f[2];
    p_quantize = (void *)(uintptr_t)f[3];
    p_workspace = (void *)(uintptr_t)f[4];
    p_layernorm = (void *)(uintptr_t)f[5];
    p_layernorm_backward = (void *)(uintptr_t)f[6];
    p_rmsnorm_backward = (void *)(uintptr_t)f[7];
    p_norm_workspace = (void *)(uintptr_t)f[8];
    p_gated = (void *)(uintptr_t)f[9];
    p_gated_workspace = (void *)(uintptr_t)f[10];
    p_backward = (void *)(uintptr_t)f[11];
    p_backward_workspace = (void *)(uintptr_t)f[12];
    p_gated_backward = (void *)(uintptr_t)f[13];
    p_gated_backward_workspace = (void *)(uintptr_t)f[14];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, NULL},
    {"product", (PyCFunction)(void (*)(void))product, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))norm, METH_FASTCALL, NULL},
    {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, NULL},
    {"layernorm", (PyCFunction)(void (*)(void))layernorm, METH_FASTCALL, NULL},
    {"gated", (PyCFunction)(void (*)(void))gated, METH_FASTCALL, NULL},
    {"product_backward", (PyCFunction)(void (*)(void))product_backward, METH_FASTCALL, NULL},
    {"gated_backward", (PyCFunction)(void (*)(void))gated_backward, METH_FASTCALL, NULL},
    {"norm_backward", (PyCFunction)(void (*)(void))norm_backward, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", NULL, -1, methods, NULL, NULL, NULL, NULL};

/* built_for: the torch and the Python whose tensors layer_tensor.cpp was compiled to read. */
PyMODINIT_FUNC PyInit__layer(void)
{
    PyObject *m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", LAYER_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
