/* fp8bq_calls.c -- the ordinary call of the 4-bit conveniences without the
 * interpreter between its steps (CPython module `_calls`).
 *
 * A product of one token takes the GPU a few microseconds; the same checks,
 * allocations and descriptor in Python take twice that.  Each function here
 * looks at its arguments as the Python conveniences do, and where they are the
 * ordinary ones (contiguous CUDA tensors of the current device that fit each
 * other) allocates the outputs through PyTorch, makes the call of the C ABI
 * and returns the outputs.  Anything else, a mistake in the arguments among
 * it, returns None with nothing done: the Python convenience then takes the
 * call, and says what is wrong.  A status of the C ABI is returned as an int.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

#include "../../include/fp8bq.h"

typedef fp8bq_status (*product_fn)(const fp8bq_fp4_matmul_desc *, cudaStream_t);
typedef fp8bq_status (*quantize_fn)(const fp8bq_fp4_desc *, int, cudaStream_t);
typedef fp8bq_status (*dequantize_fn)(const uint8_t *, const uint8_t *, int64_t, int64_t, int64_t,
                                      fp8bq_fp4_format, const float *, int64_t, void *, fp8bq_dtype,
                                      int64_t, int64_t, cudaStream_t);

static PyTypeObject *g_tensor;                      /* torch.Tensor */
static PyObject *g_uint8, *g_bf16, *g_f32;          /* dtypes */
static product_fn g_product[2];
static quantize_fn g_quantize;
static dequantize_fn g_dequantize;
static PyObject *s_shape, *s_dtype, *s_data_ptr, *s_get_device, *s_is_contiguous, *s_new_empty;
static PyObject *g_kw_dtype;                        /* ("dtype",) */

/* What the calls look at of a tensor; 0 unless it is a contiguous CUDA tensor
 * of device `dev`.  `n`: dimensions, at most 5. */
typedef struct {
    void *ptr;
    int n, type;                                    /* type: 1 uint8, 2 bf16, 3 fp32 */
    int64_t d[5];
} view;

static int as_int(PyObject *o, int64_t *v) {        /* steals o */
    if (o == NULL) return 0;
    *v = PyLong_AsLongLong(o);
    Py_DECREF(o);
    return !(*v == -1 && PyErr_Occurred());
}

static int look(PyObject *t, int64_t dev, view *v) {
    int64_t x;
    if (!PyObject_TypeCheck(t, g_tensor)) return 0;
    if (!as_int(PyObject_CallMethodNoArgs(t, s_get_device), &x) || x != dev || dev < 0) return 0;
    PyObject *o = PyObject_CallMethodNoArgs(t, s_is_contiguous);
    if (o == NULL) return 0;
    const int contiguous = o == Py_True;
    Py_DECREF(o);
    if (!contiguous) return 0;
    o = PyObject_GetAttr(t, s_dtype);
    if (o == NULL) return 0;
    v->type = o == g_uint8 ? 1 : o == g_bf16 ? 2 : o == g_f32 ? 3 : 0;
    Py_DECREF(o);
    if (v->type == 0) return 0;
    o = PyObject_GetAttr(t, s_shape);
    if (o == NULL) return 0;
    int ok = PyTuple_Check(o) && PyTuple_GET_SIZE(o) <= 5;
    if (ok) {
        v->n = (int)PyTuple_GET_SIZE(o);
        for (int i = 0; ok && i < v->n; ++i) {
            v->d[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
            ok = v->d[i] >= 0;
        }
    }
    Py_DECREF(o);
    if (!ok || !as_int(PyObject_CallMethodNoArgs(t, s_data_ptr), &x)) return 0;
    v->ptr = (void *)(uintptr_t)x;
    return 1;
}

/* The tensor's own scale: None, or one fp32 value. */
static int look_scale(PyObject *t, int64_t dev, int nvfp4, const float **p) {
    view v;
    *p = NULL;
    if (t == Py_None) return 1;
    if (!nvfp4 || !look(t, dev, &v) || v.type != 3) return 0;
    for (int i = 0; i < v.n; ++i)
        if (v.d[i] != 1) return 0;
    *p = v.ptr;
    return 1;
}

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

/* Codes and scales that go together: [(E,) rows, kb] and their tiles. */
typedef struct {
    int n;                                          /* 2, or 3 for a stack */
    int64_t E, rows, kb;
    fp8bq_fp4_operand o;
} operand;

static int look_operand(PyObject *codes, PyObject *scales, PyObject *ts, int64_t dev, int nvfp4,
                        operand *r) {
    view c, s;
    if (!look(codes, dev, &c) || !look(scales, dev, &s) || c.type != 1 || s.type != 1) return 0;
    if (c.n < 2 || c.n > 3 || s.n != c.n + 2) return 0;
    const int64_t *cd = c.d + (c.n - 2), *sd = s.d + (s.n - 4);
    r->n = c.n;
    r->E = c.n == 3 ? c.d[0] : 1;
    r->rows = cd[0];
    r->kb = cd[1];
    if ((c.n == 3 && s.d[0] != r->E) || r->kb % 16 || sd[0] != cdiv(r->rows, 128) ||
        sd[1] != cdiv(r->kb, nvfp4 ? 32 : 64) || sd[2] != 32 || sd[3] != 16)
        return 0;
    r->o.codes = c.ptr;
    r->o.scales = s.ptr;
    r->o.codes_batch_stride = r->rows * r->kb;
    r->o.scales_batch_stride = sd[0] * sd[1] * 512;
    r->o.tensor_scale_stride = 0;
    return look_scale(ts, dev, nvfp4, &r->o.tensor_scale);
}

/* like.new_empty(shape, dtype=dtype) and its address. */
static PyObject *make(PyObject *like, int n, const int64_t *d, PyObject *dtype, void **ptr) {
    PyObject *shape = PyTuple_New(n);
    if (shape == NULL) return NULL;
    for (int i = 0; i < n; ++i) {
        PyObject *x = PyLong_FromLongLong(d[i]);
        if (x == NULL) {
            Py_DECREF(shape);
            return NULL;
        }
        PyTuple_SET_ITEM(shape, i, x);
    }
    PyObject *args[3] = {like, shape, dtype};
    PyObject *t = PyObject_VectorcallMethod(s_new_empty, args, 2, g_kw_dtype);
    Py_DECREF(shape);
    int64_t x;
    if (t != NULL && !as_int(PyObject_CallMethodNoArgs(t, s_data_ptr), &x)) Py_CLEAR(t);
    if (t != NULL) *ptr = (void *)(uintptr_t)x;
    return t;
}

/* None: the Python convenience takes the call (and any Python error met while
 * looking is its to raise again). */
static PyObject *not_ordinary(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

static int ints(PyObject *const *args, int n, int64_t *v) {
    for (int i = 0; i < n; ++i) {
        v[i] = PyLong_AsLongLong(args[i]);
        if (v[i] == -1 && PyErr_Occurred()) return 0;
    }
    return 1;
}

/* product(gated, format, device, stream, a, a_scales, a_tensor_scale, b, ..., up, ..., out_dtype) */
static PyObject *calls_product(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    int64_t v[4];
    operand m[3];
    fp8bq_fp4_matmul_desc d;
    (void)self;
    if (n != 14 || !ints(args, 4, v)) return not_ordinary();
    const int count = v[0] ? 3 : 2;
    for (int i = 0; i < count; ++i)
        if (!look_operand(args[4 + 3 * i], args[5 + 3 * i], args[6 + 3 * i], v[2], v[1] == FP8BQ_NVFP4,
                          &m[i]) ||
            m[i].n != m[0].n || m[i].E != m[0].E || m[i].kb != m[0].kb || (i && m[i].rows != m[1].rows))
            return not_ordinary();
    PyObject *dtype = args[13] == Py_None ? g_bf16 : args[13];
    if (dtype != g_bf16 && dtype != g_f32) return not_ordinary();
    memset(&d, 0, sizeof d);
    d.a = m[0].o;
    d.b = m[1].o;
    if (count == 3) d.up = m[2].o;
    d.M = m[0].rows;
    d.N = d.ld_out = m[1].rows;
    d.K = 2 * m[0].kb;
    d.batch = m[0].E;
    d.out_batch_stride = d.M * d.N;
    d.format = (int32_t)v[1];
    d.dtype_out = dtype == g_bf16 ? FP8BQ_BF16 : FP8BQ_F32;
    const int64_t shape[3] = {m[0].E, d.M, d.N};
    PyObject *out = make(args[4], m[0].n, shape + 3 - m[0].n, dtype, &d.out);
    if (out == NULL) return NULL;
    fp8bq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_product[v[0] ? 1 : 0](&d, (cudaStream_t)(uintptr_t)v[3]);
    Py_END_ALLOW_THREADS
    if (st == FP8BQ_OK) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

/* quantize(format, device, stream, x, tensor_scale) -> (codes, scales) */
static PyObject *calls_quantize(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    int64_t v[3];
    view x;
    fp8bq_fp4_desc d;
    (void)self;
    if (n != 5 || !ints(args, 3, v)) return not_ordinary();
    memset(&d, 0, sizeof d);
    const int nvfp4 = v[0] == FP8BQ_NVFP4;
    if (!look(args[3], v[1], &x) || x.type < 2 || x.n < 2 || x.n > 3 ||
        !look_scale(args[4], v[1], nvfp4, &d.tensor_scale))
        return not_ordinary();
    d.x = x.ptr;
    d.batch = x.n == 3 ? x.d[0] : 1;
    d.M = x.d[x.n - 2];
    d.K = d.ld = x.d[x.n - 1];
    d.x_batch_stride = d.M * d.K;
    d.dtype_in = x.type == 2 ? FP8BQ_BF16 : FP8BQ_F32;
    d.format = (int32_t)v[0];
    const int64_t cs[3] = {d.batch, d.M, 16 * cdiv(d.K, 32)};
    const int64_t ss[5] = {d.batch, cdiv(d.M, 128), cdiv(d.K, nvfp4 ? 64 : 128), 32, 16};
    void *pc = NULL, *ps = NULL;
    PyObject *codes = make(args[3], x.n, cs + 3 - x.n, g_uint8, &pc);
    PyObject *scales = codes == NULL ? NULL : make(args[3], x.n + 2, ss + 3 - x.n, g_uint8, &ps);
    if (scales == NULL) {
        Py_XDECREF(codes);
        return NULL;
    }
    d.codes = pc;
    d.scales = ps;
    fp8bq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_quantize(&d, 1, (cudaStream_t)(uintptr_t)v[2]);
    Py_END_ALLOW_THREADS
    PyObject *r = st == FP8BQ_OK ? PyTuple_Pack(2, codes, scales) : PyLong_FromLong(st);
    Py_DECREF(codes);
    Py_DECREF(scales);
    return r;
}

/* dequantize(format, device, stream, codes, scales, tensor_scale, columns, out_dtype) */
static PyObject *calls_dequantize(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    int64_t v[3], K = 0;
    operand m;
    (void)self;
    if (n != 8 || !ints(args, 3, v) ||
        !look_operand(args[3], args[4], args[5], v[1], v[0] == FP8BQ_NVFP4, &m))
        return not_ordinary();
    if (args[6] == Py_None) K = 2 * m.kb;
    else if (!ints(args + 6, 1, &K)) return not_ordinary();
    PyObject *dtype = args[7] == Py_None ? g_bf16 : args[7];
    if ((dtype != g_bf16 && dtype != g_f32) || K < 0 || 16 * cdiv(K, 32) != m.kb)
        return not_ordinary();
    const int64_t shape[3] = {m.E, m.rows, K};
    void *p = NULL;
    PyObject *out = make(args[3], m.n, shape + 3 - m.n, dtype, &p);
    if (out == NULL) return NULL;
    fp8bq_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_dequantize(m.o.codes, m.o.scales, m.E, m.rows, K, (fp8bq_fp4_format)v[0],
                      m.o.tensor_scale, 0, p, dtype == g_bf16 ? FP8BQ_BF16 : FP8BQ_F32, K,
                      m.rows * K, (cudaStream_t)(uintptr_t)v[2]);
    Py_END_ALLOW_THREADS
    if (st == FP8BQ_OK) return out;
    Py_DECREF(out);
    return PyLong_FromLong(st);
}

/* setup(Tensor, uint8, bfloat16, float32, matmul, gated_matmul, quantize_batched, dequantize):
 * PyTorch's types, and the addresses of the loaded library's entry points. */
static PyObject *calls_setup(PyObject *self, PyObject *const *args, Py_ssize_t n) {
    int64_t f[4];
    (void)self;
    if (n != 8 || !PyType_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "setup(Tensor, uint8, bfloat16, float32, 4 addresses)");
        return NULL;
    }
    if (!ints(args + 4, 4, f)) return NULL;
    for (int i = 0; i < 4; ++i) Py_INCREF(args[i]);
    g_tensor = (PyTypeObject *)args[0];
    g_uint8 = args[1];
    g_bf16 = args[2];
    g_f32 = args[3];
    g_product[0] = (product_fn)(uintptr_t)f[0];
    g_product[1] = (product_fn)(uintptr_t)f[1];
    g_quantize = (quantize_fn)(uintptr_t)f[2];
    g_dequantize = (dequantize_fn)(uintptr_t)f[3];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))calls_setup, METH_FASTCALL, NULL},
    {"product", (PyCFunction)(void (*)(void))calls_product, METH_FASTCALL, NULL},
    {"quantize", (PyCFunction)(void (*)(void))calls_quantize, METH_FASTCALL, NULL},
    {"dequantize", (PyCFunction)(void (*)(void))calls_dequantize, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_new_empty = PyUnicode_InternFromString("new_empty");
    PyObject *dtype = PyUnicode_InternFromString("dtype");
    g_kw_dtype = dtype ? PyTuple_Pack(1, dtype) : NULL;
    if (!s_shape || !s_dtype || !s_data_ptr || !s_get_device || !s_is_contiguous || !s_new_empty ||
        !g_kw_dtype)
        return NULL;
    return PyModule_Create(&module);
}
