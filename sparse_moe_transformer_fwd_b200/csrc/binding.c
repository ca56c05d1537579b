/* The calls for a few tokens from Python: arguments checked and handed to the
 * library's functions without ctypes.  Such a call is made for a few
 * microseconds of GPU work; checked in Python and made through ctypes a linear
 * call costs 9.9 us on the host, here 6.6 (5 on a faster host).
 *
 * Each function takes the binding's arguments, returns the library's status, or
 * None where an argument is not what the call needs (or the tensors are on
 * another device than the current one): the caller in _native.py then takes its
 * own path, which says what is wrong.  Nothing is kept from one call to the
 * next but what setup() was given. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/moe_fwd.h"

static PyTypeObject *tensor_type;
static PyObject *dt_bf16, *dt_f32, *dt_i32, *dt_u8, *dt_e4m3; /* torch dtypes */
static PyObject *current_device, *current_stream;             /* of torch: (), (device) */
static PyObject *n_dtype, *n_get_device, *n_is_contiguous, *n_numel, *n_data_ptr, *n_cuda_stream;

typedef int (*gemm_fn)(const moe_linear_shape *, const uint8_t *, const float *, const void *, const float *,
                       const uint16_t *, void *, void *, size_t, void *);
typedef int (*linear_fn)(const moe_linear_shape *, const uint16_t *, const void *, const float *, const uint16_t *,
                         void *, void *, size_t, void *);
typedef int (*linear_prenorm_fn)(const moe_linear_shape *, const uint16_t *, const uint16_t *, float, const void *,
                                 const float *, void *, void *, size_t, void *);
typedef int (*few_fn)(const moe_shape *, const uint16_t *, const uint16_t *, const float *, const void *,
                      const float *, const void *, const float *, uint16_t *, int32_t *, void *, size_t, void *);
typedef int (*few_prenorm_fn)(const moe_shape *, const uint16_t *, const uint16_t *, float, const uint16_t *,
                              const float *, const void *, const float *, const void *, const float *, uint16_t *,
                              int32_t *, void *, size_t, void *);
static gemm_fn f_gemm;
static linear_fn f_linear;
static linear_prenorm_fn f_linear_prenorm;
static few_fn f_few;
static few_prenorm_fn f_few_prenorm;

enum { BF16, F32, I32, U8, CODES };

/* obj.name() as a number */
static int number(PyObject *obj, PyObject *name, unsigned long long *out) {
    PyObject *r = PyObject_CallMethodNoArgs(obj, name);
    if (!r) return 0;
    *out = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    return !PyErr_Occurred();
}

/* Address of a contiguous tensor of the wanted type on device `dev` with at
 * least `need` elements; NULL of None.  *have: its elements. */
static int address(PyObject *t, int kind, unsigned __int128 need, unsigned long long dev, void **out,
                   unsigned long long *have) {
    unsigned long long n, at;
    *out = NULL;
    if (t == Py_None) return 1;
    if (!PyObject_TypeCheck(t, tensor_type)) return 0;
    PyObject *d = PyObject_GetAttr(t, n_dtype);
    if (!d) return 0;
    Py_DECREF(d); /* (torch keeps its dtypes) */
    const int ok = kind == BF16 ? d == dt_bf16 : kind == F32 ? d == dt_f32 : kind == I32 ? d == dt_i32
                 : kind == U8   ? d == dt_u8 : d == dt_u8 || d == dt_e4m3;
    if (!ok || !number(t, n_get_device, &n) || n != dev) return 0;
    PyObject *c = PyObject_CallMethodNoArgs(t, n_is_contiguous);
    if (!c) return 0;
    Py_DECREF(c);
    if (c != Py_True || !number(t, n_numel, &n) || n < need || !number(t, n_data_ptr, &at)) return 0;
    *out = (void *)(uintptr_t)at;
    if (have) *have = n;
    return 1;
}

/* The device of x, if it is the current one, and the stream to use on it. */
static int where(PyObject *x, PyObject *stream, unsigned long long *dev, void **st) {
    unsigned long long now, s;
    if (!PyObject_TypeCheck(x, tensor_type) || !number(x, n_get_device, dev)) return 0;
    PyObject *r = PyObject_CallNoArgs(current_device);
    if (!r) return 0;
    now = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    if (PyErr_Occurred() || now != *dev) return 0;
    if (stream == Py_None) {
        PyObject *d = PyLong_FromUnsignedLongLong(*dev);
        if (!d) return 0;
        r = PyObject_CallOneArg(current_stream, d);
        Py_DECREF(d);
    } else {
        r = PyObject_GetAttr(stream, n_cuda_stream);
    }
    if (!r) return 0;
    s = PyLong_AsUnsignedLongLong(r);
    Py_DECREF(r);
    *st = (void *)(uintptr_t)s;
    return !PyErr_Occurred();
}

/* The C struct behind a ctypes one. */
static int shape_of(PyObject *obj, void *out, Py_ssize_t size) {
    Py_buffer b;
    if (PyObject_GetBuffer(obj, &b, PyBUF_SIMPLE) != 0) return 0;
    const int ok = b.len == size;
    if (ok) memcpy(out, b.buf, size);
    PyBuffer_Release(&b);
    return ok;
}

static PyObject *declined(void) {
    PyErr_Clear();
    Py_RETURN_NONE;
}

/* linear(kind, shape, x, second, eps, w, w_scales, residual, out, ws, stream);
 * kind 0: codes and their scales, 1: x, 2: h, gamma and eps */
static PyObject *linear(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    moe_linear_shape s;
    if (n != 11) return declined();
    const long kind = PyLong_AsLong(a[0]);
    const double eps = PyFloat_AsDouble(a[4]);
    unsigned long long dev, bytes = 0;
    void *x, *second, *w, *ws_, *res, *out, *ws, *st;
    if (PyErr_Occurred() || !shape_of(a[1], &s, sizeof s) || s.T < 0 || s.K < 0 || s.N < 0 || a[9] == Py_None ||
        !where(a[2], a[10], &dev, &st))
        return declined();
    typedef unsigned __int128 u;
    const u T = s.T, K = s.K, N = s.N, KB = s.K / 128;
    if (!address(a[2], kind ? BF16 : CODES, T * K, dev, &x, NULL) ||
        !address(a[3], kind ? BF16 : F32, kind == 0 ? T * KB : kind == 2 ? K : 0, dev, &second, NULL) ||
        !address(a[5], CODES, N * K, dev, &w, NULL) || !address(a[6], F32, (N + 127) / 128 * KB, dev, &ws_, NULL) ||
        !address(a[7], BF16, T * N, dev, &res, NULL) || !address(a[8], s.out_f32 ? F32 : BF16, T * N, dev, &out, NULL) ||
        !address(a[9], U8, 0, dev, &ws, &bytes))
        return declined();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if (kind == 0) rc = f_gemm(&s, x, second, w, ws_, res, out, ws, bytes, st);
    else if (kind == 1) rc = f_linear(&s, x, w, ws_, res, out, ws, bytes, st);
    else rc = f_linear_prenorm(&s, x, second, (float)eps, w, ws_, out, ws, bytes, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

/* few(prenorm, shape, x, gamma, eps, w_router, bias, w13, w13_scales, w2,
 * w2_scales, out, ws, topk_idx_out, stream) */
static PyObject *few(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    (void)self;
    moe_shape s;
    if (n != 15) return declined();
    const int prenorm = PyObject_IsTrue(a[0]);
    const double eps = PyFloat_AsDouble(a[4]);
    unsigned long long dev, bytes = 0;
    void *x, *gamma, *wr, *bias, *w13, *s13, *w2, *s2, *out, *ws, *idx, *st;
    if (PyErr_Occurred() || !shape_of(a[1], &s, sizeof s) || s.T < 0 || s.d_model < 0 || s.n_experts < 0 ||
        s.n_shared < 0 || s.d_expert < 0 || s.top_k < 0 || a[12] == Py_None || !where(a[2], a[14], &dev, &st))
        return declined();
    typedef unsigned __int128 u;
    const int fp8 = s.precision == MOE_FP8_BLOCK || s.precision == MOE_FP8_UE8M0;
    const u T = s.T, d = s.d_model, E = s.n_experts, slots = E + s.n_shared, n2 = slots * d * s.d_expert, n13 = 2 * n2;
    if (!address(a[2], BF16, T * d, dev, &x, NULL) || !address(a[3], BF16, d, dev, &gamma, NULL) ||
        !address(a[5], BF16, E * d, dev, &wr, NULL) || !address(a[6], F32, E, dev, &bias, NULL) ||
        !address(a[7], fp8 ? CODES : BF16, n13, dev, &w13, NULL) ||
        !address(a[8], F32, fp8 ? n13 / 16384 : 0, dev, &s13, NULL) ||
        !address(a[9], fp8 ? CODES : BF16, n2, dev, &w2, NULL) ||
        !address(a[10], F32, fp8 ? n2 / 16384 : 0, dev, &s2, NULL) || !address(a[11], BF16, T * d, dev, &out, NULL) ||
        !address(a[12], U8, 0, dev, &ws, &bytes) || !address(a[13], I32, T * s.top_k, dev, &idx, NULL))
        return declined();
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    if (prenorm) rc = f_few_prenorm(&s, x, gamma, (float)eps, wr, bias, w13, s13, w2, s2, out, idx, ws, bytes, st);
    else rc = f_few(&s, x, wr, bias, w13, s13, w2, s2, out, idx, ws, bytes, st);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

/* setup(Tensor, (bfloat16, float32, int32, uint8, float8_e4m3fn), device, stream,
 * (addresses of fp8_block_gemm, moe_linear, moe_linear_prenorm, moe_forward_few,
 * moe_forward_few_prenorm)) */
static PyObject *setup(PyObject *self, PyObject *args) {
    (void)self;
    PyObject *type, *dt[5];
    unsigned long long f[5];
    if (!PyArg_ParseTuple(args, "O(OOOOO)OO(KKKKK)", &type, &dt[0], &dt[1], &dt[2], &dt[3], &dt[4], &current_device,
                          &current_stream, &f[0], &f[1], &f[2], &f[3], &f[4]))
        return NULL;
    Py_INCREF(type), Py_INCREF(current_device), Py_INCREF(current_stream);
    for (int i = 0; i < 5; ++i) Py_INCREF(dt[i]);
    tensor_type = (PyTypeObject *)type;
    dt_bf16 = dt[0], dt_f32 = dt[1], dt_i32 = dt[2], dt_u8 = dt[3], dt_e4m3 = dt[4];
    f_gemm = (gemm_fn)(uintptr_t)f[0];
    f_linear = (linear_fn)(uintptr_t)f[1];
    f_linear_prenorm = (linear_prenorm_fn)(uintptr_t)f[2];
    f_few = (few_fn)(uintptr_t)f[3];
    f_few_prenorm = (few_prenorm_fn)(uintptr_t)f[4];
    Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, NULL},
                                {"linear", (PyCFunction)(void (*)(void))linear, METH_FASTCALL, NULL},
                                {"few", (PyCFunction)(void (*)(void))few, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
    n_dtype = PyUnicode_InternFromString("dtype");
    n_get_device = PyUnicode_InternFromString("get_device");
    n_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    n_numel = PyUnicode_InternFromString("numel");
    n_data_ptr = PyUnicode_InternFromString("data_ptr");
    n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
    if (PyErr_Occurred()) return NULL;
    return PyModule_Create(&module);
}
