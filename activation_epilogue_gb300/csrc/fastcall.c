/*
 * The binding's argument marshalling in C for the calls a model makes for every token (the RMS
 * norm, the 4-bit products, dropout): tensors to addresses, then the C ABI call.  The same
 * checks as the ctypes path of gemm_epi.py, which it stands in for where Python's headers were
 * there at build time: a six-tensor call costs 5.7 us of host time through ctypes, of which
 * 1.5 are the launch.
 *
 * The functions of the library are bound by address (bind), so that the library is the one the
 * rest of the binding has loaded.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "gemm_epi.h"

static __typeof__(&gemm_epi_rmsnorm) p_rmsnorm;
static __typeof__(&gemm_epi_rmsnorm_e4m3) p_rmsnorm_e4m3;
static __typeof__(&gemm_epi_rmsnorm_backward) p_rmsnorm_backward;
static __typeof__(&gemm_epi_w4_matmul) p_w4_matmul;
static __typeof__(&gemm_epi_w4_dequantize) p_w4_dequantize;
static __typeof__(&gemm_epi_dropout) p_dropout;

static PyObject *s_is_cuda, *s_is_contiguous, *s_data_ptr;

/* The arguments of one call, converted in order; the first that cannot be sets `bad`. */
typedef struct {
    PyObject* const* args;
    int bad;
} Args;

static void* pointer(Args* a, int i)
{
    PyObject* o = a->args[i];
    if (a->bad || o == Py_None) return NULL;
    PyObject* v;
    if (PyLong_Check(o)) {
        v = Py_NewRef(o);
    } else {
        v = PyObject_GetAttr(o, s_is_cuda);
        if (v && v != Py_True) PyErr_SetString(PyExc_ValueError, "tensors must be CUDA tensors");
        if (!v || v != Py_True) goto fail;
        Py_DECREF(v);
        v = PyObject_CallMethodNoArgs(o, s_is_contiguous);
        if (v && v != Py_True)
            PyErr_SetString(PyExc_ValueError, "tensors must be contiguous (row-major)");
        if (!v || v != Py_True) goto fail;
        Py_DECREF(v);
        v = PyObject_CallMethodNoArgs(o, s_data_ptr);
        if (!v) goto fail;
    }
    void* p = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(v);
    Py_DECREF(v);
    if (PyErr_Occurred()) a->bad = 1;
    return p;
fail:
    Py_XDECREF(v);
    a->bad = 1;
    return NULL;
}

static int64_t integer(Args* a, int i)
{
    if (a->bad) return 0;
    const int64_t v = PyLong_AsLongLong(a->args[i]);
    if (v == -1 && PyErr_Occurred()) a->bad = 1;
    return v;
}

/* mod 2^64 */
static uint64_t word(Args* a, int i)
{
    if (a->bad) return 0;
    const uint64_t v = PyLong_AsUnsignedLongLongMask(a->args[i]);
    if (v == (uint64_t)-1 && PyErr_Occurred()) a->bad = 1;
    return v;
}

static float real(Args* a, int i)
{
    if (a->bad) return 0.0f;
    const double v = PyFloat_AsDouble(a->args[i]);
    if (v == -1.0 && PyErr_Occurred()) a->bad = 1;
    return (float)v;
}

static int expect(Py_ssize_t n, Py_ssize_t want, const void* bound)
{
    if (n == want && bound) return 1;
    PyErr_SetString(PyExc_TypeError, bound ? "wrong number of arguments" : "call bind first");
    return 0;
}

#define CALL(expression)                      \
    do {                                      \
        gemm_epi_status st;                   \
        if (a.bad) return NULL;               \
        Py_BEGIN_ALLOW_THREADS                \
        st = (expression);                    \
        Py_END_ALLOW_THREADS                  \
        return PyLong_FromLong((long)st);     \
    } while (0)

static PyObject* rmsnorm(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 11, (const void*)p_rmsnorm)) return NULL;
    Args a = {args, 0};
    const int64_t t = integer(&a, 0), d = integer(&a, 1), dtype = integer(&a, 2);
    void *X = pointer(&a, 3), *R = pointer(&a, 4), *g = pointer(&a, 5);
    const float eps = real(&a, 6);
    void *H = pointer(&a, 7), *Y = pointer(&a, 8), *rstd = pointer(&a, 9), *stream = pointer(&a, 10);
    CALL(p_rmsnorm(t, d, (gemm_epi_dtype)dtype, X, R, g, eps, H, Y, (float*)rstd, (cudaStream_t)stream));
}

static PyObject* rmsnorm_e4m3(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 14, (const void*)p_rmsnorm_e4m3)) return NULL;
    Args a = {args, 0};
    const int64_t t = integer(&a, 0), d = integer(&a, 1), dtype = integer(&a, 2);
    void *X = pointer(&a, 3), *R = pointer(&a, 4), *g = pointer(&a, 5);
    const float eps = real(&a, 6);
    void *H = pointer(&a, 7), *Q = pointer(&a, 8);
    const int64_t mode = integer(&a, 9);
    void *scale = pointer(&a, 10), *rstd = pointer(&a, 11), *ws = pointer(&a, 12), *stream = pointer(&a, 13);
    CALL(p_rmsnorm_e4m3(t, d, (gemm_epi_dtype)dtype, X, R, g, eps, H, Q, (gemm_epi_scale_mode)mode,
                        (float*)scale, (float*)rstd, ws, (cudaStream_t)stream));
}

static PyObject* rmsnorm_backward(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 12, (const void*)p_rmsnorm_backward)) return NULL;
    Args a = {args, 0};
    const int64_t t = integer(&a, 0), d = integer(&a, 1), dtype = integer(&a, 2);
    void *dY = pointer(&a, 3), *H = pointer(&a, 4), *g = pointer(&a, 5), *rstd = pointer(&a, 6);
    void *dH = pointer(&a, 7), *dX = pointer(&a, 8), *dg = pointer(&a, 9), *ws = pointer(&a, 10);
    void* stream = pointer(&a, 11);
    CALL(p_rmsnorm_backward(t, d, (gemm_epi_dtype)dtype, dY, H, g, (const float*)rstd, dH, dX, (float*)dg,
                            ws, (cudaStream_t)stream));
}

static PyObject* w4_matmul(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 14, (const void*)p_w4_matmul)) return NULL;
    Args a = {args, 0};
    const int64_t m = integer(&a, 0), cols = integer(&a, 1), k = integer(&a, 2), group = integer(&a, 3);
    const int64_t dtype = integer(&a, 4), epilog = integer(&a, 5);
    void *A = pointer(&a, 6), *W = pointer(&a, 7), *s = pointer(&a, 8), *z = pointer(&a, 9);
    void *bias = pointer(&a, 10), *R = pointer(&a, 11), *D = pointer(&a, 12), *stream = pointer(&a, 13);
    CALL(p_w4_matmul(m, cols, k, group, (gemm_epi_dtype)dtype, (gemm_epi_epilog)epilog, A, W, s,
                     (const uint8_t*)z, bias, R, D, (cudaStream_t)stream));
}

static PyObject* w4_dequantize(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 9, (const void*)p_w4_dequantize)) return NULL;
    Args a = {args, 0};
    const int64_t cols = integer(&a, 0), k = integer(&a, 1), group = integer(&a, 2), dtype = integer(&a, 3);
    void *W = pointer(&a, 4), *s = pointer(&a, 5), *z = pointer(&a, 6), *B = pointer(&a, 7);
    void* stream = pointer(&a, 8);
    CALL(p_w4_dequantize(cols, k, group, (gemm_epi_dtype)dtype, W, s, (const uint8_t*)z, B,
                         (cudaStream_t)stream));
}

static PyObject* dropout(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 10, (const void*)p_dropout)) return NULL;
    Args a = {args, 0};
    const int64_t count = integer(&a, 0), dtype = integer(&a, 1);
    void *X = pointer(&a, 2), *R = pointer(&a, 3);
    const float p = real(&a, 4);
    const uint64_t seed = word(&a, 5), offset = word(&a, 6);
    void *od = pointer(&a, 7), *Y = pointer(&a, 8), *stream = pointer(&a, 9);
    CALL(p_dropout(count, (gemm_epi_dtype)dtype, X, R, p, seed, offset, (const uint64_t*)od, Y,
                   (cudaStream_t)stream));
}

/* bind(rmsnorm, rmsnorm_e4m3, rmsnorm_backward, w4_matmul, w4_dequantize, dropout): addresses */
static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t n)
{
    (void)self;
    if (!expect(n, 6, (const void*)args)) return NULL;
    Args a = {args, 0};
    void* p[6];
    for (int i = 0; i < 6; ++i) p[i] = (void*)(uintptr_t)word(&a, i);
    if (a.bad) return NULL;
    p_rmsnorm = (__typeof__(p_rmsnorm))p[0];
    p_rmsnorm_e4m3 = (__typeof__(p_rmsnorm_e4m3))p[1];
    p_rmsnorm_backward = (__typeof__(p_rmsnorm_backward))p[2];
    p_w4_matmul = (__typeof__(p_w4_matmul))p[3];
    p_w4_dequantize = (__typeof__(p_w4_dequantize))p[4];
    p_dropout = (__typeof__(p_dropout))p[5];
    Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(rmsnorm),   METHOD(rmsnorm_e4m3),  METHOD(rmsnorm_backward),
                                METHOD(w4_matmul), METHOD(w4_dequantize), METHOD(dropout),
                                METHOD(bind),      {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void)
{
    s_is_cuda = PyUnicode_InternFromString("is_cuda");
    s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    if (!s_is_cuda || !s_is_contiguous || !s_data_ptr) return NULL;
    return PyModule_Create(&module);
}
