// The binding's argument marshalling in C++ for the calls a model makes for every token (the RMS
// norm, the 4-bit products, dropout): torch tensors to addresses, then the C ABI call.  It does
// what the ctypes path of gemm_epi.py does, with the same checks, and stands in for it where the
// headers of Python and torch were there at build time.  Host time of a six-tensor call (GB300's
// Grace): 5.7 us through ctypes, 4.1 with the tensors' Python methods called from C, 3.0 so; the
// launch is 1.5 of it.
//
// The functions of the library are bound by address (bind), so that the library is the one the
// rest of the binding has loaded.
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>

#include "gemm_epi.h"

namespace {

decltype(&gemm_epi_rmsnorm) p_rmsnorm;
decltype(&gemm_epi_rmsnorm_e4m3) p_rmsnorm_e4m3;
decltype(&gemm_epi_rmsnorm_backward) p_rmsnorm_backward;
decltype(&gemm_epi_w4_matmul) p_w4_matmul;
decltype(&gemm_epi_w4_dequantize) p_w4_dequantize;
decltype(&gemm_epi_dropout) p_dropout;

// The arguments of one call, converted in order; the first that cannot be sets `bad` and the
// Python error.
struct Args {
    PyObject* const* args;
    bool bad = false;
    int device = -1;  // the current device, asked for once a call

    void* fail(PyObject* type, const char* what)
    {
        PyErr_SetString(type, what);
        bad = true;
        return nullptr;
    }

    // The first element of a tensor on the current device, a raw address, or None.
    void* pointer(int i)
    {
        PyObject* o = args[i];
        if (bad || o == Py_None) return nullptr;
        if (THPVariable_Check(o)) {
            const at::Tensor& t = THPVariable_Unpack(o);
            if (!t.is_cuda()) return fail(PyExc_ValueError, "tensors must be CUDA tensors");
            if (device < 0) device = c10::cuda::current_device();
            if (t.get_device() != device)
                return fail(PyExc_ValueError, "tensors must be on the current CUDA device");
            if (!t.is_contiguous()) return fail(PyExc_ValueError, "tensors must be contiguous (row-major)");
            return t.data_ptr();
        }
        if (!PyLong_Check(o)) return fail(PyExc_TypeError, "expected a tensor, an address or None");
        return reinterpret_cast<void*>(static_cast<uintptr_t>(word(i)));
    }

    // A stream's handle; None: the current torch stream of the current device.
    cudaStream_t stream(int i)
    {
        if (!bad && args[i] == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
        return reinterpret_cast<cudaStream_t>(pointer(i));
    }

    int64_t integer(int i)
    {
        if (bad) return 0;
        const int64_t v = PyLong_AsLongLong(args[i]);
        if (v == -1 && PyErr_Occurred()) bad = true;
        return v;
    }

    uint64_t word(int i)  // mod 2^64
    {
        if (bad) return 0;
        const uint64_t v = PyLong_AsUnsignedLongLongMask(args[i]);
        if (v == static_cast<uint64_t>(-1) && PyErr_Occurred()) bad = true;
        return v;
    }

    float real(int i)
    {
        if (bad) return 0.0f;
        const double v = PyFloat_AsDouble(args[i]);
        if (v == -1.0 && PyErr_Occurred()) bad = true;
        return static_cast<float>(v);
    }
};

// One call: `convert` takes the arguments, then calls the library without the interpreter's lock.
// No C++ exception leaves it.
template <typename Convert>
PyObject* call(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, bool bound, Convert convert)
{
    if (!bound || n != want) {
        PyErr_SetString(PyExc_TypeError, bound ? "wrong number of arguments" : "call bind first");
        return nullptr;
    }
    try {
        Args a{args};
        const long status = convert(a);
        return a.bad ? nullptr : PyLong_FromLong(status);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <typename Function, typename... Parameters>
long unlocked(const Args& a, Function function, Parameters... parameters)
{
    if (a.bad) return -1;
    PyThreadState* state = PyEval_SaveThread();
    const long status = static_cast<long>(function(parameters...));
    PyEval_RestoreThread(state);
    return status;
}

gemm_epi_dtype dtype_of(int64_t v) { return static_cast<gemm_epi_dtype>(v); }

PyObject* rmsnorm(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 11, p_rmsnorm != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2);
        void *X = a.pointer(3), *R = a.pointer(4), *gamma = a.pointer(5);
        const float eps = a.real(6);
        void *H = a.pointer(7), *Y = a.pointer(8), *rstd = a.pointer(9);
        const cudaStream_t stream = a.stream(10);
        return unlocked(a, p_rmsnorm, t, d, dtype_of(dtype), X, R, gamma, eps, H, Y,
                        static_cast<float*>(rstd), stream);
    });
}

PyObject* rmsnorm_e4m3(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 14, p_rmsnorm_e4m3 != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2);
        void *X = a.pointer(3), *R = a.pointer(4), *gamma = a.pointer(5);
        const float eps = a.real(6);
        void *H = a.pointer(7), *Q = a.pointer(8);
        const int64_t mode = a.integer(9);
        void *scale = a.pointer(10), *rstd = a.pointer(11), *workspace = a.pointer(12);
        const cudaStream_t stream = a.stream(13);
        return unlocked(a, p_rmsnorm_e4m3, t, d, dtype_of(dtype), X, R, gamma, eps, H, Q,
                        static_cast<gemm_epi_scale_mode>(mode), static_cast<float*>(scale),
                        static_cast<float*>(rstd), workspace, stream);
    });
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 12, p_rmsnorm_backward != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2);
        void *dY = a.pointer(3), *H = a.pointer(4), *gamma = a.pointer(5), *rstd = a.pointer(6);
        void *dH = a.pointer(7), *dX = a.pointer(8), *dgamma = a.pointer(9), *workspace = a.pointer(10);
        const cudaStream_t stream = a.stream(11);
        return unlocked(a, p_rmsnorm_backward, t, d, dtype_of(dtype), dY, H, gamma,
                        static_cast<const float*>(rstd), dH, dX, static_cast<float*>(dgamma), workspace, stream);
    });
}

PyObject* w4_matmul(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 14, p_w4_matmul != nullptr, [](Args& a) {
        const int64_t m = a.integer(0), cols = a.integer(1), k = a.integer(2), group = a.integer(3);
        const int64_t dtype = a.integer(4), epilog = a.integer(5);
        void *A = a.pointer(6), *W = a.pointer(7), *scales = a.pointer(8), *zeros = a.pointer(9);
        void *bias = a.pointer(10), *residual = a.pointer(11), *D = a.pointer(12);
        const cudaStream_t stream = a.stream(13);
        return unlocked(a, p_w4_matmul, m, cols, k, group, dtype_of(dtype),
                        static_cast<gemm_epi_epilog>(epilog), A, W, scales,
                        static_cast<const uint8_t*>(zeros), bias, residual, D, stream);
    });
}

PyObject* w4_dequantize(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 9, p_w4_dequantize != nullptr, [](Args& a) {
        const int64_t cols = a.integer(0), k = a.integer(1), group = a.integer(2), dtype = a.integer(3);
        void *W = a.pointer(4), *scales = a.pointer(5), *zeros = a.pointer(6), *B = a.pointer(7);
        const cudaStream_t stream = a.stream(8);
        return unlocked(a, p_w4_dequantize, cols, k, group, dtype_of(dtype), W, scales,
                        static_cast<const uint8_t*>(zeros), B, stream);
    });
}

PyObject* dropout(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 10, p_dropout != nullptr, [](Args& a) {
        const int64_t count = a.integer(0), dtype = a.integer(1);
        void *X = a.pointer(2), *residual = a.pointer(3);
        const float p = a.real(4);
        const uint64_t seed = a.word(5), offset = a.word(6);
        void *offset_device = a.pointer(7), *Y = a.pointer(8);
        const cudaStream_t stream = a.stream(9);
        return unlocked(a, p_dropout, count, dtype_of(dtype), X, residual, p, seed, offset,
                        static_cast<const uint64_t*>(offset_device), Y, stream);
    });
}

// bind(rmsnorm, rmsnorm_e4m3, rmsnorm_backward, w4_matmul, w4_dequantize, dropout): addresses
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 6, true, [](Args& a) {
        void* p[6];
        for (int i = 0; i < 6; ++i) p[i] = a.pointer(i);
        if (a.bad) return 0L;
        p_rmsnorm = reinterpret_cast<decltype(p_rmsnorm)>(p[0]);
        p_rmsnorm_e4m3 = reinterpret_cast<decltype(p_rmsnorm_e4m3)>(p[1]);
        p_rmsnorm_backward = reinterpret_cast<decltype(p_rmsnorm_backward)>(p[2]);
        p_w4_matmul = reinterpret_cast<decltype(p_w4_matmul)>(p[3]);
        p_w4_dequantize = reinterpret_cast<decltype(p_w4_dequantize)>(p[4]);
        p_dropout = reinterpret_cast<decltype(p_dropout)>(p[5]);
        return 0L;
    });
}

using Method = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

PyMethodDef method(const char* name, Method function)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(function)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method("rmsnorm", rmsnorm),
                         method("rmsnorm_e4m3", rmsnorm_e4m3),
                         method("rmsnorm_backward", rmsnorm_backward),
                         method("w4_matmul", w4_matmul),
                         method("w4_dequantize", w4_dequantize),
                         method("dropout", dropout),
                         method("bind", bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__fastcall(void)
{
    return PyModule_Create(&module);
}
