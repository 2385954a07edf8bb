// The binding's argument marshalling in C++ for the calls a model makes for every token (the
// norms, the 4-bit and block-scaled E4M3 products, dropout): torch tensors to addresses, then the C ABI
// call.  It does
// what the ctypes path of gemm_epi.py does, with the same checks (device, layout, and type and size
// against the call's shape), and stands in for it where the headers of Python and torch were there
// at build time.  Host time of a six-tensor call (GB300's
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
decltype(&gemm_epi_rmsnorm_workspace) p_rmsnorm_workspace;
decltype(&gemm_epi_layernorm_forward) p_layernorm_forward;
decltype(&gemm_epi_layernorm_e4m3) p_layernorm_e4m3;
decltype(&gemm_epi_layernorm_backward) p_layernorm_backward;
decltype(&gemm_epi_layernorm_workspace) p_layernorm_workspace;
decltype(&gemm_epi_e4m3_quantize) p_e4m3_quantize;
decltype(&gemm_epi_execute_operands) p_execute_operands;

// What a buffer holds: the call's 16-bit type (by its number in the ABI), fp32, E4M3 codes, 64-bit
// counters, bytes of packed whole numbers, or bytes of any tensor.
enum class Kind { kF16 = 0, kBf16 = 1, kF32, kE4m3, kInt64, kPacked, kBytes };

Kind kind16(int64_t dtype) { return dtype == 0 ? Kind::kF16 : dtype == 1 ? Kind::kBf16 : Kind::kBytes; }

int64_t bytes_per(Kind kind)
{
    switch (kind) {
    case Kind::kF16:
    case Kind::kBf16: return 2;
    case Kind::kF32: return 4;
    case Kind::kInt64: return 8;
    default: return 1;
    }
}

at::ScalarType type_of(Kind kind)
{
    switch (kind) {
    case Kind::kF16: return at::kHalf;
    case Kind::kBf16: return at::kBFloat16;
    case Kind::kF32: return at::kFloat;
    case Kind::kE4m3: return at::kFloat8_e4m3fn;
    case Kind::kInt64: return at::kLong;
    default: return at::kByte;
    }
}

// A tensor of whole numbers stands for the bits it holds; floating-point types have to be the kind's.
bool stands_for(const at::Tensor& t, Kind kind)
{
    if (kind == Kind::kBytes) return true;
    return c10::isIntegralType(t.scalar_type(), true) &&
           (kind == Kind::kPacked || static_cast<int64_t>(t.element_size()) == bytes_per(kind));
}

// a * b, 0 where either is negative (such a shape is the library's to refuse), at most 2^62.
int64_t times(int64_t a, int64_t b)
{
    if (a <= 0 || b <= 0) return 0;
    return a > (1ll << 62) / b ? 1ll << 62 : a * b;
}

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

    // The first element of a tensor on the current device that has `count` elements of `kind` at
    // least, a raw address, or None.
    void* pointer(int i, Kind kind = Kind::kBytes, int64_t count = 0)
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
            if (count > 0 && (t.scalar_type() != type_of(kind) || t.numel() < count)) {
                if (t.scalar_type() != type_of(kind) && !stands_for(t, kind))
                    return fail(PyExc_ValueError, "a tensor's type is not the one the call reads or writes there");
                if (static_cast<int64_t>(t.nbytes()) / bytes_per(kind) < count)
                    return fail(PyExc_ValueError, "a tensor has fewer elements than the call's shape");
            }
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
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d);
        const Kind k16 = kind16(dtype);
        void *X = a.pointer(3, k16, td), *R = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, t > 0 ? d : 0);
        const float eps = a.real(6);
        void *H = a.pointer(7, k16, td), *Y = a.pointer(8, k16, td), *rstd = a.pointer(9, Kind::kF32, t);
        const cudaStream_t stream = a.stream(10);
        return unlocked(a, p_rmsnorm, t, d, dtype_of(dtype), X, R, gamma, eps, H, Y,
                        static_cast<float*>(rstd), stream);
    });
}

PyObject* rmsnorm_e4m3(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 14, p_rmsnorm_e4m3 != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d);
        const Kind k16 = kind16(dtype);
        void *X = a.pointer(3, k16, td), *R = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, t > 0 ? d : 0);
        const float eps = a.real(6);
        void *H = a.pointer(7, k16, td), *Q = a.pointer(8, Kind::kE4m3, td);
        const int64_t mode = a.integer(9);
        void* scale = a.pointer(10, Kind::kF32, mode == GEMM_EPI_SCALE_ROW ? t : t > 0);
        void* rstd = a.pointer(11, Kind::kF32, t);
        void* workspace = a.pointer(12, Kind::kBytes, mode == GEMM_EPI_SCALE_TENSOR && t > 0 && !a.bad ? p_rmsnorm_workspace(t, d) : 0);
        const cudaStream_t stream = a.stream(13);
        return unlocked(a, p_rmsnorm_e4m3, t, d, dtype_of(dtype), X, R, gamma, eps, H, Q,
                        static_cast<gemm_epi_scale_mode>(mode), static_cast<float*>(scale),
                        static_cast<float*>(rstd), workspace, stream);
    });
}

PyObject* rmsnorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 12, p_rmsnorm_backward != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d);
        const Kind k16 = kind16(dtype);
        void *dY = a.pointer(3, k16, td), *H = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, t > 0 ? d : 0);
        void *rstd = a.pointer(6, Kind::kF32, t), *dH = a.pointer(7, k16, td), *dX = a.pointer(8, k16, td);
        void* dgamma = a.pointer(9, Kind::kF32, d);
        void* workspace = a.pointer(10, Kind::kBytes, t > 0 && !a.bad ? p_rmsnorm_workspace(t, d) : 0);
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
        const Kind k16 = kind16(dtype);
        const bool any = m > 0;
        const int64_t mn = times(m, cols), scaled = any && group > 0 ? times(k / group, cols) : 0;
        void *A = a.pointer(6, k16, times(m, k)), *W = a.pointer(7, Kind::kPacked, any ? times(k / 2, cols) : 0);
        void *scales = a.pointer(8, k16, scaled), *zeros = a.pointer(9, Kind::kPacked, scaled);
        void *bias = a.pointer(10, k16, any ? cols : 0), *residual = a.pointer(11, k16, mn), *D = a.pointer(12, k16, mn);
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
        const Kind k16 = kind16(dtype);
        const int64_t scaled = group > 0 ? times(k / group, cols) : 0;
        void *W = a.pointer(4, Kind::kPacked, times(k / 2, cols)), *scales = a.pointer(5, k16, scaled);
        void *zeros = a.pointer(6, Kind::kPacked, scaled), *B = a.pointer(7, k16, times(k, cols));
        const cudaStream_t stream = a.stream(8);
        return unlocked(a, p_w4_dequantize, cols, k, group, dtype_of(dtype), W, scales,
                        static_cast<const uint8_t*>(zeros), B, stream);
    });
}

PyObject* dropout(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 10, p_dropout != nullptr, [](Args& a) {
        const int64_t count = a.integer(0), dtype = a.integer(1);
        const Kind k16 = kind16(dtype);
        void *X = a.pointer(2, k16, count), *residual = a.pointer(3, k16, count);
        const float p = a.real(4);
        const uint64_t seed = a.word(5), offset = a.word(6);
        void *offset_device = a.pointer(7, Kind::kInt64, count > 0), *Y = a.pointer(8, k16, count);
        const cudaStream_t stream = a.stream(9);
        return unlocked(a, p_dropout, count, dtype_of(dtype), X, residual, p, seed, offset,
                        static_cast<const uint64_t*>(offset_device), Y, stream);
    });
}

int64_t up(int64_t v, int64_t to) { return v / to + (v % to > 0); }

PyObject* layernorm_forward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 12, p_layernorm_forward != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d), row = t > 0 ? d : 0;
        const Kind k16 = kind16(dtype);
        void *X = a.pointer(3, k16, td), *R = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, row);
        void* beta = a.pointer(6, k16, row);
        const float eps = a.real(7);
        void *H = a.pointer(8, k16, td), *Y = a.pointer(9, k16, td), *stats = a.pointer(10, Kind::kF32, times(t, 2));
        const cudaStream_t stream = a.stream(11);
        return unlocked(a, p_layernorm_forward, t, d, dtype_of(dtype), X, R, gamma, beta, eps, H, Y,
                        static_cast<float*>(stats), stream);
    });
}

PyObject* layernorm_e4m3(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 13, p_layernorm_e4m3 != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d), row = t > 0 ? d : 0;
        const Kind k16 = kind16(dtype);
        void *X = a.pointer(3, k16, td), *R = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, row);
        void* beta = a.pointer(6, k16, row);
        const float eps = a.real(7);
        void *H = a.pointer(8, k16, td), *Q = a.pointer(9, Kind::kE4m3, td);
        void* scale = a.pointer(10, Kind::kF32, d > 0 ? times(t, up(d, 128)) : 0);
        void* stats = a.pointer(11, Kind::kF32, times(t, 2));
        const cudaStream_t stream = a.stream(12);
        return unlocked(a, p_layernorm_e4m3, t, d, dtype_of(dtype), X, R, gamma, beta, eps, H, Q,
                        static_cast<float*>(scale), static_cast<float*>(stats), stream);
    });
}

PyObject* layernorm_backward(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 13, p_layernorm_backward != nullptr, [](Args& a) {
        const int64_t t = a.integer(0), d = a.integer(1), dtype = a.integer(2), td = times(t, d);
        const Kind k16 = kind16(dtype);
        void *dY = a.pointer(3, k16, td), *H = a.pointer(4, k16, td), *gamma = a.pointer(5, k16, t > 0 ? d : 0);
        void *stats = a.pointer(6, Kind::kF32, times(t, 2)), *dH = a.pointer(7, k16, td), *dX = a.pointer(8, k16, td);
        void *dgamma = a.pointer(9, Kind::kF32, d), *dbeta = a.pointer(10, Kind::kF32, d);
        void* workspace = a.pointer(11, Kind::kBytes, t > 0 && !a.bad ? p_layernorm_workspace(t, d) : 0);
        const cudaStream_t stream = a.stream(12);
        return unlocked(a, p_layernorm_backward, t, d, dtype_of(dtype), dY, H, gamma,
                        static_cast<const float*>(stats), dH, dX, static_cast<float*>(dgamma),
                        static_cast<float*>(dbeta), workspace, stream);
    });
}

PyObject* e4m3_quantize(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 10, p_e4m3_quantize != nullptr, [](Args& a) {
        const int64_t rows = a.integer(0), cols = a.integer(1), dtype = a.integer(2), block = a.integer(3);
        const bool any = rows > 0 && cols > 0 && rows < 1ll << 40 && cols < 1ll << 40;
        const int64_t rb = any ? up(rows, 128) : 0, cb = any ? up(cols, 128) : 0;
        const bool square = block == GEMM_EPI_BLOCK_128X128;
        void *X = a.pointer(4, kind16(dtype), times(rows, cols)), *Q = a.pointer(5, Kind::kE4m3, times(rows, cols));
        void* scale = a.pointer(6, Kind::kF32, times(cb, square ? rb : rows));
        void* Qt = a.pointer(7, Kind::kE4m3, any ? times(cols, up(rows, 16) * 16) : 0);
        void* scale_t = a.pointer(8, Kind::kF32, times(rb, square ? cb : cols));
        const cudaStream_t stream = a.stream(9);
        return unlocked(a, p_e4m3_quantize, rows, cols, dtype_of(dtype), static_cast<gemm_epi_block>(block), X, Q,
                        static_cast<float*>(scale), Qt, static_cast<float*>(scale_t), stream);
    });
}

// A plan with scales for blocks of 128: (plan, m, n, k, SCALE_BLOCKS, bias values, A, B, bias, residual, D,
// aux, scale_a, scale_b, stream)
PyObject* block_product(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 15, p_execute_operands != nullptr, [](Args& a) {
        void* plan = reinterpret_cast<void*>(static_cast<uintptr_t>(a.word(0)));
        const int64_t m = a.integer(1), cols = a.integer(2), k = a.integer(3), blocks = a.integer(4);
        const int64_t bias_values = a.integer(5), mn = times(m, cols), kb = mn > 0 && k > 0 ? up(k, 128) : 0;
        const int64_t any = mn > 0;
        gemm_epi_operands o = {};
        o.A = a.pointer(6, Kind::kE4m3, any * times(m, k));
        o.B = a.pointer(7, Kind::kE4m3, any * times(cols, k));
        o.bias = a.pointer(8, Kind::kBf16, any * bias_values);
        o.residual = a.pointer(9, Kind::kBf16, mn);
        o.D = a.pointer(10, Kind::kBf16, mn);
        o.aux = a.pointer(11, Kind::kBytes, any * times(m, up(cols, 32) * 4));
        o.scale_a = static_cast<const float*>(a.pointer(12, Kind::kF32, times(kb, m)));
        o.scale_b = static_cast<const float*>(
            a.pointer(13, Kind::kF32, times(kb, blocks == GEMM_EPI_SCALE_BLOCKS_ROWS ? cols : up(cols, 128))));
        const cudaStream_t stream = a.stream(14);
        return unlocked(a, p_execute_operands, static_cast<gemm_epi_plan_t>(plan),
                        static_cast<const gemm_epi_operands*>(&o), stream);
    });
}

// bind(rmsnorm, rmsnorm_e4m3, rmsnorm_backward, w4_matmul, w4_dequantize, dropout,
// rmsnorm_workspace, layernorm_forward, layernorm_e4m3, layernorm_backward, layernorm_workspace,
// e4m3_quantize, execute_operands): addresses
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    return call(args, n, 13, true, [](Args& a) {
        void* p[13];
        for (int i = 0; i < 13; ++i) p[i] = a.pointer(i);
        if (a.bad) return 0L;
        p_rmsnorm = reinterpret_cast<decltype(p_rmsnorm)>(p[0]);
        p_rmsnorm_e4m3 = reinterpret_cast<decltype(p_rmsnorm_e4m3)>(p[1]);
        p_rmsnorm_backward = reinterpret_cast<decltype(p_rmsnorm_backward)>(p[2]);
        p_w4_matmul = reinterpret_cast<decltype(p_w4_matmul)>(p[3]);
        p_w4_dequantize = reinterpret_cast<decltype(p_w4_dequantize)>(p[4]);
        p_dropout = reinterpret_cast<decltype(p_dropout)>(p[5]);
        p_rmsnorm_workspace = reinterpret_cast<decltype(p_rmsnorm_workspace)>(p[6]);
        p_layernorm_forward = reinterpret_cast<decltype(p_layernorm_forward)>(p[7]);
        p_layernorm_e4m3 = reinterpret_cast<decltype(p_layernorm_e4m3)>(p[8]);
        p_layernorm_backward = reinterpret_cast<decltype(p_layernorm_backward)>(p[9]);
        p_layernorm_workspace = reinterpret_cast<decltype(p_layernorm_workspace)>(p[10]);
        p_e4m3_quantize = reinterpret_cast<decltype(p_e4m3_quantize)>(p[11]);
        p_execute_operands = reinterpret_cast<decltype(p_execute_operands)>(p[12]);
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
                         method("layernorm_forward", layernorm_forward),
                         method("layernorm_e4m3", layernorm_e4m3),
                         method("layernorm_backward", layernorm_backward),
                         method("e4m3_quantize", e4m3_quantize),
                         method("block_product", block_product),
                         method("bind", bind),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods,
                      nullptr,               nullptr,     nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__fastcall(void)
{
    return PyModule_Create(&module);
}
