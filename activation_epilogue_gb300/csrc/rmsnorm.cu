// RMS norm with the residual's addition, forward (16-bit or E4M3 output) and backward.
#include <cuda_fp8.h>

#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

constexpr int kThreadsPerRow = 256;
constexpr float kE4m3Max = 448.0f;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: below it a row is zeros

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the block, in the same order in every call.  `part`: one float per warp.
__device__ __forceinline__ float block_sum(float v, float* part)
{
    const int warps = blockDim.x >> 5;
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < warps; ++w) s += part[w];
    return s;
}

// Largest bit pattern of |v| over the block: as integers, NaN > infinity > finite values, so
// a NaN anywhere wins.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* part)
{
    const int warps = blockDim.x >> 5;
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t s = 0;
    for (int w = 0; w < warps; ++w) s = max(s, part[w]);
    return s;
}

// scale = amax / 448 and its reciprocal; zero for a row (tensor) with nothing above 2^-100.
__device__ __forceinline__ void scale_of(float amax, float& scale, float& inv)
{
    const bool nothing = amax < kScaleFloor;
    scale = nothing ? 0.0f : amax / kE4m3Max;
    inv = nothing ? 0.0f : 1.0f / scale;
}

// Four E4M3 codes, saturated; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_kernel(const RmsnormArgs a)
{
    __shared__ float part[32];
    __shared__ uint32_t upart[32];
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t cta_max = 0;
    for (long long r = blockIdx.x; r < a.t; r += gridDim.x) {
        const uint16_t* x = static_cast<const uint16_t*>(a.X) + r * a.d;
        const uint16_t* res = static_cast<const uint16_t*>(a.residual) + r * a.d;
        uint16_t* hout = static_cast<uint16_t*>(a.H) + r * a.d;
        float s = 0.0f;
        for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
            float v[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(x + c), v);
            if (a.residual) {
                float rv[8];
                decode8<BF16>(*reinterpret_cast<const uint4*>(res + c), rv);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += rv[j];
                const uint4 w = encode8<BF16>(v);
                *reinterpret_cast<uint4*>(hout + c) = w;
                decode8<BF16>(w, v);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
        }
        const float rstd = 1.0f / sqrtf(block_sum(s, part) / static_cast<float>(a.d) + a.eps);
        if (threadIdx.x == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if (a.mode == kRmsTensor) a.ws_rstd[r] = rstd;
        }
        const uint16_t* h = a.residual ? hout : x;  // (each thread reads back what it wrote)
        const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
        float inv = 1.0f;
        if (a.mode == kRmsGiven) inv = 1.0f / __ldg(a.scale);
        if (a.mode == kRmsRow || a.mode == kRmsTensor) {
            uint32_t m = 0;
            for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
                float v[8], g[8];
                decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
                decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = max(m, __float_as_uint(v[j] * rstd * g[j]) & 0x7FFFFFFFu);
            }
            m = block_max(m, upart);
            cta_max = max(cta_max, m);
            float scale;
            scale_of(__uint_as_float(m), scale, inv);
            if (a.mode == kRmsRow && threadIdx.x == 0) a.scale[r] = scale;
        }
        if (a.mode == kRmsTensor) continue;
        for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
            float v[8], g[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
            decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
            if (a.mode == kRms16) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + r * a.d + c) = encode8<BF16>(v);
            } else {
                uint2 q;
                q.x = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
                q.y = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + r * a.d + c) = q;
            }
        }
    }
    if (a.mode == kRmsTensor && threadIdx.x == 0) a.ws_max[blockIdx.x] = cta_max;
}

// Second pass of the per-tensor scale: the first one's maxima, then the codes.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_quantise_kernel(const RmsnormArgs a, int parts)
{
    __shared__ uint32_t upart[32];
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t m = 0;
    for (int i = threadIdx.x; i < parts; i += kThreadsPerRow) m = max(m, a.ws_max[i]);
    m = block_max(m, upart);
    float scale, inv;
    scale_of(__uint_as_float(m), scale, inv);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.scale[0] = scale;
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    for (long long r = blockIdx.x; r < a.t; r += gridDim.x) {
        const uint16_t* h = static_cast<const uint16_t*>(a.residual ? a.H : a.X) + r * a.d;
        const float rstd = a.ws_rstd[r];
        for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
            float v[8], g[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
            decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
            uint2 q;
            q.x = e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            q.y = e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + r * a.d + c) = q;
        }
    }
}

// Backward: block b takes rows b, b + blocks, ... and keeps its sums of dgamma in its own row
// of ws_dgamma, every column with one thread; rmsnorm_dgamma_kernel adds the rows in order.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_backward_kernel(const RmsnormBackwardArgs a)
{
    __shared__ float part[32];
    grid_dependency_wait();
    grid_launch_dependents();
    float* dg = a.ws_dgamma + static_cast<long long>(blockIdx.x) * a.d;
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    bool first = true;
    for (long long r = blockIdx.x; r < a.t; r += gridDim.x) {
        const uint16_t* dy = static_cast<const uint16_t*>(a.dY) + r * a.d;
        const uint16_t* h = static_cast<const uint16_t*>(a.H) + r * a.d;
        const float rstd = a.rstd[r];
        float s = 0.0f;
        for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
            float y[8], v[8], g[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(dy + c), y);
            decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
            decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xh = v[j] * rstd;
                s = fmaf(y[j] * g[j], xh, s);
                dg[c + j] = fmaf(y[j], xh, first ? 0.0f : dg[c + j]);
            }
        }
        first = false;
        const float mean = block_sum(s, part) / static_cast<float>(a.d);
        for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
            float y[8], v[8], g[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(dy + c), y);
            decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
            decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = rstd * (y[j] * g[j] - v[j] * rstd * mean);
            if (a.dH) {
                float e[8];
                decode8<BF16>(*reinterpret_cast<const uint4*>(
                                  static_cast<const uint16_t*>(a.dH) + r * a.d + c), e);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] += e[j];
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dX) + r * a.d + c) = encode8<BF16>(y);
        }
    }
}

__global__ void __launch_bounds__(256) rmsnorm_dgamma_kernel(const float* ws, int parts, int d,
                                                             float* dgamma)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (c >= d) return;
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += ws[static_cast<long long>(p) * d + c];
    dgamma[c] = s;
}

}  // namespace

int rmsnorm_max_parts(long long t) { return static_cast<int>(t < kRmsMaxParts ? t : kRmsMaxParts); }
int rmsnorm_backward_parts(long long t)
{
    return static_cast<int>(t < kRmsBackwardParts ? t : kRmsBackwardParts);
}

cudaError_t rmsnorm_launch(const RmsnormArgs& a, bool bf16, cudaStream_t stream)
{
    const int grid = a.mode == kRmsTensor ? rmsnorm_max_parts(a.t) : a.t;
    cudaError_t e = bf16 ? launch_dependent(rmsnorm_kernel<true>, grid, kThreadsPerRow, 0, stream, 1, a)
                         : launch_dependent(rmsnorm_kernel<false>, grid, kThreadsPerRow, 0, stream, 1, a);
    if (e != cudaSuccess || a.mode != kRmsTensor) return e;
    return bf16 ? launch_dependent(rmsnorm_quantise_kernel<true>, grid, kThreadsPerRow, 0, stream, 1, a, grid)
                : launch_dependent(rmsnorm_quantise_kernel<false>, grid, kThreadsPerRow, 0, stream, 1, a, grid);
}

cudaError_t rmsnorm_backward_launch(const RmsnormBackwardArgs& a, bool bf16, cudaStream_t stream)
{
    const int parts = rmsnorm_backward_parts(a.t);
    const cudaError_t e =
        bf16 ? launch_dependent(rmsnorm_backward_kernel<true>, parts, kThreadsPerRow, 0, stream, 1, a)
             : launch_dependent(rmsnorm_backward_kernel<false>, parts, kThreadsPerRow, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(rmsnorm_dgamma_kernel, (a.d + 255) / 256, 256, 0, stream, 1,
                            static_cast<const float*>(a.ws_dgamma), parts, a.d, a.dgamma);
}

}  // namespace gemm_epi
