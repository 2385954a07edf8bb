// Products with 4-bit weights and group scales for a few rows of A, with the GEMM epilogs,
// and the weight written out as the 16-bit B of a plan.
#include "gelu.cuh"
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

// The epilogue of one element, from the exact functions (a few elements per thread).
__device__ __forceinline__ float w4_epilogue(float v, int epilog, float residual)
{
    switch (epilog) {
    case EPI_RELU_BIAS: return v > 0.0f || v != v ? v : 0.0f;
    case EPI_GELU_BIAS: return 0.5f * v * erfcf(-0.70710678118654752f * v);
    case EPI_TANH_BIAS: return tanhf(v);
    case EPI_BIAS_RESIDUAL: return v + residual;
    default: return v;
    }
}

// One warp per column of D; lanes take words of 8 weights, up to 8 rows of A at a time.
template <bool BF16>
__global__ void __launch_bounds__(256) w4_simple_kernel(const W4Args a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int col = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (col >= a.n) return;
    const uint16_t* A = static_cast<const uint16_t*>(a.A);
    const uint16_t* S = static_cast<const uint16_t*>(a.scales);
    const uint32_t* W = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.W) +
                                                          static_cast<long long>(col) * (a.k / 2));
    for (int m0 = 0; m0 < a.m; m0 += 8) {
        float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int w = lane; w < a.k / 8; w += 32) {
            const uint32_t q = W[w];
            const long long gi = static_cast<long long>(w * 8 / a.group) * a.n + col;
            const float s = decode16<BF16>(S[gi]);
            const int z = a.zeros ? a.zeros[gi] : 8;
            float wt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                wt[j] = static_cast<float>(static_cast<int>((q >> (4 * j)) & 15u) - z);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (m0 + i >= a.m) break;
                float x[8];
                decode8<BF16>(*reinterpret_cast<const uint4*>(A + static_cast<long long>(m0 + i) * a.k + w * 8), x);
                float d = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) d = fmaf(x[j], wt[j], d);
                acc[i] = fmaf(d, s, acc[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = acc[i];
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            const int row = m0 + i;
            if (lane == 0 && row < a.m) {
                const long long at = static_cast<long long>(row) * a.n + col;
                if (a.bias) v += decode16<BF16>(static_cast<const uint16_t*>(a.bias)[col]);
                const float r = a.residual ? decode16<BF16>(static_cast<const uint16_t*>(a.residual)[at]) : 0.0f;
                static_cast<uint16_t*>(a.D)[at] = encode16<BF16>(w4_epilogue(v, a.epilog, r));
            }
        }
    }
}

// A block writes 64 (k) x 64 (n) of B through shared memory.
template <bool BF16>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const W4Args a)
{
    __shared__ uint16_t tile[64][66];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint16_t* S = static_cast<const uint16_t*>(a.scales);
    const int k_tiles = (a.k + 63) / 64;
    const int n0 = blockIdx.x / k_tiles * 64, k0 = blockIdx.x % k_tiles * 64;
    for (int i = threadIdx.x; i < 64 * 8; i += 256) {
        const int col = n0 + i / 8, k = k0 + i % 8 * 8;
        if (col >= a.n || k >= a.k) continue;
        const uint32_t q = *reinterpret_cast<const uint32_t*>(
            static_cast<const uint8_t*>(a.W) + (static_cast<long long>(col) * a.k + k) / 2);
        const long long gi = static_cast<long long>(k / a.group) * a.n + col;
        const float s = decode16<BF16>(S[gi]);
        const int z = a.zeros ? a.zeros[gi] : 8;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            tile[k - k0 + j][col - n0] =
                encode16<BF16>(static_cast<float>(static_cast<int>((q >> (4 * j)) & 15u) - z) * s);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 64; i += 256) {
        const int k = k0 + i / 64, col = n0 + i % 64;
        if (k < a.k && col < a.n)
            static_cast<uint16_t*>(a.D)[static_cast<long long>(k) * a.n + col] = tile[i / 64][i % 64];
    }
}

}  // namespace

cudaError_t w4_matmul_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    return bf16 ? launch_dependent(w4_simple_kernel<true>, (a.n + 7) / 8, 256, 0, stream, a)
                : launch_dependent(w4_simple_kernel<false>, (a.n + 7) / 8, 256, 0, stream, a);
}

cudaError_t w4_dequantize_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    const int grid = static_cast<int>(((a.n + 63) / 64) * static_cast<long long>((a.k + 63) / 64));
    return bf16 ? launch_dependent(w4_dequantize_kernel<true>, grid, 256, 0, stream, a)
                : launch_dependent(w4_dequantize_kernel<false>, grid, 256, 0, stream, a);
}

}  // namespace gemm_epi
