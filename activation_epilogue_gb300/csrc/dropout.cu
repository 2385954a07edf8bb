// Dropout with the residual added, the mask drawn from a counter-based generator and never
// stored: Y = residual + keep * X * scale.
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

// Philox4x32-10 of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2,
// 3" (SC 2011): ten rounds of two 32 x 32 -> 64-bit products, with a Weyl sequence on the key.
__device__ __forceinline__ uint4 philox(unsigned long long counter, uint32_t k0, uint32_t k1)
{
    uint32_t x0 = static_cast<uint32_t>(counter), x1 = static_cast<uint32_t>(counter >> 32);
    uint32_t x2 = 0, x3 = 0;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long a = static_cast<unsigned long long>(x0) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(x2) * 0xCD9E8D57u;
        const uint32_t y0 = static_cast<uint32_t>(b >> 32) ^ x1 ^ k0;
        const uint32_t y2 = static_cast<uint32_t>(a >> 32) ^ x3 ^ k1;
        x0 = y0;
        x1 = static_cast<uint32_t>(b);
        x2 = y2;
        x3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
}

template <bool BF16>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned long long offset = a.offset + (a.offset_device ? *a.offset_device : 0ull);
    const uint16_t* X = static_cast<const uint16_t*>(a.X);
    const uint16_t* R = static_cast<const uint16_t*>(a.residual);
    uint16_t* Y = static_cast<uint16_t*>(a.Y);
    const long long blocks = (a.count + 7) / 8;
    const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
    for (long long b = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; b < blocks; b += stride) {
        const uint4 w = philox(offset + static_cast<unsigned long long>(b), a.key0, a.key1);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        const int left = static_cast<int>(min(8ll, a.count - b * 8));
        float x[8], r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (left == 8) {
            decode8<BF16>(*reinterpret_cast<const uint4*>(X + b * 8), x);
            if (R) decode8<BF16>(*reinterpret_cast<const uint4*>(R + b * 8), r);
        } else {
            for (int j = 0; j < 8; ++j) {
                x[j] = j < left ? decode16<BF16>(X[b * 8 + j]) : 0.0f;
                if (R && j < left) r[j] = decode16<BF16>(R[b * 8 + j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t u = j & 1 ? ww[j / 2] >> 16 : ww[j / 2] & 0xFFFFu;
            const float y = u >= a.drop ? x[j] * a.scale : 0.0f;
            x[j] = R ? y + r[j] : y;
        }
        if (left == 8) {
            *reinterpret_cast<uint4*>(Y + b * 8) = encode8<BF16>(x);
        } else {
            for (int j = 0; j < 8; ++j)
                if (j < left) Y[b * 8 + j] = encode16<BF16>(x[j]);
        }
    }
}

}  // namespace

cudaError_t dropout_launch(const DropoutArgs& a, bool bf16, int sm_count, cudaStream_t stream)
{
    const long long blocks = (a.count + 8 * 256 - 1) / (8 * 256);
    const long long cap = static_cast<long long>(sm_count) * 8;
    const int grid = static_cast<int>(blocks < cap ? blocks : cap);
    return bf16 ? launch_dependent(dropout_kernel<true>, grid, 256, 0, stream, 1, a)
                : launch_dependent(dropout_kernel<false>, grid, 256, 0, stream, 1, a);
}

}  // namespace gemm_epi
