// Dropout with the residual added, the mask drawn from a counter-based generator and never
// stored: Y = residual + keep * X * scale.
//
// One generator call gives 128 bits, 16 for each of 8 elements (one 16-byte access): with 32 bits
// an element the twenty 32-bit products a call would outweigh the bytes.  A thread issues the
// loads of two blocks of 8 before it draws their numbers, which do not depend on them.  134M
// elements of bf16 without a residual: 87.7 us, 90 % of the copy rate (116 us with one block a
// thread in a grid-wide loop); the integer pipe is 53 % busy.
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

constexpr int kThreads = 256;
constexpr int kPerThread = 2;  // generator blocks (of 8 elements) per thread

// A thread's 8 elements of generator block b, loaded; beyond the end zeros.
__device__ __forceinline__ uint4 load_block(const uint16_t* p, long long b, long long count)
{
    if (b * 8 + 8 <= count) return *reinterpret_cast<const uint4*>(p + b * 8);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (b * 8 + j < count) w[j / 2] |= static_cast<uint32_t>(p[b * 8 + j]) << (j & 1 ? 16 : 0);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned long long offset = a.offset + (a.offset_device ? *a.offset_device : 0ull);
    const uint16_t* X = static_cast<const uint16_t*>(a.X);
    const uint16_t* R = static_cast<const uint16_t*>(a.residual);
    uint16_t* Y = static_cast<uint16_t*>(a.Y);
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kPerThread) + threadIdx.x;
    uint4 x4[kPerThread], r4[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        x4[i] = load_block(X, first + i * kThreads, a.count);
        if (RES) r4[i] = load_block(R, first + i * kThreads, a.count);
    }
    // a word's upper 16 bits are >= drop when the word is >= drop << 16, its lower 16 bits when
    // the word shifted up is; drop = 65536 (keep nothing) is a threshold that zero words miss
    const bool none = a.drop >= 65536u;
    const uint32_t least = none ? 0xFFFFFFFFu : a.drop << 16;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const long long b = first + i * kThreads;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (!none) w = philox(offset + static_cast<unsigned long long>(b), a.key0, a.key1);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        float x[8], r[8];
        decode8<BF16>(x4[i], x);
        if (RES) decode8<BF16>(r4[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool keep = (j & 1 ? ww[j / 2] : ww[j / 2] << 16) >= least;
            const float y = keep ? x[j] * a.scale : 0.0f;
            x[j] = RES ? y + r[j] : y;
        }
        const uint4 y4 = encode8<BF16>(x);
        if (b * 8 + 8 <= a.count) {
            *reinterpret_cast<uint4*>(Y + b * 8) = y4;
        } else {
            const uint32_t yy[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (b * 8 + j < a.count) Y[b * 8 + j] = static_cast<uint16_t>(yy[j / 2] >> (j & 1 ? 16 : 0));
        }
    }
}

template <bool BF16, bool RES>
cudaError_t dropout_launch_one(const DropoutArgs& a, cudaStream_t stream)
{
    const long long per_block = 8ll * kThreads * kPerThread;
    return launch_dependent(dropout_kernel<BF16, RES>, static_cast<int>((a.count + per_block - 1) / per_block),
                            kThreads, 0, stream, 1, a);  // (count <= 2^40: the grid fits)
}

}  // namespace

cudaError_t dropout_launch(const DropoutArgs& a, bool bf16, cudaStream_t stream)
{
    if (a.residual) return bf16 ? dropout_launch_one<true, true>(a, stream) : dropout_launch_one<false, true>(a, stream);
    return bf16 ? dropout_launch_one<true, false>(a, stream) : dropout_launch_one<false, false>(a, stream);
}

}  // namespace gemm_epi
