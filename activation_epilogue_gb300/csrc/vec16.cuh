// Eight 16-bit values per 16-byte access, to and from fp32, with the type a template value.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gemm_epi {

template <bool BF16>
__device__ __forceinline__ float decode16(uint32_t h)
{
    if constexpr (BF16) return __uint_as_float(h << 16);
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
}

// (lower, upper) half of a word.
template <bool BF16>
__device__ __forceinline__ float2 decode16x2(uint32_t w)
{
    if constexpr (BF16)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Round to nearest even; a in the lower half.
template <bool BF16>
__device__ __forceinline__ uint32_t encode16x2(float a, float b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool BF16>
__device__ __forceinline__ void decode8(const uint4& w, float (&x)[8])
{
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const float2 f = decode16x2<BF16>(ww[h]);
        x[2 * h] = f.x;
        x[2 * h + 1] = f.y;
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 encode8(const float (&x)[8])
{
    return make_uint4(encode16x2<BF16>(x[0], x[1]), encode16x2<BF16>(x[2], x[3]),
                      encode16x2<BF16>(x[4], x[5]), encode16x2<BF16>(x[6], x[7]));
}

template <bool BF16>
__device__ __forceinline__ uint16_t encode16(float a)
{
    if constexpr (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(a));
    return __half_as_ushort(__float2half_rn(a));
}

}  // namespace gemm_epi
