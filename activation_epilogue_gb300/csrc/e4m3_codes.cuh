// E4M3 codes with a scale for a block of values: scale = largest |x| / 448, code = x / scale.
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

namespace gemm_epi {

constexpr float kE4m3Top = 448.0f;
constexpr float kBlockFloor = 7.888609052210118e-31f;  // 2^-100: a block without a value above it is zeros

// Four E4M3 codes, rounded to nearest even, saturated; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_codes4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint2 e4m3_codes8(const float (&x)[8], float inv)
{
    return make_uint2(e4m3_codes4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                      e4m3_codes4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// A block's scale, top / 448 correctly rounded (the quotient's remainder, exact in one fma, put right: Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), and its reciprocal to
// 2^-23 from its largest |x|; an infinite or NaN one goes into the scale.
__device__ __forceinline__ void block_scale(float top, float& scale, float& inv)
{
    constexpr float kInverse = 1.0f / kE4m3Top;
    const float q = top * kInverse;
    const float right = fmaf(fmaf(-q, kE4m3Top, top), kInverse, q);
    scale = top < kBlockFloor ? 0.0f : q < 1.0e36f ? right : q;  // (an infinity has no remainder)
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
    inv = top < kBlockFloor ? 0.0f : inv;
}

// The largest bit pattern of eight |x|.
__device__ __forceinline__ uint32_t abs_max8(const float (&x)[8])
{
    uint32_t m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = __float_as_uint(x[e]) & 0x7FFFFFFFu;
    return __vimax3_u32(__vimax3_u32(m[0], m[1], m[2]), __vimax3_u32(m[3], m[4], m[5]), max(m[6], m[7]));
}

// The largest of the 16 lanes of a half warp, in all of them (bit patterns of |x|: as whole numbers
// NaN > infinity > finite values, so that a NaN anywhere wins).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v)
{
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

}  // namespace gemm_epi
