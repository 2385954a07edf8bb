// What the kernels on 4-bit weights share: unpacking a word of W, the epilogue of one element,
// bounded waits.
#pragma once

#include "kernel_params.h"
#include "ptx.cuh"
#include "vec16.cuh"
#include "wait_time.h"

namespace gemm_epi {

// GELU(v) = max(v, 0) - a Phi(-a), a = |v|, with the normal tail Phi(-a) = t 2^(P(t) - a^2/(2 ln 2)),
// t = 1/(1 + 0.4 a), fitted to fp32's precision (fit_normal_tail.py): off by 1e-7 at most and, like
// the 16-bit output, by a small part of the value in the tail (1.4e-5: its exponent's rounding).
// a stops at 15, where the power underflows to 0: below -14.5 the result is 0, of minus infinity
// too; a NaN stays NaN.  Without a branch, a third of the instructions of erfcf: 48 rows of
// 16384 x 8192, groups of 64, 31.8 -> 31.1 us.
__device__ __forceinline__ float w4_gelu(float v)
{
    const float a = fminf(fabsf(v), 15.0f);
    const float t = __fdividef(1.0f, fmaf(0.4f, a, 1.0f));
    float p = 0.273933083f;
    p = fmaf(p, t, -1.40280342f);
    p = fmaf(p, t, 2.80112267f);
    p = fmaf(p, t, -2.51509929f);
    p = fmaf(p, t, 0.774154961f);
    p = fmaf(p, t, -0.2584261f);
    p = fmaf(p, t, 0.536028981f);
    p = fmaf(p, t, 1.43861222f);
    p = fmaf(p, t, -2.64752293f);
    p = fmaf(a * -0.72134752f, a, p);  // 1 / (2 ln 2)
    return fmaf(-a * t, exp2f(p), v <= 0.0f ? 0.0f : v);
}

// The epilogue of one element.
__device__ __forceinline__ float w4_epilogue(float v, int epilog, float residual)
{
    switch (epilog) {
    case EPI_RELU_BIAS: return v > 0.0f || v != v ? v : 0.0f;
    case EPI_GELU_BIAS: return w4_gelu(v);
    case EPI_TANH_BIAS: return tanhf(v);
    case EPI_BIAS_RESIDUAL: return v + residual;
    default: return v;
    }
}

__device__ __forceinline__ float2 ld_shared_cluster_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// (a & b) | c in one instruction (left to itself the compiler takes two where b and c are both
// constants).
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t sub16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// What turns a word of W into values: the bits that a pair's nibbles are set in, and with the
// zero points z of the column, what to subtract.
//   bf16 (7 bits of mantissa): nibble in bits 0-3 under 128's bits is 128 + q.
//   f16 (10 bits): nibble in bits 0-3 under 1024's bits is 1024 + q, in bits 4-7 under 64's
//   bits 64 + q, so two pairs come of each shift.
template <bool BF16>
struct W4Unpack {
    uint32_t sub_even, sub_odd;  // of pairs 0, 2 and 1, 3
    __device__ __forceinline__ void set(uint32_t z)
    {
        if constexpr (BF16) {
            sub_even = sub_odd = z * 0x10001u + 0x43004300u;
        } else {
            sub_even = z * 0x10001u + 0x64006400u;
            sub_odd = z * 0x100010u + 0x54005400u;
        }
    }
    // v[j]: q - z of nibbles j (lower half) and j + 4, exactly
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t (&v)[4]) const
    {
        if constexpr (BF16) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = sub16x2<true>(and_or(w >> (4 * j), 0x000F000Fu, 0x43004300u), sub_even);
        } else {
            const uint32_t h = w >> 8;
            v[0] = sub16x2<false>(and_or(w, 0x000F000Fu, 0x64006400u), sub_even);
            v[1] = sub16x2<false>(and_or(w, 0x00F000F0u, 0x54005400u), sub_odd);
            v[2] = sub16x2<false>(and_or(h, 0x000F000Fu, 0x64006400u), sub_even);
            v[3] = sub16x2<false>(and_or(h, 0x00F000F0u, 0x54005400u), sub_odd);
        }
    }
};

// The same with neighbouring k in a pair: v[j] = q - z of nibbles 2 j (lower half) and 2 j + 1.
// A byte permutation puts byte j of w in the lower half and the one that holds nibble 2 j + 1 in
// its low (bf16: of w >> 4) or high (f16: byte j again) half in the upper.
template <bool BF16>
struct W4UnpackInOrder {
    uint32_t sub;
    __device__ __forceinline__ void set(uint32_t z)
    {
        sub = BF16 ? z * 0x10001u + 0x43004300u : z * 0x100001u + 0x54006400u;
    }
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t* v) const
    {
        const uint32_t h = BF16 ? w >> 4 : w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t p = __byte_perm(w, h, j | (4 + j) << 8 | j << 4 | j << 12);
            v[j] = BF16 ? sub16x2<true>(and_or(p, 0x000F000Fu, 0x43004300u), sub)
                        : sub16x2<false>(and_or(p, 0x00F0000Fu, 0x54006400u), sub);
        }
    }
};

// Waits of these kernels are for copies and arithmetic of the block itself, so they end; should
// one not, `failed` is set after two seconds of the kernel's own time and the block writes NaN.
constexpr unsigned long long kW4WaitNs = 2000ull * 1000 * 1000;

// One try suspends the thread for up to kW4TryNs: a waiting warp takes no issue slots from the
// warps that work.
constexpr uint32_t kW4TryNs = 100 * 1000;

__device__ __forceinline__ bool w4_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred P1;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 P1, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, P1;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kW4TryNs)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ bool w4_wait(uint32_t bar, uint32_t parity, volatile int* failed)
{
    if (w4_try_wait(bar, parity)) return true;
    WaitTime waited(globaltimer_ns());
    for (unsigned long long poll = 1; poll < kW4WaitNs / 8; ++poll) {
        if (w4_try_wait(bar, parity)) return true;
        if (*failed || waited.at(globaltimer_ns()) > kW4WaitNs) break;
    }
    *failed = 1;
    return false;
}

// Wait a bounded time for what is in flight after a failure.
__device__ __forceinline__ void w4_drain(uint32_t bar, uint32_t parity)
{
    for (int poll = 0; poll < (1 << 22); ++poll)
        if (mbar_try_wait(bar, parity)) return;
}

}  // namespace gemm_epi
