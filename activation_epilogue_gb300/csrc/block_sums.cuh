// What the block-scaled products' summing warps use: loads from tensor memory that are waited for later, and
// fp32 arithmetic on pairs.
#pragma once

#include <cstdint>

#include "gelu.cuh"

namespace gemm_epi {

// Start loading values of this warp's accumulator lanes, valid after tmem_wait on them: 16 columns of each thread's
// lane ...
__device__ __forceinline__ void load_lane16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// ... or, of 16 lanes and 32 columns, thread t's pairs of columns 8 i + 2 (t % 4), + 1 in lanes t / 4 (r[4 i],
// r[4 i + 1]) and t / 4 + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void load_square16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// ... and of 16 lanes and 16 columns.
__device__ __forceinline__ void load_square8(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Wait for this thread's loads; r (their destination) is marked as written here, so that nothing reads it earlier.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[N])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// ... and for two of them.
template <int N>
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[2][N])
{
    tmem_wait(r[0]);
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[1][i]));
}

// Pairs of fp32 in 64-bit registers: two additions an instruction.
using Pair = unsigned long long;

__device__ __forceinline__ Pair pair_of(uint32_t a, uint32_t b)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(a), "r"(b));
    return p;
}

// (x, y) += a b
__device__ __forceinline__ void fma2(float& x, float& y, Pair a, Pair b)
{
    Pair acc;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(x), "f"(y));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
}

__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}

// (x, y) += a
__device__ __forceinline__ void add2(float& x, float& y, Pair a)
{
    Pair acc;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(x), "f"(y));
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(acc) : "l"(a));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
}

// Shared memory by its own address (through generic ones the loads' latency is much longer).
__device__ __forceinline__ Pair ld_shared_pair(uint32_t addr)
{
    Pair v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void ld_shared_pairs(uint32_t addr, Pair& a, Pair& b)
{
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ Pair pair_of(float a, float b) { return pair_of(__float_as_uint(a), __float_as_uint(b)); }

__device__ __forceinline__ float2 unpair(Pair p)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
    return v;
}

// GELU's argument from below: at -6.1 and before, GELU is within 7e-9 of 0 and so is its value there.  NaN stays NaN.
__device__ __forceinline__ float gelu_floor(float x)
{
    float y;
    asm("max.NaN.f32 %0, %1, 0fC0C33333;" : "=f"(y) : "f"(x));  // -6.1
    return y;
}

// GELU of four values by gelu_erf_fast's formula, x / (1 + 2^(x p(x^2))), with one reciprocal for the four
// denominators (1 / a0 = a1 a2 a3 / (a0 a1 a2 a3)): the special-function unit, sixteen lanes' work a cycle, and the
// instructions are what a tile's GELU waits for (2039 x 4096 x 1024 on CTA pairs: 0.7 us less than with two such
// operations a value).  With x held to -6.1 ... 8 in the exponent, where a NaN becomes 8, the exponents stop below 30:
// the product of four denominators fits fp32, and neither a NaN nor an infinity reaches its neighbours.
__device__ __forceinline__ void gelu4(float* v)
{
    const Pair k1 = pair_of(-2.3014667034f, -2.3014667034f), k3 = pair_of(-0.10654459149f, -0.10654459149f);
    const Pair k5 = pair_of(0.00098442099988f, 0.00098442099988f), one = pair_of(1.0f, 1.0f);
    Pair x[2];
    float2 a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float lo = gelu_floor(v[2 * i]), hi = gelu_floor(v[2 * i + 1]);
        x[i] = pair_of(lo, hi);
        const Pair z = pair_of(fminf(lo, 8.0f), fminf(hi, 8.0f));
        const Pair s = mul2(z, z);
        Pair p, q, d;
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(q) : "l"(s), "l"(k5), "l"(k3));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(s), "l"(q), "l"(k1));
        const float2 u = unpair(mul2(z, p));
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair_of(exp2_approx(u.x), exp2_approx(u.y))), "l"(one));
        a[i] = unpair(d);
    }
    const float ab = a[0].x * a[0].y, cd = a[1].x * a[1].y;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ab * cd));
    const float over[2] = {r * cd, r * ab};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 y = unpair(mul2(x[i], mul2(pair_of(a[i].y, a[i].x), pair_of(over[i], over[i]))));
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
    }
}

}  // namespace gemm_epi
