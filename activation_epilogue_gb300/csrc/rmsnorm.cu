// RMS norm with the residual's addition, forward (16-bit or E4M3 output) and backward.
//
//   H = X + residual (rounded), rstd = 1 / sqrt(mean H^2 + eps), Y = H rstd gamma;
//   g = dY gamma, xh = H rstd: dX = rstd (g - xh mean(g xh)) + dH, dgamma = sum dY xh.
//
// Everything is bound by the bytes: a row is read once into registers (16-byte accesses, every
// load of the row before the first use), its sum of squares and, for E4M3, its largest value are
// reduced over the row's threads, and the row is written.  Squares, sums, rstd, maxima and the
// sums of dgamma are fp32; H, Y and dX are rounded once each, E4M3 codes once from fp32 (they are
// y times the rounded reciprocal of the scale, as the header says).
// Measured (bf16, 6.79 TB/s copy): 16384 x 8192 with the residual to 16 bits 152 us and to E4M3
// with a scale per row 131 us (105 % of the copy rate), backward 163 us (97 %); 2039 x 4096 to
// E4M3 10.4 us (83 %: a start and an end of short blocks), one row of 4096 1.6 us.  One scale for
// the tensor has to read H a second time: 177 us for 16384 x 8192, at the copy rate for the 9 bytes
// an element that it moves.  Rows wider than 16384 columns are passed over again for each sum: 4096 x
// 20480 to 16 bits 119 us (83 %), row scales 115 (75 %), tensor scale 138, given 108, backward 170 (58 %);
// 2048 x 65536 206, 227, 231, 189 and 268 us.
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

// bf16 has fp32's exponents, so the squares of a row may leave fp32 where the row and its norm do not:
// then they are summed again of the row times a power of two.  far_factor: that power, or 0 where
// the sum s stands.  A sum below 2^-80 has lost up to 2^-149 a square (2^-39 of it over 2^30 columns),
// unless eps is so much larger that the sum does not matter; one past fp32 has a value above 2^48,
// which 2^-96 leaves above 2^-48 and below 2^32.  An infinity or a NaN in the row stays one.
__device__ __forceinline__ float far_factor(float s, float eps)
{
    if (s > 3.0e38f || s != s) return 1.262177448e-29f;                    // 2^-96
    return s < 8.271806126e-25f && eps < 8.881784197e-16f ? 1.208925820e24f  // 2^-80, 2^-50: 2^80
                                                          : 0.0f;
}

// rstd from the mean of the squares of the row times `factor`.
__device__ __forceinline__ float far_rstd(float mean, float factor, float eps)
{
    return factor / sqrtf(mean + eps * factor * factor);
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

// ---- rows that a block holds in registers -------------------------------------------------
// T threads per row, V vectors of 8 per thread (vector j of thread i: columns 8 (j T + i) ...):
// every load of a row is issued before any value is used, and the row is read once.  T = 32 is
// a warp per row, four rows per block and no barrier; wider rows take a block each.

template <int T>
__host__ __device__ constexpr int rms_block()
{
    return T < 128 ? 128 : T;
}

// Sum (largest bits) over the T threads of a row, the same in every call and in every one of
// them.  One barrier: rows take the words `part` in turn, so that the row after next is the first
// to write these again, and no thread gets there before all have read them.
template <int T>
__device__ __forceinline__ float row_sum(float v, float (&part)[32])
{
    v = warp_sum(v);
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) s += part[w];
    return s;
}

template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (&part)[32])
{
    v = __reduce_max_sync(0xFFFFFFFFu, v);
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) s = max(s, part[w]);
    return s;
}

template <int T, int V, bool STREAM = false>
__device__ __forceinline__ void load_row(const void* base, long long row, int d, uint4 (&w)[V])
{
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + row * d);
    const int i0 = threadIdx.x % T;
#pragma unroll
    for (int j = 0; j < V; ++j)
        w[j] = (j * T + i0) * 8 >= d ? make_uint4(0, 0, 0, 0)
               : STREAM              ? __ldcs(p + j * T + i0)
                                     : p[j * T + i0];
}

template <bool STREAM = false>
__device__ __forceinline__ void store_e4m3(uint8_t* p, const float (&y)[8], float inv)
{
    uint2 q;
    q.x = e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
    q.y = e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
    if constexpr (STREAM)
        __stcs(reinterpret_cast<uint2*>(p), q);
    else
        *reinterpret_cast<uint2*>(p) = q;
}

// A far row (bf16) from memory, where H (X without a residual) stands as the same threads stored it:
// what the kernels do for a near one.  It stands behind a near row's code, which stores nothing for it: a
// branch between the sum and the outputs took the overlap of the sum's wait with the decoding
// (ROW, 16384 x 2048: 36.9 us, 41.1 with it), a call registers.  Returns the thread's largest bits of Y.
template <int T>
__device__ __forceinline__ uint32_t far_row(const RmsnormArgs& a, int mode, long long r, float factor,
                                            float (&part)[32], uint32_t (&upart)[32])
{
    if constexpr (T > 32) __syncthreads();  // (part, upart and a mark in ws_rstd have been read)
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    const uint16_t* h = static_cast<const uint16_t*>(a.residual ? a.H : a.X) + r * a.d;
    const int i0 = threadIdx.x % T;
    float s = 0.0f;
#pragma unroll 1
    for (int c = i0 * 8; c < a.d; c += T * 8) {
        float x[8];
        decode8<true>(*reinterpret_cast<const uint4*>(h + c), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e] * factor, x[e] * factor, s);
    }
    const float rstd = far_rstd(row_sum<T>(s, part) / static_cast<float>(a.d), factor, a.eps);
    if (i0 == 0) {
        if (a.rstd) a.rstd[r] = rstd;
        if (mode == kRmsTensor) a.ws_rstd[r] = rstd;
    }
    float inv = mode == kRmsGiven ? 1.0f / a.scale[0] : 0.0f;
    uint32_t m = 0;
#pragma unroll 1
    for (int pass = mode == kRmsRow ? 0 : 1; pass < 2; ++pass) {
#pragma unroll 1
        for (int c = i0 * 8; c < a.d; c += T * 8) {
            float x[8], g[8];
            decode8<true>(*reinterpret_cast<const uint4*>(h + c), x);
            decode8<true>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * g[e];
            if (mode == kRmsTensor || pass == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
            } else if (mode == kRms16) {
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + r * a.d + c) = encode8<true>(x);
            } else {
                store_e4m3(static_cast<uint8_t*>(a.Y) + r * a.d + c, x, inv);
            }
        }
        if (mode == kRmsRow && pass == 0) {
            float scale;
            scale_of(__uint_as_float(row_max<T>(m, upart)), scale, inv);
            if (i0 == 0) a.scale[r] = scale;
        }
    }
    return m;
}

// The far ones of a block's rows, which ws_rstd marks with minus their factor (tensor scale).
template <int T>
__device__ __forceinline__ uint32_t far_rows(const RmsnormArgs& a, float (&part)[32], uint32_t (&upart)[32])
{
    constexpr int kRows = T == 32 ? rms_block<T>() / T : 1;
    uint32_t m = 0;
    if constexpr (T > 32) __syncthreads();
    __syncwarp();
#pragma unroll 1
    for (long long r = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T; r < a.t;
         r += static_cast<long long>(gridDim.x) * kRows) {
        const float factor = -a.ws_rstd[r];
        if (factor > 0.0f) m = max(m, far_row<T>(a, kRmsTensor, r, factor, part, upart));
    }
    return m;
}

// Blocks an SM (at least; 0: the compiler's choice), by measurement.  One row a block: 2048 x 2048 to 16
// bits 6.4 us with 8, 6.9 with the compiler's 12 of fewer registers; 2048 x 8192 21.4 with 4, 22.3 with 3;
// to E4M3 with row scales 18.9 with 3, 20.4 with 4; 2048 x 16384 to 16 bits 40.3 with 2, 46.1 with 1.
// Walking (tensor scale): 8192 x 4096 45.8 with 6, 52.4 with 5.
template <bool BF16, int T, int V, int MODE>
constexpr int rms_blocks()
{
    if (MODE == kRmsTensor) return !BF16 ? 0 : T == 32 ? (V < 4 ? 6 : 0) : T == 128 ? (V == 2 ? 8 : 6) : T == 256 ? 3 : 0;
    if (T == 256) return BF16 && MODE != kRmsRow ? 4 : 0;
    return (T == 128 || T == 32) && V == 2 ? 8 : T == 512 && (BF16 || MODE != kRms16) ? 2 : 0;
}

template <bool BF16, int T, int V, int MODE>
__global__ void __launch_bounds__(rms_block<T>(), rms_blocks<BF16, T, V, MODE>()) rmsnorm_kernel(const RmsnormArgs a)
{
    constexpr int kRows = rms_block<T>() / T;
    __shared__ float part[2][32];
    __shared__ uint32_t upart[2][32];
    const int i0 = threadIdx.x % T;
    grid_dependency_wait();
    grid_launch_dependents();
    uint4 gamma[V];
    load_row<T, V>(a.gamma, 0, a.d, gamma);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    const float given = MODE == kRmsGiven ? a.scale[0] : 1.0f;
    uint32_t top = 0;
    int parity = 0;
    bool any_far = false;
    // (the grid walks for the tensor scale alone)
    for (long long r = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T; r < a.t;
         r += static_cast<long long>(gridDim.x) * kRows, parity ^= 1) {
        uint4 h[V];
        // (tensor scale: X and the residual are read once, H again by the second pass)
        constexpr bool kStream = MODE == kRmsTensor;
        if (kStream && a.residual)
            load_row<T, V, true>(a.X, r, a.d, h);
        else
            load_row<T, V>(a.X, r, a.d, h);
        if (a.residual) {
            uint4 res[V];
            load_row<T, V, kStream>(a.residual, r, a.d, res);
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.H) + r * a.d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8], y[8];
                decode8<BF16>(h[j], x);
                decode8<BF16>(res[j], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] += y[e];
                h[j] = encode8<BF16>(x);
                if ((j * T + i0) * 8 < a.d) out[j * T + i0] = h[j];
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float x[8];
            decode8<BF16>(h[j], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
        }
        s = row_sum<T>(s, part[parity]);
        const float rstd = 1.0f / sqrtf(s * inv_d + a.eps);
        // a far row's outputs are left to far_row
        const float factor = BF16 ? far_factor(s, a.eps) : 0.0f;  // (the same in all of the row's threads)
        const bool far = factor != 0.0f;
        any_far |= far;
        if (i0 == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if (MODE == kRmsTensor) a.ws_rstd[r] = far ? -factor : rstd;
        }
        float inv = 1.0f / given;  // (here: a division ahead of the row's loads would hold them up)
        if constexpr (MODE == kRmsRow || MODE == kRmsTensor) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float x[8], g[8];
                decode8<BF16>(h[j], x);
                decode8<BF16>(gamma[j], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e] * rstd * g[e]) & 0x7FFFFFFFu);
            }
            if constexpr (MODE == kRmsTensor) {
                if (!far) top = max(top, m);
            } else {
                float scale;
                scale_of(__uint_as_float(row_max<T>(m, upart[parity])), scale, inv);
                if (i0 == 0) a.scale[r] = scale;
            }
        }
        if constexpr (MODE != kRmsTensor) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (j * T + i0) * 8;
                if (c >= a.d || far) continue;
                float x[8], g[8];
                decode8<BF16>(h[j], x);
                decode8<BF16>(gamma[j], g);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * g[e];
                if constexpr (MODE == kRms16)
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + r * a.d + c) = encode8<BF16>(x);
                else
                    store_e4m3(static_cast<uint8_t*>(a.Y) + r * a.d + c, x, inv);
            }
            if (far) far_row<T>(a, MODE, r, factor, part[0], upart[0]);
            break;
        }
    }
    if constexpr (MODE == kRmsTensor) {
        if (BF16 && any_far) top = max(top, far_rows<T>(a, part[0], upart[0]));
        const uint32_t m = row_max<rms_block<T>()>(top, upart[0]);
        if (threadIdx.x == 0) a.ws_max[blockIdx.x] = m;
    }
}

// Second pass of the per-tensor scale: the largest of the first pass's maxima, then the codes.
// It walks the rows from the last to the first, so that it begins with the rows of H that the
// first pass left in L2 (2 % of a call at most, as the loads and stores past L2).
template <bool BF16, int T, int V>
__global__ void __launch_bounds__(rms_block<T>()) rmsnorm_quantise_kernel(const RmsnormArgs a, int parts)
{
    constexpr int kRows = rms_block<T>() / T;
    __shared__ uint32_t upart[2][32];
    const int i0 = threadIdx.x % T;
    grid_dependency_wait();
    grid_launch_dependents();
    uint4 gamma[V];
    load_row<T, V>(a.gamma, 0, a.d, gamma);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < parts; i += rms_block<T>()) m = max(m, a.ws_max[i]);
    m = row_max<rms_block<T>()>(m, upart[0]);
    float scale, inv;
    scale_of(__uint_as_float(m), scale, inv);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.scale[0] = scale;
    for (long long q = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T; q < a.t;
         q += static_cast<long long>(gridDim.x) * kRows) {
        const long long r = a.t - 1 - q;
        const float rstd = a.ws_rstd[r];
        uint4 h[V];
        load_row<T, V, true>(a.residual ? a.H : a.X, r, a.d, h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (j * T + i0) * 8;
            if (c >= a.d) continue;
            float x[8], g[8];
            decode8<BF16>(h[j], x);
            decode8<BF16>(gamma[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * rstd * g[e];
            store_e4m3<true>(static_cast<uint8_t*>(a.Y) + r * a.d + c, x, inv);
        }
    }
}

// Backward: a block keeps the sums of dgamma of its rows in registers, every column with one
// thread (T = 32: one per warp, added in order at the end), and writes them to its row of the
// workspace; rmsnorm_dgamma_kernel adds those.  The next row is copied to shared memory while
// this one is worked on, every thread copying the vectors that it reads itself, so that the
// copies need no barrier.
template <int T, int V>
__host__ __device__ constexpr int rms_backward_smem()
{
    return 2 * 3 * V * rms_block<T>() * 16;
}

template <bool BF16, int T, int V>
__global__ void __launch_bounds__(rms_block<T>()) rmsnorm_backward_kernel(const RmsnormBackwardArgs a)
{
    constexpr int kBlock = rms_block<T>(), kRows = kBlock / T;
    extern __shared__ __align__(16) uint4 buf[];  // [2][dY, H, dH][V][thread]
    __shared__ float part[2][32];
    const int i0 = threadIdx.x % T;
    grid_dependency_wait();
    grid_launch_dependents();
    auto fetch = [&](long long r, int stage) {
        const uint16_t* src[3] = {static_cast<const uint16_t*>(a.dY), static_cast<const uint16_t*>(a.H),
                                  static_cast<const uint16_t*>(a.dH)};
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if ((s < 2 || a.dH) && (j * T + i0) * 8 < a.d)
                    cp_async_16(smem_u32(buf + ((stage * 3 + s) * V + j) * kBlock + threadIdx.x),
                                src[s] + r * a.d + (j * T + i0) * 8);
    };
    const long long step = static_cast<long long>(gridDim.x) * kRows;
    long long r = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T;
    float rstd = 0.0f;
    if (r < a.t) {
        fetch(r, 0);
        rstd = a.rstd[r];
    }
    cp_async_commit();
    uint4 gamma[V];
    load_row<T, V>(a.gamma, 0, a.d, gamma);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    float dg[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[j][e] = 0.0f;
    int parity = 0;
    for (; r < a.t; r += step, parity ^= 1) {
        float next_rstd = 0.0f;
        if (r + step < a.t) {
            fetch(r + step, parity ^ 1);
            next_rstd = a.rstd[r + step];
        }
        cp_async_commit();
        cp_async_wait_group<1>();
        const uint4* row = buf + parity * 3 * V * kBlock + threadIdx.x;
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
            float y[8], x[8], g[8];
            decode8<BF16>(row[j * kBlock], y);
            decode8<BF16>(row[(V + j) * kBlock], x);
            decode8<BF16>(gamma[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = x[e] * rstd;
                s = fmaf(y[e] * g[e], xh, s);
                dg[j][e] = fmaf(y[e], xh, dg[j][e]);
            }
        }
        const float mean = row_sum<T>(s, part[parity]) * inv_d;
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dX) + r * a.d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
            float y[8], x[8], g[8];
            decode8<BF16>(row[j * kBlock], y);
            decode8<BF16>(row[(V + j) * kBlock], x);
            decode8<BF16>(gamma[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = rstd * (y[e] * g[e] - x[e] * rstd * mean);
            if (a.dH) {
                float z[8];
                decode8<BF16>(row[(2 * V + j) * kBlock], z);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += z[e];
            }
            out[j * T + i0] = encode8<BF16>(y);
        }
        rstd = next_rstd;
    }
    if constexpr (kRows > 1) {
        __shared__ float sum[T * V * 8];
        for (int w = 0; w < kRows; ++w) {
            if (threadIdx.x / T == w) {
#pragma unroll
                for (int j = 0; j < V; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float& at = sum[(j * T + i0) * 8 + e];
                        at = w == 0 ? dg[j][e] : at + dg[j][e];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.d; c += rms_block<T>())
            a.ws_dgamma[static_cast<long long>(blockIdx.x) * a.d + c] = sum[c];
    } else {
        float4* out = reinterpret_cast<float4*>(a.ws_dgamma + static_cast<long long>(blockIdx.x) * a.d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
            out[(j * T + i0) * 2] = make_float4(dg[j][0], dg[j][1], dg[j][2], dg[j][3]);
            out[(j * T + i0) * 2 + 1] = make_float4(dg[j][4], dg[j][5], dg[j][6], dg[j][7]);
        }
    }
}

// ---- rows longer than that, read again from L1 and L2 for each pass -----------------------

template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow, 8) rmsnorm_long_kernel(const RmsnormArgs a)
{
    __shared__ float part[32];
    __shared__ uint32_t upart[32];
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t cta_max = 0;
    float far = 0.0f;  // the factor of a far row, the last of them
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
        s = block_sum(s, part);
        const float rstd = 1.0f / sqrtf(s / static_cast<float>(a.d) + a.eps);
        const float factor = BF16 ? far_factor(s, a.eps) : 0.0f;  // (the same in all threads)
        if (threadIdx.x == 0) {
            if (a.rstd) a.rstd[r] = rstd;
            if (a.mode == kRmsTensor) a.ws_rstd[r] = factor != 0.0f ? -factor : rstd;
        }
        if (factor != 0.0f) {
            far = factor;
            continue;
        }
        const uint16_t* h = a.residual ? hout : x;  // (each thread reads back what it wrote)
        const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
        float inv = 1.0f;
        if (a.mode == kRmsGiven) inv = 1.0f / a.scale[0];
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
    if (BF16 && far != 0.0f) {
        if (a.mode == kRmsTensor)
            cta_max = max(cta_max, block_max(far_rows<kThreadsPerRow>(a, part, upart), upart));
        else  // (its only row)
            far_row<kThreadsPerRow>(a, a.mode, blockIdx.x, far, part, upart);
    }
    if (a.mode == kRmsTensor && threadIdx.x == 0) a.ws_max[blockIdx.x] = cta_max;
}

// Second pass of the per-tensor scale: the first one's maxima, then the codes.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_quantise_long_kernel(const RmsnormArgs a, int parts)
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

// Backward in two passes: the mean of g xh of every row (a block per row), then dX and dgamma
// by columns, a block with 2048 columns of rows y, y + slices, ..., each column with one thread.
template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_backward_mean_kernel(const RmsnormBackwardArgs a)
{
    __shared__ float part[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const long long r = blockIdx.x;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dY) + r * a.d;
    const uint16_t* h = static_cast<const uint16_t*>(a.H) + r * a.d;
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    const float rstd = a.rstd[r];
    float s = 0.0f;
    for (int c = threadIdx.x * 8; c < a.d; c += kThreadsPerRow * 8) {
        float y[8], v[8], g[8];
        decode8<BF16>(*reinterpret_cast<const uint4*>(dy + c), y);
        decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), v);
        decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(y[j] * g[j], v[j] * rstd, s);
    }
    s = block_sum(s, part);
    if (threadIdx.x == 0) a.ws_mean[r] = s / static_cast<float>(a.d);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreadsPerRow) rmsnorm_backward_columns_kernel(const RmsnormBackwardArgs a, int slices)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int slice = blockIdx.x % slices;
    const int c = (blockIdx.x / slices * kThreadsPerRow + threadIdx.x) * 8;
    if (c >= a.d) return;
    float g[8], dg[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.gamma) + c), g);
#pragma unroll 2
    for (long long r = slice; r < a.t; r += slices) {
        const long long at = r * a.d + c;
        const float rstd = a.rstd[r], mean = a.ws_mean[r];
        float y[8], x[8], z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dY) + at), y);
        decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.H) + at), x);
        if (a.dH) decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dH) + at), z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xh = x[j] * rstd;
            dg[j] = fmaf(y[j], xh, dg[j]);
            y[j] = rstd * (y[j] * g[j] - xh * mean);
            if (a.dH) y[j] += z[j];
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dX) + at) = encode8<BF16>(y);
    }
    float4* out = reinterpret_cast<float4*>(a.ws_dgamma + static_cast<long long>(slice) * a.d + c);
    out[0] = make_float4(dg[0], dg[1], dg[2], dg[3]);
    out[1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
}

// Sums of `parts` rows of d values, in an order that depends on parts alone: a block takes 32
// columns, its warp w rows w, w + WARPS, ..., and the warps' sums meet in order.  Many parts
// take 32 warps (1024 rows of 1024 columns: 10 us with 8, 3 with 32), few 8 (64 rows of 4096:
// a whole call 3.9 us with 8, 4.8 with 32).  A warp's loads are issued together, the last one's
// row again past the end (333 x 1000: a call 4.5 -> 3.8 us, 2000 x 1024 7.2 -> 6.6), from 32
// registers a thread, so that an SM holds 64 warps (8000 x 2048: 29.4 -> 26.4, 500 x 4096 8.4 -> 7.2).
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 64 / WARPS) rmsnorm_dgamma_kernel(const float* ws, int parts, int d,
                                                                    float* dgamma)
{
    constexpr int kAtOnce = WARPS == 32 ? 12 : 16;
    __shared__ float sum[WARPS][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    grid_dependency_wait();
    grid_launch_dependents();
    float s = 0.0f;
    if (c < d) {
        for (int p = w; p < parts; p += WARPS * kAtOnce) {
            float v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                v[i] = ws[static_cast<long long>(min(p + i * WARPS, parts - 1)) * d + c];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) s += p + i * WARPS < parts ? v[i] : 0.0f;
        }
    }
    sum[w][lane] = s;
    __syncthreads();
    if constexpr (WARPS == 32) {
        // one warp per column now: its 32 partial sums
        s = warp_sum(sum[lane][w]);
        if (lane == 0 && blockIdx.x * 32 + w < d) dgamma[blockIdx.x * 32 + w] = s;
    } else if (w == 0 && c < d) {
#pragma unroll
        for (int i = 1; i < WARPS; ++i) s += sum[i][lane];
        dgamma[c] = s;
    }
}

constexpr int kRmsMaxWidth = 16384;  // widest row held in registers
constexpr int kFewRows = 2048;       // backward, d <= 512: a block per row, not a warp, up to here

// Blocks for `rows` rows, kRows at a time, at most `cap`, all with the same number of rounds.
int even_grid(long long rows, int rows_per_block, long long cap)
{
    const long long blocks = (rows + rows_per_block - 1) / rows_per_block;
    const long long rounds = blocks > cap ? (blocks + cap - 1) / cap : 1;
    return static_cast<int>((blocks + rounds - 1) / rounds);
}

template <bool BF16, int T, int V>
cudaError_t rmsnorm_launch_width(const RmsnormArgs& a, cudaStream_t stream)
{
    constexpr int kBlock = rms_block<T>(), kRows = kBlock / T;
    // A block per row (four for T = 32): 16384x8192 with E4M3 rows 131 us, against 145-163 with
    // 304 to 1024 blocks that walk the rows.  The first pass of the tensor scale walks, since
    // its blocks' maxima are read by every block of the second.
    const int grid = even_grid(a.t, kRows, a.mode == kRmsTensor ? 912 : (1ll << 31) - 1);
    switch (a.mode) {
    case kRms16: return launch_dependent(rmsnorm_kernel<BF16, T, V, kRms16>, grid, kBlock, 0, stream, 1, a);
    case kRmsRow: return launch_dependent(rmsnorm_kernel<BF16, T, V, kRmsRow>, grid, kBlock, 0, stream, 1, a);
    case kRmsGiven: return launch_dependent(rmsnorm_kernel<BF16, T, V, kRmsGiven>, grid, kBlock, 0, stream, 1, a);
    default: break;
    }
    const cudaError_t e = launch_dependent(rmsnorm_kernel<BF16, T, V, kRmsTensor>, grid, kBlock, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(rmsnorm_quantise_kernel<BF16, T, V>, grid, kBlock, 0, stream, 1, a, grid);
}

template <bool BF16>
cudaError_t rmsnorm_launch_type(const RmsnormArgs& a, cudaStream_t stream)
{
    if (a.d <= 256) return rmsnorm_launch_width<BF16, 32, 1>(a, stream);
    if (a.d <= 512) return rmsnorm_launch_width<BF16, 32, 2>(a, stream);
    if (a.d <= 1024) return rmsnorm_launch_width<BF16, 32, 4>(a, stream);
    if (a.d <= 2048) return rmsnorm_launch_width<BF16, 128, 2>(a, stream);
    // (2039 x 4096 11.1 us, 16384 x 4096 68.6; with 256 threads of two vectors 12.3 and 74.1)
    if (a.d <= 4096) return rmsnorm_launch_width<BF16, 128, 4>(a, stream);
    if (a.d <= 8192) return rmsnorm_launch_width<BF16, 256, 4>(a, stream);
    if (a.d <= kRmsMaxWidth) return rmsnorm_launch_width<BF16, 512, 4>(a, stream);
    const int grid = a.mode == kRmsTensor ? even_grid(a.t, 1, kRmsMaxParts) : a.t;
    const cudaError_t e = launch_dependent(rmsnorm_long_kernel<BF16>, grid, kThreadsPerRow, 0, stream, 1, a);
    if (e != cudaSuccess || a.mode != kRmsTensor) return e;
    return launch_dependent(rmsnorm_quantise_long_kernel<BF16>, grid, kThreadsPerRow, 0, stream, 1, a, grid);
}

// Width class of the backward kernel: its rows per block and most blocks (what fits on 152 SMs
// at once; each block's sums of dgamma are a row of the workspace).
struct BackwardShape {
    int rows, cap;
};

BackwardShape backward_shape(long long t, long long d)
{
    // (most blocks, measured: 1024x1024 4.7 us with 456, 5.3 with 608 and 912; 4096x1024 10.1 with
    // 760, 10.6 with 912, 32768x1024 47.7 and 45.3, with a warp per row 12.4 and 48.4; 4096x512
    // 7.1 with a warp per row, 7.9 with a block; 16384x2048 45.8 with
    // 608, 61.4 with 304; 16384x4096 82.9 with 456, 87.6 with 304; 16384x8192 164 with 304, 175
    // with 228; 8192x16384 161 with 152, 171 with 456)
    if (d <= 512) return t <= kFewRows ? BackwardShape{1, 456} : BackwardShape{4, 456};
    if (d <= 1024) return {1, t <= kFewRows ? 456 : 912};
    if (d <= 2048) return {1, 608};
    if (d <= 4096) return {1, 456};
    if (d <= 8192) return {1, 304};
    if (d <= kRmsMaxWidth) return {1, 152};
    return {1, static_cast<int>(kRmsMaxWidth * 64 / d) + 1};  // (times d / 2048 blocks)
}

template <bool BF16, int T, int V>
cudaError_t backward_launch_width(const RmsnormBackwardArgs& a, int parts, cudaStream_t stream)
{
    auto kernel = rmsnorm_backward_kernel<BF16, T, V>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, rms_backward_smem<T, V>(), prepared);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, parts, rms_block<T>(), rms_backward_smem<T, V>(), stream, 1, a);
}

template <bool BF16>
cudaError_t backward_launch_type(const RmsnormBackwardArgs& a, int parts, cudaStream_t stream)
{
    if (a.d <= 1024 && (a.d > 512 || a.t <= kFewRows)) return backward_launch_width<BF16, 128, 1>(a, parts, stream);
    if (a.d <= 256) return backward_launch_width<BF16, 32, 1>(a, parts, stream);
    if (a.d <= 512) return backward_launch_width<BF16, 32, 2>(a, parts, stream);
    if (a.d <= 2048) return backward_launch_width<BF16, 128, 2>(a, parts, stream);
    if (a.d <= 4096) return backward_launch_width<BF16, 256, 2>(a, parts, stream);
    if (a.d <= 8192) return backward_launch_width<BF16, 256, 4>(a, parts, stream);
    if (a.d <= kRmsMaxWidth) return backward_launch_width<BF16, 512, 4>(a, parts, stream);
    const cudaError_t e = launch_dependent(rmsnorm_backward_mean_kernel<BF16>, a.t, kThreadsPerRow, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    const int columns = (a.d + kThreadsPerRow * 8 - 1) / (kThreadsPerRow * 8);
    return launch_dependent(rmsnorm_backward_columns_kernel<BF16>, columns * parts, kThreadsPerRow, 0, stream, 1, a, parts);
}

}  // namespace

int rmsnorm_backward_parts(long long t, long long d)
{
    const BackwardShape s = backward_shape(t, d);
    return even_grid(t, s.rows, s.cap);
}

cudaError_t rmsnorm_launch(const RmsnormArgs& a, bool bf16, cudaStream_t stream)
{
    return bf16 ? rmsnorm_launch_type<true>(a, stream) : rmsnorm_launch_type<false>(a, stream);
}

cudaError_t rmsnorm_backward_launch(const RmsnormBackwardArgs& a, bool bf16, cudaStream_t stream)
{
    const int parts = rmsnorm_backward_parts(a.t, a.d);
    const cudaError_t e = bf16 ? backward_launch_type<true>(a, parts, stream)
                               : backward_launch_type<false>(a, parts, stream);
    if (e != cudaSuccess) return e;
    const float* ws = a.ws_dgamma;
    return parts > 128 ? launch_dependent(rmsnorm_dgamma_kernel<32>, (a.d + 31) / 32, 1024, 0, stream, 1, ws, parts, a.d, a.dgamma)
                       : launch_dependent(rmsnorm_dgamma_kernel<8>, (a.d + 31) / 32, 256, 0, stream, 1, ws, parts, a.d, a.dgamma);
}

}  // namespace gemm_epi
