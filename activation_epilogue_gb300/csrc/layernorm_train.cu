// LayerNorm with the residual's addition for training and block-scaled E4M3 products: forward (16-bit
// or E4M3 output, with the rows' statistics) and backward.
//
//   H = X + residual (rounded), mu = mean H, rstd = 1 / sqrt(mean (H - mu)^2 + eps),
//   Y = (H - mu) rstd gamma + beta;
//   g = dY gamma, xh = (H - mu) rstd: dX = rstd (g - mean(g) - xh mean(g xh)) + dH,
//   dgamma = sum dY xh, dbeta = sum dY.
//
// Bound by the bytes, as the RMS norm: a row is read once into registers, every load issued before the
// first use, and two sums over the row's threads stand between the loads and the stores.  The first gives
// a mean m0 in fp32; the second, of the deviations from it and of their squares, gives what m0 lacks
// (mu = m0 + mean of the deviations) and the variance about mu, so that a row far from zero loses nothing
// to the rounding of its mean.  16384 x 8192 bf16 with a residual to H and E4M3: 141.2 us, 940 MB at 6.66 TB/s,
// a copy's rate.  With E4M3 output sixteen lanes hold a block of 128 columns, whose scale
// takes four shuffles and no barrier.  Sums, statistics, maxima and scales are fp32; H, Y and dX are
// rounded once each, E4M3 codes once from fp32.
#include "e4m3_codes.cuh"
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

constexpr int kLongThreads = 256;   // rows too long for registers
constexpr int kMaxWidth = 16384;    // widest row held in registers

template <int T>
__host__ __device__ constexpr int ln_block()
{
    return T < 128 ? 128 : T;
}

// Sums of a pair of values over the T threads of a row, the same in every call and in all of them.
// `part` has a pair per warp of the block and is not used again before the next barrier.
template <int T>
__device__ __forceinline__ float2 row_sum2(float2 v, float2 (&part)[16])
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
    }
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        s.x += part[w].x;
        s.y += part[w].y;
    }
    return s;
}

template <int T>
__device__ __forceinline__ float row_sum(float v, float (&part)[16])
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (T == 32) return v;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) s += part[w];
    return s;
}

// bf16 has fp32's exponents, so that a row's sum or squares may leave fp32 where the row does not.
// far_factor: the power of two that the row is multiplied with before they are taken again, or 0 where
// they stand.  Above: a sum or a sum of squares past 2^127 of values up to 2^128 has, after 2^-96, squares
// up to 2^66 and a sum up to 2^96 over 2^30 columns.  Below: squares below 2^-80 in all have lost up to
// 2^-149 each, unless eps is so much larger that they do not matter; then no value is further than 2^-40
// from the mean, and with the mean below 2^-16 nothing passes 2^65 after 2^80.  (With the mean above that,
// two different bf16 values would be further apart: the row is constant.)
__device__ __forceinline__ float far_factor(float sum, float squares, float mean, float eps)
{
    if (!(fabsf(sum) < 1.7e38f) || !(squares < 1.7e38f)) return 1.262177448e-29f;  // 2^-96
    return squares < 8.271806126e-25f && eps < 8.881784197e-16f && fabsf(mean) < 1.52587890625e-5f
               ? 1.208925820e24f  // 2^80
               : 0.0f;
}

// The variance from the sums of the deviations from m0 and of their squares.
__device__ __forceinline__ float variance(float2 dev, float inv_d)
{
    const float more = dev.x * inv_d;
    const float var = fmaxf(dev.y * inv_d - more * more, 0.0f);
    return isnan(dev.y) ? dev.y : var;
}

template <int T, int V>
__device__ __forceinline__ void load_row(const void* base, long long row, int d, uint4 (&w)[V])
{
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + row * d);
    const int i0 = threadIdx.x % T;
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = (j * T + i0) * 8 >= d ? make_uint4(0, 0, 0, 0) : p[j * T + i0];
}

// Eight values of Y: rounded to 16 bits, or as E4M3 codes of their block of 128, which sixteen lanes hold
// (all 32 lanes of the warp call; those past the row's end with zeros and in = false).
template <bool BF16, bool E4M3>
__device__ __forceinline__ void store_y(const LayernormArgs& a, long long r, int c, bool in, const float (&y)[8])
{
    if constexpr (!E4M3) {
        if (in) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.Y) + r * a.d + c) = encode8<BF16>(y);
    } else {
        float scale, inv;
        block_scale(__uint_as_float(half_warp_max(in ? abs_max8(y) : 0u)), scale, inv);
        if (!in) return;
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.Y) + r * a.d + c) = e4m3_codes8(y, inv);
        if ((threadIdx.x & 15) == 0) a.scale[static_cast<long long>(c / 128) * a.t + r] = scale;
    }
}

// A row from memory, where H (X without a residual) stands as the same threads stored it, times `factor`
// (a far row's, or 1: a row too long for registers).  Returns the factor that the row needs instead, or 0.
template <bool BF16, int T, bool E4M3>
__device__ __forceinline__ float row_from_memory(const LayernormArgs& a, long long r, float factor, float (&part)[16],
                                                 float2 (&part2)[16])
{
    if constexpr (T > 32) __syncthreads();  // (part and part2 have been read)
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    const uint16_t* beta = static_cast<const uint16_t*>(a.beta);
    const uint16_t* h = static_cast<const uint16_t*>(a.residual ? a.H : a.X) + r * a.d;
    const int i0 = threadIdx.x % T;
    const float inv_d = 1.0f / static_cast<float>(a.d);
    float s = 0.0f;
#pragma unroll 1
    for (int c = i0 * 8; c < a.d; c += T * 8) {
        float x[8];
        decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(x[e], factor, s);
    }
    s = row_sum<T>(s, part);
    const float m0 = s * inv_d;
    float2 dev = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int c = i0 * 8; c < a.d; c += T * 8) {
        float x[8];
        decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = fmaf(x[e], factor, -m0);
            dev.x += u;
            dev.y = fmaf(u, u, dev.y);
        }
    }
    dev = row_sum2<T>(dev, part2);
    if (BF16 && factor == 1.0f) {
        const float other = far_factor(s, dev.y, m0, a.eps);
        if (other != 0.0f) return other;
    }
    const float more = dev.x * inv_d, var = variance(dev, inv_d);
    // rstd of the row times `factor`; where a large row's own variance fits fp32 (a constant row: eps
    // stands beside it) rstd of the row itself, for deviations times `back`.
    const bool own = factor < 1.0f && var < 1.355252716e-20f;  // 2^-66
    const float back = own ? 1.0f / factor : 1.0f;
    const float rstd = 1.0f / sqrtf(own ? fmaf(var * back, back, a.eps) : var + a.eps * factor * factor);
    if (i0 == 0 && a.stats) {
        a.stats[2 * r] = (m0 + more) / factor;
        a.stats[2 * r + 1] = own ? rstd : rstd * factor;
    }
    // (whole warps: sixteen lanes have a block of 128 columns)
#pragma unroll 1
    for (int c = i0 * 8; c - i0 % 32 * 8 < a.d; c += T * 8) {
        const bool in = c < a.d;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8], b[8];
        if (in) {
            decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), x);
            decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
            decode8<BF16>(*reinterpret_cast<const uint4*>(beta + c), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf((fmaf(x[e], factor, -m0) - more) * back * rstd, g[e], b[e]);
        }
        store_y<BF16, E4M3>(a, r, c, in, x);
    }
    return 0.0f;
}

// Blocks an SM (at least): what keeps enough loads on their way.  gamma and beta are read where they are used, from L1
// and L2: held in registers from the start they left two blocks of 256 threads an SM (16384 x 8192 to E4M3: 200 us;
// three blocks so 156, four 154, five 141).  2039 x 4096 to 16 bits: 8.1 us with 8, 8.5 with 6, 9.5 with 10.
template <int T, int V>
constexpr int ln_blocks()
{
    return T == 512 ? 2 : T == 256 ? 5 : V == 4 ? 8 : V == 2 ? 10 : 12;
}

template <bool BF16, int T, int V, bool E4M3>
__global__ void __launch_bounds__(ln_block<T>(), ln_blocks<T, V>()) layernorm_forward_kernel(const LayernormArgs a)
{
    constexpr int kRows = ln_block<T>() / T;
    __shared__ float part[16];
    __shared__ float2 part2[16];
    const int i0 = threadIdx.x % T;
    grid_dependency_wait();
    grid_launch_dependents();
    const long long r = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / T;
    if (r >= a.t) return;  // (T = 32: a whole warp, and no barrier below)
    uint4 h[V];
    load_row<T, V>(a.X, r, a.d, h);
    if (a.residual) {
        uint4 res[V];
        load_row<T, V>(a.residual, r, a.d, res);
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
    const float inv_d = 1.0f / static_cast<float>(a.d);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        float x[8];
        decode8<BF16>(h[j], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += x[e];
    }
    s = row_sum<T>(s, part);
    const float m0 = s * inv_d;
    float2 dev = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        if ((j * T + i0) * 8 >= a.d) continue;
        float x[8];
        decode8<BF16>(h[j], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = x[e] - m0;
            dev.x += u;
            dev.y = fmaf(u, u, dev.y);
        }
    }
    dev = row_sum2<T>(dev, part2);
    const float factor = BF16 ? far_factor(s, dev.y, m0, a.eps) : 0.0f;  // (the same in all of the row's threads)
    if (factor != 0.0f) {
        row_from_memory<BF16, T, E4M3>(a, r, factor, part, part2);
        return;
    }
    const float more = dev.x * inv_d, rstd = 1.0f / sqrtf(variance(dev, inv_d) + a.eps);
    if (i0 == 0 && a.stats) *reinterpret_cast<float2*>(a.stats + 2 * r) = make_float2(m0 + more, rstd);
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int c = (j * T + i0) * 8;
        uint4 gamma = make_uint4(0, 0, 0, 0), beta = gamma;
        if (c < a.d) {
            gamma = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.gamma) + c);
            beta = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.beta) + c);
        }
        float x[8], g[8], b[8];
        decode8<BF16>(h[j], x);
        decode8<BF16>(gamma, g);
        decode8<BF16>(beta, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf((x[e] - m0 - more) * rstd, g[e], b[e]);
        store_y<BF16, E4M3>(a, r, c, c < a.d, x);
    }
}

// Rows that do not fit registers, read again from L1 and L2 for each pass.
template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kLongThreads) layernorm_long_kernel(const LayernormArgs a)
{
    __shared__ float part[16];
    __shared__ float2 part2[16];
    grid_dependency_wait();
    grid_launch_dependents();
    const long long r = blockIdx.x;
    if (a.residual) {
        const uint16_t* x = static_cast<const uint16_t*>(a.X) + r * a.d;
        const uint16_t* res = static_cast<const uint16_t*>(a.residual) + r * a.d;
        uint16_t* out = static_cast<uint16_t*>(a.H) + r * a.d;
        for (int c = threadIdx.x * 8; c < a.d; c += kLongThreads * 8) {
            float v[8], w[8];
            decode8<BF16>(*reinterpret_cast<const uint4*>(x + c), v);
            decode8<BF16>(*reinterpret_cast<const uint4*>(res + c), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
            *reinterpret_cast<uint4*>(out + c) = encode8<BF16>(v);
        }
    }
    const float factor = row_from_memory<BF16, kLongThreads, E4M3>(a, r, 1.0f, part, part2);
    if (factor != 0.0f) row_from_memory<BF16, kLongThreads, E4M3>(a, r, factor, part, part2);
}

// ---- backward ------------------------------------------------------------------------------
// A block walks rows and keeps the sums of dgamma and dbeta of its rows in registers, every column with
// one thread (T = 32: one per warp, added in order at the end), and writes them to its row of the
// workspace; layernorm_sums_kernel adds those.  (Added up over a cluster of two to eight blocks first they
// cost more than the rows saved: 8192 x 4096 46 us without, 46 to 68 so.)  The next row is copied to shared
// memory while this one is worked on, every thread copying the vectors that it reads itself, so that the
// copies need no barrier.  16384 x 8192 in bf16 with dH: 165.8 us, 1074 MB at 6.5 TB/s (a copy's rate is 6.7);
// 333 x 1000 in f16 with dH: 6.1 us, the latency of the two launches.

// (h - mu) rstd, where h - mu may leave fp32: both are halved for rows of that size.
struct RowStats {
    float half, mean, rstd, rstd_half;
    __device__ __forceinline__ explicit RowStats(float2 s)
    {
        half = s.y < 7.888609052210118e-31f ? 0.5f : 1.0f;  // 2^-100
        mean = s.x * half;
        rstd = s.y;
        rstd_half = s.y / half;
    }
    __device__ __forceinline__ float xh(float h) const { return fmaf(h, half, -mean) * rstd_half; }
};

template <int T, int V>
__host__ __device__ constexpr int ln_backward_smem()
{
    return 2 * 3 * V * ln_block<T>() * 16;
}

// (As many registers as a block can have, but for the two blocks an SM of 8192 columns: 8192 x 4096 46 us, 59 with the
// compiler's 80; 16384 x 8192 165 us with two blocks, 174 with one.)
template <bool BF16, int T, int V>
__global__ void __launch_bounds__(ln_block<T>(), T == 256 && V == 4 ? 2 : 1)
    layernorm_backward_kernel(const LayernormBackwardArgs a)
{
    constexpr int kBlock = ln_block<T>(), kRows = kBlock / T;
    extern __shared__ __align__(16) uint4 buf[];  // [2][dY, H, dH][V][thread]
    __shared__ float2 part[2][16];
    const int i0 = threadIdx.x % T;
    grid_dependency_wait();
    grid_launch_dependents();
    const float2* stats = reinterpret_cast<const float2*>(a.stats);
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
    float2 now = make_float2(0.0f, 0.0f);
    if (r < a.t) {
        fetch(r, 0);
        now = stats[r];
    }
    cp_async_commit();
    uint4 gamma[V];
    load_row<T, V>(a.gamma, 0, a.d, gamma);
    const float inv_d = 1.0f / static_cast<float>(a.d);
    float dg[V][8], db[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dg[j][e] = db[j][e] = 0.0f;
    int parity = 0;
    for (; r < a.t; r += step, parity ^= 1) {
        float2 next = make_float2(0.0f, 0.0f);
        if (r + step < a.t) {
            fetch(r + step, parity ^ 1);
            next = stats[r + step];
        }
        cp_async_commit();
        cp_async_wait_group<1>();
        const uint4* row = buf + parity * 3 * V * kBlock + threadIdx.x;
        const RowStats st(now);
        float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
            float y[8], x[8], g[8];
            decode8<BF16>(row[j * kBlock], y);
            decode8<BF16>(row[(V + j) * kBlock], x);
            decode8<BF16>(gamma[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = st.xh(x[e]);
                const float yg = y[e] * g[e];
                s.x += yg;
                s.y = fmaf(yg, xh, s.y);
                dg[j][e] = fmaf(y[e], xh, dg[j][e]);
                db[j][e] += y[e];
            }
        }
        s = row_sum2<T>(s, part[parity]);
        const float mean_g = s.x * inv_d, mean_gx = s.y * inv_d;
        uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dX) + r * a.d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
            float y[8], x[8], g[8];
            decode8<BF16>(row[j * kBlock], y);
            decode8<BF16>(row[(V + j) * kBlock], x);
            decode8<BF16>(gamma[j], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = st.rstd * (fmaf(y[e], g[e], -mean_g) - st.xh(x[e]) * mean_gx);
            if (a.dH) {
                float z[8];
                decode8<BF16>(row[(2 * V + j) * kBlock], z);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += z[e];
            }
            out[j * T + i0] = encode8<BF16>(y);
        }
        now = next;
    }
    float4* out = reinterpret_cast<float4*>(a.ws_sums) + blockIdx.x * 2ll * (a.d / 4);  // [dgamma, dbeta][d / 4]
    auto place = [&](int j, int q) { return (q >> 1) * (a.d / 4) + (j * T + i0) * 2 + (q & 1); };
    auto value = [&](int j, int q) {  // of dgamma's eight columns, then of dbeta's
        const float* v = q < 2 ? dg[j] + 4 * q : db[j] + 4 * (q - 2);
        return make_float4(v[0], v[1], v[2], v[3]);
    };
    if constexpr (kRows > 1) {
        float4* sums = reinterpret_cast<float4*>(buf);
        cp_async_wait_group<0>();
        for (int w = 0; w < kRows; ++w) {
            __syncthreads();
            if (static_cast<int>(threadIdx.x) / T != w) continue;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if ((j * T + i0) * 8 >= a.d) continue;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 v = value(j, q);
                    float4& at = sums[place(j, q)];
                    at = w == 0 ? v : make_float4(at.x + v.x, at.y + v.y, at.z + v.z, at.w + v.w);
                }
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < a.d / 2; i += kBlock) out[i] = sums[i];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if ((j * T + i0) * 8 >= a.d) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) out[place(j, q)] = value(j, q);
        }
    }
}

// Rows longer than that, in two passes: the means of g and g xh of every row (a block per row), then dX
// and the sums by columns, a block with 2048 columns of rows y, y + slices, ..., each column with one thread.
template <bool BF16>
__global__ void __launch_bounds__(kLongThreads) layernorm_backward_means_kernel(const LayernormBackwardArgs a)
{
    __shared__ float2 part[16];
    grid_dependency_wait();
    grid_launch_dependents();
    const long long r = blockIdx.x;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dY) + r * a.d;
    const uint16_t* h = static_cast<const uint16_t*>(a.H) + r * a.d;
    const uint16_t* gamma = static_cast<const uint16_t*>(a.gamma);
    const RowStats st(reinterpret_cast<const float2*>(a.stats)[r]);
    float2 s = make_float2(0.0f, 0.0f);
    for (int c = threadIdx.x * 8; c < a.d; c += kLongThreads * 8) {
        float y[8], x[8], g[8];
        decode8<BF16>(*reinterpret_cast<const uint4*>(dy + c), y);
        decode8<BF16>(*reinterpret_cast<const uint4*>(h + c), x);
        decode8<BF16>(*reinterpret_cast<const uint4*>(gamma + c), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float yg = y[e] * g[e];
            s.x += yg;
            s.y = fmaf(yg, st.xh(x[e]), s.y);
        }
    }
    s = row_sum2<kLongThreads>(s, part);
    if (threadIdx.x == 0)
        reinterpret_cast<float2*>(a.ws_means)[r] =
            make_float2(s.x / static_cast<float>(a.d), s.y / static_cast<float>(a.d));
}

template <bool BF16>
__global__ void __launch_bounds__(kLongThreads) layernorm_backward_columns_kernel(const LayernormBackwardArgs a, int slices)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int slice = blockIdx.x % slices;
    const int c = (blockIdx.x / slices * kLongThreads + threadIdx.x) * 8;
    if (c >= a.d) return;
    float g[8], dg[8] = {0, 0, 0, 0, 0, 0, 0, 0}, db[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.gamma) + c), g);
#pragma unroll 2
    for (long long r = slice; r < a.t; r += slices) {
        const long long at = r * a.d + c;
        const RowStats st(reinterpret_cast<const float2*>(a.stats)[r]);
        const float2 mean = reinterpret_cast<const float2*>(a.ws_means)[r];
        float y[8], x[8], z[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dY) + at), y);
        decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.H) + at), x);
        if (a.dH) decode8<BF16>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.dH) + at), z);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float xh = st.xh(x[e]);
            dg[e] = fmaf(y[e], xh, dg[e]);
            db[e] += y[e];
            y[e] = st.rstd * (fmaf(y[e], g[e], -mean.x) - xh * mean.y);
            if (a.dH) y[e] += z[e];
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dX) + at) = encode8<BF16>(y);
    }
    float* sums = a.ws_sums + slice * 2ll * a.d + c;
    reinterpret_cast<float4*>(sums)[0] = make_float4(dg[0], dg[1], dg[2], dg[3]);
    reinterpret_cast<float4*>(sums)[1] = make_float4(dg[4], dg[5], dg[6], dg[7]);
    reinterpret_cast<float4*>(sums + a.d)[0] = make_float4(db[0], db[1], db[2], db[3]);
    reinterpret_cast<float4*>(sums + a.d)[1] = make_float4(db[4], db[5], db[6], db[7]);
}

// Sums of `parts` rows of 2 d values, in an order that depends on parts alone: a block takes 32 columns,
// its warp w rows w, w + WARPS, ..., and the warps' sums meet in order; the first d are dgamma.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 64 / WARPS) layernorm_sums_kernel(const float* ws, int parts, int d,
                                                                                float* dgamma, float* dbeta)
{
    constexpr int kAtOnce = WARPS == 32 ? 12 : 16;
    __shared__ float sum[WARPS][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long width = 2ll * d;
    const long long c = blockIdx.x * 32ll + lane;
    grid_dependency_wait();
    grid_launch_dependents();
    auto store = [&](long long at, float s) {
        if (at < d)
            dgamma[at] = s;
        else if (at < width)
            dbeta[at - d] = s;
    };
    float s = 0.0f;
    if (c < width) {
        for (int p = w; p < parts; p += WARPS * kAtOnce) {
            float v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) v[i] = ws[min(p + i * WARPS, parts - 1) * width + c];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) s += p + i * WARPS < parts ? v[i] : 0.0f;
        }
    }
    sum[w][lane] = s;
    __syncthreads();
    if constexpr (WARPS == 32) {
        s = sum[lane][w];  // one warp per column now: its 32 partial sums
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) store(blockIdx.x * 32ll + w, s);
    } else if (w == 0) {
#pragma unroll
        for (int i = 1; i < WARPS; ++i) s += sum[i][lane];
        store(c, s);
    }
}

// Blocks for `rows` rows, `per_block` at a time, at most `cap`, all with the same number of rounds.
int even_grid(long long rows, int per_block, long long cap)
{
    const long long blocks = (rows + per_block - 1) / per_block;
    const long long rounds = blocks > cap ? (blocks + cap - 1) / cap : 1;
    return static_cast<int>((blocks + rounds - 1) / rounds);
}

template <bool BF16, int T, int V>
cudaError_t forward_width(const LayernormArgs& a, cudaStream_t stream)
{
    constexpr int kRows = ln_block<T>() / T;
    const int grid = static_cast<int>((static_cast<long long>(a.t) + kRows - 1) / kRows);
    return a.scale ? launch_dependent(layernorm_forward_kernel<BF16, T, V, true>, grid, ln_block<T>(), 0, stream, 1, a)
                   : launch_dependent(layernorm_forward_kernel<BF16, T, V, false>, grid, ln_block<T>(), 0, stream, 1, a);
}

template <bool BF16>
cudaError_t forward_type(const LayernormArgs& a, cudaStream_t stream)
{
    if (a.d <= 256) return forward_width<BF16, 32, 1>(a, stream);
    if (a.d <= 512) return forward_width<BF16, 32, 2>(a, stream);
    if (a.d <= 1024) return forward_width<BF16, 32, 4>(a, stream);
    if (a.d <= 2048) return forward_width<BF16, 128, 2>(a, stream);
    if (a.d <= 4096) return forward_width<BF16, 128, 4>(a, stream);
    if (a.d <= 8192) return forward_width<BF16, 256, 4>(a, stream);
    if (a.d <= kMaxWidth) return forward_width<BF16, 512, 4>(a, stream);
    return a.scale ? launch_dependent(layernorm_long_kernel<BF16, true>, a.t, kLongThreads, 0, stream, 1, a)
                   : launch_dependent(layernorm_long_kernel<BF16, false>, a.t, kLongThreads, 0, stream, 1, a);
}

// Width class of the backward kernel: its rows per block and most blocks (what fits on 152 SMs at once;
// each block's sums are a row of the workspace).
struct BackwardShape {
    int rows, cap;
};

BackwardShape backward_shape(long long t, long long d)
{
    // (most blocks, measured: 8192 x 1024 18.1 us with 912, 18.9 with 608; 8192 x 2048 27.9 with 760, 29.5 with 608, 33.8
    // with 456; 8192 x 4096 46 with 304, 51 with 608, 56 with 456: more than are there at once make a second wave)
    if (d <= 512) return t <= 2048 ? BackwardShape{1, 456} : BackwardShape{4, 456};
    if (d <= 1024) return {1, t <= 2048 ? 456 : 912};
    if (d <= 2048) return {1, 760};
    if (d <= 8192) return {1, 304};
    if (d <= kMaxWidth) return {1, 152};
    return {1, static_cast<int>(kMaxWidth * 64 / d) + 1};  // (times d / 2048 blocks)
}

template <bool BF16, int T, int V>
cudaError_t backward_width(const LayernormBackwardArgs& a, int parts, cudaStream_t stream)
{
    auto kernel = layernorm_backward_kernel<BF16, T, V>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, ln_backward_smem<T, V>(), prepared);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, parts, ln_block<T>(), ln_backward_smem<T, V>(), stream, 1, a);
}

template <bool BF16>
cudaError_t backward_type(const LayernormBackwardArgs& a, int parts, cudaStream_t stream)
{
    if (a.d <= 1024 && (a.d > 512 || a.t <= 2048)) return backward_width<BF16, 128, 1>(a, parts, stream);
    if (a.d <= 256) return backward_width<BF16, 32, 1>(a, parts, stream);
    if (a.d <= 512) return backward_width<BF16, 32, 2>(a, parts, stream);
    if (a.d <= 2048) return backward_width<BF16, 128, 2>(a, parts, stream);
    if (a.d <= 4096) return backward_width<BF16, 256, 2>(a, parts, stream);
    if (a.d <= 8192) return backward_width<BF16, 256, 4>(a, parts, stream);
    if (a.d <= kMaxWidth) return backward_width<BF16, 512, 4>(a, parts, stream);
    const cudaError_t e = launch_dependent(layernorm_backward_means_kernel<BF16>, a.t, kLongThreads, 0, stream, 1, a);
    if (e != cudaSuccess) return e;
    const int columns = (a.d + kLongThreads * 8 - 1) / (kLongThreads * 8);
    return launch_dependent(layernorm_backward_columns_kernel<BF16>, columns * parts, kLongThreads, 0, stream, 1, a, parts);
}

}  // namespace

int layernorm_backward_parts(long long t, long long d)
{
    const BackwardShape s = backward_shape(t, d);
    return even_grid(t, s.rows, s.cap);
}

cudaError_t layernorm_forward_launch(const LayernormArgs& a, bool bf16, cudaStream_t stream)
{
    return bf16 ? forward_type<true>(a, stream) : forward_type<false>(a, stream);
}

cudaError_t layernorm_backward_launch(const LayernormBackwardArgs& a, bool bf16, cudaStream_t stream)
{
    const int parts = layernorm_backward_parts(a.t, a.d);
    const cudaError_t e = bf16 ? backward_type<true>(a, parts, stream) : backward_type<false>(a, parts, stream);
    if (e != cudaSuccess) return e;
    const float* ws = a.ws_sums;
    const int grid = static_cast<int>((2ll * a.d + 31) / 32);
    return parts > 128 ? launch_dependent(layernorm_sums_kernel<32>, grid, 1024, 0, stream, 1, ws, parts, a.d, a.dgamma, a.dbeta)
                       : launch_dependent(layernorm_sums_kernel<8>, grid, 256, 0, stream, 1, ws, parts, a.d, a.dgamma, a.dbeta);
}

}  // namespace gemm_epi
