// Products with 4-bit weights and group scales for a few rows of A, with the GEMM epilogs,
// and the weight written out as the 16-bit B of a plan.
//
// The product, D^T = W A^T, streams the weight once: W's rows (columns of D) are the 16 MMA
// rows of mma.m16n8k16, rows of A its 8 columns, so even one row of A uses the tensor cores
// and every weight is unpacked once for up to 64 rows.  For a few rows that is 4 bits of
// traffic per 2 m flops, bound by the weight's bytes.
//
//   * A block takes 16 MT CW columns of D and all of k, in stages of 128 KW values of k
//     (CW KW = 8 warps): the stage's weights, rows of A, scales and zero points are copied
//     with cp.async into a ring, each byte by one thread.
//   * Warp (cw, kw) multiplies its 16 MT columns by its 128 values of k.  In a row's 64 bytes
//     of those, chunk i (16 bytes) holds k = 32 i .. 32 i + 31, and ldmatrix hands word t of
//     row r to lane 4 r + t: eight values of k for MMA row r.  A word's halves-apart nibbles
//     (j, j + 4) become a register pair of 16-bit values by one shift and one and-or with the
//     bits of 128 (bf16) or 1024 (f16), whose last mantissa bit is 1; subtracting 128 + z
//     (1024 + z) leaves q - z, exactly.  The rows of A are paired in the same order (the order
//     of k inside an MMA is free as long as both operands have it).
//   * A group's sum is complete in the accumulator (groups are whole MMAs, all of whose lanes
//     are in one group), so the scale multiplies an fp32 sum, and no weight is ever rounded.
//   * The KW warps' sums meet in shared memory, in order; then the epilogue.
#include "gelu.cuh"
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

constexpr int kWarps = 8;
constexpr int kBlockK = 128;  // values of k per warp and stage: 64 bytes of each row of W

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

// 16 bytes to shared memory, or zeros where `live` is false (src must be readable either way).
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_async_8_or_zero(uint32_t dst, const void* src, bool live)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8 : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait_group()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                     "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                     "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 16-bit type's bits of 128 (bf16) or 1024 (f16), in both halves.
template <bool BF16>
__device__ constexpr uint32_t w4_magic()
{
    return BF16 ? 0x43004300u : 0x64006400u;
}

// q - z of nibbles (j, j + 4) of a word as a register pair; zoff = magic + z in both halves.
template <bool BF16, int J>
__device__ __forceinline__ uint32_t w4_pair(uint32_t w, uint32_t zoff)
{
    const uint32_t v = ((w >> (4 * J)) & 0x000F000Fu) | w4_magic<BF16>();
    if constexpr (BF16) {
        const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                         *reinterpret_cast<const __nv_bfloat162*>(&zoff));
        return *reinterpret_cast<const uint32_t*>(&d);
    }
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&zoff));
    return *reinterpret_cast<const uint32_t*>(&d);
}

// Shared-memory layout of one stage, in bytes, for m rows of A.
template <int MT, int CW, int G>
struct W4Stage {
    static constexpr int kKW = kWarps / CW;
    static constexpr int kCols = 16 * MT * CW;
    static constexpr int kStageK = kBlockK * kKW;
    static constexpr int kGroups = kStageK / G;
    static constexpr int kW = kCols * kKW * 64;           // [kw][column][64 bytes], chunks swizzled
    static constexpr int kScales = kGroups * kCols * 2;   // [group][column]
    static constexpr int kZeros = kGroups * kCols;        // [group][column]
    static constexpr int kARow = kStageK * 2 + 64;        // a row of A, padded by half a bank cycle
    static constexpr int kA = kW + kScales + kZeros;
    static __host__ __device__ int bytes(int m) { return kA + m * kARow; }
};

constexpr int kMaxStages = 6;

template <bool BF16, int NT, int MT, int CW, int G>
__global__ void __launch_bounds__(kWarps * 32) w4_matmul_kernel(const W4Args a, int stages)
{
    using S = W4Stage<MT, CW, G>;
    constexpr int KW = S::kKW;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cw = warp % CW, kw = warp / CW;
    const int n0 = blockIdx.x * S::kCols;
    const int stage_bytes = S::bytes(a.m);
    const int steps = (a.k + S::kStageK - 1) / S::kStageK;

    grid_dependency_wait();
    grid_launch_dependents();

    const uint8_t* W = static_cast<const uint8_t*>(a.W);
    const uint16_t* A = static_cast<const uint16_t*>(a.A);
    const uint16_t* scales = static_cast<const uint16_t*>(a.scales);
    auto load = [&](int step) {
        const uint32_t st = sbase + (step % stages) * stage_bytes;
        const int k0 = step * S::kStageK;
        // weights: chunk = 16 bytes = 32 values of k
        constexpr int kRowChunks = KW * 4;
        for (int i = tid; i < S::kCols * kRowChunks; i += kWarps * 32) {
            const int col = i / kRowChunks, c = i % kRowChunks;
            const int k = k0 + c * 32;
            const bool live = n0 + col < a.n && k < a.k;
            const uint8_t* src = live ? W + (static_cast<long long>(n0 + col) * a.k + k) / 2 : W;
            const uint32_t dst = st + ((c / 4) * S::kCols + col) * 64 + (((c & 3) ^ ((col >> 1) & 3)) << 4);
            cp_async_16_or_zero(dst, src, live);
        }
        // rows of A: chunk = 8 values
        constexpr int kAChunks = S::kStageK / 8;
        for (int i = tid; i < a.m * kAChunks; i += kWarps * 32) {
            const int row = i / kAChunks, c = i % kAChunks;
            const int k = k0 + c * 8;
            const bool live = k < a.k;
            const uint16_t* src = live ? A + static_cast<long long>(row) * a.k + k : A;
            cp_async_16_or_zero(st + S::kA + row * S::kARow + c * 16, src, live);
        }
        // scales and zero points: 8 columns each
        for (int i = tid; i < S::kGroups * (S::kCols / 8); i += kWarps * 32) {
            const int g = i / (S::kCols / 8), c = i % (S::kCols / 8) * 8;
            const bool live = n0 + c < a.n && k0 + g * G < a.k;
            const long long at = live ? static_cast<long long>(k0 / G + g) * a.n + n0 + c : 0;
            cp_async_16_or_zero(st + S::kW + (g * S::kCols + c) * 2, scales + at, live);
            if (a.zeros) cp_async_8_or_zero(st + S::kW + S::kScales + g * S::kCols + c, a.zeros + at, live);
        }
    };

    float total[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) total[i][j][c] = 0.0f;

    for (int s = 0; s < stages - 1; ++s) {
        if (s < steps) load(s);
        cp_async_commit();
    }
    const int r = lane >> 2, t = lane & 3;
    for (int step = 0; step < steps; ++step) {
        // this step's copies (of this thread, then of all) have landed, and every warp is done
        // with the stage that the next load overwrites
        switch (stages) {
        case 2: cp_async_wait_group<0>(); break;
        case 3: cp_async_wait_group<1>(); break;
        case 4: cp_async_wait_group<2>(); break;
        case 5: cp_async_wait_group<3>(); break;
        default: cp_async_wait_group<4>(); break;
        }
        __syncthreads();
        if (step + stages - 1 < steps) load(step + stages - 1);
        cp_async_commit();
        const uint32_t st = sbase + (step % stages) * stage_bytes;
        const uint8_t* stp = smem + (step % stages) * stage_bytes;
        // this warp's weights: chunk i of row (lane & 7) [+ 8] for ldmatrix
        uint32_t w[MT][2][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = (cw * MT + i) * 16 + h * 8 + (lane & 7);
                ldmatrix_x4(w[i][h], st + (kw * S::kCols + col) * 64 + (((lane >> 3) ^ ((col >> 1) & 3)) << 4));
            }
        float part[MT][NT][4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int g = kw * (kBlockK / G) + c * 32 / G;  // group within the stage
            if (c * 32 % G == 0) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) part[i][j][e] = 0.0f;
            }
            // rows of A: 8 values of k per lane, paired (k, k + 4)
            uint32_t b[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int row = min(j * 8 + r, a.m - 1);  // (rows past m: columns nobody reads)
                const uint4 v = *reinterpret_cast<const uint4*>(stp + S::kA + row * S::kARow + kw * 256 + c * 64 + t * 16);
                b[j][0] = __byte_perm(v.x, v.z, 0x5410);
                b[j][1] = __byte_perm(v.x, v.z, 0x7632);
                b[j][2] = __byte_perm(v.y, v.w, 0x5410);
                b[j][3] = __byte_perm(v.y, v.w, 0x7632);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int col = (cw * MT + i) * 16 + r;
                uint32_t z0 = 8, z1 = 8;
                if (a.zeros) {
                    const uint8_t* zp = stp + S::kW + S::kScales + g * S::kCols + col;
                    z0 = zp[0];
                    z1 = zp[8];
                }
                z0 = z0 * 0x10001u + w4_magic<BF16>();
                z1 = z1 * 0x10001u + w4_magic<BF16>();
                const uint32_t lo = w[i][0][c], hi = w[i][1][c];
                const uint32_t p0 = w4_pair<BF16, 0>(lo, z0), p1 = w4_pair<BF16, 1>(lo, z0);
                const uint32_t p2 = w4_pair<BF16, 2>(lo, z0), p3 = w4_pair<BF16, 3>(lo, z0);
                const uint32_t q0 = w4_pair<BF16, 0>(hi, z1), q1 = w4_pair<BF16, 1>(hi, z1);
                const uint32_t q2 = w4_pair<BF16, 2>(hi, z1), q3 = w4_pair<BF16, 3>(hi, z1);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma_16816<BF16>(part[i][j], p0, q0, p1, q1, b[j][0], b[j][1]);
                    mma_16816<BF16>(part[i][j], p2, q2, p3, q3, b[j][2], b[j][3]);
                }
                if ((c + 1) * 32 % G == 0) {
                    const uint16_t* sp = reinterpret_cast<const uint16_t*>(stp + S::kW) + g * S::kCols + col;
                    const float s0 = decode16<BF16>(sp[0]), s1 = decode16<BF16>(sp[8]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        total[i][j][0] = fmaf(part[i][j][0], s0, total[i][j][0]);
                        total[i][j][1] = fmaf(part[i][j][1], s0, total[i][j][1]);
                        total[i][j][2] = fmaf(part[i][j][2], s1, total[i][j][2]);
                        total[i][j][3] = fmaf(part[i][j][3], s1, total[i][j][3]);
                    }
                }
            }
        }
    }

    // The k-warps' sums: [kw][row of A][column], then one thread per element adds them in order.
    cp_async_wait_group<0>();
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    constexpr int kRedRow = S::kCols + 1;  // (odd: a warp's stores to 8 rows fall in 8 banks)
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = j * 8 + 2 * t + (e & 1);
                const int col = (cw * MT + i) * 16 + r + (e >> 1) * 8;
                red[(kw * NT * 8 + row) * kRedRow + col] = total[i][j][e];
            }
    __syncthreads();
    for (int i = tid; i < a.m * S::kCols; i += kWarps * 32) {
        const int row = i / S::kCols, col = i % S::kCols;
        if (n0 + col >= a.n) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < KW; ++q) v += red[(q * NT * 8 + row) * kRedRow + col];
        const long long at = static_cast<long long>(row) * a.n + n0 + col;
        if (a.bias) v += decode16<BF16>(static_cast<const uint16_t*>(a.bias)[n0 + col]);
        const float res = a.residual ? decode16<BF16>(static_cast<const uint16_t*>(a.residual)[at]) : 0.0f;
        static_cast<uint16_t*>(a.D)[at] = encode16<BF16>(w4_epilogue(v, a.epilog, res));
    }
}

template <bool BF16, int NT, int MT, int CW, int G>
cudaError_t w4_launch_one(const W4Args& a, cudaStream_t stream)
{
    using S = W4Stage<MT, CW, G>;
    constexpr int kMaxSmem = 227 * 1024;
    auto kernel = w4_matmul_kernel<BF16, NT, MT, CW, G>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, kMaxSmem, prepared);
    if (e != cudaSuccess) return e;
    const int steps = (a.k + S::kStageK - 1) / S::kStageK;
    int stages = steps + 1 < kMaxStages ? steps + 1 : kMaxStages;
    if (stages < 2) stages = 2;
    while (stages > 2 && stages * S::bytes(a.m) > 100 * 1024) --stages;
    int smem = stages * S::bytes(a.m);
    const int red = S::kKW * NT * 8 * (S::kCols + 1) * 4;
    if (smem < red) smem = red;
    return launch_dependent(kernel, (a.n + S::kCols - 1) / S::kCols, kWarps * 32, smem, stream, a, stages);
}

template <bool BF16, int NT, int MT, int CW>
cudaError_t w4_launch_group(const W4Args& a, cudaStream_t stream)
{
    if (a.group == 32) return w4_launch_one<BF16, NT, MT, CW, 32>(a, stream);
    if (a.group == 64) return w4_launch_one<BF16, NT, MT, CW, 64>(a, stream);
    return w4_launch_one<BF16, NT, MT, CW, 128>(a, stream);
}

template <bool BF16>
cudaError_t w4_launch_type(const W4Args& a, cudaStream_t stream)
{
    if (a.m <= 2) return w4_launch_group<BF16, 1, 1, 1>(a, stream);
    if (a.m <= 8) return w4_launch_group<BF16, 1, 1, 2>(a, stream);
    if (a.m <= 16) return w4_launch_group<BF16, 2, 1, 4>(a, stream);
    if (a.m <= 32) return w4_launch_group<BF16, 4, 2, 4>(a, stream);
    if (a.m <= 48) return w4_launch_group<BF16, 6, 2, 4>(a, stream);
    return w4_launch_group<BF16, 8, 2, 4>(a, stream);
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
    return bf16 ? w4_launch_type<true>(a, stream) : w4_launch_type<false>(a, stream);
}

cudaError_t w4_dequantize_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    (void)sm_count;
    const int grid = static_cast<int>(((a.n + 63) / 64) * static_cast<long long>((a.k + 63) / 64));
    return bf16 ? launch_dependent(w4_dequantize_kernel<true>, grid, 256, 0, stream, a)
                : launch_dependent(w4_dequantize_kernel<false>, grid, 256, 0, stream, a);
}

}  // namespace gemm_epi
