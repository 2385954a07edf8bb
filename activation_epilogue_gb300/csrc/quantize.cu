// E4M3 codes of a 16-bit matrix with a scale for each block of 1 x 128 or 128 x 128 values, row-major
// and / or transposed in one pass (the products' A and transposed B in every direction of training).
//
// Bound by the bytes: 2 read and 1 written per value and output.  16384 x 8192 both ways in 128 x 128 blocks
// 79.7 us, 537 MB at 6.7 TB/s, a copy's rate; 2039 x 4096 both ways in 1 x 128 blocks 9.2 us, 34 MB, of which
// 5 are the bytes and the rest a launch and a tile's two barriers.
//   * 1 x 128, row-major alone: sixteen lanes have a block, eight values each, and four rows at a time,
//     every load issued first; no shared memory and no barrier.
//   * everything else: a block of threads has a 128 x 128 tile in registers, a thread 8 rows x 8
//     columns of it, so that both the codes of a row (8 columns) and of a transposed row (8 rows) are
//     8 bytes of one thread.  Largest values are taken on the 16-bit patterns, two at once.  The
//     transposed codes pass through 16 KB of shared memory, in 8-byte chunks swizzled by the column, to
//     be written 128 bytes a column.
#include "e4m3_codes.cuh"
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"

namespace gemm_epi {

namespace {

constexpr int kRowsAtOnce = 4;  // 1 x 128 blocks: rows of a thread

// Largest |x| of eight values as a pair of 16-bit patterns.
__device__ __forceinline__ uint32_t abs_max2(const uint4& w)
{
    constexpr uint32_t m = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(w.x & m, w.y & m), __vmaxu2(w.z & m, w.w & m));
}

template <bool BF16>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const QuantizeArgs a)
{
    grid_dependency_wait();
    grid_launch_dependents();
    const int blocks = (a.cols + 127) / 128;
    const long long item = static_cast<long long>(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const long long r0 = item / blocks * kRowsAtOnce;
    const int b = static_cast<int>(item % blocks);
    const int c = b * 128 + (threadIdx.x & 15) * 8;
    const bool in = c < a.cols;
    uint4 w[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        w[i] = make_uint4(0, 0, 0, 0);
        if (in && r0 + i < a.rows)
            w[i] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.X) + (r0 + i) * a.cols + c);
    }
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
        const uint32_t m2 = abs_max2(w[i]);
        const uint32_t top = half_warp_max(max(m2 & 0xFFFFu, m2 >> 16));
        float scale, inv, x[8];
        block_scale(decode16<BF16>(top), scale, inv);
        if (r0 + i >= a.rows) continue;
        decode8<BF16>(w[i], x);
        if (in) *reinterpret_cast<uint2*>(a.Q + (r0 + i) * a.cols + c) = e4m3_codes8(x, inv);
        if ((threadIdx.x & 15) == 0) a.scale[static_cast<long long>(b) * a.rows + r0 + i] = scale;
    }
}

// (four blocks an SM: 16384 x 8192 both ways 92 us, 98 with three, 101 with five)
template <bool BF16, bool SQUARE>
__global__ void __launch_bounds__(256, 4) quantize_tile_kernel(const QuantizeArgs a)
{
    __shared__ uint2 codes[128 * 16];     // transposed: [column][chunk of 8 rows ^ (column / 8)]
    __shared__ uint4 column_max[8][16];   // [warp][8 columns as pairs]; SQUARE: the warps' maxima in .x of the first
    __shared__ float inv_t[128];
    grid_dependency_wait();
    grid_launch_dependents();
    const int blocks = (a.cols + 127) / 128;
    const int b = static_cast<int>(blockIdx.x % blocks);
    const long long tile = blockIdx.x / blocks;
    const long long r0 = tile * 128;
    const int warp = threadIdx.x >> 5;
    const int part = threadIdx.x & 15, rows8 = threadIdx.x >> 4;  // this thread's 8 columns, its 8 rows
    const int c = b * 128 + part * 8;
    const bool in = c < a.cols;
    uint4 w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long r = r0 + rows8 * 8 + j;
        w[j] = make_uint4(0, 0, 0, 0);
        if (in && r < a.rows) w[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.X) + r * a.cols + c);
    }
    float square_inv = 0.0f;
    if constexpr (SQUARE) {
        uint32_t m2 = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m2 = __vmaxu2(m2, abs_max2(w[j]));
        uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(m2 & 0xFFFFu, m2 >> 16));
        if ((threadIdx.x & 31) == 0) column_max[0][warp].x = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, column_max[0][i].x);
        float scale;
        block_scale(decode16<BF16>(top), scale, square_inv);
        if (threadIdx.x == 0) {
            const long long row_tiles = (a.rows + 127) / 128;
            if (a.Q) a.scale[b * row_tiles + tile] = scale;
            if (a.Qt) a.scale_t[tile * blocks + b] = scale;
        }
    } else if (a.Qt) {
        constexpr uint32_t m = 0x7FFF7FFFu;
        uint4 t = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            t.x = __vmaxu2(t.x, w[j].x & m);
            t.y = __vmaxu2(t.y, w[j].y & m);
            t.z = __vmaxu2(t.z, w[j].z & m);
            t.w = __vmaxu2(t.w, w[j].w & m);
        }
        t.x = __vmaxu2(t.x, __shfl_xor_sync(0xFFFFFFFFu, t.x, 16));
        t.y = __vmaxu2(t.y, __shfl_xor_sync(0xFFFFFFFFu, t.y, 16));
        t.z = __vmaxu2(t.z, __shfl_xor_sync(0xFFFFFFFFu, t.z, 16));
        t.w = __vmaxu2(t.w, __shfl_xor_sync(0xFFFFFFFFu, t.w, 16));
        if ((threadIdx.x & 31) < 16) column_max[warp][part] = t;
        __syncthreads();
        if (threadIdx.x < 128) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max(top, static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(column_max[i])[threadIdx.x]));
            float scale, inv;
            block_scale(decode16<BF16>(top), scale, inv);
            inv_t[threadIdx.x] = inv;
            if (b * 128 + threadIdx.x < a.cols) a.scale_t[tile * a.cols + b * 128 + threadIdx.x] = scale;
        }
    }
    if (a.Q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long r = r0 + rows8 * 8 + j;
            float inv = square_inv;
            if constexpr (!SQUARE) {
                const uint32_t m2 = abs_max2(w[j]);
                float scale;
                block_scale(decode16<BF16>(half_warp_max(max(m2 & 0xFFFFu, m2 >> 16))), scale, inv);
                if (part == 0 && r < a.rows) a.scale[static_cast<long long>(b) * a.rows + r] = scale;
            }
            float x[8];
            decode8<BF16>(w[j], x);
            if (in && r < a.rows) *reinterpret_cast<uint2*>(a.Q + r * a.cols + c) = e4m3_codes8(x, inv);
        }
    }
    if (!a.Qt) return;
    if constexpr (!SQUARE) __syncthreads();
    const int rows_here = static_cast<int>(min(8ll, a.rows - r0 - rows8 * 8));
#pragma unroll
    for (int h = 0; h < 4; ++h) {  // two columns at once
        float lo[8], hi[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t word = h == 0 ? w[j].x : h == 1 ? w[j].y : h == 2 ? w[j].z : w[j].w;
            const float2 v = decode16x2<BF16>(word);
            lo[j] = v.x;
            hi[j] = v.y;
        }
        const int col = part * 8 + 2 * h;
        uint2 q[2] = {e4m3_codes8(lo, SQUARE ? square_inv : inv_t[col]),
                      e4m3_codes8(hi, SQUARE ? square_inv : inv_t[col + 1])};
        if (rows_here < 8) {  // (a NaN scale makes NaN codes of what pads the transposed rows)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                q[i].x &= rows_here >= 4 ? ~0u : rows_here <= 0 ? 0u : (1u << 8 * rows_here) - 1;
                q[i].y &= rows_here <= 4 ? 0u : (1u << 8 * (rows_here - 4)) - 1;
            }
        }
        codes[col * 16 + (rows8 ^ part)] = q[0];
        codes[(col + 1) * 16 + (rows8 ^ part)] = q[1];
    }
    __syncthreads();
    const long long ld = (a.rows + 15) / 16 * 16;
    const int chunk = threadIdx.x & 7;  // of 16 rows
    if (r0 + chunk * 16 >= ld) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int col = (threadIdx.x >> 3) + 32 * i;
        if (b * 128 + col >= a.cols) break;
        const int swap = col >> 3;
        uint4 q = *reinterpret_cast<const uint4*>(codes + col * 16 + ((2 * chunk ^ swap) & ~1));
        if (swap & 1) q = make_uint4(q.z, q.w, q.x, q.y);
        *reinterpret_cast<uint4*>(a.Qt + (b * 128 + col) * ld + r0 + chunk * 16) = q;
    }
}

}  // namespace

cudaError_t quantize_launch(const QuantizeArgs& a, bool bf16, cudaStream_t stream)
{
    const long long blocks = (a.cols + 127) / 128;
    if (!a.Qt && !a.square) {
        const long long items = (a.rows + kRowsAtOnce - 1) / kRowsAtOnce * blocks;
        const int grid = static_cast<int>((items + 15) / 16);
        return bf16 ? launch_dependent(quantize_rows_kernel<true>, grid, 256, 0, stream, 1, a)
                    : launch_dependent(quantize_rows_kernel<false>, grid, 256, 0, stream, 1, a);
    }
    const int grid = static_cast<int>((a.rows + 127) / 128 * blocks);
    if (a.square)
        return bf16 ? launch_dependent(quantize_tile_kernel<true, true>, grid, 256, 0, stream, 1, a)
                    : launch_dependent(quantize_tile_kernel<false, true>, grid, 256, 0, stream, 1, a);
    return bf16 ? launch_dependent(quantize_tile_kernel<true, false>, grid, 256, 0, stream, 1, a)
                : launch_dependent(quantize_tile_kernel<false, false>, grid, 256, 0, stream, 1, a);
}

}  // namespace gemm_epi
