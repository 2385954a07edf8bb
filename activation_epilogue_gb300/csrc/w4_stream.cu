// Products with a large 4-bit weight for up to 4 rows of A: the weight streams from memory straight
// to the registers of the warps that multiply it.
//
// D^T = W A^T with W's rows (columns of D) as the 16 MMA rows of mma.m16n8k16 and the rows of A as
// its 8 columns, as in the kernel that stages everything in shared memory (w4.cu).  Bound by the
// weight's bytes and, near them, by the instructions that unpack it; so what surrounds those is
// kept small:
//
//   * A block takes 8 to 32 columns of D, in groups of 8 spread evenly over blocks that are a
//     multiple of the SMs, and its eight warps every eighth 128 values of k.  A lane loads
//     its own words of its rows (one in each group) (16 or 8 bytes at a time: as much as keeps the lanes of an
//     MMA inside one group of the scales), three blocks of 128 k ahead, in registers; no barrier
//     and no copy through shared memory.  The order of k inside an MMA is free as long as both
//     operands have it.
//   * The rows of A, scales and zero points of a long stretch of k are put in shared memory once,
//     A in the order that the unpacked words come in (eight values of k as the pairs (j, j + 4)),
//     so that one 16-byte load serves two MMAs.
//   * A group's sum is complete in the accumulator, so the scale multiplies an fp32 sum, and
//     no weight is ever rounded.
//   * The warps' sums meet in shared memory in order, those of a cluster that splits k over
//     distributed shared memory; then the epilogue.
// Measured (bf16, groups of 128, one row; the staged kernel in brackets): 8192 columns, k 16384
// 17.2 us (22.7), 16384 x 8192 19.7 (23.4), 8192 x 8192 10.0 (12.4), 5120 x 5120 5.5 (8.0);
// 4096 x 1024 2.8 (2.3: its longer code and its first barrier cost a short call more).  For
// 8192 columns with k 16384 that is 59 % of the copy rate; the loads alone take 14.9 us (a kernel
// that only reads as many bytes in order: 14.3), the arithmetic alone 14.9.  Tried at 18.0 us, before
// the hint to L2: two steps loaded ahead 19.9, four (168 registers' worth in 128) 21.9; several
// blocks of 128 k in a row per warp, for longer pieces of a row of W, 18.9 to 19.1.
// A further row of A costs some 0.8 us at k 8192 and 1.5 at 16384: every block reads all of A from
// L2.  Blocks of twice the warps and columns, one an SM, halve that (4 rows, 8192 columns, k 16384:
// 23.0 -> 21.3 us), but a call no longer overlaps the end of the one before (one row: 16384 x 8192
// 20.0 -> 21.9, 5120 x 5120 5.5 -> 6.3), nor does loading A ahead of W's first words help (19.5).
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"
#include "w4_mma.cuh"
#include "w4_segment.h"
#include "w4_unpack.cuh"

namespace gemm_epi {

namespace {

constexpr int kWarps = kStreamWarps;
constexpr int kThreads = kWarps * 32;
constexpr int kCols = kStreamCols;
constexpr int kBlockK = kStreamBlockK;
constexpr int kStepK = kStreamStepK;
constexpr int kUnroll = kStreamUnroll;
constexpr int kAhead = kUnroll - 1;           // steps loaded ahead
constexpr int kMaxSmem = kStreamMaxSmem;

// Ask for `bytes` (a multiple of 16) from src (16-byte aligned) to be brought into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// Words (8 values of k) of a lane in a block of 128 k: word i of lane t holds k = k_of(t, i) ..
// + 7.  With groups of 128 a lane has 32 consecutive values, of 64 twice 16.
template <int G>
__device__ __forceinline__ int k_of(int t, int i)
{
    static_assert(G == 128 || G == 64, "groups");
    return G == 128 ? 32 * t + 8 * i : 64 * (i >> 1) + 16 * t + 8 * (i & 1);
}

// The four words of one row (src: the row's first byte of the block), zeros from `left` on.
template <int G>
__device__ __forceinline__ void load_words(const uint8_t* src, int t, int left, uint32_t (&w)[4])
{
    if constexpr (G == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + t * 16);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint2 v = make_uint2(0, 0);
            if (64 * h < left) v = *reinterpret_cast<const uint2*>(src + 32 * h + t * 8);
            w[2 * h] = v.x;
            w[2 * h + 1] = v.y;
        }
    }
}

// The sums of this block's share of k: NQ groups of 8 columns (MMA rows 0-7, 8-15 of one or two
// MMAs; the upper half of the last is zeros where NQ is odd).
template <bool BF16, int G, int NQ>
__device__ __forceinline__ void stream_columns(const W4Args& a, uint8_t* smem, int n0, int first, int steps,
                                               int seg_steps, float (&total)[2][4])
{
    using S = Segment<G>;
    constexpr int kMT = (NQ + 1) / 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, t = lane & 3;
    const int k0 = first * kStepK + warp * kBlockK;  // this warp's first
    const int mine = min(steps, (a.k - k0 + kStepK - 1) / kStepK);  // steps in which it has any

    const uint8_t* src[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
        src[q] = static_cast<const uint8_t*>(a.W) + (static_cast<long long>(n0 + q * 8 + r) * a.k + k0) / 2;
    int load_left = a.k - k0, loaded = 0;
    uint32_t w[kUnroll][NQ][4];
    auto load = [&](uint32_t (&to)[NQ][4]) {
        if (loaded < mine) {
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                load_words<G>(src[q], t, load_left, to[q]);
                src[q] += kStepK / 2;
            }
        }
        load_left -= kStepK;
        ++loaded;
    };

    // Ahead of the wait only L2 is asked for the first words of each row (a hint: what is written
    // until the wait ends is read after it).  From 8 steps on: 8192 x 8192 10.5 -> 10.0 us, 8192
    // columns with k 16384 18.1 -> 17.2, 16384 x 8192 20.6 -> 19.7; with 4 steps 11264 x 4096
    // 10.2 -> 10.7.  One step 17.4, six 17.9 (k 16384), all of a row 20.8.
    if (steps >= 8 && tid < NQ * 8)
        prefetch_l2_bulk(static_cast<const uint8_t*>(a.W) +
                             (static_cast<long long>(n0 + tid) * a.k + static_cast<long long>(first) * kStepK) / 2,
                         kAhead * kStepK / 2);
    grid_dependency_wait();
    grid_launch_dependents();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(w[u]);

    for (int seg = 0; seg < steps; seg += seg_steps) {
        const int count = min(seg_steps, steps - seg);
        const int kseg = (first + seg) * kStepK;
        const int pitch = S::pitch(count), o_scales = S::scales(a.m, count), o_zeros = S::zeros(a.m, count);
        if (seg > 0) __syncthreads();  // every warp is done with the segment before
        // scales and zero points: 8 columns of one group at a time
        const int groups = count * S::kGroups, g0 = kseg / G, g_end = a.k / G;
        for (int i = tid; i < groups * (kCols / 8); i += kThreads) {
            const int g = i / (kCols / 8), c = i % (kCols / 8) * 8;
            uint8_t* s_at = smem + o_scales + (g * kCols + c) * 2;
            if (g0 + g < g_end && c < NQ * 8) {
                const long long at = static_cast<long long>(g0 + g) * a.n + n0 + c;
                cp_async_16(smem_u32(s_at), static_cast<const uint16_t*>(a.scales) + at);
                if (a.zeros) cp_async_8(smem_u32(smem + o_zeros + g * kCols + c), a.zeros + at);
            } else {
                *reinterpret_cast<uint4*>(s_at) = make_uint4(0, 0, 0, 0);
            }
        }
        // rows of A: 8 values at a time, four loads in flight per thread
        const int chunks = count * (kStepK / 8);
        int row = 0, c = tid;
        while (c >= chunks) {
            c -= chunks;
            ++row;
        }
        while (row < a.m) {
            uint4 v[4];
            int to[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                to[j] = -1;
                v[j] = make_uint4(0, 0, 0, 0);  // (zeros past the end of k)
                if (row < a.m) {
                    to[j] = row * pitch + (G == 128 ? c ^ (c >> 3 & 1) : c) * 16;
                    if (kseg + c * 8 < a.k)
                        v[j] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.A) +
                                                               static_cast<long long>(row) * a.k + kseg + c * 8);
                }
                c += kThreads;
                while (c >= chunks) {
                    c -= chunks;
                    ++row;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (to[j] >= 0)
                    *reinterpret_cast<uint4*>(smem + to[j]) =
                        make_uint4(__byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                                   __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
        }
        cp_async_wait_all();
        __syncthreads();
        // (rows past m: columns of the product that nobody reads)
        const uint8_t* act = smem + min(r, a.m - 1) * pitch + warp * (kBlockK * 2);
        const uint8_t* sp = smem + o_scales + (warp * (kBlockK / G) * kCols + r) * 2;
        const uint8_t* zp = smem + o_zeros + warp * (kBlockK / G) * kCols + r;
        for (int s4 = seg; s4 < seg + count; s4 += kUnroll) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (s4 + u >= mine || s4 + u >= seg + count) break;
                load(w[(u + kAhead) % kUnroll]);
                float part[kMT][4];
                W4Unpack<BF16> unpack[kMT][2];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    constexpr int kWords = G / 32;  // of a lane in a group
                    const int g = i / kWords;
                    if (i % kWords == 0) {
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) {
                            unpack[mt][0].set(a.zeros ? zp[g * kCols + mt * 16] : 8u);
                            unpack[mt][1].set(a.zeros ? zp[g * kCols + mt * 16 + 8] : 8u);
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[mt][e] = 0.0f;
                        }
                    }
                    const int c = k_of<G>(t, i) / 8;
                    const uint4 b = *reinterpret_cast<const uint4*>(act + (G == 128 ? c ^ (c >> 3 & 1) : c) * 16);
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) {
                        uint32_t p[4], q[4] = {0, 0, 0, 0};
                        unpack[mt][0](w[u][2 * mt][i], p);
                        if constexpr (NQ % 2 == 0) {
                            unpack[mt][1](w[u][2 * mt + 1][i], q);
                        } else {
                            if (2 * mt + 1 < NQ) unpack[mt][1](w[u][2 * mt + 1 < NQ ? 2 * mt + 1 : 0][i], q);
                        }
                        mma_16816<BF16>(part[mt], p[0], q[0], p[1], q[1], b.x, b.y);
                        mma_16816<BF16>(part[mt], p[2], q[2], p[3], q[3], b.z, b.w);
                    }
                    if ((i + 1) % kWords == 0) {
#pragma unroll
                        for (int mt = 0; mt < kMT; ++mt) {
                            const uint16_t* s16 = reinterpret_cast<const uint16_t*>(sp) + g * kCols + mt * 16;
                            const float s0 = decode16<BF16>(s16[0]), s1 = decode16<BF16>(s16[8]);
                            total[mt][0] = fmaf(part[mt][0], s0, total[mt][0]);
                            total[mt][1] = fmaf(part[mt][1], s0, total[mt][1]);
                            total[mt][2] = fmaf(part[mt][2], s1, total[mt][2]);
                            total[mt][3] = fmaf(part[mt][3], s1, total[mt][3]);
                        }
                    }
                }
                act += kStepK * 2;
                sp += S::kGroups * kCols * 2;
                zp += S::kGroups * kCols;
            }
        }
    }
}

template <bool BF16, int G>
__global__ void __launch_bounds__(kThreads, 2) w4_stream_kernel(const W4Args a, int cluster, int seg_steps)
{
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = lane >> 2, t = lane & 3;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    // this block's columns: the n / 8 groups of 8 spread evenly over the blocks, 1 to 4 each
    const int tile = static_cast<int>(blockIdx.x) / cluster, tiles = static_cast<int>(gridDim.x) / cluster;
    const int each = a.n / 8 / tiles, more = a.n / 8 % tiles;
    const int n0 = (tile * each + min(tile, more)) * 8, nq = each + (tile < more);
    const int all_steps = (a.k + kStepK - 1) / kStepK;
    const int first = static_cast<int>(static_cast<long long>(all_steps) * rank / cluster);
    const int steps = static_cast<int>(static_cast<long long>(all_steps) * (rank + 1) / cluster) - first;
    float total[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) total[i][e] = 0.0f;
    switch (nq) {
    case 4: stream_columns<BF16, G, 4>(a, smem, n0, first, steps, seg_steps, total); break;
    case 3: stream_columns<BF16, G, 3>(a, smem, n0, first, steps, seg_steps, total); break;
    case 2: stream_columns<BF16, G, 2>(a, smem, n0, first, steps, seg_steps, total); break;
    default: stream_columns<BF16, G, 1>(a, smem, n0, first, steps, seg_steps, total); break;
    }

    // The warps' sums: [warp][row of A][column], then one thread per element adds them in order.
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    constexpr int kRedRow = kCols + 1;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[(warp * 8 + 2 * t + (e & 1)) * kRedRow + mt * 16 + r + (e >> 1) * 8] = total[mt][e];
    __syncthreads();
    const int elements = a.m * kCols;  // (at most one per thread)
    float v = 0.0f;
    const int row = tid / kCols, col = n0 + tid % kCols, at_red = row * kRedRow + tid % kCols;
    const bool stored = tid < elements && tid % cluster == rank && tid % kCols < nq * 8;
    if (tid < elements) {
#pragma unroll
        for (int q = 0; q < kWarps; ++q) v += red[q * 8 * kRedRow + at_red];
    }
    if (cluster > 1) {
        if (tid < elements) red[at_red] = v;  // (its own eight values: no other thread reads them)
        cluster_sync_all();
        if (stored) {
            v = 0.0f;
            for (int q = 0; q < cluster; ++q) v += ld_shared_cluster_f32(map_shared_rank(sbase + at_red * 4, q));
        }
    }
    if (stored) {
        const long long at = static_cast<long long>(row) * a.n + col;
        if (a.bias) v += decode16<BF16>(static_cast<const uint16_t*>(a.bias)[col]);
        const float res = a.residual ? decode16<BF16>(static_cast<const uint16_t*>(a.residual)[at]) : 0.0f;
        static_cast<uint16_t*>(a.D)[at] = encode16<BF16>(w4_epilogue(v, a.epilog, res));
    }
    if (cluster > 1) cluster_sync_all();  // the peers' shared memory stays until it is read
}

template <bool BF16, int G>
cudaError_t launch_one(const W4Args& a, int sms, cudaStream_t stream)
{
    using S = Segment<G>;
    auto kernel = w4_stream_kernel<BF16, G>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, kMaxSmem, prepared);
    if (e != cudaSuccess) return e;
    const int steps = (a.k + kStepK - 1) / kStepK;
    int tiles = (a.n + kCols - 1) / kCols;
    // k split over a cluster while that leaves an SM for every block; otherwise as many blocks as
    // give every SM the same number, the columns spread evenly over them (5120 columns: 304 blocks
    // of 16 or 24 columns, not 160 of 32 on 152 SMs)
    int cluster = 1;
    while (cluster < 8 && tiles * cluster * 2 <= sms && steps >= 2 * cluster) cluster *= 2;
    if (cluster == 1) {
        tiles = (tiles + sms - 1) / sms * sms;
        if (tiles > a.n / 8) tiles = a.n / 8;
    }
    const int seg = S::steps_for(a.m, (steps + cluster - 1) / cluster);
    int smem = S::bytes(a.m, seg);
    constexpr int kRed = kWarps * 8 * (kCols + 1) * 4;
    if (smem < kRed) smem = kRed;
    return launch_dependent(kernel, tiles * cluster, kThreads, smem, stream, cluster, a, cluster, seg);
}

template <bool BF16>
cudaError_t launch_type(const W4Args& a, int sms, cudaStream_t stream)
{
    if (a.group == 64) return launch_one<BF16, 64>(a, sms, stream);
    return launch_one<BF16, 128>(a, sms, stream);
}

}  // namespace

cudaError_t w4_stream_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    return bf16 ? launch_type<true>(a, sm_count, stream) : launch_type<false>(a, sm_count, stream);
}

}  // namespace gemm_epi
