// E4M3 products with a scale for each block of 128 of k, few rows of A: D^T = B A^T with 128
// columns of D as the MMA's rows and NP rows of A (16 to 128) as its columns, so that a product of
// few rows streams B through every SM without computing rows that are not there.
//
// As in the CTA-pair kernel (gemm_block_pair.cuh) each K block's sum is an accumulator of its own,
// here one of four in turn, which the summing warps read, scale and add up in fp32.  Accumulator
// lanes are columns of D and its columns rows of A.  The warps stage the scales of A eight K blocks
// at a time in shared memory (times the scale of B's block, which the whole tile shares, with
// SQUARE; otherwise with the scales of B's rows), and a thread's values are loaded as four lanes of
// a quarter of the rows of A, so that it reads a quarter of their scales (all of them, by every lane,
// took 256 cycles of shared memory a K block of 64 rows, as many as the copies).  K may be split over
// the blocks of a cluster, which add their sums in rank order through distributed shared memory, each
// for every cluster-th row, so that the result does not depend on timing.
//
// Bound by B's bytes: one row with n = 8192, k = 16384 takes 24.2 us, 134 MB at 5.5 TB/s (28.8 with one
// block an SM), 48 rows with n = 16384, k = 8192 27.4 us (29.6); launch, first copies and the last sums are
// the four microseconds that a copy of these bytes does not have.
#include "block_sums.cuh"
#include "gemm_kernel.cuh"
#include "launch.h"

namespace gemm_epi {

namespace {

constexpr int kRowsB = 128;   // columns of D per block: MMA rows
constexpr int kAccs = 4;
constexpr int kGroup = 8;     // K blocks whose scales are staged together
constexpr int kMaxStages = 12;
constexpr int kAloneSmem = 200 * 1024;  // with this much a block has an SM to itself
constexpr int kRedRow = kRowsB + 4;  // (a warp's sums meet different banks)
// What a block of a cluster that gave up on a wait leaves for the others in the place of its sums: a NaN that no sum is
// (arithmetic makes 0x7FFFFFFF).  Its flag read by them in a load of its own took 0.2 us a call.
constexpr uint32_t kGaveUp = 0x7FC0DEADu;

enum : int { kFull = 0, kEmpty = kMaxStages, kAccFull = 2 * kMaxStages, kAccEmpty = kAccFull + kAccs,
             kStall = kAccEmpty + kAccs, kDrain, kBars };

template <int NP, bool SQUARE>
struct Layout {
    static constexpr int kParts = NP >= 64 ? 2 : 1;       // warps per lane quarter, NP / kParts rows of A each
    static constexpr int kOwn = NP / kParts;
    static constexpr int kSumWarps = 4 * kParts;
    static constexpr int kSumThreads = 32 * kSumWarps;
    static constexpr int kProducerWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
    static constexpr int kThreads = kSumThreads + 128;    // (the last two warps help with the epilogue)
    static constexpr int kB = kRowsB * 128, kA = NP * 128;
    static constexpr int kStage = kB + kA;
    // Two blocks an SM (one of 128 rows, whose sums need the registers): twice the K slices, and a call's last
    // blocks share the SMs with the next call's first.
    static constexpr int kPerSm = NP == 128 ? 1 : 2;
    static constexpr int kStagesRaw = (NP == 128 ? 200 : 96) * 1024 / kStage;
    static constexpr int kStages = kStagesRaw > kMaxStages ? kMaxStages : kStagesRaw;
    static constexpr int kChunk = kOwn < 32 ? 16 : 32;    // rows of A per load from tensor memory
    static constexpr int kScaleBytes = kGroup * (NP + (SQUARE ? 0 : kRowsB)) * 4;
    static constexpr int kOffScale = kStages * kStage;    // [2][kGroup][NP], then [kGroup][columns of D]
    static constexpr int kOffBar = kOffScale + 2 * kScaleBytes;
    static constexpr int kBytes = 1024 + kOffBar + kBars * 8 + 16;
    static constexpr int kTmem = kAccs * NP;
    static_assert(kPerSm * (kBytes + 1024) <= 228 * 1024, "shared memory");
    static_assert(NP * kRedRow * 4 <= kStages * kStage, "the sums fit the ring");
    static_assert(kTmem <= 512 && kTmem >= 32, "tensor memory");
    static constexpr int kStaged = kGroup * NP / kSumThreads;  // scales that a thread stages for a group
    static_assert(kGroup * NP % kSumThreads == 0, "staging");
};

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float2 ld_shared_cluster_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v) { st_shared_u32(addr, __float_as_uint(v)); }

__device__ __forceinline__ void load_values(uint32_t taddr, uint32_t (&r)[16]) { load_square16(taddr, r); }
__device__ __forceinline__ void load_values(uint32_t taddr, uint32_t (&r)[8]) { load_square8(taddr, r); }

__device__ __forceinline__ float apply(float v, int epilog)
{
    if (epilog == EPI_RELU_BIAS || epilog == EPI_RELU_AUX_BIAS) return v > 0.0f ? v : 0.0f;
    return epilog == EPI_GELU_BIAS ? gelu_erf_fast(gelu_floor(v)) : v;  // (as gelu4; minus infinity is no NaN either)
}

template <int NP, bool SQUARE>
__global__ void __launch_bounds__(Layout<NP, SQUARE>::kThreads, Layout<NP, SQUARE>::kPerSm)
    block_swapped_kernel(const __grid_constant__ GemmParams p)
{
    using L = Layout<NP, SQUARE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + L::kOffBar;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::kOffBar + kBars * 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;
    const int rank = static_cast<int>(blockIdx.x) % split;
    const int tile = static_cast<int>(blockIdx.x) / split;
    const int n0 = tile / p.tiles_n * kRowsB;  // (the row tiles of one panel of B next to each other)
    const int m0 = tile % p.tiles_n * NP;
    const int first = static_cast<int>(static_cast<long long>(p.k_blocks) * rank / split);
    const int blocks = static_cast<int>(static_cast<long long>(p.k_blocks) * (rank + 1) / split) - first;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&p.tm_A);
        prefetch_tensormap(&p.tm_B);
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar0 + 8 * (kFull + s), 1);
            mbar_init(bar0 + 8 * (kEmpty + s), 1);
        }
        for (int a = 0; a < kAccs; ++a) {
            mbar_init(bar0 + 8 * (kAccFull + a), 1);
            mbar_init(bar0 + 8 * (kAccEmpty + a), L::kSumWarps);
        }
        mbar_init(bar0 + 8 * kStall, 1);
        mbar_init(bar0 + 8 * kDrain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == L::kMmaWarp) {
        tmem_alloc(smem_u32(holder), L::kTmem);
        tmem_relinquish_alloc_permit();
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = *holder;
    if (threadIdx.x == 0) grid_launch_dependents();
    const bool stall = p.debug_stall == 1 || (p.debug_stall == 2 && rank == split - 1);
    if (stall) {
        if (threadIdx.x == 0 && !wait_bounded(bar0 + 8 * kStall, 0, abort_flag, p.wait_limit_ns, false))
            record_failure(p.status, abort_flag, kRoleStallTest);
        __syncthreads();
    }

    float sum[L::kOwn];
#pragma unroll
    for (int i = 0; i < L::kOwn; ++i) sum[i] = 0.0f;

    if (warp == L::kProducerWarp) {
        if (lane == 0 && !stall) {
            int issued = 0;
            auto copy = [&](int i, bool b, bool a) {
                const int s = i % L::kStages;
                const uint32_t full = bar0 + 8 * (kFull + s);
                if (b) {
                    mbar_arrive_expect_tx(full, L::kStage);
                    tma_load_2d(sbase + s * L::kStage, &p.tm_B, full, (first + i) * 128, n0);
                }
                if (a) tma_load_2d(sbase + s * L::kStage + L::kB, &p.tm_A, full, (first + i) * 128, m0);
            };
            const int ahead = min(blocks, L::kStages);
            // (ahead of the wait: B itself where that is promised, otherwise B into L2, which needs no promise)
            for (int i = 0; i < ahead; ++i) {
                if (p.b_ready)
                    copy(i, true, false);
                else
                    tma_prefetch_2d(&p.tm_B, (first + i) * 128, n0);
            }
            grid_dependency_wait();
            for (int i = 0; i < ahead; ++i) copy(i, !p.b_ready, true);
            issued = ahead;
            for (int i = ahead; i < blocks; ++i) {
                if (!wait_bounded(bar0 + 8 * (kEmpty + i % L::kStages), (i / L::kStages & 1) ^ 1, abort_flag,
                                  p.wait_limit_ns)) {
                    if (!*abort_flag) record_failure(p.status, abort_flag, kRoleProducer);
                    break;
                }
                copy(i, true, true);
                ++issued;
            }
            // the copies on their way land before the block's shared memory is given back (also where another role
            // gives up after the last of them)
            for (int i = max(0, issued - L::kStages); i < issued; ++i)
                wait_bounded(bar0 + 8 * (kFull + i % L::kStages), i / L::kStages & 1, abort_flag, kDrainLimitNs, false);
        }
        __syncwarp();
    } else if (warp == L::kMmaWarp) {
        if (lane == 0 && !stall) {
            constexpr uint32_t idesc = make_idesc_e4m3(kRowsB, NP);
            grid_dependency_wait();  // (A does not land earlier: the wait limit does not count the previous grid's time)
            int i = 0;
            for (; i < blocks; ++i) {
                const int s = i % L::kStages, acc = i % kAccs;
                if (!wait_bounded(bar0 + 8 * (kAccEmpty + acc), (i / kAccs & 1) ^ 1, abort_flag, p.wait_limit_ns) ||
                    !wait_bounded(bar0 + 8 * (kFull + s), i / L::kStages & 1, abort_flag, p.wait_limit_ns)) {
                    if (!*abort_flag) record_failure(p.status, abort_flag, kRoleMma);
                    break;
                }
                tcgen05_fence_after_sync();
                const uint32_t sb = sbase + s * L::kStage, sa = sb + L::kB;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8_ss(tmem + acc * NP, make_sdesc_sw128(sb + kk * 32, 0, 1024),
                              make_sdesc_sw128(sa + kk * 32, 0, 1024), idesc, kk > 0 ? 1u : 0u);
                mma_commit(bar0 + 8 * (kEmpty + s));
                mma_commit(bar0 + 8 * (kAccFull + acc));
            }
            if (i > 0) {
                // every MMA issued completes, and its commits arrive, before the block leaves
                mma_commit(bar0 + 8 * kDrain);
                wait_bounded(bar0 + 8 * kDrain, 0, abort_flag, kDrainLimitNs, false);
            }
        }
        __syncwarp();
    } else if (warp < L::kSumWarps && !stall) {
        const int quarter = warp & 3, part = warp >> 2;
        const long long sb_row = SQUARE ? (p.n - 1) / 128 + 1 : p.n;  // (n + 127 may pass 32 bits)
        const uint32_t staged = sbase + L::kOffScale;
        float next[L::kStaged], next_b[SQUARE ? 1 : kGroup];
        auto load_scales = [&](int g) {  // of group g of this block's K blocks (the last one's again past the end)
#pragma unroll
            for (int e = 0; e < L::kStaged; ++e) {
                const int at = threadIdx.x + e * L::kSumThreads;
                const int b = first + min(g * kGroup + at / NP, blocks - 1);
                next[e] = p.scale_a[static_cast<long long>(b) * p.m + min(m0 + at % NP, p.m - 1)];
                if (SQUARE) next[e] *= p.scale_b[static_cast<long long>(b) * sb_row + n0 / 128];
            }
            if (!SQUARE && threadIdx.x < kRowsB) {
#pragma unroll
                for (int e = 0; e < kGroup; ++e)
                    next_b[e] = p.scale_b[static_cast<long long>(first + min(g * kGroup + e, blocks - 1)) * sb_row +
                                          min(n0 + static_cast<int>(threadIdx.x), p.n - 1)];
            }
        };
        grid_dependency_wait();
        load_scales(0);
        const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * L::kOwn;
        bool ok = true;
        for (int g = 0; g * kGroup < blocks; ++g) {
            const uint32_t mine = staged + (g & 1) * L::kScaleBytes;
#pragma unroll
            for (int e = 0; e < L::kStaged; ++e) st_shared_f32(mine + 4 * (threadIdx.x + e * L::kSumThreads), next[e]);
            if (!SQUARE && threadIdx.x < kRowsB) {
#pragma unroll
                for (int e = 0; e < kGroup; ++e)
                    st_shared_f32(mine + kGroup * NP * 4 + 4 * (e * kRowsB + threadIdx.x), next_b[e]);
            }
            // (a buffer is written again two groups on: by then every thread has passed the barrier between)
            named_barrier_sync(1, L::kSumThreads);
            if ((g + 1) * kGroup < blocks) load_scales(g + 1);
#pragma unroll 1
            for (int e = 0; e < kGroup; ++e) {
                const int i = g * kGroup + e, acc = i % kAccs;
                if (i >= blocks || !ok) continue;
                // (the warp gives up as one: what follows is for all of its lanes)
                const uint32_t bar = bar0 + 8 * (kAccFull + acc), parity = i / kAccs & 1;
                if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity)) &&
                    !__all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, p.wait_limit_ns))) {
                    if (!*abort_flag) record_failure(p.status, abort_flag, kRoleEpilogue);
                    ok = false;
                    continue;
                }
                tcgen05_fence_after_sync();
                const uint32_t fa = mine + (e * NP + part * L::kOwn + 2 * (lane & 3)) * 4;
                Pair fb[4];  // lanes lane / 4 + 8 j
                if constexpr (!SQUARE) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int at = kGroup * NP + e * kRowsB + quarter * 32 + 8 * j + (lane >> 2);
                        const uint32_t v = ld_shared_u32(mine + at * 4);
                        fb[j] = pair_of(v, v);
                    }
                }
                constexpr int kLoads = 2 * L::kOwn / L::kChunk;  // chunk of columns, half of the lanes
                uint32_t r[2][L::kChunk / 2];
                auto load = [&](int c) { load_values(t_lane + acc * NP + ((c & 1) << 20) + (c >> 1) * L::kChunk, r[c & 1]); };
                load(0);
                Pair f[L::kChunk / 8];
#pragma unroll
                for (int c = 0; c < kLoads; ++c) {
                    if (c % 2 == 0) {
#pragma unroll
                        for (int q = 0; q < L::kChunk / 8; ++q) f[q] = ld_shared_pair(fa + ((c >> 1) * L::kChunk + 8 * q) * 4);
                    }
                    tmem_wait(r[c & 1]);
                    if (c + 1 < kLoads) {
                        load(c + 1);
                    } else {
                        tcgen05_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar0 + 8 * (kAccEmpty + acc));
                    }
#pragma unroll
                    for (int q = 0; q < L::kChunk / 2; q += 2) {
                        float* s = sum + c * (L::kChunk / 2) + q;
                        const Pair x = pair_of(r[c & 1][q], r[c & 1][q + 1]);
                        if constexpr (SQUARE)
                            fma2(s[0], s[1], x, f[q / 4]);
                        else
                            fma2(s[0], s[1], x, mul2(f[q / 4], fb[2 * (c & 1) + (q >> 1 & 1)]));
                    }
                }
            }
        }
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == L::kMmaWarp) {
        tcgen05_fence_after_sync();
        tmem_dealloc(tmem, L::kTmem);
    }
    grid_dependency_wait();
    // The sums as [row of A][column of D] in shared memory, then the epilogue over all threads; with K split,
    // block `rank` of the cluster takes every split-th set of rows and adds the blocks' sums in order.  A block that
    // gave up on a wait has kGaveUp in the place of its sums, and nothing of the tile is stored by any of them.
    float* red = reinterpret_cast<float*>(smem);
    const bool failed = *abort_flag;
    if (warp < L::kSumWarps) {
#pragma unroll
        for (int i = 0; i < L::kOwn; ++i) {
            const int c = i / (L::kChunk / 2), e = i % (L::kChunk / 2);  // the load, its value (see load_values)
            const int row = (warp >> 2) * L::kOwn + (c >> 1) * L::kChunk + (e >> 2) * 8 + 2 * (lane & 3) + (e & 1);
            red[row * kRedRow + (warp & 3) * 32 + (c & 1) * 16 + (e >> 1 & 1) * 8 + (lane >> 2)] =
                failed ? __uint_as_float(kGaveUp) : sum[i];
        }
    }
    if (split > 1)
        cluster_sync_all();
    else
        __syncthreads();
    constexpr int kRowsAtOnce = L::kThreads / (kRowsB / 2);
    const int c2 = threadIdx.x % (kRowsB / 2) * 2, col = n0 + c2;
    const bool there = col < p.n && !failed;  // (n is even)
    const bool along_cols = p.bias_layout == 1, has_bias = p.epilog != EPI_NONE;
    float2 bias = make_float2(0.0f, 0.0f);
    if (there && has_bias && along_cols)
        bias = make_float2(load_16bit(p.bias, col, 1), load_16bit(p.bias, col + 1, 1));
    const int rows = min(NP, p.m - m0);
    for (int r = static_cast<int>(threadIdx.x) / (kRowsB / 2) + rank * kRowsAtOnce; r < rows; r += split * kRowsAtOnce) {
        float2 v = make_float2(0.0f, 0.0f);
        bool store = there;
        if (split == 1) {
            v = *reinterpret_cast<const float2*>(red + r * kRedRow + c2);
        } else {
            for (int q = 0; q < split; ++q) {
                const float2 w = ld_shared_cluster_f32x2(map_shared_rank(sbase + (r * kRedRow + c2) * 4, q));
                v.x += w.x;
                v.y += w.y;
                store = store && __float_as_uint(w.x) != kGaveUp;
            }
        }
        const long long row = m0 + r;
        if (there && has_bias && !along_cols) bias.x = bias.y = load_16bit(p.bias, row, 1);
        v.x += bias.x;
        v.y += bias.y;
        if (p.epilog == EPI_RELU_AUX_BIAS) {
            // lanes 0-15 have the 32 columns of one word, lanes 16-31 those of the next
            uint32_t word = there ? ((v.x > 0.0f ? 1u : 0u) | (v.y > 0.0f ? 2u : 0u)) << (2 * (lane & 15)) : 0u;
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) word |= __shfl_xor_sync(0xFFFFFFFFu, word, o);
            if (store && (lane & 15) == 0) static_cast<uint32_t*>(p.aux)[row * p.aux_ld + col / 32] = word;
        }
        v.x = apply(v.x, p.epilog);
        v.y = apply(v.y, p.epilog);
        if (!store) continue;
        const long long at = row * p.n + col;
        if (p.epilog == EPI_BIAS_RESIDUAL) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.residual) + at);
            v.x += __uint_as_float(w << 16);
            v.y += __uint_as_float(w & 0xFFFF0000u);
        }
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.D) + at) = pack2(v.x, v.y, 1);
    }
    if (split > 1) cluster_sync_all();  // the peers' shared memory stays until it is read
}

template <int NP, bool SQUARE>
cudaError_t launch_one(const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    auto kernel = block_swapped_kernel<NP, SQUARE>;
    if (prepare) {
        constexpr int most = Layout<NP, SQUARE>::kBytes > kAloneSmem ? Layout<NP, SQUARE>::kBytes : kAloneSmem;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                    cudaSharedmemCarveoutMaxShared);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(Layout<NP, SQUARE>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = Layout<NP, SQUARE>::kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.split > 1 ? p.split : 1);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Clusters of `split` blocks that the GPU holds at once, kPerSm blocks an SM: what it holds with one an SM (asked for
// with shared memory that makes it so; the answer for two is one's too), times kPerSm.
template <int NP>
int max_clusters(int split)
{
    auto kernel = block_swapped_kernel<NP, true>;
    if (launch_one<NP, true>(GemmParams{}, 0, nullptr, false, true) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
    cfg.blockDim = dim3(Layout<NP, true>::kThreads, 1, 1);
    cfg.dynamicSmemBytes = kAloneSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess ? n * Layout<NP, true>::kPerSm : 0;
}

template <bool SQUARE>
cudaError_t launch_np(int np, const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    switch (np) {
    case 16: return launch_one<16, SQUARE>(p, grid, stream, pdl, prepare);
    case 32: return launch_one<32, SQUARE>(p, grid, stream, pdl, prepare);
    case 64: return launch_one<64, SQUARE>(p, grid, stream, pdl, prepare);
    case 128: return launch_one<128, SQUARE>(p, grid, stream, pdl, prepare);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

// (Asked for once a process: its devices are taken to be the same GPU model, as elsewhere in the planner.)
int block_swapped_max_clusters(int np, int split)
{
    static std::atomic<int> known[4][9];  // (0: not asked yet; else the answer + 1)
    std::atomic<int>& at = known[np == 16 ? 0 : np == 32 ? 1 : np == 64 ? 2 : 3][split];
    int v = at.load(std::memory_order_relaxed);
    if (v == 0) {
        v = 1 + (np == 16   ? max_clusters<16>(split)
                 : np == 32 ? max_clusters<32>(split)
                 : np == 64 ? max_clusters<64>(split)
                            : max_clusters<128>(split));
        at.store(v, std::memory_order_relaxed);
    }
    return v - 1;
}

cudaError_t block_swapped(int np, bool square, const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    return square ? launch_np<true>(np, p, grid, stream, pdl, prepare) : launch_np<false>(np, p, grid, stream, pdl, prepare);
}

int block_swapped_smem(int np)
{
    return np == 16   ? Layout<16, true>::kBytes
           : np == 32 ? Layout<32, true>::kBytes
           : np == 64 ? Layout<64, true>::kBytes
                      : Layout<128, true>::kBytes;
}

int block_swapped_stages(int np)
{
    return np == 16   ? Layout<16, true>::kStages
           : np == 32 ? Layout<32, true>::kStages
           : np == 64 ? Layout<64, true>::kStages
                      : Layout<128, true>::kStages;
}

}  // namespace gemm_epi
