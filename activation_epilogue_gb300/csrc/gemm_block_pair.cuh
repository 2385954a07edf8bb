// E4M3 products with a scale for each block of 128 of k, run by CTA pairs on 256 x 256 tiles:
//
//   D = epi(sum_b sa[b][i] sb[b][j] sum_{k in block b} A_ik B_jk + bias),
//
// with one scale per row of A and block (sa, m fp32 for each block of k) and one per 128 rows of
// the transposed B (SQUARE, n / 128 of them for each block) or per row of it (n of them).
//
// The tensor cores cannot apply such scales to a sum that they keep, so the sum of each block of
// 128 k is a sum of its own: the MMA thread starts every K block with a cleared accumulator and
// hands it over, alternating between the two that tensor memory holds, and the epilogue warps read
// it, multiply it by its scales and add it to the tile's sums in fp32 registers: 128 a thread (two
// warps a lane quarter, 128 columns each, so that with SQUARE a warp's columns share one scale and
// a thread has one factor a block).  A block's MMAs take 512 cycles (256 x 256 x 128 on the pair);
// reading 128 x 256 fp32 from tensor memory takes 256 of them and the additions, two columns an
// instruction, 128 issue slots a scheduler (256 where every column has its scale), so the
// promotion hides behind the next block's MMAs.  The copies, the tile order and the stores are
// those of the CTA-pair kernel for one scale.
#pragma once

#include "gemm_kernel.cuh"

namespace gemm_epi {

namespace block_pair {

using C = TileCfg<256, true>;
constexpr int kCols = 128;                    // columns of D per epilogue warp
// Four warps of copies and MMAs (two of them idle), then the eight that sum: the registers are
// given out by warpgroup, and the sums need more than an even share of the block's 384 x 168.
constexpr int kBlockThreads = 384;
constexpr int kIssueRegs = 56, kSumRegs = 224;
static_assert(128 * kIssueRegs + 256 * kSumRegs <= 384 * 168, "a split of the registers that the block starts with");
constexpr int kScaleDepth = 3;                // a scale for each row of B: blocks of scales in flight
static_assert(kCols * (1 + kScaleDepth) * 4 <= 2048, "a warp's staging area");

// (x, y) += (a, b) * s
__device__ __forceinline__ void fma2(float& x, float& y, float a, float b, float s)
{
    unsigned long long acc, v, ss;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(ss));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
}

// (a, b) * (u, v)
__device__ __forceinline__ float2 mul2(float a, float b, float u, float v)
{
    unsigned long long x, y;
    float2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(u), "f"(v));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ void issue_blocks(const GemmParams& p, uint32_t sbase, uint32_t bar0, uint32_t tmem_base,
                                        volatile int* abort_flag)
{
    constexpr uint32_t idesc = make_idesc_e4m3(2 * kBM, 256);
    const WorkRange w = work_range<true>(p);
    if (w.pair_rank != 0) return;
    const uint32_t self = cluster_ctarank();
    const uint16_t mask_self = static_cast<uint16_t>(1u << self);
    const uint16_t mask_pair = static_cast<uint16_t>(3u << self);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t block = 0;  // K blocks so far, over all tiles
    bool issued_any = false;
    bool ok = true;
    int tile = w.first;
    for (int j = 0; ok; ++j) {
        if (j > 0 && !sched_take(bar0, j, tile, abort_flag, p.wait_limit_ns)) {
            if (!*abort_flag) record_failure(p.status, abort_flag, kRoleMma);
            ok = false;
            break;
        }
        if (tile >= w.end) break;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++block) {
            const uint32_t acc = block & 1u;
            if (!wait_bounded<true>(bar0 + 8u * (kBarTmemEmpty + acc), ((block >> 1) & 1u) ^ 1u, abort_flag,
                                    p.wait_limit_ns) ||
                !wait_bounded(bar0 + 8u * (kBarFull + stage), phase, abort_flag, p.wait_limit_ns)) {
                if (!*abort_flag) record_failure(p.status, abort_flag, kRoleMma);
                ok = false;
                break;
            }
            tcgen05_fence_after_sync();
            const uint32_t sa = sbase + stage * C::kStageBytes;
            const uint32_t sb = sa + C::kABytes;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                mma_f8_ss_pair(tmem_base + acc * 256u, make_sdesc_sw128(sa + kk * 32, 0, 1024),
                               make_sdesc_sw128(sb + kk * 32, 0, 1024), idesc, kk > 0 ? 1u : 0u);
            issued_any = true;
            mma_commit_pair(bar0 + 8u * (kBarEmpty + stage), mask_pair);
            mma_commit_pair(bar0 + 8u * (kBarTmemFull + acc), mask_pair);
            if (++stage == C::kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && issued_any) {
        // every MMA issued completes before tensor memory is released
        mma_commit_pair(bar0 + 8u * kBarDrain, mask_self);
        wait_bounded(bar0 + 8u * kBarDrain, 0, abort_flag, kDrainLimitNs, false);
    }
}

template <bool SQUARE, int EPI>
__device__ __forceinline__ void sum_blocks(const GemmParams& p, uint8_t* smem, uint32_t sbase, uint32_t bar0,
                                             uint32_t tmem_base, volatile int* abort_flag)
{
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int ew = warp - 4;
    const int quarter = warp & 3, half = ew >> 2;
    const WorkRange w = work_range<true>(p);
    float* sbias = reinterpret_cast<float*>(smem + C::kOffBias) + ew * 512;  // this warp's own, as all of its areas
    float* sscale = sbias + kCols;
    const uint32_t sscale_u32 = sbase + C::kOffBias + ew * 2048 + kCols * 4;
    uint8_t* box = smem + C::kOffEpi + ew * 2048;
    const uint32_t box_u32 = sbase + C::kOffEpi + ew * 2048;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * kCols;
    const uint32_t empty0 = map_shared_rank(bar0 + 8u * kBarTmemEmpty, cluster_ctarank() & ~1u);
    const long long sb_row = SQUARE ? (p.n + 127) / 128 : p.n;
    constexpr bool kBias = EPI != EPI_NONE;
    grid_dependency_wait();

    uint32_t block = 0;
    int tile = w.first;
    for (int j = 0;; ++j) {
        if (j > 0 && !sched_take_warp(bar0, j, tile, abort_flag, p.wait_limit_ns)) {
            if (!*abort_flag) record_failure(p.status, abort_flag, kRoleEpilogue);
            break;
        }
        if (tile >= w.end) break;
        int tm, tn;
        tile_coords(tile, p, tm, tn);
        const int row0 = tm * 2 * kBM + w.pair_rank * kBM + quarter * 32;
        const int row = row0 + lane;
        const int col0 = tn * 256 + half * kCols;
        const bool live = row0 < p.m && col0 < p.n;  // this warp has something to store
        float lb = 0.0f;
        if (kBias && p.bias_layout == 1) {
            __syncwarp();
            for (int i = lane; i < kCols; i += 32)
                sbias[i] = col0 + i < p.n ? load_16bit(p.bias, col0 + i, 1) : 0.0f;
        } else if (kBias && row < p.m) {
            lb = load_16bit(p.bias, row, 1);
        }
        const float* sa = p.scale_a + min(row, p.m - 1);
        const float* sb = p.scale_b + (SQUARE ? min(col0 / kCols, static_cast<int>(sb_row) - 1) : 0);
        // the scales of four blocks of k at a time, loaded while those before are worked on
        float next_a[4], next_b[4];
        auto load_scales = [&](int kb) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = min(kb + i, p.k_blocks - 1);
                next_a[i] = sa[static_cast<long long>(b) * p.m];
                if (SQUARE) next_b[i] = sb[static_cast<long long>(b) * sb_row];
            }
        };
        auto copy_scales = [&](int kb) {  // (a scale for each row of B; columns past n stay as they are)
            if (kb < p.k_blocks && col0 + 4 * lane < p.n)
                cp_async_16(sscale_u32 + (kb % kScaleDepth) * (kCols * 4) + lane * 16,
                            p.scale_b + static_cast<long long>(kb) * sb_row + col0 + 4 * lane);
            cp_async_commit();
        };
        load_scales(0);
        if constexpr (!SQUARE) {
            __syncwarp();
            copy_scales(0);
            copy_scales(1);
        }
        float sum[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
        bool ok = true;
        for (int kb0 = 0; kb0 < p.k_blocks && ok; kb0 += 4) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = SQUARE ? next_a[i] * next_b[i] : next_a[i];
            if (kb0 + 4 < p.k_blocks) load_scales(kb0 + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int kb = kb0 + i;
                if (kb >= p.k_blocks) break;
                const float* cs = nullptr;
                if constexpr (!SQUARE) {
                    copy_scales(kb + 2);
                    cp_async_wait_group<2>();
                    __syncwarp();
                    cs = sscale + (kb % kScaleDepth) * kCols;
                }
                const uint32_t acc = block & 1u;
                // (the warp gives up as one: what follows is for all of its lanes)
                if (!__all_sync(0xFFFFFFFFu, wait_bounded(bar0 + 8u * (kBarTmemFull + acc), (block >> 1) & 1u,
                                                          abort_flag, p.wait_limit_ns))) {
                    if (!*abort_flag) record_failure(p.status, abort_flag, kRoleEpilogue);
                    ok = false;
                    break;
                }
                ++block;
                tcgen05_fence_after_sync();
#pragma unroll
                for (int c = 0; c < kCols / 32; ++c) {
                    uint32_t r[32];
                    __syncwarp();
                    if (live) tmem_load_32cols(t_lane + acc * 256u + c * 32, r);
                    if (c == kCols / 32 - 1) {
                        tcgen05_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(empty0 + 8u * acc);
                    }
                    if (!live) continue;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        float* s = sum + c * 32 + e;
                        const float x[4] = {__uint_as_float(r[e]), __uint_as_float(r[e + 1]),
                                            __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3])};
                        if constexpr (SQUARE) {
                            fma2(s[0], s[1], x[0], x[1], f[i]);
                            fma2(s[2], s[3], x[2], x[3], f[i]);
                        } else {
                            const float4 v = *reinterpret_cast<const float4*>(cs + c * 32 + e);
                            const float2 y = mul2(x[0], x[1], v.x, v.y), z = mul2(x[2], x[3], v.z, v.w);
                            fma2(s[0], s[1], y.x, y.y, f[i]);
                            fma2(s[2], s[3], z.x, z.y, f[i]);
                        }
                    }
                }
            }
        }
        if (!ok) break;
        if (!live) continue;
        // ---- the tile's sums: bias, activation, residual, one rounding ----
        if (kBias) __syncwarp();  // (sbias)
#pragma unroll
        for (int c = 0; c < kCols / 32; ++c) {
            const int at = col0 + c * 32;
            if (at >= p.n) break;
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = sum[c * 32 + e];
            uint4 res[4];
            const bool whole = row < p.m && at + 32 <= p.n;
            const uint16_t* R = static_cast<const uint16_t*>(p.residual) + static_cast<long long>(row) * p.n + at;
            if (EPI == EPI_BIAS_RESIDUAL && whole) {
#pragma unroll
                for (int q = 0; q < 4; ++q) res[q] = reinterpret_cast<const uint4*>(R)[q];
            }
            if constexpr (kBias) add_bias<32>(v, sbias + c * 32, p.bias_layout == 1, lb);
            if constexpr (EPI == EPI_RELU_AUX_BIAS) {
                uint32_t word = 0;
#pragma unroll
                for (int e = 0; e < 32; ++e) word |= (v[e] > 0.0f && at + e < p.n) ? (1u << e) : 0u;
                if (row < p.m)
                    static_cast<uint32_t*>(p.aux)[static_cast<long long>(row) * p.aux_ld + at / 32] = word;
            }
            activate(v, EPI);
            if constexpr (EPI == EPI_BIAS_RESIDUAL) {
                if (whole) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t ww[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            v[q * 8 + 2 * h] += __uint_as_float(ww[h] << 16);
                            v[q * 8 + 2 * h + 1] += __uint_as_float(ww[h] & 0xFFFF0000u);
                        }
                    }
                } else if (row < p.m) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (at + e < p.n) v[e] += load_16bit(R, e, 1);
                }
            }
            // 32 rows x 32 columns, 64-byte rows with the 64-byte swizzle
            if (lane == 0) bulk_wait_group_read<0>();  // this warp's last box is read
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                    make_uint4(pack2(v[8 * q], v[8 * q + 1], 1), pack2(v[8 * q + 2], v[8 * q + 3], 1),
                               pack2(v[8 * q + 4], v[8 * q + 5], 1), pack2(v[8 * q + 6], v[8 * q + 7], 1));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(&p.tm_D, box_u32, at, row0);
                bulk_commit_group();
            }
        }
    }
    if constexpr (!SQUARE) cp_async_wait_all();
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
}

template <bool SQUARE, int EPI>
__global__ void __launch_bounds__(kBlockThreads, 1) block_pair_kernel(const __grid_constant__ GemmParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::kOffBar;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffBar + kOffHolder);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + kOffAbort);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&p.tm_A);
        prefetch_tensormap(&p.tm_B);
        prefetch_tensormap(&p.tm_D);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(bar0 + 8u * (kBarFull + s), 1);
            mbar_init(bar0 + 8u * (kBarEmpty + s), 1);
        }
        for (int s = 0; s < kSchedSlots; ++s) {
            mbar_init(bar0 + 8u * (kBarSchedFull + s), 1);
            mbar_init(bar0 + 8u * (kBarSchedEmpty + s), sched_consumers<kEpiWarps>());
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar0 + 8u * (kBarTmemFull + a), 1);
            mbar_init(bar0 + 8u * (kBarTmemEmpty + a), 2 * kEpiWarps);  // a lane of every epilogue warp of the pair
        }
        mbar_init(bar0 + 8u * kBarStall, 1);
        mbar_init(bar0 + 8u * kBarDrain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_holder), C::kTmemCols);
        tmem_relinquish_alloc_permit_pair();
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // the pair's barriers are initialised before either signals the other's
    tcgen05_fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    if (threadIdx.x == 0) grid_launch_dependents();
    if (p.debug_stall) {
        if (threadIdx.x == 0 &&
            !wait_bounded(bar0 + 8u * kBarStall, 0, abort_flag, p.wait_limit_ns, false))
            record_failure(p.status, abort_flag, kRoleStallTest);
        __syncthreads();
    }
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0 && !*abort_flag) {
            if (lane == 0) run_producer<256, false, true, false, true>(p, sbase, bar0, abort_flag, 0);
        } else if (warp == 1 && !*abort_flag) {
            if (lane == 0) issue_blocks(p, sbase, bar0, tmem_base, abort_flag);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        if (!*abort_flag) sum_blocks<SQUARE, EPI>(p, smem, sbase, bar0, tmem_base, abort_flag);
    }
    tcgen05_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // neither CTA leaves while the other may signal its barriers or write its tensor memory
    if (warp == 1) {
        tcgen05_fence_after_sync();
        tmem_dealloc_pair(tmem_base, C::kTmemCols);
    }
    if (p.sched != nullptr && threadIdx.x == 0 && (cluster_ctarank() & 1u) == 0) sched_finish(p);
}

template <bool SQUARE, int EPI>
cudaError_t launch_one(const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    if (prepare)
        return cudaFuncSetAttribute(block_pair_kernel<SQUARE, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    C::kSmemBytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kBlockThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;  // one CTA pair
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, block_pair_kernel<SQUARE, EPI>, p);
}

// Launch the kernel of `epilog`, or (prepare) set its shared memory.
template <bool SQUARE>
cudaError_t launch_epilog(int epilog, const GemmParams& p, int grid, cudaStream_t stream, bool pdl, bool prepare)
{
    switch (epilog) {
    case EPI_BIAS: return launch_one<SQUARE, EPI_BIAS>(p, grid, stream, pdl, prepare);
    case EPI_RELU_BIAS: return launch_one<SQUARE, EPI_RELU_BIAS>(p, grid, stream, pdl, prepare);
    case EPI_GELU_BIAS: return launch_one<SQUARE, EPI_GELU_BIAS>(p, grid, stream, pdl, prepare);
    case EPI_RELU_AUX_BIAS: return launch_one<SQUARE, EPI_RELU_AUX_BIAS>(p, grid, stream, pdl, prepare);
    case EPI_BIAS_RESIDUAL: return launch_one<SQUARE, EPI_BIAS_RESIDUAL>(p, grid, stream, pdl, prepare);
    case EPI_NONE: return launch_one<SQUARE, EPI_NONE>(p, grid, stream, pdl, prepare);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace block_pair

}  // namespace gemm_epi
