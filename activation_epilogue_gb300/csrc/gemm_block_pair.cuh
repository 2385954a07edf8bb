// E4M3 products with a scale for each block of 128 of k, run by CTA pairs on 256 x 256 tiles:
//
//   D = epi(sum_b sa[b][i] sb[b][j] sum_{k in block b} A_ik B_jk + bias),
//
// with one scale per row of A and block (sa, m fp32 for each block of k) and one per 128 rows of
// the transposed B (SQUARE, n / 128 of them for each block) or per row of it (n of them).
//
// The tensor cores cannot apply such scales to a sum that they keep, so the sum of each block of
// 128 k is a sum of its own: the MMA warp starts every K block with cleared accumulators and hands
// them over, and the summing warps read them, multiply them by their scales and add them to the
// tile's sums in fp32 registers.  What bounds it is this hand-over and the additions: 256 x 256 x 128
// take 512 cycles of the pair's tensor cores, a block in all about 660 (SQUARE) and 1090.
//   * Four accumulators of 128 columns, half a tile each: a half's MMAs run while the three before
//     it are read, so that no MMA waits for a round trip through barriers (a whole tile's, two in
//     turn: 1977 us for 16384 x 8192 x 8192).
//   * Eight summing warps (a lane quarter, half the tile's columns each), 128 sums a thread, two added
//     an instruction.  A block is one chain of steps for each warp: its accumulators' barrier, four
//     loads of 32 columns, the arrival that frees them.  What is in that chain counts, not the
//     instructions: barriers tested ahead of their use, addresses that need no arithmetic.
//   * SQUARE: a warp's columns share one scale, a thread (a row) has one factor a block.  Otherwise
//     every column has its own, and a thread's values are loaded as four rows of 32 columns, so that
//     32 scales a block come from shared memory for them and not 128 (whose 1024 cycles a block
//     would bound it); each value then takes the product of its two scales (formed first: it alone has to be
//     finite) before its addition, 512 cycles of the fp32 pipes.  (Without the reads of the columns' scales a block
//     would take 90 cycles less, without the products 15; wider reads, scales by asynchronous copies and other orders
//     of the products: 1 to 2 %.  The loads of sixteen lanes are not what costs: 84.0 us for 84.4 with SQUARE's, which
//     itself takes 73.6 for 64.4 with these.)
//   * One warp brings the scales of all blocks into a ring in shared memory, ahead of the sums.
// 16384 x 8192 x 8192: 854 us, 2.57 PFLOP/s, where the power limit holds (717 in a short burst); 4096 x 8192 x
// 2064 64.4 us, 2.15 PFLOP/s, 84.4 with a scale for each row of B.
#pragma once

#include "block_sums.cuh"
#include "gemm_kernel.cuh"

namespace gemm_epi {

namespace block_pair {

using C = TileCfg<256, true>;
constexpr int kCols = 128;                    // columns of D per accumulator
constexpr int kHalfBytes = 64 * 128;          // a CTA's rows of B for half a tile's columns, in a stage
constexpr int kStages = 5;
constexpr int kStageBytes = C::kStageBytes;
// Four warps of copies, MMAs (two) and scales, then those that sum: the registers are
// given out by warpgroup, and the sums need more than an even share of the block's 384 x 168.
constexpr int kSumWarps = 8;
constexpr int kBlockThreads = 128 + 32 * kSumWarps;
constexpr int kIssueRegs = 88, kSumRegs = 208;
static_assert(128 * kIssueRegs + 32 * kSumWarps * kSumRegs <= kBlockThreads * 168,
              "a split of the registers that the block starts with");
// Blocks of scales on their way: SQUARE, the rows' factors for the tile's two halves (a row's scale times
// the block's of B); otherwise the rows' scales and those of 256 columns.
constexpr int kGroup = 4;                     // K blocks of scales that are handed over together
constexpr int kScaleGroups = 2;
constexpr int kScaleFloats = 3 * 128;
// Shared memory: the stages, 2 KB boxes for each summing warp (one is filled while the other is read: 4096 x 8192 x
// 2064 64.0 us with five stages and two boxes, 66.6 with six and one), the bias of three tiles' columns (a tile's is
// staged with its first scales, two groups ahead of their use at most: when those of tile j + 3 are, the epilogue
// of tile j is over), the scales.
constexpr int kBoxes = 2;
constexpr int kBiasTiles = 3;
constexpr int kOffBox = kStages * kStageBytes;
constexpr int kOffBias = kOffBox + kSumWarps * kBoxes * 2048;
constexpr int kOffScale = kOffBias + kBiasTiles * 256 * 4;
constexpr int kOffBar = kOffScale + kScaleGroups * kGroup * kScaleFloats * 4;
constexpr int kSmemBytes = 1024 + kOffBar + C::kBarBytes;  // (1024: alignment)
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr int kBarAccFull = kBarTmemFull;     // [4], in place of the one-scale kernel's four
constexpr int kBarAccEmpty = 44;              // [4], behind the tile indices
constexpr int kBarScaleFull = 48;             // [2]
constexpr int kBarScaleEmpty = kBarScaleFull + kScaleGroups;
constexpr int kBarDrain2 = kBarScaleEmpty + kScaleGroups;  // (the second issuing warp's kBarDrain)
static_assert(kBarAccFull + 4 == kBarStall && kOffSchedSlot + 4 * kSchedSlots <= kBarAccEmpty * 8 &&
                  (kBarDrain2 + 1) * 8 <= C::kBarBytes,
              "barrier area");

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// Whether a barrier's phase is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// A whole warp's wait (it gives up as one: what follows is for all of its lanes): one try in line, the loop out of
// the way (a loop of tries in its place took 1040 us for 16384 x 8192 x 8192 instead of 885).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int* abort_flag,
                                          unsigned long long limit_ns)
{
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag, limit_ns));
}

// The pair's tile j (j >= 1), for a whole warp: in the static order everyone knows it (handed over like the other
// order's, by writes and reads ordered over the cluster, it kept the copies and the sums waiting: 4096 x 8192 x 2064
// 81.5 us, 70.5 so); otherwise the even CTA's producer says it, as in the one-scale kernel.
__device__ __forceinline__ bool next_tile(const GemmParams& p, const WorkRange& w, uint32_t bar0, int j, int& tile,
                                          const volatile int* abort_flag)
{
    if (p.sched != nullptr) return sched_take_warp(bar0, j, tile, abort_flag, p.wait_limit_ns);
    const long long at = static_cast<long long>(tile) + w.stride;
    tile = at < w.end ? static_cast<int>(at) : w.end;
    return true;
}

// One thread of each CTA: the K blocks of every tile into the ring of stages, the even CTA's barriers
// counting both CTAs' bytes.  A CTA's 128 rows of B are 64 of each half of the tile's columns, so that the
// pair's MMA of a half (64 rows from either CTA) makes 128 columns next to each other.  The even CTA also
// tells the tiles to everyone else, a tile ahead (see the one-scale kernel's producer).
__device__ __forceinline__ void copy_operands(const GemmParams& p, uint32_t sbase, uint32_t bar0, volatile int* abort_flag)
{
    const WorkRange w = work_range<true>(p);
    const uint32_t rank = static_cast<uint32_t>(w.pair_rank);
    const bool even = rank == 0, dyn = p.sched != nullptr;
    const uint32_t full0 = map_shared_rank(bar0 + 8u * kBarFull, cluster_ctarank() & ~1u);
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    bool ok = true;
    int tile = w.first, next = w.end;
    grid_dependency_wait();
    for (int j = 0; ok; ++j) {
        if (j > 0) {
            if (even || !dyn)
                tile = next;
            else if (!sched_take(bar0, j, tile, abort_flag, p.wait_limit_ns))
                ok = false;
        }
        if (!ok || tile >= w.end) break;
        const unsigned ticket = even && dyn ? atomicAdd(p.sched, 1u) : 0u;  // (needed a few K blocks later)
        if (!dyn) next = static_cast<int>(min(static_cast<long long>(tile) + w.stride, static_cast<long long>(w.end)));
        const int publish_at = min(2, p.k_blocks - 1);
        int tm, tn;
        tile_coords(tile, p, tm, tn);
        const int arow = tm * 2 * kBM + static_cast<int>(rank) * kBM, brow = tn * 256 + static_cast<int>(rank) * 64;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
            ok = wait_bounded(bar0 + 8u * (kBarEmpty + stage), phase ^ 1u, abort_flag, p.wait_limit_ns);
            if (!ok) break;
            const uint32_t sa = sbase + stage * kStageBytes, full = full0 + 8u * stage;
            if (even) mbar_arrive_expect_tx(bar0 + 8u * (kBarFull + stage), 2 * kStageBytes);
            tma_load_2d_pair(sa, &p.tm_A, full, kb * 128, arow);
            tma_load_2d_pair(sa + C::kABytes, &p.tm_B, full, kb * 128, brow);
            tma_load_2d_pair(sa + C::kABytes + kHalfBytes, &p.tm_B, full, kb * 128, brow + 128);
            ++issued;
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
            if (even && dyn && kb == publish_at) {
                const long long at = static_cast<long long>(w.stride) + ticket;
                next = at < w.end ? static_cast<int>(at) : w.end;
                ok = sched_publish(bar0, j + 1, next, abort_flag, p.wait_limit_ns);
                if (!ok) break;
            }
        }
    }
    if (!ok && !*abort_flag) record_failure(p.status, abort_flag, kRoleProducer);
    if (!even) return;
    // the copies on their way land before the CTA can leave, also where another role gives up after this one's
    // last copy (the even CTA's barriers count both CTAs' copies)
    for (long long f = issued > kStages ? issued - kStages : 0; f < issued; ++f)
        wait_bounded(bar0 + 8u * (kBarFull + static_cast<int>(f % kStages)), static_cast<uint32_t>(f / kStages & 1),
                     abort_flag, kDrainLimitNs, false);
}

// Arrive on an mbarrier of the even CTA (a shared::cluster address).  What it orders are this warp's reads
// of tensor memory, which the tcgen05 fences around the barrier order; a release at cluster scope would
// wait for the warp's loads and stores of memory as well, a microsecond in every K block (before the later
// steps 1980 us for 16384 x 8192 x 8192 with it, 1012 so).
__device__ __forceinline__ void arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Two warps, one for each half of a tile's columns: a wait for a barrier that is long there takes 90 cycles and
// four MMAs with their commits 160, so that one warp's round for a block, 790 cycles, was longer than the MMAs'.
// The whole warp runs the loop, so that what the instructions take is uniform over it (in one thread's branch each
// operand is moved to uniform registers first); one elected lane issues.
__device__ __forceinline__ void issue_blocks(const GemmParams& p, uint32_t sbase, uint32_t bar0, uint32_t tmem_base,
                                             int h, volatile int* abort_flag)
{
    constexpr uint32_t idesc = make_idesc_e4m3(2 * kBM, kCols);
    const WorkRange w = work_range<true>(p);
    if (w.pair_rank != 0) return;
    const uint32_t self = cluster_ctarank();
    const uint16_t mask_self = static_cast<uint16_t>(1u << self);
    const uint16_t mask_pair = static_cast<uint16_t>(3u << self);
    grid_dependency_wait();  // (no copy lands earlier: the wait limit does not count the previous grid's time)
    const bool elected = elect_one();
    const uint64_t desc0 = make_sdesc_sw128(sbase, 0, 1024);
    const uint32_t b_at = static_cast<uint32_t>((C::kABytes + h * kHalfBytes) >> 4);
    int stage = 0;
    uint32_t phase = 0;
    uint32_t block = 0;  // K blocks so far, over all tiles
    bool ok = true;
    int tile = w.first;
    for (int j = 0; ok; ++j) {
        if (j > 0 && !next_tile(p, w, bar0, j, tile, abort_flag)) {
            ok = false;
            break;
        }
        if (tile >= w.end) break;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++block) {
            const uint64_t desc = desc0 + static_cast<uint32_t>(stage * (kStageBytes >> 4));
            const uint32_t acc = 2 * (block & 1u) + h;
            const uint32_t full = bar0 + 8u * (kBarFull + stage), empty = bar0 + 8u * (kBarAccEmpty + acc);
            const uint32_t turn = ((block >> 1) & 1u) ^ 1u;
            // (both at once: either takes 90 cycles)
            const bool there = mbar_try_wait(full, phase), free = mbar_try_wait(empty, turn);
            if (!__all_sync(0xFFFFFFFFu, there && free)) {
                ok = warp_wait(full, phase, abort_flag, p.wait_limit_ns) &&
                     warp_wait(empty, turn, abort_flag, p.wait_limit_ns);
                if (!ok) break;
            }
            tcgen05_fence_after_sync();
            if (elected) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_f8_ss_pair(tmem_base + acc * kCols, desc + kk * 2, desc + b_at + kk * 2, idesc, kk > 0 ? 1u : 0u);
                mma_commit_pair(bar0 + 8u * (kBarAccFull + acc), mask_pair);
                mma_commit_pair(bar0 + 8u * (kBarEmpty + stage), mask_pair);
            }
            __syncwarp();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    if (!ok && !*abort_flag) record_failure(p.status, abort_flag, kRoleMma);
    // every MMA issued completes before tensor memory is released (also where the sums gave up on them)
    const uint32_t drain = bar0 + 8u * (h ? kBarDrain2 : kBarDrain);
    if (elected) mma_commit_pair(drain, mask_self);
    __syncwarp();
    wait_bounded(drain, 0, abort_flag, kDrainLimitNs, false);
}

// One warp: the scales of every K block of every tile into the ring, and each tile's bias along the columns (read by
// the summing warps themselves it held up every tile: 2039 x 4096 x 1024 15.1 us, 14.4 so).
template <bool SQUARE>
__device__ __forceinline__ void stage_scales(const GemmParams& p, uint32_t sbase, uint32_t bar0, volatile int* abort_flag)
{
    const int lane = threadIdx.x & 31;
    const WorkRange w = work_range<true>(p);
    const long long sb_row = SQUARE ? (p.n - 1) / 128 + 1 : p.n;  // (n + 127 may pass 32 bits)
    constexpr int kB = SQUARE ? 2 : 8;        // scales of B of a lane and block
    constexpr int kAtOnce = SQUARE ? 4 : 2;   // blocks whose loads are on their way together
    const bool bias_along_cols = p.epilog != EPI_NONE && p.bias_layout == 1;
    grid_dependency_wait();
    uint32_t group = 0;
    int tile = w.first;
    for (int j = 0;; ++j) {
        if (j > 0 && !next_tile(p, w, bar0, j, tile, abort_flag)) {
            if (!*abort_flag) record_failure(p.status, abort_flag, kRoleProducer);
            return;
        }
        if (tile >= w.end) return;
        int tm, tn;
        tile_coords(tile, p, tm, tn);
        const int row0 = tm * 2 * kBM + w.pair_rank * kBM;
        int ia[4], ib[kB];  // (those past the matrix are the last ones again: their sums are not stored)
#pragma unroll
        for (int i = 0; i < 4; ++i) ia[i] = min(row0 + lane + 32 * i, p.m - 1);
#pragma unroll
        for (int i = 0; i < kB; ++i)
            ib[i] = SQUARE ? min(tn * 2 + i, static_cast<int>(sb_row) - 1) : min(tn * 256 + lane + 32 * i, p.n - 1);
        float bias[8];
        if (bias_along_cols) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int col = tn * 256 + lane + 32 * i;
                bias[i] = col < p.n ? load_16bit(p.bias, col, 1) : 0.0f;
            }
        }
        for (int kb0 = 0; kb0 < p.k_blocks; kb0 += kGroup, ++group) {
            const uint32_t slot = group % kScaleGroups;
#pragma unroll
            for (int q0 = 0; q0 < kGroup; q0 += kAtOnce) {
                float a[kAtOnce][4], b[kAtOnce][kB];
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) {
                    const long long kb = min(kb0 + q0 + q, p.k_blocks - 1);
                    const float* sa = p.scale_a + kb * p.m;
                    const float* sb = p.scale_b + kb * sb_row;
#pragma unroll
                    for (int i = 0; i < 4; ++i) a[q][i] = sa[ia[i]];
#pragma unroll
                    for (int i = 0; i < kB; ++i) b[q][i] = sb[ib[i]];
                }
                if (q0 == 0 && !warp_wait(bar0 + 8u * (kBarScaleEmpty + slot), (group / kScaleGroups & 1u) ^ 1u, abort_flag,
                                               p.wait_limit_ns)) {
                    if (!*abort_flag) record_failure(p.status, abort_flag, kRoleProducer);
                    return;
                }
                if (bias_along_cols && kb0 == 0 && q0 == 0) {
                    const uint32_t to = sbase + kOffBias + (j % kBiasTiles * 256 + lane) * 4;
#pragma unroll
                    for (int i = 0; i < 8; ++i) st_shared_u32(to + 128 * i, __float_as_uint(bias[i]));
                }
#pragma unroll
                for (int q = 0; q < kAtOnce; ++q) {
                    const uint32_t to = sbase + kOffScale + ((slot * kGroup + q0 + q) * kScaleFloats + lane) * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        st_shared_u32(to + 128 * i, __float_as_uint(SQUARE ? a[q][i] * b[q][0] : a[q][i]));
                        if (SQUARE) st_shared_u32(to + 512 + 128 * i, __float_as_uint(a[q][i] * b[q][1]));
                    }
                    if constexpr (!SQUARE) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) st_shared_u32(to + 512 + 128 * i, __float_as_uint(b[q][i]));
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar0 + 8u * (kBarScaleFull + slot));
        }
    }
}

template <int N, int EPI>
__device__ __forceinline__ void activate_block(float (&v)[N])
{
    if constexpr (EPI == EPI_GELU_BIAS) {
#pragma unroll
        for (int i = 0; i < N; i += 4) gelu4(v + i);
    } else {
        activate(v, EPI);
    }
}

// The place of a thread's sums: with SQUARE sum[e] is column e of its lane's row; otherwise sum
// 32 b + 16 a + 4 i + 2 u + v is row lane / 4 + 16 a + 8 u, column 32 b + 8 i + 2 (lane % 4) + v.

// The epilogue of 32 of the warp's columns, `at` on, and their store through the warp's box.
template <bool SQUARE, int EPI>
__device__ __forceinline__ void store_chunk(const GemmParams& p, const float* sum, uint32_t bias, int row0, int at,
                                            uint32_t box)
{
    const int lane = threadIdx.x & 31;
    constexpr bool kBias = EPI != EPI_NONE;
    const bool along_cols = p.bias_layout == 1;
    // (a thread's rows: one, or four)
    auto row_of = [&](int q) { return SQUARE ? row0 + lane : row0 + lane / 4 + 8 * q; };
    if (lane == 0) bulk_wait_group_read<kBoxes - 1>();  // this box has been read
    __syncwarp();
    if constexpr (SQUARE) {
        const int row = row_of(0);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = sum[e];
        if (kBias && along_cols) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                Pair a, b;
                ld_shared_pairs(bias + 4 * e, a, b);
                add2(v[e], v[e + 1], a);
                add2(v[e + 2], v[e + 3], b);
            }
        } else if (kBias) {
            const float b = row < p.m ? load_16bit(p.bias, row, 1) : 0.0f;
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] += b;
        }
        if constexpr (EPI == EPI_RELU_AUX_BIAS) {
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 32; ++e) word |= (v[e] > 0.0f && at + e < p.n) ? (1u << e) : 0u;
            if (row < p.m) static_cast<uint32_t*>(p.aux)[static_cast<long long>(row) * p.aux_ld + at / 32] = word;
        }
        activate_block<32, EPI>(v);
        const uint16_t* R = static_cast<const uint16_t*>(p.residual) + static_cast<long long>(row) * p.n + at;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (EPI == EPI_BIAS_RESIDUAL && row < p.m && at + 8 * q < p.n) {  // (n is a multiple of 8)
                const uint4 w = *reinterpret_cast<const uint4*>(R + 8 * q);
                const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    v[8 * q + 2 * h] += __uint_as_float(ww[h] << 16);
                    v[8 * q + 2 * h + 1] += __uint_as_float(ww[h] & 0xFFFF0000u);
                }
            }
            st_shared_v4(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), pack2(v[8 * q], v[8 * q + 1], 1),
                         pack2(v[8 * q + 2], v[8 * q + 3], 1), pack2(v[8 * q + 4], v[8 * q + 5], 1),
                         pack2(v[8 * q + 6], v[8 * q + 7], 1));
        }
    } else {
        const int c2 = 2 * (lane & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // rows lane / 4 + 8 q
            const int row = row_of(q);
            const float lb = kBias && !along_cols && row < p.m ? load_16bit(p.bias, row, 1) : 0.0f;
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 b =
                    kBias && along_cols ? unpair(ld_shared_pair(bias + 4 * (8 * i + c2))) : make_float2(lb, lb);
                v[2 * i] = sum[16 * (q >> 1) + 4 * i + 2 * (q & 1)] + b.x;
                v[2 * i + 1] = sum[16 * (q >> 1) + 4 * i + 2 * (q & 1) + 1] + b.y;
            }
            if constexpr (EPI == EPI_RELU_AUX_BIAS) {
                uint32_t word = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + 8 * i < p.n)
                        word |= ((v[2 * i] > 0.0f ? 1u : 0u) | (v[2 * i + 1] > 0.0f ? 2u : 0u)) << (8 * i + c2);
                word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
                word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2);
                if (c2 == 0 && row < p.m)
                    static_cast<uint32_t*>(p.aux)[static_cast<long long>(row) * p.aux_ld + at / 32] = word;
            }
            activate_block<8, EPI>(v);
            const uint16_t* R = static_cast<const uint16_t*>(p.residual) + static_cast<long long>(row) * p.n + at + c2;
            const int r32 = lane / 4 + 8 * q;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (EPI == EPI_BIAS_RESIDUAL && row < p.m && at + 8 * i < p.n) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(R + 8 * i);
                    v[2 * i] += __uint_as_float(w << 16);
                    v[2 * i + 1] += __uint_as_float(w & 0xFFFF0000u);
                }
                st_shared_u32(box + r32 * 64 + ((i ^ ((r32 >> 1) & 3)) << 4) + 2 * c2, pack2(v[2 * i], v[2 * i + 1], 1));
            }
        }
    }
    // 32 rows x 32 columns, 64-byte rows with the 64-byte swizzle
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(&p.tm_D, box, at, row0);
        bulk_commit_group();
    }
}

template <bool SQUARE, int EPI>
__device__ __forceinline__ void sum_blocks(const GemmParams& p, uint32_t sbase, uint32_t bar0,
                                           uint32_t tmem_base, volatile int* abort_flag)
{
    const int lane = threadIdx.x & 31;
    const int sw = static_cast<int>(threadIdx.x >> 5) - 4;
    const int quarter = sw & 3, half = sw >> 2;
    const WorkRange w = work_range<true>(p);
    const uint32_t box = sbase + kOffBox + sw * (kBoxes * 2048);
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t empty0 = map_shared_rank(bar0 + 8u * kBarAccEmpty, cluster_ctarank() & ~1u);
    // this thread's row's factor, or its four rows' scales and its columns'
    const uint32_t rows = sbase + kOffScale + 4 * (quarter * 32 + (SQUARE ? half * 128 + lane : lane / 4));
    const uint32_t columns = sbase + kOffScale + 4 * (128 + half * 128 + 2 * (lane & 3));
    grid_dependency_wait();

    uint32_t block = 0, group = 0;  // K blocks and groups of scales so far, over all tiles
    uint32_t stored = 0;            // boxes so far
    auto failed = [&]() {
        if (!*abort_flag) record_failure(p.status, abort_flag, kRoleEpilogue);
        return false;
    };
    // the MMAs into accumulator `a` (0 or 1, of this half) are done
    auto ready = [&](uint32_t bar, uint32_t parity) {
        const bool ok = warp_wait(bar, parity, abort_flag, p.wait_limit_ns);
        tcgen05_fence_after_sync();
        return ok || failed();
    };
    // the scales of the next group of K blocks are there
    auto scales_ready = [&]() {
        return warp_wait(bar0 + 8u * (kBarScaleFull + group % kScaleGroups), group / kScaleGroups & 1u, abort_flag,
                         p.wait_limit_ns) || failed();
    };
    // this warp has read its part of an accumulator
    auto release = [&](uint32_t bar) {
        tcgen05_fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_pair(bar);
    };
    // ... and a group's scales
    auto release_scales = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar0 + 8u * (kBarScaleEmpty + group % kScaleGroups));
        ++group;
    };

    int tile = w.first;
    for (int j = 0;; ++j) {
        if (j > 0 && !next_tile(p, w, bar0, j, tile, abort_flag)) {
            if (!*abort_flag) record_failure(p.status, abort_flag, kRoleEpilogue);
            break;
        }
        if (tile >= w.end) break;
        int tm, tn;
        tile_coords(tile, p, tm, tn);
        const int row0 = tm * 2 * kBM + w.pair_rank * kBM + quarter * 32;
        const int col0 = tn * 256 + half * kCols;
        bool ok = true;
        if (row0 >= p.m || col0 >= p.n) {  // nothing of the tile for this warp to store
            for (int kb = 0; kb < p.k_blocks && ok; ++kb, ++block) {
                const uint32_t at = 2 * (block & 1u) + half;
                ok = (kb % kGroup != 0 || scales_ready()) && ready(bar0 + 8u * (kBarAccFull + at), block >> 1 & 1u);
                if (!ok) break;
                release(empty0 + 8u * at);
                if (kb % kGroup == kGroup - 1 || kb == p.k_blocks - 1) release_scales();
            }
            if (!ok) break;
            continue;
        }
        float sum[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) sum[i] = 0.0f;
        // Columns 32 c on, as two loads (SQUARE: half of the columns; otherwise half of the lanes each).  The blocks
        // are walked in groups, as their scales come, so that every address and parity within one is a constant
        // next to a few registers.  (Sixteen values on their way while sixteen are added were no quicker; the next
        // block's first ones ahead of this one's end, and sums held as pairs, cost copies of registers.)
        uint32_t r[2][16];
        auto load = [&](uint32_t from, int c) {
            if constexpr (SQUARE) {
                load_lane16(from + c * 32, r[0]);
                load_lane16(from + c * 32 + 16, r[1]);
            } else {
                load_square16(from + c * 32, r[0]);
                load_square16(from + c * 32 + (16u << 16), r[1]);
            }
        };
        // the accumulators that this tile's even and odd blocks use, their barriers' parities (the same in every group)
        const uint32_t even = 2 * (block & 1u) + half, odd = even ^ 2u;
        const uint32_t from[2] = {t_lane + even * kCols, t_lane + odd * kCols};
        const uint32_t full[2] = {bar0 + 8u * (kBarAccFull + even), bar0 + 8u * (kBarAccFull + odd)};
        const uint32_t empty[2] = {empty0 + 8u * even, empty0 + 8u * odd};
        const uint32_t parity[2] = {block >> 1 & 1u, (block + 1) >> 1 & 1u};
        block += p.k_blocks;
        bool soon = false;  // whether the next block was done when this one's last values had been read
        for (int left = p.k_blocks; left > 0 && ok; left -= kGroup) {
            ok = scales_ready();
            if (!ok) break;
            const uint32_t at = group % kScaleGroups * (kGroup * kScaleFloats * 4);
#pragma unroll
            for (int q = 0; q < kGroup; ++q) {
                if (q >= left) break;
                Pair f[SQUARE ? 1 : 4], g[4];
#pragma unroll
                for (int i = 0; i < (SQUARE ? 1 : 4); ++i) {
                    const uint32_t v = ld_shared_u32(rows + at + q * (kScaleFloats * 4) + 32 * i);
                    f[i] = pair_of(v, v);
                }
                if (__all_sync(0xFFFFFFFFu, soon)) {
                    tcgen05_fence_after_sync();
                } else {
                    ok = ready(full[q & 1], parity[q & 1] ^ (q >> 1));
                    if (!ok) break;
                }
                load(from[q & 1], 0);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (!SQUARE) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            g[i] = ld_shared_pair(columns + at + q * (kScaleFloats * 4) + 128 * c + 32 * i);
                    }
                    tmem_wait(r);
                    if (c == 3) {
                        release(empty[q & 1]);
                        soon = mbar_test(full[(q + 1) & 1], parity[(q + 1) & 1] ^ ((q + 1) >> 1 & 1));
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float* s = sum + c * 32 + h * 16 + e;
                            const Pair x = pair_of(r[h][e], r[h][e + 1]);
                            if constexpr (SQUARE)
                                fma2(s[0], s[1], x, f[0]);
                            else
                                fma2(s[0], s[1], x, mul2(g[e / 4], f[2 * h + (e >> 1 & 1)]));
                        }
                    }
                    if (c < 3) load(from[q & 1], c + 1);
                }
            }
            release_scales();
        }
        if (!ok) break;
        const uint32_t bias = sbase + kOffBias + (j % kBiasTiles * 256 + half * kCols) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (col0 + c * 32 < p.n) {
                store_chunk<SQUARE, EPI>(p, sum + c * 32, bias + c * 128, row0, col0 + c * 32,
                                         box + stored++ % kBoxes * 2048);
            }
    }
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
    const uint32_t bar0 = sbase + kOffBar;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kOffBar + kOffHolder);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffBar + kOffAbort);
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_tensormap(&p.tm_A);
        prefetch_tensormap(&p.tm_B);
        prefetch_tensormap(&p.tm_D);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar0 + 8u * (kBarFull + s), 1);
            mbar_init(bar0 + 8u * (kBarEmpty + s), 2);  // (a commit of each half)
        }
        for (int s = 0; s < kSchedSlots; ++s) {
            mbar_init(bar0 + 8u * (kBarSchedFull + s), 1);
            mbar_init(bar0 + 8u * (kBarSchedEmpty + s), sched_consumers<kSumWarps>() + 3);  // (and the scales' warps, the second half's MMAs)
        }
        for (int s = 0; s < kScaleGroups; ++s) {
            mbar_init(bar0 + 8u * (kBarScaleFull + s), 1);
            mbar_init(bar0 + 8u * (kBarScaleEmpty + s), kSumWarps);
        }
        for (int a = 0; a < 4; ++a) {
            mbar_init(bar0 + 8u * (kBarAccFull + a), 1);
            mbar_init(bar0 + 8u * (kBarAccEmpty + a), kSumWarps);  // a lane of each warp of this half, of both CTAs
        }
        mbar_init(bar0 + 8u * kBarStall, 1);
        mbar_init(bar0 + 8u * kBarDrain, 1);
        mbar_init(bar0 + 8u * kBarDrain2, 1);
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
            if (lane == 0) copy_operands(p, sbase, bar0, abort_flag);
        } else if ((warp == 1 || warp == 3) && !*abort_flag) {
            issue_blocks(p, sbase, bar0, tmem_base, warp >> 1, abort_flag);
        } else if (warp == 2 && !*abort_flag) {
            stage_scales<SQUARE>(p, sbase, bar0, abort_flag);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
        if (!*abort_flag) sum_blocks<SQUARE, EPI>(p, sbase, bar0, tmem_base, abort_flag);
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
                                    kSmemBytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kBlockThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmemBytes;
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
