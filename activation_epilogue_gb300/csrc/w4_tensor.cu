// Products with 4-bit weights for 9 to 64 rows of A (from 5 on of the largest weights), on tcgen05:
// D^T = W A^T with 128 columns of D as the MMA's rows and the rows of A as its columns.
//
// mma.sync takes 16 cycles for 16 x 8 x 16 on this part, an eighth of tcgen05's rate, so that
// from two 8-row tiles of A on it, and not the weight's bytes, bounds a product (16384x8192,
// 48 rows: 72 us; this kernel's figures stand at its launch).  tcgen05 reads its first operand from
// tensor memory, where a thread's lane is the MMA's row: the thread that unpacks a row of W
// writes it there with tcgen05.st, and the unpacked weight never passes through shared memory
// (whose bandwidth it would exhaust: 128 x 128 values written and read again are 512 cycles of
// it, the block's share of the weight's bytes 370).
//
//   * The producer (one thread) copies blocks of 128 k of A by TMA (128-byte swizzle, rows past
//     m and k past the end read as zeros).
//   * Four chains (three with groups below 128) take every fourth (third) block each, with a block of
//     tensor memory (two halves), one or two accumulators and an issuing warp of their own.
//     (One issuer's own instructions took 1300 cycles a block, nearly all of a call: 48 us for
//     16384x8192 with 48 rows; two chains 31 us, four 26.6, and 25.1 with a group's MMAs issued
//     in a row, without a check between them.)
//   * A chain's four unpacking warps have a quarter of the 128 rows each: a block's 2 KB of a
//     quarter come through a ring of the warp's own in shared memory (cp.async, no barrier but
//     the warp's), each thread unpacks its row's 64 bytes to q - z, exactly, two neighbouring k
//     per 32-bit word, and stores them to tensor memory, half a block at a time.
//   * The chain's issuer runs the MMAs of one group of the scales after another.
//   * Eight warps (a quarter of the lanes, half of the rows of A each), with groups below 128 two
//     times eight with every other group each, read the groups' sums, of the chains in turn,
//     multiply them by the group's scales (one per lane: the lane is the column of D) and add them
//     up in fp32, two rows of A per instruction; at the end all threads apply the epilogue and
//     store D.
// A chain's waits are for its own earlier blocks alone, in order, so that no wait can take an
// older phase of a barrier for the one it needs.
// Measured (16384x8192, bf16, 48 rows): 24.5 us with groups of 128, 30.5 with 64, 39.0 with 32
// (a group's hand-over from the issuer to the summing warps costs more than its MMAs); about
// 6 us of each is start and end (4096x1024: 6.8 us), the rest 580 cycles a block of 128 x 128
// against some 370 for the unpacking instructions alone and for the weight's bytes.  A block takes
// 2000 warp instructions with groups of 128, 2600 with 64 (1080 of them unpacking), on 66 to 70 %
// of the issue slots.  Tried and left: all columns of a group loaded at once (64: 32.2 us, 32:
// 45.6), the sums as 64-bit pairs throughout (32.3, 42.2: more moves), one fma a column (31.4,
// 40.4), 1024 threads with 96 registers for eight summing warps of all columns (37.1, 53.5).
#include "kernel_params.h"
#include "launch.h"
#include "plan.h"
#include "ptx.cuh"
#include "w4_unpack.cuh"

namespace gemm_epi {

namespace {

constexpr int kCols = 128;                  // columns of D per block: MMA rows
constexpr int kBlockK = 128;                // k per block of the pipeline
constexpr int kMostChains = 4;
constexpr int kWDepth = 3;                  // blocks in flight per unpacking warp
constexpr int kMaxBSlots = 8;               // blocks of A in shared memory (most)
constexpr int kScaleDepth = 3;              // rounds of the chains' scales in flight per summing warp

// barriers (8 bytes each), then the tensor memory address and the failure flag
enum : int {
    kAFull = 0,
    kAEmpty = kAFull + 2 * kMostChains,
    kBFull = kAEmpty + 2 * kMostChains,
    kBEmpty = kBFull + kMaxBSlots,
    kAccFull = kBEmpty + kMaxBSlots,
    kAccEmpty = kAccFull + 2 * kMostChains,
    kDrain = kAccEmpty + 2 * kMostChains,
    kBars = kDrain + kMostChains
};
constexpr int kHeader = 512;
static_assert(kBars * 8 + 8 <= kHeader, "header");

template <int NP, int G>
struct Layout {
    static constexpr int kGroups = kBlockK / G;
    // Warps.  With groups of 128 the unpacking bounds a call: four chains.  With smaller groups the
    // summing does (some 240 cycles of waiting for a group, and two for each of its columns): three
    // chains, which leave room for a second set of summing warps, each with every other group.
    // 16384x8192 with 16, 32, 48 and 64 rows, groups of 64: 26.7, 29.0, 30.5 and 36.7 us (four
    // chains and one set 27.3, 29.9, 33.6, 36.7), of 32: 31.0, 34.6, 39.2, 51.2 (39.7, 44.2, 47.1, 54.8).
    static constexpr int kChains = G == 128 ? 4 : 3;
    static constexpr int kSets = G == 128 ? 1 : 2;
    static constexpr int kSumWarps = 8 * kSets;       // set, half of the rows of A, quarter of the lanes
    static constexpr int kUnpackWarps = 4 * kChains;  // chain, quarter of the lanes
    static constexpr int kProducerWarp = kSumWarps + kUnpackWarps;
    static constexpr int kIssuerWarp = kProducerWarp + 1;  // one thread each
    static constexpr int kThreads = 32 * (kIssuerWarp + kChains);
    // Tensor memory: a block of the unpacked weight for each chain, then its accumulators.
    static constexpr int kTmemAcc = kChains * (kBlockK / 2);
    static constexpr int kAccPer = 2 * kChains * NP <= 512 - kTmemAcc ? 2 : 1;
    static constexpr int kBarPer = kAccPer > kSets ? kAccPer : kSets;  // barriers for them, in turn
    static_assert(kChains <= kMostChains && kTmemAcc + kChains * kAccPer * NP <= 512, "tensor memory");
    // Shared memory: blocks of A, a ring of each unpacking warp (32 rows' 64 bytes of W, and the
    // groups' zero points), a ring of each summing warp (its groups' scales of its 32 columns).
    static constexpr int kB = NP * kBlockK * 2;
    static constexpr int kBSlots = NP == 64 ? kChains : 2 * kChains;  // (a multiple of the chains)
    static constexpr int kWSlot = 32 * 64 + kGroups * 32;
    static constexpr int kSetGroups = kGroups / kSets;                // of a block, for each set
    static constexpr int kSSlot = kChains * kSetGroups * 64;
    static constexpr int kOffW = kBSlots * kB;
    static constexpr int kOffS = kOffW + kUnpackWarps * kWDepth * kWSlot;
    static constexpr int kOffBar = kOffS + kSumWarps * kScaleDepth * kSSlot;
    static constexpr int kBytes = 1024 + kOffBar + kHeader;  // (1024: alignment)
    static_assert(kBSlots <= kMaxBSlots, "slots");
    static_assert(kBytes <= 227 * 1024, "shared memory");
    static_assert(kOffBar >= kSets * NP * kCols * 4, "the sums fit the rings");
};

__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

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

// mbar_arrive in the lanes that `take` part, without a branch.
__device__ __forceinline__ void mbar_arrive_if(uint32_t bar, bool take)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
        "r"(static_cast<uint32_t>(take))
        : "memory");
}

// Store 16 words of this thread's lane (no wait).
__device__ __forceinline__ void tmem_store_16cols_async(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
          "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
          "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Start loading 8 columns of this thread's lane; valid after tmem_wait_ld8 on them.
__device__ __forceinline__ void tmem_load_8cols_async(uint32_t taddr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}

// (x, y) += (a, b) * s
__device__ __forceinline__ void fma2(float& x, float& y, uint32_t a, uint32_t b, float s)
{
    unsigned long long acc, v, ss;
    asm("mov.b64 %0, {%1, %2};" : "=l"(acc) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(a), "r"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(ss));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(acc));
}


template <bool BF16, int NP, int G>
__global__ void __launch_bounds__(Layout<NP, G>::kThreads, 1) w4_tensor_kernel(const __grid_constant__ W4Args a,
                                                                const __grid_constant__ CUtensorMap tm_A,
                                                                int cluster)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_u32(smem);
    using L = Layout<NP, G>;
    constexpr int kB = L::kB, kBSlots = L::kBSlots;
    constexpr int kGroups = L::kGroups;  // per block
    constexpr int kChains = L::kChains, kSets = L::kSets, kSumWarps = L::kSumWarps, kBarPer = L::kBarPer;
    constexpr int kProducerWarp = L::kProducerWarp, kIssuerWarp = L::kIssuerWarp, kThreads = L::kThreads;
    const uint32_t bar0 = sbase + L::kOffBar;
    uint32_t* holder = reinterpret_cast<uint32_t*>(smem + L::kOffBar + kBars * 8);
    volatile int* failed = reinterpret_cast<volatile int*>(holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    const int n0 = static_cast<int>(blockIdx.x) / cluster * kCols;
    const int all_blocks = (a.k + kBlockK - 1) / kBlockK;
    const int first = static_cast<int>(static_cast<long long>(all_blocks) * rank / cluster);
    const int blocks = static_cast<int>(static_cast<long long>(all_blocks) * (rank + 1) / cluster) - first;
    const int groups = min(blocks * kGroups, a.k / G - first * kGroups);  // of this block's part of k

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * kChains; ++i) {
            mbar_init(bar0 + 8 * (kAFull + i), 4);
            mbar_init(bar0 + 8 * (kAEmpty + i), 1);
        }
        for (int i = 0; i < kBSlots; ++i) {
            mbar_init(bar0 + 8 * (kBFull + i), 1);
            mbar_init(bar0 + 8 * (kBEmpty + i), 1);
        }
        for (int i = 0; i < kChains * kBarPer; ++i) {
            mbar_init(bar0 + 8 * (kAccFull + i), 1);
            mbar_init(bar0 + 8 * (kAccEmpty + i), 8);
        }
        for (int i = 0; i < kChains; ++i) mbar_init(bar0 + 8 * (kDrain + i), 1);
        *failed = 0;
        fence_mbar_init();
    }
    if (warp == kIssuerWarp) {
        tmem_alloc(smem_u32(holder), 512);
        tmem_relinquish_alloc_permit();
    }
    if (warp == kProducerWarp && lane == 0 && blocks > 0) prefetch_tensormap(&tm_A);
    tcgen05_fence_before_sync();
    __syncthreads();
    tcgen05_fence_after_sync();
    const uint32_t tmem = *holder;
    grid_dependency_wait();
    grid_launch_dependents();

    float total[NP / 2];
#pragma unroll
    for (int j = 0; j < NP / 2; ++j) total[j] = 0.0f;

    if (warp == kProducerWarp) {
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < blocks; ++i) {
                const int slot = i % kBSlots;
                if (!w4_wait(bar0 + 8 * (kBEmpty + slot), (i / kBSlots & 1) ^ 1, failed)) break;
                const uint32_t full = bar0 + 8 * (kBFull + slot);
                mbar_arrive_expect_tx(full, kB);
                tma_load_2d(sbase + slot * kB, &tm_A, full, (first + i) * kBlockK, 0);
                tma_load_2d(sbase + slot * kB + kB / 2, &tm_A, full, (first + i) * kBlockK + 64, 0);
                ++issued;
            }
            if (*failed) {
                // the copies on their way land before the block's shared memory is given back
                for (int i = max(0, issued - kBSlots); i < issued; ++i)
                    w4_drain(bar0 + 8 * (kBFull + i % kBSlots), i / kBSlots & 1);
            }
        }
        __syncwarp();
    } else if (warp >= kIssuerWarp) {
        // The whole warp runs the loop, so that what the instructions take is uniform over it (in
        // one thread's branch each MMA's operands are moved to uniform registers first); one
        // elected lane issues.
        const bool elected = elect_one();
        constexpr uint32_t idesc = make_idesc_f16(BF16 ? 1u : 0u, 0u, 0u, kCols, NP);
        bool issued = false;
        const uint64_t desc0 = make_sdesc_sw128(sbase, 0, 1024);
        const int chain = __shfl_sync(0xFFFFFFFFu, warp - kIssuerWarp, 0);
        int last = -1;
        uint32_t n = 0;  // groups of this chain so far
        int bs = chain;
        uint32_t phase = 0, b_phase = 0;
        bool ok = true;
        for (int i = chain; i < blocks && ok; i += kChains, phase ^= 1) {
            const uint64_t desc = desc0 + static_cast<uint32_t>(bs * kB >> 4);
            uint32_t d_tmem = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ok = ok && w4_wait(bar0 + 8 * (kAFull + 2 * chain + h), phase, failed);
                if (h == 0) ok = ok && w4_wait(bar0 + 8 * (kBFull + bs), b_phase, failed);
                if (!ok) break;
                tcgen05_fence_after_sync();
                constexpr int kSteps = G / 16 < 4 ? G / 16 : 4;  // of a group, in half a block
#pragma unroll
                for (int s = 0; s < 4; s += kSteps) {
                    const int k16 = 4 * h + s;  // 16 k within the block
                    if (i * kGroups + k16 * 16 / G >= groups) break;
                    if (k16 * 16 % G == 0) {
                        const uint32_t before = n - L::kAccPer;  // the group that this accumulator held
                        if (n >= L::kAccPer)
                            ok = w4_wait(bar0 + 8 * (kAccEmpty + chain * kBarPer + before % kBarPer),
                                         before / kBarPer & 1, failed);
                        if (!ok) break;
                        tcgen05_fence_after_sync();
                        d_tmem = tmem + L::kTmemAcc + (chain * L::kAccPer + n % L::kAccPer) * NP;
                    }
                    const bool whole = (k16 + kSteps) * 16 % G == 0;  // the group ends here
                    if (elected) {
#pragma unroll
                        for (int j = 0; j < kSteps; ++j)
                            mma_f16_ts(d_tmem, tmem + chain * 64 + (k16 + j) * 8,
                                       desc + ((h * (kB / 2) + (s + j) * 32) >> 4), idesc,
                                       (k16 + j) * 16 % G > 0);
                        if (whole) mma_commit(bar0 + 8 * (kAccFull + chain * kBarPer + n % kBarPer));
                    }
                    issued = true;
                    if (whole) ++n;
                }
                if (!ok) break;
                if (elected) {
                    mma_commit(bar0 + 8 * (kAEmpty + 2 * chain + h));
                    if (h == 1) mma_commit(bar0 + 8 * (kBEmpty + bs));
                }
            }
            if (!ok) break;
            last = i;
            bs += kChains;
            if (bs >= kBSlots) {
                bs -= kBSlots;
                b_phase ^= 1;
            }
        }
        // (the last commits arrive before the block leaves)
        if (last >= 0 && !*failed) w4_wait(bar0 + 8 * (kBEmpty + last % kBSlots), last / kBSlots & 1, failed);
        __syncwarp();
        if (*failed && issued) {
            // every MMA issued completes before tensor memory is released
            if (elected) mma_commit(bar0 + 8 * (kDrain + chain));
            w4_drain(bar0 + 8 * (kDrain + chain), 0);
        }
        __syncwarp();
    } else if (warp >= kSumWarps) {
        // ---- unpacking: this warp's quarter (its tensor memory lanes) of its chain's blocks ----
        const int quarter = warp & 3, chain = (warp - kSumWarps) >> 2;
        const int ring = L::kOffW + (warp - kSumWarps) * (kWDepth * L::kWSlot);
        // copies: 16-byte chunk lane % 4 of rows lane / 4 + 8 j; 8 zero points of one group
        const int crow = lane >> 2, chunk = lane & 3;
        const uint8_t* src[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            src[j] = static_cast<const uint8_t*>(a.W) +
                     (static_cast<long long>(min(n0 + quarter * 32 + crow + 8 * j, a.n - 1)) * a.k +
                      static_cast<long long>(first + chain) * kBlockK) / 2 + chunk * 16;
        const uint32_t dst = crow * 64 + ((chunk ^ ((crow >> 1) & 3)) << 4);  // (+ 8 rows: + 512)
        const int k_first = (first + chain) * kBlockK;
        int k_left = a.k - k_first;
        const int zgroup = lane >> 2, zcol = (lane & 3) * 8;
        const bool copies_zeros = a.zeros != nullptr && zgroup < kGroups && n0 + quarter * 32 + zcol < a.n;
        const uint8_t* zsrc = a.zeros + static_cast<long long>(k_first / G + zgroup) * a.n + n0 + quarter * 32 + zcol;
        const long long z_step = static_cast<long long>(kChains * kGroups) * a.n;
        const int mine = blocks > chain ? (blocks - chain + kChains - 1) / kChains : 0;
        auto fetch = [&](int slot) {
            const uint32_t to = sbase + ring + slot * L::kWSlot;
            if (chunk * 32 < k_left) {
#pragma unroll
                for (int j = 0; j < 4; ++j) cp_async_16(to + dst + j * 512, src[j]);
            }
            if (copies_zeros && zgroup * G < k_left) cp_async_8(to + 2048 + zgroup * 32 + zcol, zsrc);
#pragma unroll
            for (int j = 0; j < 4; ++j) src[j] += kChains * kBlockK / 2;
            zsrc += z_step;
            k_left -= kChains * kBlockK;
        };
#pragma unroll
        for (int j = 0; j < kWDepth - 1; ++j) {
            if (j < mine) fetch(j);
            cp_async_commit();
        }
        const uint32_t t_lane = tmem + chain * 64 + (static_cast<uint32_t>(quarter * 32) << 16);
        int slot = 0, fill = kWDepth - 1;
        uint32_t phase = 1;
        bool ok = true;
        for (int b = 0; b < mine && ok; ++b, phase ^= 1) {
            if (b + kWDepth - 1 < mine) fetch(fill);
            cp_async_commit();
            if (++fill == kWDepth) fill = 0;
            cp_async_wait_group<kWDepth - 1>();
            __syncwarp();
            const uint8_t* mem = smem + ring + slot * L::kWSlot;
            if (++slot == kWDepth) slot = 0;
            W4UnpackInOrder<BF16> unpack[kGroups];
#pragma unroll
            for (int q = 0; q < kGroups; ++q) unpack[q].set(a.zeros ? mem[2048 + q * 32 + lane] : 8u);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 w4[2];
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    w4[c] = *reinterpret_cast<const uint4*>(mem + lane * 64 + (((2 * h + c) ^ ((lane >> 1) & 3)) << 4));
                ok = w4_wait(bar0 + 8 * (kAEmpty + 2 * chain + h), phase, failed);
                if (!ok) break;
                tcgen05_fence_after_sync();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint32_t w[4] = {w4[c].x, w4[c].y, w4[c].z, w4[c].w};
                    uint32_t v[16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) unpack[(2 * h + c) * 32 / G](w[j], v + 4 * j);
                    tmem_store_16cols_async(t_lane + (2 * h + c) * 16, v);
                }
                tmem_wait_st();
                tcgen05_fence_before_sync();
                __syncwarp();  // (also: the slot is read before its next copy is issued)
                mbar_arrive_if(bar0 + 8 * (kAFull + 2 * chain + h), lane == 0);
            }
        }
        cp_async_wait_group<0>();
    } else {
        // ---- the groups' sums, scaled and added ----
        const int quarter = warp & 3, set = warp >> 3;
        const int ring = L::kOffS + warp * (kScaleDepth * L::kSSlot);
        // group q of the set in a round of the chains' blocks: of chain q / kSetGroups
        auto in_round = [&](int q) { return q / L::kSetGroups * kGroups + q % L::kSetGroups * kSets + set; };
        const int scol = (lane & 3) * 8;
        const bool copies = n0 + quarter * 32 + scol < a.n;
        const uint16_t* src = static_cast<const uint16_t*>(a.scales) +
                              static_cast<long long>(first * kGroups) * a.n + n0 + quarter * 32 + scol;
        const long long s_step = static_cast<long long>(kChains * kGroups) * a.n;
        const int rounds = (blocks + kChains - 1) / kChains;
        int left = groups;  // from the next round to copy on
        auto fetch = [&](int slot) {
#pragma unroll
            for (int j = 0; j < kChains * L::kSetGroups; j += 8) {
                const int q = j + (lane >> 2);
                if (copies && q < kChains * L::kSetGroups && in_round(q) < left)
                    cp_async_16(sbase + ring + slot * L::kSSlot + q * 64 + scol * 2,
                                src + static_cast<long long>(in_round(q)) * a.n);
            }
            src += s_step;
            left -= kChains * kGroups;
        };
#pragma unroll
        for (int j = 0; j < kScaleDepth - 1; ++j) {
            if (j < rounds) fetch(j);
            cp_async_commit();
        }
        const uint32_t t_lane = tmem + L::kTmemAcc + (static_cast<uint32_t>(quarter * 32) << 16) + (warp >> 2 & 1) * (NP / 2);
        for (int i = 0; i < rounds; ++i) {
            if (i + kScaleDepth - 1 < rounds) fetch((i + kScaleDepth - 1) % kScaleDepth);
            cp_async_commit();
            cp_async_wait_group<kScaleDepth - 1>();
            __syncwarp();
            const uint16_t* scales = reinterpret_cast<const uint16_t*>(smem + ring + (i % kScaleDepth) * L::kSSlot) + lane;
            const int here = groups - i * (kChains * kGroups);  // groups from this round on
            bool ok = true;
#pragma unroll
            for (int p = 0; p < kChains * L::kSetGroups; ++p) {
                const int chain = p % kChains;  // the chains in turn
                const int q = chain * L::kSetGroups + p / kChains;
                if (in_round(q) >= here) continue;
                // (unsigned: its remainders are masks)
                const uint32_t n = i * kGroups + p / kChains * kSets + set;  // of the chain
                const uint32_t bar = chain * kBarPer + n % kBarPer;
                const float sc = decode16<BF16>(scales[q * 32]);
                if (!w4_wait(bar0 + 8 * (kAccFull + bar), n / kBarPer & 1, failed)) {
                    ok = false;
                    break;
                }
                tcgen05_fence_after_sync();
                const uint32_t t_acc = t_lane + (chain * L::kAccPer + n % L::kAccPer) * NP;
                uint32_t r[2][8];
                tmem_load_8cols_async(t_acc, r[0]);
#pragma unroll
                for (int j = 0; j < NP / 16; ++j) {
                    tmem_wait_ld8(r[j & 1]);
                    if (j + 1 < NP / 16) {
                        tmem_load_8cols_async(t_acc + (j + 1) * 8, r[(j + 1) & 1]);
                    } else {
                        tcgen05_fence_before_sync();
                        __syncwarp();
                        mbar_arrive_if(bar0 + 8 * (kAccEmpty + bar), lane == 0);
                    }
#pragma unroll
                    for (int e = 0; e < 8; e += 2)
                        fma2(total[j * 8 + e], total[j * 8 + e + 1], r[j & 1][e], r[j & 1][e + 1], sc);
                }
            }
            if (!ok) break;
            __syncwarp();  // the slot is read before its next copy is issued
        }
        cp_async_wait_group<0>();
    }

    tcgen05_fence_before_sync();
    __syncthreads();
    if (warp == kIssuerWarp) {
        tcgen05_fence_after_sync();
        tmem_dealloc(tmem, 512);
    }
    // The sums as [row][column] in shared memory, then the epilogue in a loop over all threads (one
    // copy of its code: unrolled over the rows it took 8 us a call to fetch).  With k split over a
    // cluster, block r of it takes every cluster-th element and adds the blocks' sums in order.
    float* red = reinterpret_cast<float*>(smem);
    if (warp < kSumWarps) {
        const bool gave_up = *failed != 0;
#pragma unroll
        for (int j = 0; j < NP / 2; ++j)
            red[((warp >> 3) * NP + (warp >> 2 & 1) * (NP / 2) + j) * kCols + (warp & 3) * 32 + lane] = gave_up ? __int_as_float(0x7FC00000) : total[j];
    }
    if (cluster > 1)
        cluster_sync_all();
    else
        __syncthreads();
    // a thread has two neighbouring columns of rows first_row, first_row + step, ...
    constexpr int kRowsAtOnce = kThreads / (kCols / 2);
    const int c2 = threadIdx.x % (kCols / 2) * 2, col = n0 + c2;
    const int first_row = static_cast<int>(threadIdx.x) / (kCols / 2) + rank * kRowsAtOnce;
    if (threadIdx.x < kRowsAtOnce * (kCols / 2) && col < a.n) {  // (n is even)
        float2 bias = make_float2(0.0f, 0.0f);
        if (a.bias) {
            const uint16_t* p = static_cast<const uint16_t*>(a.bias) + col;
            bias = make_float2(decode16<BF16>(p[0]), decode16<BF16>(p[1]));
        }
#pragma unroll 2
        for (int row = first_row; row < a.m; row += cluster * kRowsAtOnce) {
            float2 v = make_float2(0.0f, 0.0f);
            const int at_red = row * kCols + c2;
            if (cluster == 1) {
#pragma unroll
                for (int set = 0; set < kSets; ++set) {
                    const float2 w = *reinterpret_cast<const float2*>(red + set * NP * kCols + at_red);
                    v.x += w.x;
                    v.y += w.y;
                }
            } else {
                for (int q = 0; q < cluster * kSets; ++q) {
                    const float2 w = ld_shared_cluster_f32x2(map_shared_rank(sbase + (q % kSets * NP * kCols + at_red) * 4, q / kSets));
                    v.x += w.x;
                    v.y += w.y;
                }
            }
            const long long at = static_cast<long long>(row) * a.n + col;
            float2 res = make_float2(0.0f, 0.0f);
            if (a.residual) res = decode16x2<BF16>(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.residual) + at));
            *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.D) + at) =
                encode16x2<BF16>(w4_epilogue(v.x + bias.x, a.epilog, res.x), w4_epilogue(v.y + bias.y, a.epilog, res.y));
        }
    }
    if (cluster > 1) cluster_sync_all();  // the peers' shared memory stays until it is read
}

template <bool BF16, int NP, int G>
cudaError_t launch_one(const W4Args& a, const CUtensorMap& map, int sms, cudaStream_t stream)
{
    auto kernel = w4_tensor_kernel<BF16, NP, G>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, Layout<NP, G>::kBytes, prepared);
    if (e != cudaSuccess) return e;
    const int tiles = (a.n + kCols - 1) / kCols, blocks = (a.k + kBlockK - 1) / kBlockK;
    // (48 rows, k 8192, groups of 128: 8192 columns in clusters of two 16.4 us, 9856 to 16384 with a block
    // each 24.4 to 24.6, 20480 with a second wave 48.9)
    int cluster = sms / tiles;
    if (cluster > 8) cluster = 8;
    if (cluster > blocks / 4) cluster = blocks / 4;
    if (cluster < 1) cluster = 1;
    return launch_dependent(kernel, tiles * cluster, Layout<NP, G>::kThreads, Layout<NP, G>::kBytes, stream, cluster, a, map, cluster);
}

template <bool BF16, int NP>
cudaError_t launch_group(const W4Args& a, const CUtensorMap& map, int sms, cudaStream_t stream)
{
    if (a.group == 32) return launch_one<BF16, NP, 32>(a, map, sms, stream);
    if (a.group == 64) return launch_one<BF16, NP, 64>(a, map, sms, stream);
    return launch_one<BF16, NP, 128>(a, map, sms, stream);
}

template <bool BF16>
cudaError_t launch_type(const W4Args& a, const CUtensorMap& map, int sms, cudaStream_t stream)
{
    if (a.m <= 16) return launch_group<BF16, 16>(a, map, sms, stream);
    if (a.m <= 32) return launch_group<BF16, 32>(a, map, sms, stream);
    if (a.m <= 48) return launch_group<BF16, 48>(a, map, sms, stream);
    return launch_group<BF16, 64>(a, map, sms, stream);
}

}  // namespace

cudaError_t w4_tensor_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    CUtensorMap map = {};
    const uint32_t rows = static_cast<uint32_t>((a.m + 15) / 16 * 16);
    if (a.k > 0 &&
        !gemm_epi_impl::encode_2d(&map, a.A, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                  static_cast<uint64_t>(a.k), static_cast<uint64_t>(a.m), 64, rows,
                                  CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    return bf16 ? launch_type<true>(a, map, sm_count, stream) : launch_type<false>(a, map, sm_count, stream);
}

}  // namespace gemm_epi
