// Products with 4-bit weights and group scales for a few rows of A, with the GEMM epilogs,
// and the weight written out as the 16-bit B of a plan.
//
// The product, D^T = W A^T, streams the weight once: W's rows (columns of D) are the 16 MMA
// rows of mma.m16n8k16, rows of A its 8 columns, so even one row of A uses the tensor cores
// and every weight is unpacked once for the up to 16 rows that this kernel takes (more, and the
// larger weights, go to w4_stream.cu and w4_tensor.cu).  For a few rows that is 4 bits of
// traffic per 2 m flops, bound by the weight's bytes.
//
//   * A block takes 16 MT CW columns of D and all of k (or a cluster's share of it), in stages of
//     128 KW values of k (CW KW = 8 warps): the stage's weights, rows of A, scales and zero points are copied
//     with cp.async into a ring, each byte by one thread.
//   * Warp (cw, kw) multiplies its 16 MT columns by its 128 values of k.  In a row's 64 bytes
//     of those, chunk i (16 bytes) holds k = 32 i .. 32 i + 31, and ldmatrix hands word t of
//     row r to lane 4 r + t: eight values of k for MMA row r.  A word's halves-apart nibbles
//     (j, j + 4) become a register pair of 16-bit values by a shift and one and-or with the bits
//     of a power of two whose last mantissa bits hold them; a subtraction leaves q - z, exactly
//     (W4Unpack).  The rows of A are paired in the same order (the order
//     of k inside an MMA is free as long as both operands have it).
//   * A group's sum is complete in the accumulator (groups are whole MMAs, all of whose lanes
//     are in one group), so the scale multiplies an fp32 sum, and no weight is ever rounded.
//   * The KW warps' sums meet in shared memory, in order; then the epilogue.
// Measured (bf16, groups of 128, weights from DRAM): 4096 x 4096 with one row 5.0 us, 4096 x 1024
// 2.8; 8 rows of 8192 x 8192 14.0 us, with groups of 64 of 16384 x 8192 26.3 (40 % of the copy rate
// for the weight's bytes); groups of 32 with one row 5.3 us, 2.9, and 8192 x 8192 13.2.  With one row of
// 8192 columns, k 16384, the loads alone took 13.4 us, the arithmetic alone 17.6, both 22.7: the larger
// weights of up to 4 rows have a kernel of their own.  Tried and left: bulk copies of rows by one warp
// (33 us: 75 cycles for each copy of 512 bytes), 16 warps a block (26.6), 256 values of k per warp and
// stage (22.8).
#include "kernel_params.h"
#include "launch.h"
#include "ptx.cuh"
#include "vec16.cuh"
#include "w4_mma.cuh"
#include "w4_unpack.cuh"

namespace gemm_epi {

namespace {

constexpr int kWarps = 8;
constexpr int kThreadsW4 = kWarps * 32;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kBlockK = 128;  // values of k per warp and stage: 64 bytes of each row of W

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// One stage in shared memory for m rows of A, in bytes.  Rows are padded so that eight rows'
// 16-byte pieces (ldmatrix), or two rows' 64 bytes (rows of A), fall in different banks.
template <int MT, int CW, int G>
struct W4Stage {
    static constexpr int kKW = kWarps / CW;
    static constexpr int kCols = 16 * MT * CW;
    static constexpr int kStageK = kBlockK * kKW;
    static constexpr int kGroups = kStageK / G;
    static constexpr int kWRow = kKW * 64 + 16;
    static constexpr int kARow = kStageK * 2 + 64;
    static constexpr int kScales = kCols * kWRow;                  // [group][column] 16 bits
    static constexpr int kZeros = kScales + kGroups * kCols * 2;   // [group][column] bytes
    static constexpr int kA = kZeros + kGroups * kCols;
    static __host__ __device__ constexpr int bytes(int m) { return kA + m * kARow; }
};

// cluster: CTAs of a cluster that split k (their sums meet over distributed shared memory).
template <bool BF16, int NT, int MT, int CW, int G, int STAGES>
__global__ void __launch_bounds__(kThreadsW4) w4_matmul_kernel(const W4Args a, int cluster)
{
    using S = W4Stage<MT, CW, G>;
    constexpr int KW = S::kKW;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cw = warp % CW, kw = warp / CW;
    const int rank = static_cast<int>(blockIdx.x) % cluster;
    const int n0 = static_cast<int>(blockIdx.x) / cluster * S::kCols;
    const int cols = min(S::kCols, a.n - n0);
    const int stage_bytes = S::bytes(a.m);
    const int all_steps = (a.k + S::kStageK - 1) / S::kStageK;
    const int first = static_cast<int>(static_cast<long long>(all_steps) * rank / cluster);
    const int steps = static_cast<int>(static_cast<long long>(all_steps) * (rank + 1) / cluster) - first;

    // What this thread copies in every stage.  W: kWCopies 16-byte chunks (32 values of k) of
    // column wcol, kWLanes chunks apart; columns past n copy the last one's (nobody reads what
    // comes of them).  A: chunk ac (8 values) of rows arow, arow + kARows, ...  Scales and zero
    // points: 8 columns of one group, the first half of the block and the second.
    constexpr int kWLanes = kThreadsW4 / S::kCols;
    constexpr int kWCopies = KW * 4 / kWLanes;
    constexpr int kAChunks = S::kStageK / 8;
    constexpr int kARows = kThreadsW4 / kAChunks;
    constexpr int kSChunks = S::kGroups * (S::kCols / 8);
    static_assert(kThreadsW4 % S::kCols == 0 && KW * 4 % kWLanes == 0 && kThreadsW4 % kAChunks == 0 &&
                      2 * kSChunks <= kThreadsW4, "every thread has a fixed part in the copies");
    const int wcol = tid / kWLanes, wc = tid % kWLanes;
    const int ac = tid % kAChunks, arow = tid / kAChunks;
    const int sc = tid % (kThreadsW4 / 2);
    const int sgroup = sc / (S::kCols / 8), scol = sc % (S::kCols / 8) * 8;
    const bool copies_scales = tid < kSChunks;
    const bool copies_zeros = a.zeros != nullptr && tid >= kThreadsW4 / 2 && sc < kSChunks;
    const uint8_t* wsrc = static_cast<const uint8_t*>(a.W) +
                          (static_cast<long long>(min(n0 + wcol, a.n - 1)) * a.k + first * S::kStageK) / 2 + wc * 16;
    const uint16_t* asrc = static_cast<const uint16_t*>(a.A) + static_cast<long long>(arow) * a.k + first * S::kStageK + ac * 8;
    const long long a_step = static_cast<long long>(kARows) * a.k;
    const long long s_step = static_cast<long long>(S::kGroups) * a.n;
    const long long sat = static_cast<long long>(first * S::kGroups + sgroup) * a.n + min(n0 + scol, a.n - 8);
    const uint16_t* ssrc = static_cast<const uint16_t*>(a.scales) + sat;
    const uint8_t* zsrc = a.zeros + sat;
    const uint32_t wdst = wcol * S::kWRow + wc * 16;
    const uint32_t adst = S::kA + arow * S::kARow + ac * 16;
    int load_left = a.k - first * S::kStageK;  // values of k from the next stage to load on

    auto load = [&](uint32_t st) {
        // (past the end of k nothing is copied, and nothing of it is read)
        const bool whole = load_left >= S::kStageK;
#pragma unroll
        for (int i = 0; i < kWCopies; ++i)
            if (whole || (wc + i * kWLanes) * 32 < load_left)
                cp_async_16(st + wdst + i * kWLanes * 16, wsrc + i * kWLanes * 16);
        wsrc += S::kStageK / 2;
        if (whole || ac * 8 < load_left) {
            const uint16_t* ap = asrc;
            uint32_t dst = st + adst;
            for (int row = arow; row < a.m; row += kARows) {
                cp_async_16(dst, ap);
                ap += a_step;
                dst += kARows * S::kARow;
            }
        }
        asrc += S::kStageK;
        if (whole || sgroup * G < load_left) {
            if (copies_scales) cp_async_16(st + S::kScales + (sgroup * S::kCols + scol) * 2, ssrc);
            if (copies_zeros) cp_async_8(st + S::kZeros + sgroup * S::kCols + scol, zsrc);
        }
        ssrc += s_step;
        zsrc += s_step;
        load_left -= S::kStageK;
    };

    float total[MT][NT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) total[i][j][c] = 0.0f;

    grid_dependency_wait();
    grid_launch_dependents();
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (s < steps) load(sbase + s * stage_bytes);
        cp_async_commit();
    }
    const int r = lane >> 2, t = lane & 3;
    // byte offsets in a stage of what this lane reads
    const uint32_t woff = (cw * MT * 16 + (lane & 7)) * S::kWRow + kw * 64 + ((lane >> 3) << 4);
    int aoff[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)  // (rows past m: columns of the product that nobody reads)
        aoff[j] = S::kA + min(j * 8 + r, a.m - 1) * S::kARow + kw * 256 + t * 16;
    const int soff = S::kScales + (kw * (kBlockK / G) * S::kCols + cw * MT * 16 + r) * 2;
    const int zat = S::kZeros + kw * (kBlockK / G) * S::kCols + cw * MT * 16 + r;
    int k_left = a.k - first * S::kStageK - kw * kBlockK;  // from this warp's part of the stage on
    int slot = 0, fill = (STAGES - 1) * stage_bytes;       // byte offsets of stages
    for (int step = 0; step < steps; ++step, k_left -= S::kStageK) {
        // this step's copies (of this thread, then of all) have landed, and every warp is done
        // with the stage that the next load overwrites
        cp_async_wait_group<STAGES - 2>();
        __syncthreads();
        if (step + STAGES - 1 < steps) load(sbase + fill);
        cp_async_commit();
        fill = fill == (STAGES - 1) * stage_bytes ? 0 : fill + stage_bytes;
        const uint8_t* stp = smem + slot;
        const uint32_t st = sbase + slot;
        slot = slot == (STAGES - 1) * stage_bytes ? 0 : slot + stage_bytes;
        auto block = [&](int chunks) {
            uint32_t w[MT][2][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) ldmatrix_x4(w[i][h], st + woff + (i * 16 + h * 8) * S::kWRow);
            float part[MT][NT][4];
            W4Unpack<BF16> unpack[MT][2];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (c >= chunks) break;
                const int g = c * 32 / G;  // this warp's group
                if (c * 32 % G == 0) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        unpack[i][0].set(a.zeros ? stp[zat + g * S::kCols + i * 16] : 8);
                        unpack[i][1].set(a.zeros ? stp[zat + g * S::kCols + i * 16 + 8] : 8);
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int e = 0; e < 4; ++e) part[i][j][e] = 0.0f;
                    }
                }
                // rows of A: 8 values of k per lane, paired (k, k + 4)
                uint32_t b[NT][4];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 v = *reinterpret_cast<const uint4*>(stp + aoff[j] + c * 64);
                    b[j][0] = __byte_perm(v.x, v.z, 0x5410);
                    b[j][1] = __byte_perm(v.x, v.z, 0x7632);
                    b[j][2] = __byte_perm(v.y, v.w, 0x5410);
                    b[j][3] = __byte_perm(v.y, v.w, 0x7632);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    uint32_t p[4], q[4];
                    unpack[i][0](w[i][0][c], p);
                    unpack[i][1](w[i][1][c], q);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        mma_16816<BF16>(part[i][j], p[0], q[0], p[1], q[1], b[j][0], b[j][1]);
                        mma_16816<BF16>(part[i][j], p[2], q[2], p[3], q[3], b[j][2], b[j][3]);
                    }
                    if ((c + 1) * 32 % G == 0) {
                        const uint16_t* s16 = reinterpret_cast<const uint16_t*>(stp + soff) + g * S::kCols + i * 16;
                        const float s0 = decode16<BF16>(s16[0]), s1 = decode16<BF16>(s16[8]);
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
        };
        if (k_left >= kBlockK)
            block(4);
        else if (k_left > 0)
            block(k_left / 32);  // (k ends on a group's border)
    }
    cp_async_wait_group<0>();

    // The k-warps' sums: [kw][row of A][column], then one thread per element adds them in order.
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
    const int elements = a.m * S::kCols;
    if (cluster > 1) {
        for (int i = tid; i < elements; i += kThreadsW4) {
            const int at = i / S::kCols * kRedRow + i % S::kCols;
            float v = red[at];
#pragma unroll
            for (int q = 1; q < KW; ++q) v += red[q * NT * 8 * kRedRow + at];
            red[at] = v;
        }
        cluster_sync_all();
    }
    for (int i = rank * kThreadsW4 + tid; i < elements; i += kThreadsW4 * cluster) {
        const int row = i / S::kCols, col = i % S::kCols;
        if (col >= cols) continue;
        const int ra = row * kRedRow + col;
        float v = 0.0f;
        if (cluster > 1) {
            for (int q = 0; q < cluster; ++q) v += ld_shared_cluster_f32(map_shared_rank(sbase + ra * 4, q));
        } else {
#pragma unroll
            for (int q = 0; q < KW; ++q) v += red[q * NT * 8 * kRedRow + ra];
        }
        const long long at = static_cast<long long>(row) * a.n + n0 + col;
        if (a.bias) v += decode16<BF16>(static_cast<const uint16_t*>(a.bias)[n0 + col]);
        const float res = a.residual ? decode16<BF16>(static_cast<const uint16_t*>(a.residual)[at]) : 0.0f;
        static_cast<uint16_t*>(a.D)[at] = encode16<BF16>(w4_epilogue(v, a.epilog, res));
    }
    if (cluster > 1) cluster_sync_all();  // the peers' shared memory stays until it is read
}

template <bool BF16, int NT, int MT, int CW, int G, int STAGES>
cudaError_t w4_launch_one(const W4Args& a, int sms, cudaStream_t stream)
{
    using S = W4Stage<MT, CW, G>;
    auto kernel = w4_matmul_kernel<BF16, NT, MT, CW, G, STAGES>;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(kernel, kMaxSmem, prepared);
    if (e != cudaSuccess) return e;
    const int steps = (a.k + S::kStageK - 1) / S::kStageK;
    const int tiles = (a.n + S::kCols - 1) / S::kCols;
    int smem = STAGES * S::bytes(a.m);
    const int red = S::kKW * NT * 8 * (S::kCols + 1) * 4;
    if (smem < red) smem = red;
    // k split over a cluster while that leaves an SM for every block (1024 columns, k 4096, one row:
    // 4.5 us whole, 3.9 in 2, 3.75 in 4, 4.2 in 8; 12 rows 12.7, 8.4, 5.4 and 4.85; 4096x4096, one row,
    // where 128 blocks have 128 SMs: 5.0 whole, 5.4 in 2, 8.3 in 4; 8 rows 5.5, 5.7 and 9.0)
    int cluster = 1;
    while (cluster < 8 && tiles * cluster * 2 <= sms && steps >= 2 * cluster) cluster *= 2;
    return launch_dependent(kernel, tiles * cluster, kThreadsW4, smem, stream, cluster, a, cluster);
}

template <bool BF16, int NT, int MT, int CW, int STAGES>
cudaError_t w4_launch_group(const W4Args& a, int sms, cudaStream_t stream)
{
    if (a.group == 32) return w4_launch_one<BF16, NT, MT, CW, 32, STAGES>(a, sms, stream);
    if (a.group == 64) return w4_launch_one<BF16, NT, MT, CW, 64, STAGES>(a, sms, stream);
    return w4_launch_one<BF16, NT, MT, CW, 128, STAGES>(a, sms, stream);
}

template <bool BF16>
cudaError_t w4_launch_type(const W4Args& a, int sms, cudaStream_t stream)
{
    const long long weights = static_cast<long long>(a.n) * a.k;
    // up to 4 rows of a large weight: without the stages in shared memory (one row, groups of
    // 128: 8192x8192 10.0 us there, 12.4 here, 4096x4096 4.3 and 4.4, 4096x1024 2.8 and 2.3;
    // groups of 64: 8192x8192 11.4 and 12.9, 5120x5120 8.2 and 8.2; 8 rows 16.0 and 13.9)
    if (a.m <= 4 && a.group >= 64 && weights >= (a.group == 128 ? 20ll : 60ll) << 20)
        return w4_stream_launch(a, BF16, sms, stream);
    if (a.m <= 4) return w4_launch_group<BF16, 1, 2, 1, 4>(a, sms, stream);
    // 5 to 8 rows: tcgen05's lower rate of instructions outweighs its longer start only where the
    // weight is large and the groups are few (8 rows, groups of 128: 16384x8192 26.6 us here, 23.0
    // there, 8192x16384 25.7 and 24.3, 8192x8192 14.2 and 14.9; groups of 64: 26.9 and 26.6, 26.2
    // and 27.8)
    if (a.m <= 8 && (a.group < 128 || weights < 96ll << 20)) return w4_launch_group<BF16, 1, 2, 1, 3>(a, sms, stream);
    // 9 to 16 rows: this kernel's second tile of rows costs a small weight less than tcgen05's
    // longer start (12 rows: 4096x1024 4.4 us here, 5.4 there, 1024x4096 4.9 and 6.2), a large one
    // more (4096x4096 8.4 and 7.7, 8192x8192 24.6 and 15.0)
    if (a.m <= 16 && weights <= 12ll << 20)
        return w4_launch_group<BF16, 2, 1, 4, 4>(a, sms, stream);
    return w4_tensor_launch(a, BF16, sms, stream);
}

// The weight written out: a block turns 128 (k) x TN (n) of W, column by column in memory, into
// rows of B.  A thread unpacks 32 values of k of two neighbouring columns, so that a
// (k, two columns) word is one 4-byte store to shared memory; the words of a row are permuted
// by 8 times the number of its 32 rows, which puts the four rows a warp stores to at a time in
// different banks.  (q - z) is exact in 16 bits, and the 16-bit product with the scale is the
// exact product rounded once.  Bound by B's bytes.
constexpr int kDequantK = 128;

template <bool BF16>
__device__ __forceinline__ uint32_t mul16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16)
        asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <bool BF16, int TN>
__global__ void __launch_bounds__(2 * TN) w4_dequantize_kernel(const W4Args a)
{
    extern __shared__ uint32_t tile[];  // [kDequantK][TN / 2]
    const int n_tiles = (a.n + TN - 1) / TN;
    const int n0 = blockIdx.x % n_tiles * TN, k0 = blockIdx.x / n_tiles * kDequantK;
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = threadIdx.x & 3, pair = threadIdx.x >> 2;
    const int col = n0 + 2 * pair, k = k0 + 32 * t;
    if (col < a.n && k < a.k) {  // (n is even, k a multiple of 32)
        const uint8_t* src = static_cast<const uint8_t*>(a.W) + (static_cast<long long>(col) * a.k + k) / 2;
        const uint4 w0 = __ldcs(reinterpret_cast<const uint4*>(src));
        const uint4 w1 = __ldcs(reinterpret_cast<const uint4*>(src + a.k / 2));
        const long long at = static_cast<long long>(k / a.group) * a.n + col;
        const uint32_t s = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.scales) + at);
        const uint32_t z = a.zeros ? *reinterpret_cast<const uint16_t*>(a.zeros + at) : 0x0808u;
        const uint32_t s0 = __byte_perm(s, s, 0x1010), s1 = __byte_perm(s, s, 0x3232);
        W4Unpack<BF16> u0, u1;
        u0.set(z & 0xFFu);
        u1.set(z >> 8);
        const uint32_t ww0[4] = {w0.x, w0.y, w0.z, w0.w}, ww1[4] = {w1.x, w1.y, w1.z, w1.w};
        uint32_t* to = tile + 32 * t * (TN / 2) + (pair ^ (8 * t));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v0[4], v1[4];
            u0(ww0[i], v0);
            u1(ww1[i], v1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = mul16x2<BF16>(v0[j], s0), y = mul16x2<BF16>(v1[j], s1);
                to[(8 * i + j) * (TN / 2)] = __byte_perm(x, y, 0x5410);
                to[(8 * i + j + 4) * (TN / 2)] = __byte_perm(x, y, 0x7632);
            }
        }
    }
    __syncthreads();
    constexpr int kPerRow = TN / 8, kRowsAtOnce = 2 * TN / kPerRow;
    const int c = threadIdx.x % kPerRow * 8;
    if (n0 + c >= a.n) return;  // (n is a multiple of 8)
    const int rows = min(kDequantK, a.k - k0);
    uint16_t* out = static_cast<uint16_t*>(a.D) + static_cast<long long>(k0) * a.n + n0 + c;
#pragma unroll
    for (int i = 0; i < kDequantK / kRowsAtOnce; ++i) {
        const int row = i * kRowsAtOnce + threadIdx.x / kPerRow;
        if (row < rows) {
            const uint4 v = *reinterpret_cast<const uint4*>(tile + row * (TN / 2) + ((c / 2) ^ (8 * (row / 32))));
            uint4* p = reinterpret_cast<uint4*>(out + static_cast<long long>(row) * a.n);
            if (a.streams)
                __stcs(p, v);
            else
                *p = v;
        }
    }
}

template <bool BF16, int TN>
cudaError_t w4_dequantize_one(const W4Args& a, cudaStream_t stream)
{
    constexpr int kSmem = kDequantK * TN * 2;
    static std::atomic<unsigned long long> prepared;
    const cudaError_t e = allow_smem(w4_dequantize_kernel<BF16, TN>, kSmem, prepared);
    if (e != cudaSuccess) return e;
    const long long n_tiles = (a.n + TN - 1) / TN, k_tiles = (a.k + kDequantK - 1) / kDequantK;
    return launch_dependent(w4_dequantize_kernel<BF16, TN>, static_cast<int>(n_tiles * k_tiles), 2 * TN, kSmem, stream, 1, a);
}

}  // namespace

cudaError_t w4_matmul_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    return bf16 ? w4_launch_type<true>(a, sm_count, stream) : w4_launch_type<false>(a, sm_count, stream);
}

cudaError_t w4_dequantize_launch(const W4Args& a, bool bf16, int sm_count, cudaStream_t stream)
{
    // 256 columns a block where that leaves two blocks per SM (8192x16384: 54.4 us, 63.7 with 128
    // columns; 4096x1024: 3.5 us, 2.9 with 128); a B that L2 cannot hold is stored past it
    const long long blocks = ((a.n + 255) / 256) * static_cast<long long>((a.k + kDequantK - 1) / kDequantK);
    W4Args b = a;
    b.streams = static_cast<long long>(a.n) * a.k * 2 > 64ll << 20;
    if (blocks >= 2ll * sm_count)
        return bf16 ? w4_dequantize_one<true, 256>(b, stream) : w4_dequantize_one<false, 256>(b, stream);
    return bf16 ? w4_dequantize_one<true, 128>(b, stream) : w4_dequantize_one<false, 128>(b, stream);
}

}  // namespace gemm_epi
