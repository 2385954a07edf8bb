// Shared memory of the streaming 4-bit product: how much of k a block holds of A and of the scales at
// a time.  Plain arithmetic, for the host's launch and the kernel alike.
#pragma once

#ifdef __CUDACC__
#define W4_HOST_DEVICE __host__ __device__
#else
#define W4_HOST_DEVICE
#endif

namespace gemm_epi {

constexpr int kStreamCols = 32;                           // columns of D per block (most)
constexpr int kStreamWarps = 8;
constexpr int kStreamBlockK = 128;                        // k per warp at a time
constexpr int kStreamStepK = kStreamWarps * kStreamBlockK;  // k per step of the block
constexpr int kStreamUnroll = 4;                          // steps in the kernel's unrolled loop
constexpr int kStreamMaxSmem = 100 * 1024;                // two blocks per SM
constexpr int kStreamMaxRows = 4;

// A segment of `steps` steps for m rows of A.  A row is padded, and with groups of 128 its 16-byte
// pieces exchanged in pairs, so that the eight lanes that read at a time (two rows, four pieces) find
// eight different banks.
template <int G>
struct Segment {
    static constexpr int kPad = G == 128 ? 32 : 16;
    static constexpr int kGroups = kStreamStepK / G;  // per step
    static W4_HOST_DEVICE int pitch(int steps) { return steps * kStreamStepK * 2 + kPad; }
    static W4_HOST_DEVICE int scales(int m, int steps) { return m * pitch(steps); }
    static W4_HOST_DEVICE int zeros(int m, int steps) { return scales(m, steps) + steps * kGroups * kStreamCols * 2; }
    static W4_HOST_DEVICE int bytes(int m, int steps) { return zeros(m, steps) + steps * kGroups * kStreamCols; }

    // Steps in a segment for a block with `needed` steps of k (up to 2^20): all of them, rounded up to
    // the unrolled loop's, or as many as fit.  (From the bytes of one step: those of all of a long k
    // may pass 2^31.)
    static W4_HOST_DEVICE int steps_for(int m, int needed)
    {
        const int per_step = m * kStreamStepK * 2 + kGroups * kStreamCols * 3;
        const int most = (kStreamMaxSmem - m * kPad) / per_step / kStreamUnroll * kStreamUnroll;
        const int all = (needed + kStreamUnroll - 1) / kStreamUnroll * kStreamUnroll;
        return all < kStreamUnroll ? kStreamUnroll : all < most ? all : most;
    }
    static_assert(kPad % 16 == 0 && (kStreamMaxRows * (kStreamStepK * 2 + kPad) + kGroups * kStreamCols * 3) * kStreamUnroll <=
                                        kStreamMaxSmem, "one round of the unrolled loop fits");
};

}  // namespace gemm_epi
