// Reads lines "group rows steps" and prints the streaming 4-bit product's segment for them: its steps,
// its bytes, and the bytes of a segment of one more round of the unrolled loop.
#include <cstdio>

#include "w4_segment.h"

template <int G>
static void print(int m, int steps)
{
    using S = gemm_epi::Segment<G>;
    const int seg = S::steps_for(m, steps);
    std::printf("%d %d %d\n", seg, S::bytes(m, seg), S::bytes(m, seg + gemm_epi::kStreamUnroll));
}

int main()
{
    int g, m, steps;
    while (std::scanf("%d %d %d", &g, &m, &steps) == 3) {
        if (g == 128)
            print<128>(m, steps);
        else
            print<64>(m, steps);
    }
    return 0;
}
