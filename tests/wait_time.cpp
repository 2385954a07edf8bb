// Reads steps between two looks at a clock, in nanoseconds, and how many of each, and prints the time that
// a wait has counted.
#include <cstdio>

#include "wait_time.h"

int main()
{
    unsigned long long now = 5, step, repeat, total = 0;
    gemm_epi::WaitTime waited(now);
    while (std::scanf("%llu %llu", &step, &repeat) == 2)
        for (unsigned long long i = 0; i < repeat; ++i) total = waited.at(now += step);
    std::printf("%llu\n", total);
    return 0;
}
