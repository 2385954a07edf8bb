"""The streaming 4-bit product's shared memory over the whole range of k (no GPU): the kernel's own size
arithmetic, compiled for the host."""
import os
import subprocess

import pytest

from activation_epilogue_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
MAX_SMEM, STEP_K, UNROLL = 100 * 1024, 1024, 4


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("w4") / "sizes")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-I", libbuild.CSRC, os.path.join(HERE, "w4_stream_sizes.cpp"), "-o", exe], check=True)
    return exe


def test_segments_fit_and_are_the_largest_that_do(program):
    # steps of a block: k = 2^30 at most, a cluster of 8 at most; every size near the limits of shared
    # memory and of 32 bits (4 rows: 2^31 bytes are 2^18 steps)
    counts = sorted({*range(0, 80), *(2 ** i + j for i in range(6, 20) for j in (-1, 0, 1)), 2 ** 20 - 1, 2 ** 20})
    asked = [(g, m, s) for g in (64, 128) for m in (1, 2, 3, 4) for s in counts]
    out = subprocess.run([program], input="".join("%d %d %d\n" % a for a in asked), capture_output=True, text=True, check=True)
    rows = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    assert len(rows) == len(asked)
    for (g, m, steps), (seg, size, larger) in zip(asked, rows):
        pad = 32 if g == 128 else 16
        assert size == m * (seg * STEP_K * 2 + pad) + seg * (STEP_K // g) * 32 * 3
        assert seg >= UNROLL and seg % UNROLL == 0 and size <= MAX_SMEM, (g, m, steps, seg, size)
        # all of k, or the next round would not fit
        assert seg >= steps or larger > MAX_SMEM, (g, m, steps, seg)
        assert seg < max(steps, 1) + UNROLL
