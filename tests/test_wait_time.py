"""What a kernel's bounded wait counts as waited: its own time, not that of a context which another one
displaced (no GPU; the kernels' own arithmetic, compiled for the host)."""
import os
import subprocess

import pytest

from activation_epilogue_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
LIMIT = 2 * 10 ** 9


@pytest.fixture(scope="module")
def waited(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("wait") / "time")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", libbuild.CSRC,
                    os.path.join(HERE, "wait_time.cpp"), "-o", exe], check=True)

    def run(*steps):
        text = "".join("%d %d\n" % s for s in steps)
        return int(subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout)
    return run


def test_a_running_kernel_s_time_counts_in_full(waited):
    # one look in 100 us, a suspension's limit: the wait ends after two seconds
    assert waited((100_000, 20_000)) == LIMIT
    assert waited((37, 1000)) == 37_000


def test_time_displaced_from_the_gpu_does_not(waited):
    assert waited((100_000, 10), (60 * 10 ** 9, 1), (100_000, 10)) == 3_000_000
    assert waited(*[(60 * 10 ** 9, 1), (100_000, 10)] * 50) == 100_000_000


def test_a_wait_ends_however_rarely_it_looks(waited):
    assert waited((10 ** 9, 2001)) > LIMIT
