"""The 64-bit references of the sub-layer operators, pinned without a GPU: the generator to its
published vectors, gradients to differences, the 4-bit layout to a loop."""
import numpy as np
import pytest
import torch

import sublayer_reference as ref


@pytest.mark.parametrize("counter,key,want", [
    # published known answers of Philox4x32-10
    ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
    ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
    ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
     [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
])
def test_philox_known_answers(counter, key, want):
    assert [int(w[0]) for w in ref.philox4x32([[c] for c in counter], key)] == want


def test_dropout_keep_rate_and_windows():
    keep = ref.dropout_keep(0, 200001, 0.3, seed=2 ** 63 + 5, offset=2 ** 64 - 100)
    assert abs(keep.mean() - 0.7) < 5 * np.sqrt(0.21 / keep.size)
    assert np.array_equal(keep[8000:9000], ref.dropout_keep(8000, 1000, 0.3, 2 ** 63 + 5, 2 ** 64 - 100))
    assert ref.dropout_keep(0, 99, 0.0, 1, 2).all() and not ref.dropout_keep(0, 99, 1.0, 1, 2).any()


def test_rmsnorm_backward_against_differences():
    g = torch.Generator().manual_seed(3)
    h, dy, dh = (torch.randn(3, 16, generator=g, dtype=torch.float64) for _ in range(3))
    gamma = torch.rand(16, generator=g, dtype=torch.float64) + 0.5

    def f(hh, gg):
        return float((ref.rmsnorm(hh, gg, 1e-3)[0] * dy).sum() + (hh * dh).sum())
    dx, dgamma, _, _ = ref.rmsnorm_backward(dy, h, gamma, ref.rmsnorm(h, gamma, 1e-3)[1], dh)
    step = 1e-5
    for i, j in ((0, 0), (1, 7), (2, 15)):
        e = torch.zeros_like(h)
        e[i, j] = step
        assert abs((f(h + e, gamma) - f(h - e, gamma)) / (2 * step) - float(dx[i, j])) < 1e-7
    for j in (0, 9):
        e = torch.zeros_like(gamma)
        e[j] = step
        assert abs((f(h, gamma + e) - f(h, gamma - e)) / (2 * step) - float(dgamma[j])) < 1e-7


def test_w4_layout_by_hand():
    p = ref.w4_problem(2, 8, 64, 32, "f16", True, 1)
    B = ref.w4_weight(p["q"], p["scales"], p["zeros"], 32)
    for i, j in ((0, 0), (33, 5), (63, 7), (31, 2)):
        byte = int(p["W"][j, i // 2])
        q = byte >> 4 if i % 2 else byte & 15
        want = (q - int(p["zeros"][i // 32, j])) * float(p["scales"][i // 32, j])
        assert float(B[i, j]) == want
