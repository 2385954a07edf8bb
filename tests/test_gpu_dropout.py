"""Dropout from the counter-based generator (+ residual): the mask bit for bit, the values
against 64 bits."""
import numpy as np
import pytest
import torch

import sublayer_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import TD

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(count, dtype, seed, residual):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(count, generator=g)
    X = torch.where(X == 0, 1.0, X).to(TD[dtype])
    return X, torch.randn(count, generator=g).to(TD[dtype]) if residual else None


def _run(X, R, p, seed, offset, dtype, offset_device=None):
    Y = torch.full((X.numel() + 9,), 7.0, dtype=TD[dtype], device="cuda")
    gemm_epi.gemm_epi_dropout(X.numel(), dtype, X.cuda(), None if R is None else R.cuda(), p, seed, offset, Y,
                              offset_device)
    torch.cuda.synchronize()
    assert (Y[X.numel():] == 7.0).all()
    return Y[:X.numel()].cpu()


@pytest.mark.parametrize("count", [1, 7, 8, 9, 250, 2048, 2049, 100003, 1 << 20])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout(count, dtype, residual):
    X, R = _inputs(count, dtype, count, residual)
    p, seed, offset = 0.3, 0xFEDCBA9876543210 ^ count, 2 ** 32 - 3   # the counter's low word wraps
    keep = ref.dropout_keep(0, count, p, seed, offset)
    Y = _run(X, R, p, seed, offset, dtype)
    if not residual:
        assert np.array_equal((Y != 0).numpy(), keep)
    want = ref.dropout(X, R, keep, p)
    size = X.double().abs() * 65536 / (65536 - ref.dropped(p)) + (0 if R is None else R.double().abs())
    ref.check_16(Y, want, dtype, 2 * ref.F32 * size, "Y")


@pytest.mark.parametrize("p", [0.0, 1.0, 2.0 ** -17, 1e-5, 0.5, 1 - 2.0 ** -16, 1 - 2.0 ** -18])
def test_dropout_probabilities(p):
    X, R = _inputs(5000, "bf16", 3, True)
    keep = ref.dropout_keep(0, 5000, p, 12, 34)
    Y = _run(X, R, p, 12, 34, "bf16")
    want = ref.dropout(X, R, keep, p)
    size = want.abs() + R.double().abs()
    ref.check_16(Y, want, "bf16", 4 * ref.F32 * size, "Y")
    if p == 0.0:
        assert torch.equal(_run(X, None, p, 1, 2, "bf16"), X)
    if p == 1.0:
        assert torch.equal(Y, R) and (_run(X, None, p, 1, 2, "bf16") == 0).all()


def test_dropout_backward_is_the_same_mask():
    X, _ = _inputs(10007, "f16", 8, False)
    dY, _ = _inputs(10007, "f16", 9, False)
    Y = _run(X, None, 0.25, 77, 5, "f16")
    dX = _run(dY, None, 0.25, 77, 5, "f16")
    assert torch.equal(Y == 0, dX == 0)
    # Y is linear in X: the directional difference of the call is the call on the direction
    step = _run((X.float() + 1).half(), None, 0.25, 77, 5, "f16").double() - Y.double()
    moved = (X.float() + 1).half().double() - X.double()
    assert ((step - moved * (dX.double() / dY.double())).abs() <= 2.0 ** -9 * (Y.double().abs() + 2)).all()


def test_dropped_values_do_not_matter_and_in_place():
    X, R = _inputs(4096, "bf16", 10, True)
    keep = ref.dropout_keep(0, 4096, 0.5, 1, 0)
    bad = X.clone()
    bad[torch.from_numpy(~keep)] = float("nan")
    assert torch.equal(_run(bad, R, 0.5, 1, 0, "bf16"), _run(X, R, 0.5, 1, 0, "bf16"))
    for target in ("X", "R"):
        Xg, Rg = X.cuda(), R.cuda()
        out = Xg if target == "X" else Rg
        gemm_epi.gemm_epi_dropout(4096, "bf16", Xg, Rg, 0.5, 1, 0, out)
        assert torch.equal(out.cpu(), _run(X, R, 0.5, 1, 0, "bf16"))


def test_dropout_counters_continue():
    # two calls, the second's offset ceil(count / 8) further on, draw one longer call's mask
    X, _ = _inputs(8016, "bf16", 11, False)
    whole = _run(X, None, 0.4, 5, 2 ** 64 - 500, "bf16")        # the 64-bit counter wraps
    parts = [_run(X[:4000].contiguous(), None, 0.4, 5, 2 ** 64 - 500, "bf16"),
             _run(X[4000:].clone(), None, 0.4, 5, 0, "bf16")]
    assert torch.equal(whole, torch.cat(parts))


def test_dropout_offset_on_the_device_in_a_graph():
    X, R = _inputs(3000, "f16", 12, True)
    Xg, Rg = X.cuda(), R.cuda()
    Y = torch.zeros(3000, dtype=torch.float16, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gemm_epi.gemm_epi_dropout(3000, "f16", Xg, Rg, 0.2, 9, 100, Y, step)
        step.add_(375)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y.cpu(), _run(X, R, 0.2, 9, 100 + 375 * i, "f16")), i


@pytest.mark.slow
def test_dropout_offsets_past_32_bits():
    count = 2 ** 32 + 13
    X = torch.ones(count, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(count, dtype=torch.bfloat16, device="cuda")
    gemm_epi.gemm_epi_dropout(count, "bf16", X, None, 0.5, 3, 7, Y)
    for first in (0, 2 ** 31 - 1000, 2 ** 32 - 1000 + 1000 % 8):
        n = min(5000, count - first)
        keep = ref.dropout_keep(first, n, 0.5, 3, 7)
        assert np.array_equal(Y[first:first + n].float().cpu().numpy(), 2.0 * keep)
