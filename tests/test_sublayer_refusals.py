"""The RMS norm, 4-bit-weight and dropout calls: what they refuse, and the empty problems they
accept, before any device is touched (no GPU)."""
import ctypes

import pytest
import torch

from activation_epilogue_gb300 import build as libbuild
from activation_epilogue_gb300 import gemm_epi

P = 1 << 20          # an aligned address that no call may read
INVALID, SHAPE, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    gemm_epi.load_library()


def _status(call, **kw):
    with pytest.raises(gemm_epi.GemmEpiError) as e:
        call(**kw, stream=0)
    return e.value.status


NORM = dict(t=4, d=64, dtype="bf16", X=P, residual=P, gamma=P, eps=1e-6, H=P, Y=2 * P)


@pytest.mark.parametrize("change,status", [
    (dict(dtype="e4m3"), INVALID), (dict(t=-1), SHAPE), (dict(d=12), SHAPE), (dict(d=0), SHAPE),
    (dict(t=2 ** 31), SHAPE), (dict(t=1, d=2 ** 30 + 8), SHAPE), (dict(t=2 ** 30, d=8192), SHAPE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(X=None), INVALID),
    (dict(gamma=None), INVALID), (dict(Y=None), INVALID), (dict(H=None), INVALID),
    (dict(residual=None), INVALID), (dict(Y=P, H=P), INVALID), (dict(X=P + 8), MISALIGNED),
    (dict(gamma=P + 2), MISALIGNED), (dict(H=P + 8), MISALIGNED), (dict(Y=P + 8), MISALIGNED),
    (dict(residual=P + 8), MISALIGNED), (dict(rstd=P + 2), MISALIGNED),
])
def test_rmsnorm_refusals(change, status):
    assert _status(gemm_epi.gemm_epi_rmsnorm, **{**NORM, **change}) == status


NORM8 = dict(t=4, d=64, dtype="f16", X=P, residual=None, gamma=P, eps=1e-6, H=None, Q=2 * P,
             mode="TENSOR", scale=P, workspace=P)


@pytest.mark.parametrize("change,status", [
    (dict(scale=None), INVALID), (dict(workspace=None), INVALID), (dict(Q=P), INVALID),
    (dict(scale=P + 2), MISALIGNED), (dict(workspace=P + 8), MISALIGNED), (dict(Q=P + 8), MISALIGNED),
    (dict(d=4), SHAPE), (dict(dtype="e4m3"), INVALID), (dict(mode="ROW", scale=None), INVALID),
    (dict(residual=2 * P, H=3 * P), INVALID),
])
def test_rmsnorm_e4m3_refusals(change, status):
    assert _status(gemm_epi.gemm_epi_rmsnorm_e4m3, **{**NORM8, **change}) == status


def test_rmsnorm_e4m3_bad_mode():
    lib = gemm_epi.load_library()
    for mode in (-1, 3):
        assert lib.gemm_epi_rmsnorm_e4m3(4, 64, 1, P, None, P, 1e-6, None, 2 * P, mode, P, None, P,
                                         None) == INVALID


BWD = dict(t=4, d=64, dtype="bf16", dY=P, H=2 * P, gamma=P, rstd=P, dH=None, dX=3 * P, dgamma=P,
           workspace=P)


@pytest.mark.parametrize("change,status", [
    (dict(dtype="e4m3"), INVALID), (dict(d=20), SHAPE), (dict(dY=None), INVALID),
    (dict(H=None), INVALID), (dict(gamma=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dX=None), INVALID), (dict(dgamma=None), INVALID), (dict(workspace=None), INVALID),
    (dict(dX=2 * P), INVALID), (dict(dY=P + 8), MISALIGNED), (dict(rstd=P + 2), MISALIGNED),
    (dict(dH=P + 8), MISALIGNED), (dict(dgamma=P + 2), MISALIGNED),
    (dict(workspace=P + 8), MISALIGNED),
])
def test_rmsnorm_backward_refusals(change, status):
    assert _status(gemm_epi.gemm_epi_rmsnorm_backward, **{**BWD, **change}) == status


def test_rmsnorm_workspace_sizes():
    ws = gemm_epi.gemm_epi_rmsnorm_workspace
    assert ws(4, 12) == 0 and ws(-1, 8) == 0 and ws(4, 0) == 0
    assert ws(0, 8) >= 0 and ws(1, 8) > 0
    for t, d in ((1, 8), (100000, 8), (7, 65536)):
        assert ws(t, d) % 16 == 0


W4 = dict(m=2, n=64, k=128, group=32, dtype="bf16", epilog="BIAS", A=P, W=P, scales=P, zeros=None,
          bias=P, residual=None, D=P)


@pytest.mark.parametrize("change,status", [
    (dict(group=16), SHAPE), (dict(group=0), SHAPE), (dict(k=48), SHAPE), (dict(n=12), SHAPE),
    (dict(m=65), SHAPE), (dict(m=-1), SHAPE), (dict(n=-8), SHAPE), (dict(k=-32), SHAPE),
    (dict(n=2 ** 31), SHAPE), (dict(n=8, k=2 ** 30 + 32), SHAPE),
    (dict(dtype="e4m3"), INVALID), (dict(epilog="RELU_AUX_BIAS"), INVALID),
    (dict(epilog="GELU_AUX_BIAS"), INVALID), (dict(epilog="LN_GELU_BIAS"), INVALID),
    (dict(epilog="DRELU_BGRAD"), INVALID), (dict(A=None), INVALID), (dict(W=None), INVALID),
    (dict(scales=None), INVALID), (dict(D=None), INVALID), (dict(bias=None), INVALID),
    (dict(residual=P), INVALID), (dict(epilog="BIAS_RESIDUAL"), INVALID),
    (dict(epilog="NONE"), INVALID), (dict(A=P + 8), MISALIGNED), (dict(W=P + 4), MISALIGNED),
    (dict(D=P + 8), MISALIGNED), (dict(scales=P + 2), MISALIGNED), (dict(bias=P + 1), MISALIGNED),
    (dict(zeros=P + 4), MISALIGNED),
])
def test_w4_refusals(change, status):
    assert _status(gemm_epi.gemm_epi_w4_matmul, **{**W4, **change}) == status


@pytest.mark.parametrize("change,status", [
    (dict(group=48), SHAPE), (dict(k=96, group=64), SHAPE), (dict(n=4), SHAPE), (dict(W=None), INVALID),
    (dict(scales=None), INVALID), (dict(B=None), INVALID), (dict(B=P + 2), MISALIGNED),
    (dict(W=P + 8), MISALIGNED), (dict(dtype="e4m3"), INVALID),
])
def test_w4_dequantize_refusals(change, status):
    base = dict(n=64, k=128, group=32, dtype="f16", W=P, scales=P, zeros=None, B=P)
    assert _status(gemm_epi.gemm_epi_w4_dequantize, **{**base, **change}) == status


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), SHAPE), (dict(dtype="e4m3"), INVALID), (dict(p=-0.1), INVALID),
    (dict(p=1.5), INVALID), (dict(p=float("nan")), INVALID), (dict(X=None), INVALID),
    (dict(Y=None), INVALID), (dict(X=P + 2), MISALIGNED), (dict(Y=P + 8), MISALIGNED),
    (dict(residual=P + 2), MISALIGNED), (dict(offset_device=P + 4), MISALIGNED),
])
def test_dropout_refusals(change, status):
    base = dict(count=100, dtype="bf16", X=P, residual=None, p=0.1, seed=1, offset=0, Y=P)
    assert _status(gemm_epi.gemm_epi_dropout, **{**base, **change}) == status


def _apart(**kw):
    """kw with an address of its own, 16 MiB apart, for every buffer that is True."""
    at = iter(range(16, 10 ** 6, 16))
    return {k: next(at) << 20 if v is True else v for k, v in kw.items()}


NORM_A = _apart(t=4, d=64, dtype="bf16", X=True, residual=True, gamma=True, eps=1e-6, H=True, Y=True, rstd=True)
NORM8_A = dict({k: v for k, v in NORM_A.items() if k != "Y"}, Q=500 << 20, scale=501 << 20, workspace=502 << 20)
BWD_A = _apart(t=4, d=64, dtype="bf16", dY=True, H=True, gamma=True, rstd=True, dH=True, dX=True,
               dgamma=True, workspace=True)
W4_A = _apart(m=2, n=128, k=128, group=32, dtype="bf16", epilog="BIAS_RESIDUAL", A=True, W=True, scales=True,
              zeros=True, bias=True, residual=True, D=True)
DEQ_A = _apart(n=128, k=128, group=32, dtype="bf16", W=True, scales=True, zeros=True, B=True)
DROP_A = _apart(count=256, dtype="bf16", X=True, residual=True, p=0.1, seed=1, offset=0, Y=True,
                offset_device=True)


@pytest.mark.parametrize("call,base,out,over,by", [
    # (output, what it may not overlap, bytes into that): the whole of it, or its last 16 bytes
    *[("rmsnorm", NORM_A, out, over, by) for out, over, by in (
        ("H", "X", 16), ("H", "residual", 496), ("Y", "X", 496), ("Y", "residual", 16), ("H", "Y", 0), ("Y", "H", 496),
        ("H", "gamma", 0), ("Y", "gamma", 112), ("rstd", "X", 508), ("rstd", "gamma", 0), ("rstd", "H", 0),
        ("rstd", "Y", 508))],
    *[("rmsnorm_e4m3", dict(NORM8_A, mode=mode), out, over, by) for mode in ("ROW", "TENSOR", "GIVEN") for out, over, by in (
        ("Q", "X", 0), ("Q", "residual", 496), ("H", "Q", 240), ("Q", "gamma", 0), ("scale", "H", 0),
        ("scale", "Q", 252), ("scale", "rstd", 0))],
    ("rmsnorm_e4m3", dict(NORM8_A, mode="ROW"), "scale", "X", 0),
    ("rmsnorm_e4m3", dict(NORM8_A, mode="ROW"), "rstd", "scale", 12),
    ("rmsnorm_e4m3", dict(NORM8_A, mode="TENSOR"), "workspace", "X", 496),
    ("rmsnorm_e4m3", dict(NORM8_A, mode="TENSOR"), "Q", "workspace", 16),
    *[("rmsnorm_backward", BWD_A, out, over, by) for out, over, by in (
        ("dX", "H", 0), ("dX", "H", 496), ("dX", "dY", 16), ("dX", "dH", 496), ("dX", "gamma", 0), ("dX", "rstd", 0),
        ("dgamma", "dX", 0), ("dgamma", "dY", 508), ("dgamma", "gamma", 0), ("workspace", "dY", 0),
        ("dgamma", "workspace", 0))],
    *[("w4_matmul", W4_A, "D", over, by) for over, by in (
        ("A", 0), ("A", 496), ("W", 0), ("W", 8176), ("scales", 0), ("zeros", 496), ("bias", 0), ("residual", 16))],
    *[("w4_dequantize", DEQ_A, "B", over, by) for over, by in (("W", 0), ("W", 8176), ("scales", 0), ("zeros", 496))],
    *[("dropout", DROP_A, "Y", over, by) for over, by in (("X", 16), ("residual", 496), ("offset_device", 0))],
])
def test_overlaps_are_refused(call, base, out, over, by):
    assert _status(getattr(gemm_epi, "gemm_epi_" + call), **{**base, out: base[over] + by}) == INVALID
    if by == 0 and out not in ("rstd", "scale"):  # (those end within 16 bytes)
        # the other way round: the output begins first
        assert _status(getattr(gemm_epi, "gemm_epi_" + call), **{**base, over: base[out] + 16}) == INVALID


def test_empty_problems_launch_nothing():
    none = dict(stream=0)
    gemm_epi.gemm_epi_rmsnorm(0, 64, "bf16", None, None, None, 1e-6, None, None, **none)
    gemm_epi.gemm_epi_rmsnorm_e4m3(0, 64, "bf16", None, None, None, 1e-6, None, None, "TENSOR", None, **none)
    gemm_epi.gemm_epi_w4_matmul(0, 64, 128, 32, "bf16", "BIAS", None, None, None, None, None, None, None, **none)
    gemm_epi.gemm_epi_w4_matmul(2, 0, 128, 32, "bf16", "BIAS", None, None, None, None, None, None, None, **none)
    gemm_epi.gemm_epi_w4_dequantize(64, 0, 32, "bf16", None, None, None, None, **none)
    gemm_epi.gemm_epi_dropout(0, "f16", None, None, 0.5, 1, 2, None, **none)


def test_binding_refuses_tensors_it_cannot_pass():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        gemm_epi.gemm_epi_rmsnorm(4, 64, "bf16", x, None, x, 1e-6, None, x, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        gemm_epi.gemm_epi_dropout(256, "bf16", x, None, 0.5, 1, 2, x, stream=0)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    class Tensor:
        is_cuda = True

        def get_device(self):
            return 1

        def is_contiguous(self):
            return True

        def data_ptr(self):
            return P

    monkeypatch.setattr(gemm_epi, "_current_device", lambda: 0)
    slow = gemm_epi._CtypesCalls(gemm_epi.load_library())
    with pytest.raises(ValueError, match="current CUDA device"):
        slow.dropout(0, 1, Tensor(), None, 0.5, 1, 2, None, P, 0)
    monkeypatch.setattr(gemm_epi, "_current_device", lambda: 1)
    assert slow.dropout(0, 1, Tensor(), None, 0.5, 1, 2, None, P, 0) == 0


def test_both_marshalling_paths_agree():
    """The C marshalling is there (its sources build with the library) and answers as the ctypes
    path does: the same statuses, the same refusals of arguments."""
    fast = gemm_epi._bind_calls()
    assert fast.__name__.endswith("_fastcall")
    slow = gemm_epi._CtypesCalls(gemm_epi.load_library())
    rows = [("rmsnorm", (0, 64, 1, None, None, None, 1e-6, None, None, None, 0), 0),
            ("rmsnorm", (4, 12, 1, P, None, P, 1e-6, None, P, None, 0), SHAPE),
            ("rmsnorm", (4, 64, 1, P, None, P, -1.0, None, P, None, 0), INVALID),
            ("rmsnorm_e4m3", (4, 64, 1, P, None, P, 1e-6, None, 2 * P, 1, P, None, None, 0), INVALID),
            ("rmsnorm_backward", (4, 64, 1, P, P, P, P, None, P + 8, P, P, 0), MISALIGNED),
            ("w4_matmul", (65, 64, 64, 64, 1, 0, P, P, P, None, P, None, P, 0), SHAPE),
            ("w4_dequantize", (64, 64, 64, 1, P, P, P + 4, P, 0), MISALIGNED),
            ("dropout", (0, 1, None, None, 0.5, 2 ** 64 + 3, -1, None, None, 0), 0),
            ("dropout", (8, 1, P, None, 1.5, 1, 2, None, P, 0), INVALID)]
    for name, args, want in rows:
        assert getattr(fast, name)(*args) == want == getattr(slow, name)(*args), name
    for bad in (torch.zeros(4, 64, dtype=torch.bfloat16), "x", 1.5):
        for calls in (fast, slow):
            with pytest.raises((ValueError, TypeError, AttributeError, ctypes.ArgumentError)):
                calls.dropout(8, 1, bad, None, 0.5, 1, 2, None, P, 0)
    with pytest.raises(TypeError):
        fast.rmsnorm(1, 2, 3)
    with pytest.raises((TypeError, OverflowError)):
        fast.rmsnorm(2 ** 70, 64, 1, P, None, P, 1e-6, None, P, None, 0)


# The tensors of one call each, as (argument's place, type, elements); every other argument in order.
TYPED_CALLS = [
    ("rmsnorm", (4, 64, 1, None, None, None, 1e-6, None, None, None, 0),
     {3: ("bfloat16", 256), 4: ("bfloat16", 256), 5: ("bfloat16", 64), 7: ("bfloat16", 256), 8: ("bfloat16", 256),
      9: ("float32", 4)}),
    ("rmsnorm_e4m3", (4, 64, 0, None, None, None, 1e-6, None, None, 0, None, None, None, 0),
     {3: ("float16", 256), 4: ("float16", 256), 5: ("float16", 64), 7: ("float16", 256), 8: ("float8_e4m3fn", 256),
      10: ("float32", 4), 11: ("float32", 4)}),
    ("rmsnorm_e4m3", (4, 64, 0, None, None, None, 1e-6, None, None, 1, None, None, None, 0),
     {3: ("float16", 256), 5: ("float16", 64), 8: ("float8_e4m3fn", 256), 10: ("float32", 1), 12: (None, 4112)}),
    ("rmsnorm_backward", (4, 64, 1, None, None, None, None, None, None, None, None, 0),
     {3: ("bfloat16", 256), 4: ("bfloat16", 256), 5: ("bfloat16", 64), 6: ("float32", 4), 7: ("bfloat16", 256),
      8: ("bfloat16", 256), 9: ("float32", 64), 10: (None, 4112)}),
    ("w4_matmul", (2, 128, 64, 32, 0, 4, None, None, None, None, None, None, None, 0),
     {6: ("float16", 128), 7: ("uint8", 4096), 8: ("float16", 256), 9: ("uint8", 256), 10: ("float16", 128),
      11: ("float16", 256), 12: ("float16", 256)}),
    ("w4_dequantize", (128, 64, 32, 1, None, None, None, None, 0),
     {4: ("uint8", 4096), 5: ("bfloat16", 256), 6: ("uint8", 256), 7: ("bfloat16", 8192)}),
    ("dropout", (100, 1, None, None, 0.5, 1, 2, None, None, 0),
     {2: ("bfloat16", 100), 3: ("bfloat16", 100), 7: ("int64", 1), 8: ("bfloat16", 100)}),
]


def typed_refusals(calls, tensor):
    """Calls that are right but for one tensor, of another type or one element short; `tensor` makes one.
    (None: a workspace, bytes of any tensor.)"""
    for name, args, tensors in TYPED_CALLS:
        full = list(args)
        for i, (dtype, count) in tensors.items():
            full[i] = tensor(dtype or "uint8", count)
        for i, (dtype, count) in tensors.items():
            wrong = [tensor(dtype or "uint8", count - 1)]
            if dtype:
                wrong += [tensor(other, 2 * count + 8) for other in ("float64", "float16", "bfloat16", "float32", "uint8")
                          if other != dtype and (other, dtype) != ("uint8", "float8_e4m3fn")]
            for bad in wrong:
                with pytest.raises(ValueError, match="type|fewer"):
                    getattr(calls, name)(*full[:i], bad, *full[i + 1:])


def test_binding_refuses_other_types_and_short_tensors(monkeypatch):
    class Tensor:
        is_cuda = True

        def __init__(self, dtype, count):
            self.dtype, self.count = getattr(torch, dtype), count

        def get_device(self):
            return 0

        def is_contiguous(self):
            return True

        def element_size(self):
            return self.dtype.itemsize

        def numel(self):
            return self.count

        def is_floating_point(self):
            return self.dtype.is_floating_point

        def is_complex(self):
            return self.dtype.is_complex

        def data_ptr(self):
            return P

    monkeypatch.setattr(gemm_epi, "_current_device", lambda: 0)
    typed_refusals(gemm_epi._CtypesCalls(gemm_epi.load_library()), Tensor)
