"""The LayerNorm calls for training, the block-scaled quantisation and products: what they refuse, and
the empty problems they accept, before any device is touched (no GPU)."""
import pytest
import torch

from activation_epilogue_gb300 import build as libbuild
from activation_epilogue_gb300 import gemm_epi

INVALID, SHAPE, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    gemm_epi.load_library()


def _status(call, **kw):
    with pytest.raises(gemm_epi.GemmEpiError) as e:
        getattr(gemm_epi, "gemm_epi_" + call)(**kw, stream=0)
    return e.value.status


def _apart(**kw):
    """kw with an address of its own, 16 MiB apart, for every buffer that is True."""
    at = iter(range(16, 10 ** 6, 16))
    return {k: next(at) << 20 if v is True else v for k, v in kw.items()}


FWD = _apart(t=4, d=64, dtype="bf16", X=True, residual=True, gamma=True, beta=True, eps=1e-5, H=True, Y=True, stats=True)
E4M3 = dict({k: v for k, v in FWD.items() if k != "Y"}, Q=500 << 20, scale=501 << 20)
BWD = _apart(t=4, d=64, dtype="f16", dY=True, H=True, gamma=True, stats=True, dH=True, dX=True, dgamma=True, dbeta=True,
             workspace=True)
QUANT = _apart(rows=40, cols=64, dtype="bf16", block="1X128", X=True, Q=True, scale=True, Qt=True, scale_t=True)


@pytest.mark.parametrize("call,base", [("layernorm_forward", FWD), ("layernorm_e4m3", E4M3)])
@pytest.mark.parametrize("change,status", [
    (dict(dtype="e4m3"), INVALID), (dict(t=-1), SHAPE), (dict(d=12), SHAPE), (dict(d=0), SHAPE), (dict(t=2 ** 31), SHAPE),
    (dict(t=1, d=2 ** 30 + 8), SHAPE), (dict(t=2 ** 30, d=8192), SHAPE), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(X=None), INVALID),
    (dict(gamma=None), INVALID), (dict(beta=None), INVALID), (dict(H=None), INVALID), (dict(residual=None), INVALID),
    (dict(X=8), MISALIGNED), (dict(gamma=2), MISALIGNED), (dict(beta=8), MISALIGNED), (dict(H=8), MISALIGNED),
    (dict(residual=8), MISALIGNED), (dict(stats=4), MISALIGNED),
])
def test_layernorm_refusals(call, base, change, status):
    assert _status(call, **{**base, **change}) == status


@pytest.mark.parametrize("change,status", [
    (dict(scale=None), INVALID), (dict(Q=None), INVALID), (dict(scale=2), MISALIGNED), (dict(Q=8), MISALIGNED),
    (dict(Q=E4M3["X"]), INVALID), (dict(Q=E4M3["residual"]), INVALID), (dict(Q=E4M3["H"]), INVALID),
])
def test_layernorm_e4m3_refusals(change, status):
    assert _status("layernorm_e4m3", **{**E4M3, **change}) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype="e4m3"), INVALID), (dict(d=20), SHAPE), (dict(t=-1), SHAPE), (dict(dY=None), INVALID),
    (dict(H=None), INVALID), (dict(gamma=None), INVALID), (dict(stats=None), INVALID), (dict(dX=None), INVALID),
    (dict(dgamma=None), INVALID), (dict(dbeta=None), INVALID), (dict(workspace=None), INVALID), (dict(dY=8), MISALIGNED),
    (dict(stats=4), MISALIGNED), (dict(dH=8), MISALIGNED), (dict(dgamma=2), MISALIGNED), (dict(dbeta=2), MISALIGNED),
    (dict(workspace=8), MISALIGNED), (dict(dX=8), MISALIGNED),
])
def test_layernorm_backward_refusals(change, status):
    assert _status("layernorm_backward", **{**BWD, **change}) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype="e4m3"), INVALID), (dict(rows=-1), SHAPE), (dict(rows=2 ** 31), SHAPE), (dict(cols=8), SHAPE),
    (dict(cols=0), SHAPE), (dict(cols=72), SHAPE), (dict(cols=2 ** 30 + 16), SHAPE), (dict(rows=2 ** 30, cols=2048), SHAPE),
    (dict(X=None), INVALID), (dict(Q=None), INVALID), (dict(scale=None), INVALID), (dict(Qt=None), INVALID),
    (dict(scale_t=None), INVALID), (dict(Q=None, scale=None, Qt=None, scale_t=None), INVALID), (dict(X=8), MISALIGNED),
    (dict(Q=8), MISALIGNED), (dict(Qt=8), MISALIGNED), (dict(scale=2), MISALIGNED), (dict(scale_t=2), MISALIGNED),
])
def test_quantize_refusals(change, status):
    assert _status("e4m3_quantize", **{**QUANT, **change}) == status


def test_bad_block():
    lib = gemm_epi.load_library()
    for block in (-1, 2):
        assert lib.gemm_epi_e4m3_quantize(4, 64, 1, block, 16 << 20, 32 << 20, 48 << 20, None, None, None) == INVALID


@pytest.mark.parametrize("call,base,out,over,by", [
    # (output, what it may not overlap, bytes into that): the whole of it, or its last bytes
    *[("layernorm_forward", FWD, out, over, by) for out, over, by in (
        ("H", "X", 16), ("H", "residual", 496), ("Y", "X", 496), ("Y", "residual", 16), ("H", "Y", 0), ("Y", "H", 496),
        ("H", "gamma", 0), ("Y", "gamma", 112), ("Y", "beta", 0), ("H", "beta", 112), ("stats", "X", 504), ("stats", "gamma", 0),
        ("stats", "H", 0), ("stats", "Y", 504))],
    *[("layernorm_e4m3", E4M3, out, over, by) for out, over, by in (
        ("Q", "X", 0), ("Q", "residual", 496), ("H", "Q", 240), ("Q", "beta", 0), ("scale", "H", 0), ("scale", "Q", 252),
        ("scale", "stats", 0), ("scale", "X", 508))],
    *[("layernorm_backward", BWD, out, over, by) for out, over, by in (
        ("dX", "H", 0), ("dX", "H", 496), ("dX", "dY", 16), ("dX", "dH", 496), ("dX", "gamma", 0), ("dX", "stats", 16),
        ("dgamma", "dX", 0), ("dgamma", "dY", 508), ("dgamma", "gamma", 0), ("dbeta", "dX", 0), ("dbeta", "dgamma", 252),
        ("dbeta", "H", 0), ("workspace", "dY", 0), ("dgamma", "workspace", 0), ("dbeta", "workspace", 0))],
    *[("e4m3_quantize", QUANT, out, over, by) for out, over, by in (
        ("Q", "X", 0), ("Q", "X", 5104), ("Qt", "X", 0), ("Qt", "Q", 2544), ("Q", "Qt", 3056), ("scale", "X", 0),
        ("scale", "Q", 2556), ("scale_t", "Qt", 3068), ("scale_t", "scale", 156), ("scale", "Qt", 0))],
])
def test_overlaps_are_refused(call, base, out, over, by):
    assert _status(call, **{**base, out: base[over] + by}) == INVALID


def test_workspace_sizes():
    ws = gemm_epi.gemm_epi_layernorm_workspace
    assert ws(4, 12) == 0 and ws(-1, 8) == 0 and ws(4, 0) == 0
    assert ws(0, 8) >= 0 and ws(1, 8) > 0
    for t, d in ((1, 8), (100000, 8), (7, 65536), (2 ** 31 - 1, 8)):
        assert ws(t, d) % 16 == 0


def test_empty_problems_launch_nothing():
    gemm_epi.gemm_epi_layernorm_forward(0, 64, "bf16", None, None, None, None, 1e-5, None, None, stream=0)
    gemm_epi.gemm_epi_layernorm_e4m3(0, 64, "f16", None, None, None, None, 1e-5, None, None, None, stream=0)
    gemm_epi.gemm_epi_e4m3_quantize(0, 64, "bf16", "128X128", None, stream=0)


P = 1 << 20
CALLS = [  # arguments in order, and the tensors among them: (place, type, elements)
    ("layernorm_forward", (4, 64, 1, None, None, None, None, 1e-5, None, None, None, 0),
     {3: ("bfloat16", 256), 4: ("bfloat16", 256), 5: ("bfloat16", 64), 6: ("bfloat16", 64), 8: ("bfloat16", 256),
      9: ("bfloat16", 256), 10: ("float32", 8)}),
    ("layernorm_e4m3", (4, 200, 0, None, None, None, None, 1e-5, None, None, None, None, 0),
     {3: ("float16", 800), 5: ("float16", 200), 6: ("float16", 200), 9: ("float8_e4m3fn", 800), 10: ("float32", 8),
      11: ("float32", 8)}),
    ("layernorm_backward", (4, 64, 1, None, None, None, None, None, None, None, None, None, 0),
     {3: ("bfloat16", 256), 4: ("bfloat16", 256), 5: ("bfloat16", 64), 6: ("float32", 8), 7: ("bfloat16", 256),
      8: ("bfloat16", 256), 9: ("float32", 64), 10: ("float32", 64), 11: (None, 2080)}),
    ("e4m3_quantize", (40, 144, 1, 0, None, None, None, None, None, 0),
     {4: ("bfloat16", 5760), 5: ("float8_e4m3fn", 5760), 6: ("float32", 80), 7: ("float8_e4m3fn", 144 * 48),
      8: ("float32", 144)}),
    ("e4m3_quantize", (200, 144, 0, 1, None, None, None, None, None, 0),
     {4: ("float16", 28800), 5: ("float8_e4m3fn", 28800), 6: ("float32", 4), 7: ("float8_e4m3fn", 144 * 208),
      8: ("float32", 4)}),
    ("block_product", (0, 3, 136, 144, 1, 136, None, None, None, None, None, None, None, None, 0),
     {6: ("float8_e4m3fn", 432), 7: ("float8_e4m3fn", 136 * 144), 8: ("bfloat16", 136), 9: ("bfloat16", 408),
      10: ("bfloat16", 408), 11: (None, 60), 12: ("float32", 6), 13: ("float32", 4)}),
    ("block_product", (0, 3, 136, 144, 2, 3, None, None, None, None, None, None, None, None, 0),
     {8: ("bfloat16", 3), 13: ("float32", 272)}),
]


def typed_refusals(calls, tensor):
    """Calls that are right but for one tensor, of another type or one element short; `tensor` makes one.
    (None: bytes of any tensor.)"""
    for name, args, tensors in CALLS:
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


def test_both_marshalling_paths_agree():
    fast = gemm_epi._bind_calls()
    assert fast.__name__.endswith("_fastcall")
    slow = gemm_epi._CtypesCalls(gemm_epi.load_library())
    q = [i * 16 << 20 for i in range(1, 12)]
    rows = [("layernorm_forward", (0, 64, 1, None, None, None, None, 1e-5, None, None, None, 0), 0),
            ("layernorm_forward", (4, 12, 1, P, None, P, P, 1e-5, None, P, None, 0), SHAPE),
            ("layernorm_e4m3", (4, 64, 1, q[0], None, q[1], q[2], 1e-5, None, q[3], None, None, 0), INVALID),
            ("layernorm_backward", (4, 64, 1, *q[:4], None, q[4] + 8, q[5], q[6], q[7], 0), MISALIGNED),
            ("e4m3_quantize", (40, 64, 1, 0, q[0], q[1], q[2], None, q[3], 0), INVALID),
            ("e4m3_quantize", (0, 64, 1, 1, None, None, None, None, None, 0), 0),
            ("block_product", (0, 4, 64, 128, 1, 64, *q[:8], 0), INVALID)]
    for name, args, want in rows:
        assert getattr(fast, name)(*args) == want == getattr(slow, name)(*args), name
    for bad in (torch.zeros(4, 64, dtype=torch.bfloat16), "x", 1.5):
        for calls in (fast, slow):
            with pytest.raises((ValueError, TypeError, AttributeError)):
                calls.e4m3_quantize(4, 64, 1, 0, bad, q[1], q[2], None, None, 0)


def test_widths_next_to_the_largest_integer():
    q = [i * 16 << 20 for i in range(1, 8)]
    for calls in (gemm_epi._bind_calls(), gemm_epi._CtypesCalls(gemm_epi.load_library())):
        for d in (2 ** 63 - 8, 2 ** 63 - 128):
            assert calls.layernorm_e4m3(4, d, 1, q[0], None, q[1], q[2], 1e-5, None, q[3], q[4], None, 0) == SHAPE
            assert calls.layernorm_forward(4, d, 1, q[0], None, q[1], q[2], 1e-5, None, q[3], None, 0) == SHAPE
            assert calls.e4m3_quantize(4, d, 1, 0, q[0], q[1], q[2], q[3], q[4], 0) == SHAPE
            assert calls.e4m3_quantize(d, 16, 1, 0, q[0], q[1], q[2], q[3], q[4], 0) == SHAPE
