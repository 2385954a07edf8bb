"""LayerNorm for training (forward to 16 bits and to block-scaled E4M3, backward) against the same in
64 bits."""
import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import F32, TD

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
# every width class of the kernels, their edges, and rows too long for registers
WIDTHS = [8, 24, 256, 264, 512, 520, 1000, 1032, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 16392, 40968]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _problem(t, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + t * d)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x = normal(t, d) * torch.exp(normal(t, 1)) + 3 * normal(t, 1)
    r = normal(t, d) * (1 + 20 * (torch.rand(d, generator=g, device="cuda") < 0.01)) + normal(1, d)
    return {"X": x.to(TD[dtype]), "R": r.to(TD[dtype]), "gamma": (1 + 0.3 * normal(d)).to(TD[dtype]),
            "beta": (0.5 * normal(d)).to(TD[dtype]), "dY": normal(t, d).to(TD[dtype]), "dH": normal(t, d).to(TD[dtype])}


def _forward(p, dtype, eps, residual=True, e4m3=False, stats=True):
    t, d = p["X"].shape
    H = torch.empty_like(p["X"]) if residual else None
    st = torch.full((t, 2), float("nan"), device="cuda") if stats else None
    R = p["R"] if residual else None
    if e4m3:
        Y = torch.full((t, d), 0x55, dtype=torch.uint8, device="cuda").view(E4M3)
        scale = torch.full((-(-d // 128), t), -1.0, device="cuda")
        gemm_epi.gemm_epi_layernorm_e4m3(t, d, dtype, p["X"], R, p["gamma"], p["beta"], eps, H, Y, scale, st)
        return H, Y, st, scale
    Y = torch.full_like(p["X"], float("nan"))
    gemm_epi.gemm_epi_layernorm_forward(t, d, dtype, p["X"], R, p["gamma"], p["beta"], eps, H, Y, st)
    return H, Y, st, None


def _check_forward(p, dtype, eps, H, Y, stats, scale):
    h = p["X"] if H is None else H
    if H is not None:
        assert torch.equal(H, (p["X"].float() + p["R"].float()).to(TD[dtype]))
    y, mean, rstd, error = ref.layernorm(h, p["gamma"], p["beta"], eps)
    S = ref.sum_error(h.shape[1])
    if stats is not None:
        dev = (h.double() - mean[:, None]).abs().mean(1)
        assert torch.all((stats[:, 0].double() - mean).abs() <= 2 * F32 * mean.abs() + 2 * S * dev + S * S * h.double().abs().mean(1))
        lacks = S * h.double().abs().mean(1)
        # (2^-149: a step of fp32 below 2^-126, where a row next to the largest value has its rstd)
        assert torch.all((stats[:, 1].double() - rstd).abs() <= rstd * (S + 8 * F32 + 2 * S * lacks ** 2 * rstd ** 2) + 2.0 ** -149)
    if scale is None:
        ref.check(Y, y, error, dtype)
        return
    top = ref.tops(y, "1X128")
    off = ref.tops(error, "1X128")
    assert torch.all((scale.double() - top / 448).abs() <= off / 448 + 2 * F32 * top / 448)
    s = ref.spread(scale, "1X128", *y.shape)
    s = torch.where(s > 0, s, 1.0)
    ref.check_codes(Y, y / s, error / s + 4 * F32 * (y / s).abs(), "codes")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward(d, dtype, e4m3):
    for t, residual in ((1, True), (5, False), (133, True)):
        p = _problem(t, d, dtype)
        _check_forward(p, dtype, 1e-5, *_forward(p, dtype, 1e-5, residual, e4m3))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [264, 2056, 8192, 16392])
def test_rows_far_from_zero(d, e4m3):
    """A mean far above the deviations, and constant rows (variance 0: only eps stands below)."""
    for dtype, mean in (("f16", 1000.0), ("bf16", 96.0)):
        p = _problem(6, d, dtype)
        p["X"] = (mean + torch.randn(6, d, device="cuda")).to(TD[dtype])
        p["X"][4] = mean
        p["X"][5] = 0
        H, Y, st, scale = _forward(p, dtype, 1e-5, False, e4m3)
        _check_forward(p, dtype, 1e-5, H, Y, st, scale)
        assert st[4, 0] == mean and st[5, 0] == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [24, 1000, 2056, 8192, 16384, 16392])
def test_rows_whose_sums_leave_fp32(d, e4m3):
    p = _problem(9, d, "bf16")
    g = torch.Generator(device="cuda").manual_seed(d)
    unit = torch.randn(9, d, generator=g, device="cuda", dtype=torch.float64).clamp(-3, 3)
    size = torch.tensor([2.0 ** e for e in (126, 120, 70, 64, -45, -60, -100, -120, 0)], device="cuda", dtype=torch.float64)
    p["X"] = (unit * size[:, None]).to(torch.bfloat16)
    p["X"][0, ::2] += 2.0 ** 127  # a sum far past fp32 (and, from 3 * 2^126 + 2^127 on, infinities)
    H, Y, st, scale = _forward(p, "bf16", 0.0, False, e4m3)
    whole = torch.isfinite(p["X"].float()).all(1)
    assert Y[~whole].float().isnan().all() and whole[1:].all()
    Y, st, p["X"], scale = Y[whole], st[whole], p["X"][whole], scale if scale is None else scale[:, whole]
    y, mean, rstd, error = ref.layernorm(p["X"], p["gamma"], p["beta"], 0.0)
    fine = rstd < 2.0 ** 128  # (past that the statistic itself leaves fp32)
    assert torch.isfinite(Y.float()).all()
    S = ref.sum_error(d)
    assert torch.all((st[:, 1].double() - rstd).abs()[fine] <= ((S + 8 * F32) * rstd + 2.0 ** -149)[fine])
    if not e4m3:
        ref.check(Y, y, error, "bf16")
    else:
        s = ref.spread(scale, "1X128", *y.shape)
        ref.check_codes(Y, y / s, error / s + 4 * F32 * (y / s).abs(), "codes")
    with_eps = _forward(p, "bf16", 1e-5, False, e4m3)
    if not e4m3:
        y, _, _, error = ref.layernorm(p["X"], p["gamma"], p["beta"], 1e-5)
        ref.check(with_eps[1], y, error, "bf16")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [24, 1000, 8192, 16392])
def test_rows_next_to_the_largest_value(d, e4m3):
    """Sums far past fp32, of one sign and of both."""
    p = _problem(4, d, "bf16")
    top = torch.finfo(torch.bfloat16).max
    unit = torch.rand(4, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(d))
    p["X"] = (top * (0.5 + 0.5 * unit)).to(torch.bfloat16)
    p["X"][1] *= -1
    p["X"][2, ::3] *= -1
    p["X"][3] = top
    H, Y, st, scale = _forward(p, "bf16", 1e-5, False, e4m3)
    _check_forward(p, "bf16", 1e-5, H, Y, st, scale)


@pytest.mark.parametrize("d", [264, 2056, 16392])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nan_and_infinity(d, dtype):
    p = _problem(6, d, dtype)
    p["X"][1, 3], p["X"][2, d - 1], p["X"][3, 0] = float("nan"), float("inf"), float("-inf")
    bad = torch.tensor([0, 1, 1, 1, 0, 0], dtype=torch.bool, device="cuda")
    _, Y, st, _ = _forward(p, dtype, 1e-5, False)
    assert Y[bad].isnan().all() and torch.isfinite(Y[~bad]).all()
    assert st[bad, 1].isnan().all()
    _, Q, _, scale = _forward(p, dtype, 1e-5, False, e4m3=True)
    assert Q.float()[bad].isnan().all() and scale[:, bad].isnan().all()
    assert torch.isfinite(Q.float()[~bad]).all() and torch.isfinite(scale[:, ~bad]).all()


@pytest.mark.parametrize("d", [264, 4096, 16392])
def test_in_place_and_without_statistics(d):
    p = _problem(33, d, "bf16")
    H, Y, st, _ = _forward(p, "bf16", 1e-5)
    _, Y2, _, _ = _forward(p, "bf16", 1e-5, stats=False)
    assert torch.equal(Y, Y2)
    for h, y in (("X", "R"), ("R", "X")):
        q = {k: v.clone() for k, v in p.items()}
        gemm_epi.gemm_epi_layernorm_forward(33, d, "bf16", q["X"], q["R"], q["gamma"], q["beta"], 1e-5, q[h], q[y])
        assert torch.equal(q[h], H) and torch.equal(q[y], Y)
    q = p["X"].clone()
    gemm_epi.gemm_epi_layernorm_forward(33, d, "bf16", q, None, p["gamma"], p["beta"], 1e-5, None, q)
    assert torch.equal(q, _forward(p, "bf16", 1e-5, residual=False)[1])
    # zero blocks: nothing of a row left by gamma and beta
    p["gamma"][:128], p["beta"][:128] = 0, 0
    _, Q, _, scale = _forward(p, "bf16", 1e-5, e4m3=True)
    assert not scale[0].any() and not Q.float()[:, :128].any()


def _backward(p, dtype, stats, dh=True, dX=None):
    t, d = p["X"].shape
    dX = torch.full_like(p["X"], float("nan")) if dX is None else dX
    dgamma, dbeta = torch.full((d,), float("nan"), device="cuda"), torch.full((d,), float("nan"), device="cuda")
    ws = torch.full((gemm_epi.gemm_epi_layernorm_workspace(t, d),), 0xFF, dtype=torch.uint8, device="cuda")
    gemm_epi.gemm_epi_layernorm_backward(t, d, dtype, p["dY"], p["X"], p["gamma"], stats, p["dH"] if dh else None,
                                         dX, dgamma, dbeta, ws)
    return dX, dgamma, dbeta


def _check_backward(p, dtype, stats, dh, dX, dgamma, dbeta):
    want = ref.layernorm_backward(p["dY"], p["X"], p["gamma"], stats, p["dH"] if dh else None)
    ref.check(dX, want[0], want[3], dtype, "dX")
    assert torch.all((dgamma.double() - want[1]).abs() <= want[4]), "dgamma"
    assert torch.all((dbeta.double() - want[2]).abs() <= want[5]), "dbeta"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", WIDTHS)
def test_backward(d, dtype):
    for t, dh in ((1, True), (5, False), (700, True)):
        p = _problem(t, d, dtype)
        stats = _forward(p, dtype, 1e-5, residual=False)[2]
        _check_backward(p, dtype, stats, dh, *_backward(p, dtype, stats, dh))


@pytest.mark.parametrize("t,d", [(2500, 24), (2500, 512), (5000, 1000), (3000, 2048)])
def test_backward_of_many_rows(t, d):
    p = _problem(t, d, "bf16")
    stats = _forward(p, "bf16", 1e-5, residual=False)[2]
    out = _backward(p, "bf16", stats)
    _check_backward(p, "bf16", stats, True, *out)
    for got, want in zip(_backward(p, "bf16", stats), out):  # the same bits in every call
        assert torch.equal(got, want)


def test_backward_in_place_and_empty():
    p = _problem(50, 1000, "bf16")
    stats = _forward(p, "bf16", 1e-5, residual=False)[2]
    want = _backward(p, "bf16", stats)
    for name in ("dY", "dH"):
        q = {k: v.clone() for k, v in p.items()}
        got = _backward(q, "bf16", stats, dX=q[name])
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    dgamma, dbeta = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    gemm_epi.gemm_epi_layernorm_backward(0, 64, "bf16", None, None, None, None, None, None, dgamma, dbeta, None)
    assert not dgamma.any() and not dbeta.any()


def test_backward_of_large_rows():
    """Rows whose deviations leave fp32 in their difference with the mean."""
    p = _problem(4, 264, "bf16")
    p["X"][:] = torch.where(torch.rand(4, 264, device="cuda") < 0.2, -3e38, 3e38).to(torch.bfloat16)
    p["X"][2:] *= 2.0 ** -30
    stats = _forward(p, "bf16", 1e-5, residual=False)[2]
    _check_backward(p, "bf16", stats, True, *_backward(p, "bf16", stats))


def test_against_differences():
    """The formula that the kernel is held to, by autograd and by differences of the forward pass."""
    p = _problem(3, 40, "f16", seed=5)
    x, gamma, beta = (p[k].double().requires_grad_() for k in ("X", "gamma", "beta"))
    dy, dh = p["dY"].double(), p["dH"].double()

    def loss(x, gamma, beta):
        mean = x.mean(1, keepdim=True)
        rstd = ((x - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return (((x - mean) * rstd * gamma + beta) * dy).sum() + (x * dh).sum()

    grads = torch.autograd.grad(loss(x, gamma, beta), (x, gamma, beta))
    assert torch.autograd.gradcheck(loss, (x, gamma, beta))
    h = x.detach()
    mean = h.mean(1)
    stats = torch.stack((mean, ((h - mean[:, None]).square().mean(1) + 1e-5).rsqrt()), 1)
    formula = ref.layernorm_backward(dy, h, gamma.detach(), stats, dh)
    for got, want in zip(formula, grads):
        assert torch.allclose(got, want, rtol=1e-9, atol=1e-9)
    st = _forward(p, "f16", 1e-5, residual=False)[2]
    _check_backward(p, "f16", st, True, *_backward(p, "f16", st))
