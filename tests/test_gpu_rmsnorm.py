"""RMS norm (+ residual), forward in 16 bits and E4M3 and backward, against 64 bits."""
import numpy as np
import pytest
import torch

import sublayer_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import TD

pytestmark = pytest.mark.gpu

# rows shorter than a warp's width of vectors, odd widths, and widths on both sides of every
# power of two that a kernel may hold a row in
SHAPES = [(1, 8), (3, 72), (37, 264), (5, 1000), (300, 1024), (2, 2048), (7, 4104), (129, 4096),
          (11, 2056), (4, 4088), (1, 8192), (3, 8200), (2, 16384), (1, 16392), (2, 40000)]
MODES = ["ROW", "TENSOR", "GIVEN"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _inputs(t, d, dtype, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(t, d, generator=g)
    R = torch.randn(t, d, generator=g) * torch.exp(torch.randn(d, generator=g)) if residual else None
    gamma = 1 + 0.3 * torch.randn(d, generator=g)
    return X.to(TD[dtype]), None if R is None else R.to(TD[dtype]), gamma.to(TD[dtype])


def _cuda(*tensors):
    return [None if v is None else v.cuda() for v in tensors]


def _forward(X, R, gamma, eps, dtype, mode=None, scale=None):
    """One call on the GPU; (H, Y or codes, scale, rstd) on the CPU."""
    t, d = X.shape
    Xg, Rg, gg = _cuda(X, R, gamma)
    H = torch.full((t, d), float("nan"), dtype=TD[dtype], device="cuda") if R is not None else None
    rstd = torch.full((t,), float("nan"), device="cuda")
    if mode is None:
        Y = torch.full((t, d), float("nan"), dtype=TD[dtype], device="cuda")
        gemm_epi.gemm_epi_rmsnorm(t, d, dtype, Xg, Rg, gg, eps, H, Y, rstd)
    else:
        Y = torch.full((t, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        if mode == "GIVEN":
            scale = torch.tensor([scale], device="cuda")
        else:
            scale = torch.full((t if mode == "ROW" else 1,), float("nan"), device="cuda")
        ws = torch.full((gemm_epi.gemm_epi_rmsnorm_workspace(t, d),), 0xFF, dtype=torch.uint8, device="cuda")
        gemm_epi.gemm_epi_rmsnorm_e4m3(t, d, dtype, Xg, Rg, gg, eps, H, Y, mode, scale, rstd, ws)
    torch.cuda.synchronize()
    return (None if H is None else H.cpu()), Y.cpu(), (None if scale is None else scale.cpu()), rstd.cpu()


def _check_h(H, X, R, dtype):
    want = X.double() + R.double()
    ref.check_16(H, want, dtype, ref.F32 * want.abs(), "H")


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm(t, d, dtype, residual):
    X, R, gamma = _inputs(t, d, dtype, t + d, residual)
    H, Y, _, rstd = _forward(X, R, gamma, 1e-6, dtype)
    if residual:
        _check_h(H, X, R, dtype)
    want, wr = ref.rmsnorm(H if residual else X, gamma, 1e-6)
    rel = ref.sum_error(d) / 2 + 4 * ref.F32
    assert ((rstd.double() - wr).abs() <= rel * wr).all()
    ref.check_16(Y, want, dtype, (rel + 4 * ref.F32) * want.abs(), "Y")


@pytest.mark.parametrize("t,d", SHAPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype,residual", [("bf16", True), ("f16", False)])
def test_rmsnorm_e4m3(t, d, mode, dtype, residual):
    X, R, gamma = _inputs(t, d, dtype, t + d + 1, residual)
    H, Q, scale, rstd = _forward(X, R, gamma, 1e-5, dtype, mode, 0.01)
    if residual:
        _check_h(H, X, R, dtype)
    want, wr = ref.rmsnorm(H if residual else X, gamma, 1e-5)
    rel = ref.sum_error(d) / 2 + 4 * ref.F32
    assert ((rstd.double() - wr).abs() <= rel * wr).all()
    if mode != "GIVEN":
        top = want.abs().amax(1) if mode == "ROW" else want.abs().amax().view(1)
        assert ((scale.double() - top / 448).abs() <= (rel + 8 * ref.F32) * top / 448).all()
        # the largest value lands on the largest code
        codes = Q.float().abs()
        assert ((codes.amax(1) if mode == "ROW" else codes.amax()) == 448).all()
    s = scale.double().view(-1, 1)
    ref.check_e4m3(Q, want / s, rel + 12 * ref.F32, f"{mode} codes")


def test_rmsnorm_rstd_is_optional_and_rows_are_alike():
    # the same row gives the same bits wherever it stands and whatever else is asked for
    X, R, gamma = _inputs(1, 1000, "bf16", 5)
    H1, Y1, _, r1 = _forward(X, R, gamma, 1e-6, "bf16")
    for t in (2, 40, 700):
        H, Y, _, r = _forward(X.expand(t, -1).contiguous(), R.expand(t, -1).contiguous(), gamma, 1e-6, "bf16")
        assert torch.equal(Y, Y[:1].expand(t, -1)) and torch.equal(r, r[:1].expand(t))
        assert torch.equal(H, H1.expand(t, -1))
    Xg, Rg, gg = _cuda(X, R, gamma)
    H, Y = torch.empty_like(Xg), torch.empty_like(Xg)
    gemm_epi.gemm_epi_rmsnorm(1, 1000, "bf16", Xg, Rg, gg, 1e-6, H, Y)
    assert torch.equal(Y.cpu(), Y1)


@pytest.mark.parametrize("d", [1000, 20000])
@pytest.mark.parametrize("which", ["H=X,Y=R", "H=R,Y=X", "H=R", "Y=X"])
def test_rmsnorm_in_place(d, which):
    t, dtype = 9, "bf16"
    X, R, gamma = _inputs(t, d, dtype, 8)
    H0, Y0, _, _ = _forward(X, R, gamma, 1e-6, dtype)
    Xg, Rg, gg = _cuda(X, R, gamma)
    H, Y = torch.empty_like(Xg), torch.empty_like(Xg)
    for part in which.split(","):
        name, target = part.split("=")
        if name == "H":
            H = Xg if target == "X" else Rg
        else:
            Y = Xg if target == "X" else Rg
    gemm_epi.gemm_epi_rmsnorm(t, d, dtype, Xg, Rg, gg, 1e-6, H, Y)
    assert torch.equal(H.cpu(), H0) and torch.equal(Y.cpu(), Y0)


@pytest.mark.parametrize("mode", [None] + MODES)
def test_rmsnorm_writes_its_rows_only(mode):
    t, d, more = 5, 264, 3
    X, R, gamma = _inputs(t, d, "bf16", 4)
    Xg, Rg, gg = _cuda(X, R, gamma)
    H = torch.full((t + more, d), 7.0, dtype=torch.bfloat16, device="cuda")
    rstd = torch.full((t + more,), 7.0, device="cuda")
    scale = torch.full((t + more,), 7.0, device="cuda")
    if mode is None:
        Y = torch.full((t + more, d), 7.0, dtype=torch.bfloat16, device="cuda")
        gemm_epi.gemm_epi_rmsnorm(t, d, "bf16", Xg, Rg, gg, 1e-6, H, Y, rstd)
    else:
        Y = torch.full((t + more, d), 7.0, device="cuda").to(torch.float8_e4m3fn)
        size = gemm_epi.gemm_epi_rmsnorm_workspace(t, d)
        ws = torch.full((size + 64,), 0x55, dtype=torch.uint8, device="cuda")
        gemm_epi.gemm_epi_rmsnorm_e4m3(t, d, "bf16", Xg, Rg, gg, 1e-6, H, Y, mode, scale, rstd, ws)
        assert (ws[size:] == 0x55).all()
        written = {"ROW": t, "TENSOR": 1, "GIVEN": 0}[mode]
        assert (scale[written:] == 7.0).all()
    assert (H[t:] == 7.0).all() and (Y[t:].float() == 7.0).all() and (rstd[t:] == 7.0).all()


def test_rmsnorm_zero_rows_and_nonfinite():
    d = 264
    X = torch.randn(6, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    X[1] = 0
    X[2, 5] = float("nan")
    X[3, 7] = float("inf")
    X[4] *= 2.0 ** -60                # far below eps
    gamma = torch.ones(d, dtype=torch.bfloat16)
    _, Y, _, rstd = _forward(X, None, gamma, 1e-6, "bf16")
    assert (Y[1] == 0).all() and abs(float(rstd[1]) - 1e3) < 1e-3
    assert Y[2].isnan().all()
    assert Y[3, 7].isnan() and (Y[3, :7] == 0).all() and (Y[3, 8:] == 0).all()
    _, Q, scale, _ = _forward(X, None, gamma, 1e-6, "bf16", "ROW")
    q = Q.float()
    assert (q[1] == 0).all() and scale[1] == 0
    assert q[2].isnan().all() and scale[2].isnan()
    assert q[3].isnan().all() and scale[3].isnan()
    for i in (0, 4, 5):                 # the other rows do not see them
        want, _ = ref.rmsnorm(X[i:i + 1], gamma, 1e-6)
        ref.check_e4m3(Q[i:i + 1], want / scale[i].double(), ref.sum_error(d) + 12 * ref.F32, "row")
    _, Q, scale, _ = _forward(X, None, gamma, 1e-6, "bf16", "TENSOR")
    assert scale.isnan().all() and Q.float().isnan().all()
    _, Q, scale, _ = _forward(torch.zeros(3, d, dtype=torch.bfloat16), None, gamma, 1e-6, "bf16", "TENSOR")
    assert scale[0] == 0 and (Q.float() == 0).all()


def test_rmsnorm_given_scale_saturates():
    d = 64
    X = torch.randn(2, d, generator=torch.Generator().manual_seed(2)).to(torch.float16)
    X[0, 3] = float("nan")
    _, Q, _, _ = _forward(X, None, torch.ones(d, dtype=torch.float16), 1e-6, "f16", "GIVEN", 1e-6)
    q = Q.float()
    assert q[0].isnan().all()
    big = X[1].float().abs() > 0.01
    assert (q[1][big].abs() == 448).all() and (torch.sign(q[1]) == torch.sign(X[1].float())).all()


# rows of a bf16 norm whose squares leave fp32: large, largest, one large value among ordinary ones,
# small, and the smallest normal numbers; ordinary rows between them
def _far_rows(d, eps):
    g = torch.Generator().manual_seed(d)
    X = torch.randn(8, d, generator=g, dtype=torch.float64)
    X[0] *= 2.0 ** 70
    X[1] = torch.where(X[1] < 0, -1.0, 1.0) * torch.finfo(torch.bfloat16).max
    X[2, d // 2] = 2.0 ** 120
    X[4] *= 2.0 ** -50
    X[5] *= 2.0 ** -100
    X[6] = torch.where(X[6] < 0, -1.0, 1.0) * 2.0 ** -126
    gamma = (1 + 0.3 * torch.randn(d, generator=g)).to(torch.bfloat16)
    return X.to(torch.bfloat16), gamma


@pytest.mark.parametrize("d", [72, 264, 1000, 2048, 4096, 8192, 16384, 20000])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("mode", [None, "ROW"])
def test_rmsnorm_of_rows_far_from_one(d, eps, mode):
    X, gamma = _far_rows(d, eps)
    _, Y, scale, rstd = _forward(X, None, gamma, eps, "bf16", mode)
    want, wr = ref.rmsnorm(X, gamma, eps)
    # (a subnormal rstd, of rows around 2^127, is off by up to 2^-150)
    rel = ref.sum_error(d) / 2 + 6 * ref.F32 + 2.0 ** -150 / wr
    assert ((rstd.double() - wr).abs() <= rel * wr).all()
    rel = rel[:, None] + 4 * ref.F32
    if mode is None:
        ref.check_16(Y, want, "bf16", rel * want.abs() + 2.0 ** -149, "Y")
        return
    top = want.abs().amax(1)
    assert ((scale.double() - top / 448).abs() <= (rel[:, 0] + 8 * ref.F32) * top / 448 + 2.0 ** -149)[top > 2.0 ** -90].all()
    for i in range(8):
        if top[i] < 2.0 ** -100:    # (eps is larger than such a row's squares: zeros, as documented)
            assert scale[i] == 0 and (Y[i].float() == 0).all()
        else:
            ref.check_e4m3(Y[i], want[i] / scale[i].double(), float(rel[i]) + 12 * ref.F32, f"codes of row {i}")


@pytest.mark.parametrize("d", [72, 1000, 4096, 16384, 20000])
@pytest.mark.parametrize("which", ["H=X,Y=R", "H=R,Y=X", "H=R", "Y=X"])
def test_rmsnorm_of_far_rows_in_place(d, which):
    X, gamma = _far_rows(d, 0.0)
    R = X.flip(1).contiguous() if "H" in which else None
    H0, Y0, _, r0 = _forward(X, R, gamma, 0.0, "bf16")
    want, wr = ref.rmsnorm(X if R is None else H0, gamma, 0.0)
    near = (wr > 0) & (wr < 2.0 ** 126)     # (not the row that X + R overflows, nor subnormal ones)
    rel = ref.sum_error(d) / 2 + 10 * ref.F32 + 2.0 ** -150 / wr
    ref.check_16(Y0[near], want[near], "bf16", rel[near, None] * want[near].abs() + 2.0 ** -149, "Y")
    bufs = dict(X=X.cuda(), R=None if R is None else R.cuda())
    out = dict(H=None if R is None else torch.empty_like(bufs["X"]), Y=torch.empty_like(bufs["X"]))
    out.update({part[0]: bufs[part[2]] for part in which.split(",")})
    rstd = torch.empty(8, device="cuda")
    gemm_epi.gemm_epi_rmsnorm(8, d, "bf16", bufs["X"], bufs["R"], gamma.cuda(), 0.0, out["H"], out["Y"], rstd)
    same = torch.equal(out["Y"].cpu().view(torch.int16), Y0.view(torch.int16)) and torch.equal(rstd.cpu(), r0)
    assert same and (R is None or torch.equal(out["H"].cpu(), H0))


def test_rmsnorm_of_far_rows_many_in_a_block():
    # the blocks of the tensor-scale pass walk the rows: far and ordinary ones in turn, in one block
    d, eps = 2048, 0.0
    X, gamma = _far_rows(d, eps)
    X = X.repeat(700, 1)
    _, Q, scale, rstd = _forward(X, None, gamma, eps, "bf16", "TENSOR")
    want, wr = ref.rmsnorm(X[:8], gamma, eps)
    rel = ref.sum_error(d) / 2 + 6 * ref.F32 + 2.0 ** -150 / wr
    assert ((rstd[:8].double() - wr).abs() <= rel * wr).all()
    assert torch.equal(rstd, rstd[:8].repeat(700))
    assert torch.equal(Q.view(torch.uint8), Q[:8].repeat(700, 1).view(torch.uint8))
    top = want.abs().max()
    assert abs(float(scale) - top / 448) <= (rel.max() + 8 * ref.F32) * top / 448
    ref.check_e4m3(Q[:8], want / scale.double(), float(rel.max()) + 16 * ref.F32, "codes")


def test_rmsnorm_backward_of_far_rows():
    X, gamma = _far_rows(1000, 0.0)
    _, _, _, rstd = _forward(X, None, gamma, 0.0, "bf16")
    keep = rstd < 2.0 ** 100        # (the gradient of the smallest rows leaves bf16)
    X, rstd = X[keep].contiguous(), rstd[keep].contiguous()
    dy, _, _, _, dh = _bwd_inputs(X.shape[0], 1000, "bf16", 5)
    dX, dgamma = _backward(dy, X, gamma, rstd, dh, "bf16")
    _check_bwd(dX, dgamma, dy, X, gamma, rstd, dh, "bf16")


@pytest.mark.parametrize("t,d", [(37, 264), (300, 1024), (7, 4104), (3, 20000)])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rmsnorm_codes_are_products_with_the_reciprocal(t, d, mode, dtype):
    """The codes bit for bit, from the call's own H, rstd and scale: fp32 products in the header's order,
    times the rounded reciprocal of the scale, rounded once to E4M3."""
    X, R, gamma = _inputs(t, d, dtype, t * d)
    H, Q, scale, rstd = _forward(X, R, gamma, 1e-6, dtype, mode, 0.007)
    y = H.float() * rstd[:, None] * gamma.float()
    inv = 1.0 / scale.float().view(-1, 1)
    want = (y * inv).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(Q.view(torch.uint8), want.view(torch.uint8))


# ---- backward -------------------------------------------------------------------------------

def _backward(dy, h, gamma, rstd, dh, dtype, dx=None):
    t, d = h.shape
    a = _cuda(dy, h, gamma, rstd, dh)
    dX = torch.full((t, d), float("nan"), dtype=TD[dtype], device="cuda")
    if dx == "dY":
        dX = a[0]
    elif dx == "dH":
        dX = a[4]
    dgamma = torch.full((d,), float("nan"), device="cuda")
    size = gemm_epi.gemm_epi_rmsnorm_workspace(t, d)
    ws = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    gemm_epi.gemm_epi_rmsnorm_backward(t, d, dtype, *a, dX, dgamma, ws)
    torch.cuda.synchronize()
    assert (ws[size:] == 0xFF).all()
    return dX.cpu(), dgamma.cpu()


def _bwd_inputs(t, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(t, d, generator=g) * torch.exp(0.5 * torch.randn(d, generator=g))).to(TD[dtype])
    dy = (0.1 * torch.randn(t, d, generator=g)).to(TD[dtype])
    dh = (0.1 * torch.randn(t, d, generator=g)).to(TD[dtype])
    gamma = (1 + 0.3 * torch.randn(d, generator=g)).to(TD[dtype])
    rstd = ref.rmsnorm(h, gamma, 1e-6)[1].float()
    return dy, h, gamma, rstd, dh


def _check_bwd(dX, dgamma, dy, h, gamma, rstd, dh, dtype):
    t, d = h.shape
    want, wg, size, gsize = ref.rmsnorm_backward(dy, h, gamma, rstd, dh)
    ref.check_16(dX, want, dtype, (ref.sum_error(d) + 8 * ref.F32) * size, "dX")
    # a column's chain: its rows of one block, then the blocks in order
    assert ((dgamma.double() - wg).abs() <= (min(t, 1024) + t / 32 + 8) * ref.F32 * gsize + 1e-40).all()


@pytest.mark.parametrize("t,d", SHAPES + [(2000, 264), (700, 1024), (400, 5120)])
@pytest.mark.parametrize("dtype,with_dh", [("bf16", True), ("f16", True), ("bf16", False)])
def test_rmsnorm_backward(t, d, dtype, with_dh):
    dy, h, gamma, rstd, dh = _bwd_inputs(t, d, dtype, t * 3 + d)
    dh = dh if with_dh else None
    dX, dgamma = _backward(dy, h, gamma, rstd, dh, dtype)
    _check_bwd(dX, dgamma, dy, h, gamma, rstd, dh, dtype)


@pytest.mark.parametrize("t,d", [(2049, 264), (4100, 72), (5000, 512), (2049, 520), (3001, 1000), (6000, 1024),
                                 (1900, 2048), (1000, 4096), (700, 8192)])
def test_rmsnorm_backward_many_rows(t, d):
    """Several rounds of every block, the last of them not full."""
    dy, h, gamma, rstd, dh = _bwd_inputs(t, d, "bf16", t + d)
    dX, dgamma = _backward(dy, h, gamma, rstd, dh, "bf16")
    _check_bwd(dX, dgamma, dy, h, gamma, rstd, dh, "bf16")
    again = _backward(dy, h, gamma, rstd, dh, "bf16")
    assert torch.equal(dX, again[0]) and torch.equal(dgamma, again[1])


@pytest.mark.parametrize("dx", ["dY", "dH"])
@pytest.mark.parametrize("t,d", [(40, 1000), (400, 1024), (3, 20000)])
def test_rmsnorm_backward_in_place_and_repeatable(t, d, dx):
    dy, h, gamma, rstd, dh = _bwd_inputs(t, d, "bf16", 11)
    first = _backward(dy, h, gamma, rstd, dh, "bf16")
    again = _backward(dy, h, gamma, rstd, dh, "bf16", dx)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_rmsnorm_backward_empty_zeroes_dgamma():
    dgamma = torch.full((64,), 3.0, device="cuda")
    gemm_epi.gemm_epi_rmsnorm_backward(0, 64, "bf16", None, None, None, None, None, None, dgamma, None)
    assert (dgamma == 0).all()


def test_rmsnorm_backward_against_differences_of_the_forward_call():
    # the library's own forward in 16 bits is too coarse to difference: the formula's gradient
    # is pinned to differences in 64 bits (CPU), and here the pair of calls to that formula
    t, d, dtype = 6, 264, "bf16"
    X, R, gamma = _inputs(t, d, dtype, 21)
    H, _, _, rstd = _forward(X, R, gamma, 1e-6, dtype)
    dy, _, _, _, dh = _bwd_inputs(t, d, dtype, 22)
    dX, dgamma = _backward(dy, H, gamma, rstd, dh, dtype)
    h64 = H.double().requires_grad_()
    g64 = gamma.double().requires_grad_()
    y = h64 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + 1e-6) * g64
    ((y * dy.double()).sum() + (h64 * dh.double()).sum()).backward()
    _, _, size, gsize = ref.rmsnorm_backward(dy, H, gamma, rstd, dh)
    # rstd itself is rounded to fp32
    ref.check_16(dX, h64.grad, dtype, 3 * (ref.sum_error(d) + 8 * ref.F32) * size, "dX")
    assert ((dgamma.double() - g64.grad).abs() <= (ref.sum_error(d) + 2 * t * ref.F32) * gsize).all()


# ---- streams, graphs, long buffers --------------------------------------------------------------

def test_rmsnorm_on_another_stream_and_in_a_graph():
    t, d, dtype = 33, 1000, "bf16"
    X, R, gamma = _inputs(t, d, dtype, 31)
    H0, Q0, s0, _ = _forward(X, R, gamma, 1e-6, dtype, "TENSOR")
    Xg, Rg, gg = _cuda(X, R, gamma)
    H, Q = torch.empty_like(Xg), torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.zeros(1, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(stream=None):
        gemm_epi.gemm_epi_rmsnorm_e4m3(t, d, dtype, Xg, Rg, gg, 1e-6, H, Q, "TENSOR", scale, None, ws, stream)
    call(side)
    side.synchronize()
    assert torch.equal(Q.cpu().view(torch.uint8), Q0.view(torch.uint8)) and torch.equal(scale.cpu(), s0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    Xg.mul_(2)          # new inputs at replay
    Rg.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    H2, Q2, s2, _ = _forward(Xg.cpu(), Rg.cpu(), gamma, 1e-6, dtype, "TENSOR")
    assert torch.equal(Q.cpu().view(torch.uint8), Q2.view(torch.uint8)) and torch.equal(scale.cpu(), s2)
    assert torch.equal(H.cpu(), H2)


def test_rmsnorm_calls_on_two_streams_at_once():
    t, d = 400, 4096
    sets, want = [], []
    for seed in (1, 2):
        X, R, gamma = _inputs(t, d, "bf16", seed)
        want.append(_forward(X, R, gamma, 1e-6, "bf16", "TENSOR"))
        sets.append(_cuda(X, R, gamma) + [torch.empty(t, d, dtype=torch.bfloat16, device="cuda"),
                    torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda"), torch.zeros(1, device="cuda"),
                    torch.empty(gemm_epi.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8, device="cuda")])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (X, R, gamma, H, Q, scale, ws) in zip(streams, sets):
            gemm_epi.gemm_epi_rmsnorm_e4m3(t, d, "bf16", X, R, gamma, 1e-6, H, Q, "TENSOR", scale, None, ws, s)
    torch.cuda.synchronize()
    for (X, R, gamma, H, Q, scale, ws), (H0, Q0, s0, _) in zip(sets, want):
        assert torch.equal(scale.cpu(), s0) and torch.equal(H.cpu(), H0)
        assert torch.equal(Q.cpu().view(torch.uint8), Q0.view(torch.uint8))


@pytest.mark.slow
def test_rmsnorm_offsets_past_32_bits():
    t, d = 2 ** 18 + 3, 16384           # 4.3e9 elements
    X = torch.zeros(t, d, dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 2 ** 17, t - 2, t - 1]
    some = torch.randn(len(rows), d, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    X[rows] = some.cuda()
    gamma = torch.ones(d, dtype=torch.bfloat16)
    Y = torch.empty_like(X)
    rstd = torch.empty(t, device="cuda")
    gemm_epi.gemm_epi_rmsnorm(t, d, "bf16", X, None, gamma.cuda(), 1e-6, None, Y, rstd)
    want, _ = ref.rmsnorm(some, gamma, 1e-6)
    ref.check_16(Y[rows], want, "bf16", (ref.sum_error(d) + 8 * ref.F32) * want.abs(), "Y")
    dgamma = torch.empty(d, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    dX = torch.empty_like(X)
    gemm_epi.gemm_epi_rmsnorm_backward(t, d, "bf16", X, X, gamma.cuda(), rstd, Y, dX, dgamma, ws)
    dx, dg, size, gsize = ref.rmsnorm_backward(some, some, gamma, rstd[rows].cpu(), Y[rows].cpu())
    ref.check_16(dX[rows], dx, "bf16", (ref.sum_error(d) + 8 * ref.F32) * size, "dX")
    assert ((dgamma.cpu().double() - dg).abs() <= 1100 * ref.F32 * gsize).all()   # zero rows add nothing
