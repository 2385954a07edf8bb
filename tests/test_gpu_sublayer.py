"""The RMS norm, the 4-bit and E4M3 products and dropout run together, as a model's
feed-forward sub-layer uses them."""
import numpy as np
import pytest
import torch

import oracle
import sublayer_reference as ref
from activation_epilogue_gb300 import gemm_epi
from parity_helpers import TOL, rel_err
from sublayer_reference import TD
from test_sublayer_refusals import typed_refusals

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gelu(v):
    return 0.5 * v * torch.special.erfc(-v / np.sqrt(2.0))


@pytest.mark.parametrize("epilog", ["BIAS", "RELU_BIAS", "GELU_BIAS", "RELU_AUX_BIAS", "BIAS_RESIDUAL", "NONE"])
@pytest.mark.parametrize("m,n,k,opts", [(300, 520, 208, {}), (1, 8, 16, {}), (1000, 776, 272, {"TILE_N": 224}),
                                        (2304, 264, 128, {"GRID": 4, "TILE_ORDER": 2})])
def test_row_scaled_plan(epilog, m, n, k, opts):
    g = torch.Generator().manual_seed(m + n)
    A = torch.randn(m, k, generator=g).to(torch.float8_e4m3fn)
    Bt = torch.randn(n, k, generator=g).to(torch.float8_e4m3fn)
    sa = torch.exp(torch.randn(m, generator=g)) / 8
    sb = torch.tensor([0.25 / np.sqrt(k)])
    bias = torch.randn(n, generator=g).to(torch.bfloat16) if epilog != "NONE" else None
    R = torch.randn(m, n, generator=g).to(torch.bfloat16) if epilog == "BIAS_RESIDUAL" else None
    D = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    aux = torch.empty(m, (n + 31) // 32, dtype=torch.int32, device="cuda") if epilog == "RELU_AUX_BIAS" else None
    cuda = [None if v is None else v.cuda() for v in (A, Bt, bias, R, sa.float(), sb.float())]
    with gemm_epi.Plan(m, n, k, "e4m3", epilog, "1N", SCALE_A_ROWS=1, **opts) as plan:
        plan.execute(cuda[0], cuda[1], cuda[2], D, aux=aux, residual=cuda[3], scales=(cuda[4], cuda[5]))
        assert plan.sync_status() == 0
        unfused = torch.empty_like(D)
        if epilog == "NONE":
            pre = torch.empty_like(D)
            plan.execute_unfused(cuda[0], cuda[1], None, pre, unfused, scales=(cuda[4], cuda[5]))
            assert torch.equal(unfused, D)
    want = sa.float().double()[:, None] * sb.float().double() * (A.double() @ Bt.double().t())
    want = want if bias is None else want + bias.double()
    if epilog in ("RELU_BIAS", "RELU_AUX_BIAS"):
        want = want.clamp(min=0)
    elif epilog == "GELU_BIAS":
        want = _gelu(want)
    elif epilog == "BIAS_RESIDUAL":
        want = want + R.double()
    assert rel_err(D, want.numpy()) <= TOL["bf16"]


def test_row_scale_option_is_for_e4m3_plans():
    for dtype, value in (("bf16", 1), ("e4m3", -1), ("e4m3", 2)):
        with pytest.raises(gemm_epi.GemmEpiError) as e:
            gemm_epi.Plan(64, 64, 64, dtype, "BIAS", "1N", SCALE_A_ROWS=value)
        assert e.value.status == 1
    gemm_epi.Plan(64, 64, 64, "bf16", "BIAS", "1N", SCALE_A_ROWS=0).free()


def test_row_scaled_plan_refuses_short_scales():
    A, Bt = (torch.zeros(64, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    D = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    one, rows = torch.ones(1, device="cuda"), torch.ones(64, device="cuda")
    with gemm_epi.Plan(64, 64, 64, "e4m3", "NONE", SCALE_A_ROWS=1) as plan:
        plan.execute(A, Bt, None, D, scales=(rows, one))
        for scales in ((one, one), (rows[:63], one), (rows.double(), one), (rows, one[:0])):
            with pytest.raises(ValueError, match="type|fewer"):
                plan.execute(A, Bt, None, D, scales=scales)
            with pytest.raises(ValueError, match="type|fewer"):
                plan.execute_unfused(A, Bt, None, D, D, scales=scales)
        plan.set_option("SCALE_A_ROWS", 0)
        plan.execute(A, Bt, None, D, scales=(one, one))
        assert plan.sync_status() == 0


@pytest.mark.parametrize("mode", ["ROW", "TENSOR"])
def test_norm_into_e4m3_product(mode):
    """H = X + R, Q = E4M3(RMS norm), D = GELU(dequantised Q . W + b) in one stream."""
    t, d, f = 300, 1024, 520
    g = torch.Generator().manual_seed(2)
    X, R = (torch.randn(t, d, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    gamma = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda()
    Wt = (torch.randn(f, d, generator=g) * 2).to(torch.float8_e4m3fn).cuda()
    b = torch.randn(f, generator=g).to(torch.bfloat16).cuda()
    sb = torch.full((1,), 0.5 / np.sqrt(d), dtype=torch.float32, device="cuda")
    H = torch.empty_like(X)
    Q = torch.empty(t, d, dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(t if mode == "ROW" else 1, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    D = torch.empty(t, f, dtype=torch.bfloat16, device="cuda")
    with gemm_epi.Plan(t, f, d, "e4m3", "GELU_BIAS", "1N", SCALE_A_ROWS=int(mode == "ROW")) as plan:
        gemm_epi.gemm_epi_rmsnorm_e4m3(t, d, "bf16", X, R, gamma, 1e-6, H, Q, mode, scale, None, ws)
        plan.execute(Q, Wt, b, D, scales=(scale, sb))
        assert plan.sync_status() == 0
    y = Q.double().cpu() * scale.double().cpu().view(-1, 1)
    want = _gelu(y @ Wt.double().cpu().t() * float(sb) + b.double().cpu())
    assert rel_err(D, want.numpy()) <= TOL["bf16"]
    # and the codes stand for the norm within E4M3's half step
    yn, _ = ref.rmsnorm(H.cpu(), gamma.cpu(), 1e-6)
    ref.check_e4m3(Q.cpu(), yn / scale.double().cpu().view(-1, 1), 1e-5, "codes")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", [1, 6, 64, 200])
def test_decode_sublayer_with_4bit_weights(dtype, t):
    """Two layers of H = X + R; Y = RMS norm(H); D = H + GELU(Y . W1 + b1) . W2 + b2, captured in
    one graph; t over the 4-bit call's limit goes through the written-out weight and a plan."""
    d, f, group = 512, 1024, 64
    g = torch.Generator().manual_seed(t)
    layers = []
    for i in range(2):
        w1 = ref.w4_problem(1, f, d, group, dtype, True, 10 + i)
        w2 = ref.w4_problem(1, d, f, group, dtype, False, 20 + i)
        gamma = (1 + 0.1 * torch.randn(d, generator=g)).to(TD[dtype])
        layers.append((gamma, w1, w2))
    X, R = (torch.randn(t, d, generator=g).to(TD[dtype]) for _ in range(2))
    names = [name + str(i) for i in range(2) for name in "HYGD"]
    bufs = {name: torch.empty(t, f if name[0] == "G" else d, dtype=TD[dtype], device="cuda")
            for name in ["X", "R"] + names}
    bufs["X"].copy_(X)
    bufs["R"].copy_(R)
    gpu = [(gm.cuda(), {k: v.cuda() for k, v in a.items() if v is not None},
            {k: v.cuda() for k, v in b.items() if v is not None}) for gm, a, b in layers]
    plans, Bs = {}, {}
    if t > gemm_epi.W4_MAX_ROWS:
        plans = {"GELU_BIAS": gemm_epi.Plan(t, f, d, dtype, "GELU_BIAS"),
                 "BIAS_RESIDUAL": gemm_epi.Plan(t, d, f, dtype, "BIAS_RESIDUAL")}
        Bs = {"GELU_BIAS": torch.empty(d, f, dtype=TD[dtype], device="cuda"),
              "BIAS_RESIDUAL": torch.empty(f, d, dtype=TD[dtype], device="cuda")}

    def product(n, k, epilog, A, w, residual, D):
        if not plans:
            gemm_epi.gemm_epi_w4_matmul(t, n, k, group, dtype, epilog, A, w["W"], w["scales"],
                                        w.get("zeros"), w["bias"], residual, D)
            return
        gemm_epi.gemm_epi_w4_dequantize(n, k, group, dtype, w["W"], w["scales"], w.get("zeros"), Bs[epilog])
        plans[epilog].execute(A, Bs[epilog], w["bias"], D, residual=residual)

    def step():
        x, r = bufs["X"], bufs["R"]
        for i, (gm, w1, w2) in enumerate(gpu):
            H, Y, G, D = (bufs[name + str(i)] for name in "HYGD")
            gemm_epi.gemm_epi_rmsnorm(t, d, dtype, x, r, gm, 1e-6, H, Y)
            product(f, d, "GELU_BIAS", Y, w1, None, G)
            product(d, f, "BIAS_RESIDUAL", G, w2, H, D)
            x, r = D, H
    step()
    torch.cuda.synchronize()
    eager = {k: v.clone() for k, v in bufs.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for name in names:
        bufs[name].fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in names:
        assert torch.equal(bufs[name], eager[name]), name
    # each step against 64 bits, from the 16-bit values that the step before stored
    x, r = X, R
    for i, (gm, w1, w2) in enumerate(layers):
        h = bufs[f"H{i}"].cpu()
        ref.check_16(h, x.double() + r.double(), dtype, ref.F32 * (x.double().abs() + r.double().abs()), "H")
        y, _ = ref.rmsnorm(h, gm, 1e-6)
        ref.check_16(bufs[f"Y{i}"], y, dtype, (ref.sum_error(d) + 8 * ref.F32) * y.abs(), "Y")
        for name, a, w, epilog in (("G", "Y", w1, "GELU_BIAS"), ("D", "G", w2, "BIAS_RESIDUAL")):
            w = dict(w, A=bufs[f"{a}{i}"].cpu(), R=h)
            want, error = ref.w4_matmul(w, group, epilog)
            if plans:
                # the written-out weight is rounded to 16 bits (half a step of each), and the
                # plans' GELU is the library's fitted one (3.1e-5 max(1, |x|))
                B = ref.w4_weight(w["q"], w["scales"], w["zeros"], group).abs()
                error = error + 1.13 * ref.HALF[dtype] * (w["A"].double().abs() @ B)
                if epilog == "GELU_BIAS":
                    error = error + 3.2e-5 * (1 + w["A"].double().abs() @ B + w["bias"].double().abs())
            ref.check_16(bufs[f"{name}{i}"], want, dtype, error, f"{name}{i}")
        x, r = bufs[f"D{i}"].cpu(), h
    for p in plans.values():
        p.free()


def test_training_sublayer():
    """Forward: H = X + R, Y = RMS norm(H), U = Y . W + b, O = H + dropout(U).  Backward from dO:
    dU = dropout(dO), dY = dU . W^T, dH (shared by X and R) and dgamma from the norm, with dO
    arriving at H past the norm; against 64-bit autograd on the stored H with the same mask."""
    t, d, p, seed = 200, 264, 0.2, 99
    g = torch.Generator().manual_seed(7)
    X, R, dO = (torch.randn(t, d, generator=g).to(torch.bfloat16) for _ in range(3))
    gamma = (1 + 0.1 * torch.randn(d, generator=g)).to(torch.bfloat16)
    W = (torch.randn(d, d, generator=g) / np.sqrt(d)).to(torch.bfloat16)
    b = torch.randn(d, generator=g).to(torch.bfloat16)
    Xg, Rg, dOg, gg, Wg, bg = (v.cuda() for v in (X, R, dO, gamma, W, b))
    Wt = Wg.t().contiguous()
    H, Y, U, O, dU, dY, dH = (torch.empty_like(Xg) for _ in range(7))
    rstd, dgamma = torch.empty(t, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    with gemm_epi.Plan(t, d, d, "bf16", "BIAS") as fwd, gemm_epi.Plan(t, d, d, "bf16", "NONE") as bwd:
        gemm_epi.gemm_epi_rmsnorm(t, d, "bf16", Xg, Rg, gg, 1e-6, H, Y, rstd)
        fwd.execute(Y, Wg, bg, U)
        gemm_epi.gemm_epi_dropout(t * d, "bf16", U, H, p, seed, 0, O)
        gemm_epi.gemm_epi_dropout(t * d, "bf16", dOg, None, p, seed, 0, dU)
        bwd.execute(dU, Wt, None, dY)
        gemm_epi.gemm_epi_rmsnorm_backward(t, d, "bf16", dY, H, gg, rstd, dOg, dH, dgamma, ws)
        assert fwd.sync_status() == 0 and bwd.sync_status() == 0
    keep = torch.from_numpy(ref.dropout_keep(0, t * d, p, seed, 0)).view(t, d)
    scale = 65536 / (65536 - ref.dropped(p))
    h = H.cpu().double().requires_grad_()
    g64 = gamma.double().requires_grad_()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * g64
    o = h + keep * (y @ W.double() + b.double()) * scale
    (o * dO.double()).sum().backward()
    assert rel_err(O, o.detach().numpy()) <= TOL["bf16"]
    assert rel_err(dH, h.grad.numpy()) <= TOL["bf16"]
    # dgamma sums t terms, each with the relative error of dY's bf16 roundings (dU, dY): at most
    # 2 * 2^-8 of the terms' magnitudes, of dY's own sum over d products
    dU64 = (keep * dO.double() * scale)
    size = ((dU64.abs() @ W.double().abs().t()) * (h.detach() * rstd.cpu().double()[:, None]).abs()).sum(0)
    assert ((dgamma.cpu().double() - g64.grad).abs() <= 2.1 * 2.0 ** -8 * size).all()


def test_both_marshalling_paths_refuse_other_types_and_short_tensors():
    def tensor(dtype, count):
        return torch.zeros(count, device="cuda").to(getattr(torch, dtype))

    typed_refusals(gemm_epi._CtypesCalls(gemm_epi.load_library()), tensor)
    typed_refusals(gemm_epi._bind_calls(), tensor)


def test_tensors_of_whole_numbers_stand_for_their_bits():
    # 16-bit values as int16, codes as uint8: what a program that packs its own buffers passes
    X, R = (torch.randn(4, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    gamma = torch.rand(64, device="cuda").to(torch.bfloat16)
    outs = []
    for cast in (lambda v, t: v, lambda v, t: v.view(t)):
        H = torch.empty_like(X)
        Q = torch.empty(4, 64, dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(4, device="cuda")
        gemm_epi.gemm_epi_rmsnorm_e4m3(4, 64, "bf16", cast(X, torch.int16), cast(R, torch.int16),
                                       cast(gamma, torch.int16), 1e-6, cast(H, torch.int16), cast(Q, torch.uint8),
                                       "ROW", cast(scale, torch.int32))
        outs.append((H, Q.view(torch.uint8), scale))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
