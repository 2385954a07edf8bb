"""LayerNorm, the block-scaled quantisation and products run together, as a pre-norm layer in 8 bits uses
them, serving and training; and what a plan with block scales refuses."""
import math

import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import F32
from test_block_refusals import typed_refusals

pytestmark = pytest.mark.gpu
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _codes(rows, cols, square=False):
    """Buffers for the codes and scales of a matrix."""
    return (torch.empty(rows, cols, dtype=E4M3, device="cuda"),
            torch.empty(ref.up(cols, 128) // 128, ref.up(rows, 128) // 128 if square else rows, device="cuda"))


def _value(q, s, block):
    return q.double() * ref.spread(s, block, *q.shape)


@pytest.mark.parametrize("t", [1, 40, 500])
def test_feed_forward_serving(t):
    """H = X + R, Q = LN(H), G = GELU(Q W1 + b1), Z = quantised G times W2 + b2 + H, eager and from a graph."""
    d, f, eps = 272, 1040, 1e-5
    g = torch.Generator(device="cuda").manual_seed(t)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)

    X, R, gamma, beta = normal(t, d), normal(t, d), normal(d, scale=0.3) + 1, normal(d, scale=0.1)
    W1, b1, W2, b2 = normal(d, f, scale=1 / math.sqrt(d)), normal(f), normal(f, d, scale=1 / math.sqrt(f)), normal(d)
    Wq1, s1 = _codes(f, d, True)
    Wq2, s2 = _codes(d, f, True)
    gemm_epi.gemm_epi_e4m3_quantize(d, f, "bf16", "128X128", W1, Qt=Wq1, scale_t=s1)
    gemm_epi.gemm_epi_e4m3_quantize(f, d, "bf16", "128X128", W2, Qt=Wq2, scale_t=s2)
    (Q, sq), (Gq, sg) = _codes(t, d), _codes(t, f)
    H, G, Z = torch.empty_like(X), torch.empty(t, f, dtype=BF16, device="cuda"), torch.empty_like(X)
    with gemm_epi.Plan(t, f, d, "e4m3", "GELU_BIAS", SCALE_BLOCKS=1) as p1, \
            gemm_epi.Plan(t, d, f, "e4m3", "BIAS_RESIDUAL", SCALE_BLOCKS=1) as p2:
        def step():
            gemm_epi.gemm_epi_layernorm_e4m3(t, d, "bf16", X, R, gamma, beta, eps, H, Q, sq)
            p1.execute(Q, Wq1, b1, G, scales=(sq, s1))
            gemm_epi.gemm_epi_e4m3_quantize(t, f, "bf16", "1X128", G, Gq, sg)
            p2.execute(Gq, Wq2, b2, Z, residual=H, scales=(sg, s2))
        step()
        torch.cuda.synchronize()
        eager = [v.clone() for v in (H, G, Z)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for v in (H, G, Z):
            v.fill_(float("nan"))
        for _ in range(3):
            graph.replay()
        assert p1.sync_status() == 0 and p2.sync_status() == 0
    for got, want in zip((H, G, Z), eager):
        assert torch.equal(got, want)
    # each step against 64 bits, from what the step before stored
    y, _, _, error = ref.layernorm(H, gamma, beta, eps)
    s = ref.spread(sq, "1X128", t, d)
    ref.check_codes(Q, y / s, error / s + 4 * F32 * (y / s).abs(), "Q")
    ref.check_quantized(W1.t(), "128X128", Wq1, s1)
    want, _, error = ref.product({"A": Q, "B": Wq1, "sa": sq, "sb": s1, "bias": b1}, 1, "GELU_BIAS")
    ref.check(G, want, error, what="G")
    ref.check_quantized(G, "1X128", Gq, sg, "G's codes")
    want, _, error = ref.product({"A": Gq, "B": Wq2, "sa": sg, "sb": s2, "bias": b2, "R": H}, 1, "BIAS_RESIDUAL")
    ref.check(Z, want, error, what="Z")


@pytest.mark.parametrize("t", [200, 1031])
def test_linear_training(t):
    """Forward: H = X + R, Y = LN(H), U = Y W + b.  Backward from dU and dH: dY = dU W^T, dW = Y^T dU, and dX,
    dgamma, dbeta of the norm; the products in block-scaled 8 bits, against 64 bits on the codes they read."""
    d, f, eps = 272, 528, 1e-5
    g = torch.Generator(device="cuda").manual_seed(t)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)

    X, R, dU, dH = normal(t, d), normal(t, d), normal(t, f), normal(t, d)
    gamma, beta, W, b = normal(d, scale=0.3) + 1, normal(d, scale=0.1), normal(d, f, scale=1 / math.sqrt(d)), normal(f)
    ldt = ref.up(t, 16)
    (Y8, sy), (Yt, syt), (dU8, sd), (dUt, sdt) = _codes(t, d), _codes(d, ldt), _codes(t, f), _codes(f, ldt)
    (Wt8, swt), (W8, sw) = _codes(f, d, True), _codes(d, f, True)
    H, Y, dY, dX = (torch.empty_like(X) for _ in range(4))
    U, dW = torch.empty(t, f, dtype=BF16, device="cuda"), torch.empty(d, f, dtype=BF16, device="cuda")
    stats, dgamma, dbeta = (torch.empty(*s, device="cuda") for s in ((t, 2), (d,), (d,)))
    ws = torch.empty(gemm_epi.gemm_epi_layernorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    with gemm_epi.Plan(t, f, d, "e4m3", "BIAS", SCALE_BLOCKS=1) as fwd, \
            gemm_epi.Plan(t, d, f, "e4m3", "NONE", SCALE_BLOCKS=1) as bwd, \
            gemm_epi.Plan(d, f, ldt, "e4m3", "NONE", SCALE_BLOCKS=2) as wgrad:
        def step():
            gemm_epi.gemm_epi_e4m3_quantize(d, f, "bf16", "128X128", W, W8, sw, Wt8, swt)
            gemm_epi.gemm_epi_layernorm_forward(t, d, "bf16", X, R, gamma, beta, eps, H, Y, stats)
            gemm_epi.gemm_epi_e4m3_quantize(t, d, "bf16", "1X128", Y, Y8, sy, Yt, syt)
            fwd.execute(Y8, Wt8, b, U, scales=(sy, swt))
            gemm_epi.gemm_epi_e4m3_quantize(t, f, "bf16", "1X128", dU, dU8, sd, dUt, sdt)
            bwd.execute(dU8, W8, None, dY, scales=(sd, sw))
            wgrad.execute(Yt, dUt, None, dW, scales=(syt, sdt))
            gemm_epi.gemm_epi_layernorm_backward(t, d, "bf16", dY, H, gamma, stats, dH, dX, dgamma, dbeta, ws)
        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=side):
            step()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in (U, dY, dW, dX, dgamma, dbeta)]
        step()
        assert all(p.sync_status() == 0 for p in (fwd, bwd, wgrad))
    for got, want in zip((U, dY, dW, dX, dgamma, dbeta), replayed):
        assert torch.equal(got, want)
    y, _, _, error = ref.layernorm(H, gamma, beta, eps)
    ref.check(Y, y, error, what="Y")
    for what, got, problem, blocks in (("U", U, (Y8, Wt8, sy, swt), 1), ("dY", dY, (dU8, W8, sd, sw), 1),
                                       ("dW", dW, (Yt, dUt, syt, sdt), 2)):
        p = dict(zip(("A", "B", "sa", "sb"), problem), bias=b)
        want, _, error = ref.product(p, blocks, "BIAS" if what == "U" else "NONE")
        ref.check(got, want, error, what=what)
    # the codes stand for Y and dU within half a step of E4M3 each: dW is the gradient to that
    full = Y.double().t() @ dU.double()
    size = Y.double().abs().t() @ dU.double().abs()
    assert torch.all((dW.double() - full).abs() <= (2.2 * 2.0 ** -4 + 2.0 ** -8) * size + 1e-2)
    want = ref.layernorm_backward(dY, H, gamma, stats, dH)
    ref.check(dX, want[0], want[3], what="dX")
    assert torch.all((dgamma.double() - want[1]).abs() <= want[4])
    assert torch.all((dbeta.double() - want[2]).abs() <= want[5])


def _status(call):
    with pytest.raises(gemm_epi.GemmEpiError) as e:
        call()
    return e.value.status


def test_options():
    for dtype, value in (("bf16", 1), ("e4m3", 3), ("e4m3", -1)):
        assert _status(lambda: gemm_epi.Plan(64, 64, 64, dtype, "BIAS", SCALE_BLOCKS=value)) == 1
    assert _status(lambda: gemm_epi.Plan(64, 64, 64, "e4m3", "BIAS", SCALE_A_ROWS=1, SCALE_BLOCKS=1)) == 1
    assert _status(lambda: gemm_epi.Plan(64, 64, 64, "e4m3", "BIAS", SCALE_BLOCKS=1, SCALE_A_ROWS=1)) == 1
    for opts in (dict(VARIANT=1), dict(VARIANT=5), dict(VARIANT=3, TILE_N=224), dict(VARIANT=2, TILE_N=256)):
        assert _status(lambda: gemm_epi.Plan(64, 64, 64, "e4m3", "BIAS", SCALE_BLOCKS=2, **opts)) == 1, opts
    # back to one scale for the tensor
    p = ref.product_problem(20, 264, 144, 1, seed=1, device="cuda")
    one = torch.ones(1, device="cuda")
    D = torch.empty(20, 264, dtype=BF16, device="cuda")
    with gemm_epi.Plan(20, 264, 144, "e4m3", "NONE", SCALE_BLOCKS=1) as plan:
        plan.set_option("SCALE_BLOCKS", 0)
        assert "variant=row-pair" in plan.describe()
        plan.execute(p["A"], p["B"], None, D, scales=(one, one))
        assert plan.sync_status() == 0
    p["sa"], p["sb"] = torch.ones_like(p["sa"]), torch.ones_like(p["sb"])
    want, _, error = ref.product(p, 1, "NONE")
    ref.check(D, want, error)


@pytest.mark.parametrize("m", [20, 700])
def test_operand_refusals(m):
    n, k = 264, 144
    p = ref.product_problem(m, n, k, 2, seed=1, device="cuda")
    D = torch.empty(m, n, dtype=BF16, device="cuda")
    raw = {name: v.data_ptr() for name, v in p.items()}
    with gemm_epi.Plan(m, n, k, "e4m3", "BIAS_RESIDUAL", SCALE_BLOCKS=2) as plan:
        def call(**change):
            v = dict(raw, D=D.data_ptr(), **{})
            v.update(change)
            plan.execute(v["A"], v["B"], v["bias"], v["D"], residual=v["R"], scales=(v["sa"], v["sb"]))
        for change, status in ((dict(sa=None), 1), (dict(sb=None), 1), (dict(A=None), 1), (dict(B=None), 1),
                               (dict(bias=None), 1), (dict(R=None), 1), (dict(D=None), 1), (dict(sb=raw["sb"] + 4), 3),
                               (dict(sa=raw["sa"] + 2), 3), (dict(A=raw["A"] + 8), 3), (dict(D=D.data_ptr() + 8), 3),
                               (dict(D=raw["A"]), 1), (dict(D=raw["B"]), 1), (dict(D=raw["bias"] // 16 * 16), 1),
                               (dict(D=raw["sa"]), 1), (dict(D=raw["sb"]), 1), (dict(D=raw["R"] + 16), 1)):
            assert _status(lambda: call(**change)) == status, change
        call(D=raw["R"])  # the residual itself
        assert plan.sync_status() == 0
        with pytest.raises(ValueError):
            plan.execute(p["A"], p["B"], p["bias"], D, residual=p["R"], scales=(p["sa"][:-1].contiguous(), p["sb"]))
        with pytest.raises(ValueError):
            plan.execute(p["A"].float(), p["B"], p["bias"], D, residual=p["R"], scales=(p["sa"], p["sb"]))
        with pytest.raises(ValueError):
            plan.execute(p["A"], p["B"], p["bias"].cpu(), D, residual=p["R"], scales=(p["sa"], p["sb"]))
    want, _, error = ref.product(dict(p, R=ref.product_problem(m, n, k, 2, seed=1, device="cuda")["R"]), 2, "BIAS_RESIDUAL")
    ref.check(p["R"], want, error)


@pytest.mark.parametrize("m", [20, 700])
@pytest.mark.parametrize("blocks", [1, 2])
def test_unfused_empty_and_k_0(m, blocks):
    n, k = 264, 400
    p = ref.product_problem(m, n, k, blocks, seed=2, device="cuda")
    D, pre = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2))
    with gemm_epi.Plan(m, n, k, "e4m3", "RELU_BIAS", SCALE_BLOCKS=blocks) as plan:
        plan.execute_unfused(p["A"], p["B"], p["bias"], pre, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, blocks, "NONE")
    ref.check(pre, want, error)
    assert torch.equal(D, (pre.float() + p["bias"].float()).clamp(min=0).to(BF16))
    # nothing to sum: the bias alone; no rows: nothing at all
    with gemm_epi.Plan(m, n, 0, "e4m3", "BIAS", SCALE_BLOCKS=blocks) as plan:
        plan.execute(None, None, p["bias"], D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    assert torch.equal(D, p["bias"].expand(m, n))
    with gemm_epi.Plan(0, n, k, "e4m3", "BIAS", SCALE_BLOCKS=blocks) as plan:
        plan.execute(None, None, None, None)
    with gemm_epi.Plan(m, 0, k, "e4m3", "BIAS", SCALE_BLOCKS=blocks) as plan:
        plan.execute(None, None, None, None)


@pytest.mark.parametrize("opts", [dict(VARIANT=2, SPLIT_K=3), dict(VARIANT=3)])
def test_a_wait_that_runs_out_is_reported(opts):
    p = ref.product_problem(40, 264, 1040, 1, seed=3, device="cuda")
    D = torch.full((40, 264), 7.0, dtype=BF16, device="cuda")
    with gemm_epi.Plan(40, 264, 1040, "e4m3", "NONE", SCALE_BLOCKS=1, **opts, WAIT_LIMIT_US=2000, DEBUG_STALL=1) as plan:
        plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 8
        assert (D == 7).all()
        plan.set_option("DEBUG_STALL", 0)
        plan.set_option("WAIT_LIMIT_US", 0)
        plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, 1, "NONE")
    ref.check(D, want, error)


@pytest.mark.parametrize("m,opts", [(3, {}), (3, dict(B_READY=1)), (100, dict(B_READY=1, SPLIT_K=2)), (700, {})])
def test_back_to_back(m, opts):
    """Products that follow one another on a stream, each reading what the one before wrote."""
    n = k = 528
    p = ref.product_problem(m, n, k, 1, seed=4, device="cuda")
    D = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(6)]
    Q, s = _codes(m, n)
    Q.copy_(p["A"])
    s.copy_(p["sa"])
    with gemm_epi.Plan(m, n, k, "e4m3", "BIAS", SCALE_BLOCKS=1, **opts) as plan:
        for out in D:
            plan.execute(Q, p["B"], p["bias"], out, scales=(s, p["sb"]))
            gemm_epi.gemm_epi_e4m3_quantize(m, n, "bf16", "1X128", out, Q, s)
        assert plan.sync_status() == 0
        Q.copy_(p["A"])
        s.copy_(p["sa"])
        for out in D:
            again = torch.empty_like(out)
            plan.execute(Q, p["B"], p["bias"], again, scales=(s, p["sb"]))
            torch.cuda.synchronize()
            assert torch.equal(again, out)
            gemm_epi.gemm_epi_e4m3_quantize(m, n, "bf16", "1X128", out, Q, s)
            torch.cuda.synchronize()
    want, _, error = ref.product(p, 1, "BIAS")
    ref.check(D[0], want, error)


def test_nan_and_infinite_scales_stay_in_their_rows():
    for m in (20, 700):
        p = ref.product_problem(m, 264, 400, 2, seed=5, device="cuda")
        p["sa"][1, 3], p["sb"][2, 70] = float("nan"), float("inf")
        D = torch.empty(m, 264, dtype=BF16, device="cuda")
        with gemm_epi.Plan(m, 264, 400, "e4m3", "NONE", SCALE_BLOCKS=2) as plan:
            plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
            assert plan.sync_status() == 0
        fine = torch.isfinite(D.float())
        assert not fine[3].any() and not fine[:, 70].any()
        fine[3], fine[:, 70] = True, True
        assert fine.all()


def test_both_marshalling_paths_refuse_other_types_and_short_tensors():
    def tensor(dtype, count):
        return torch.zeros(count, device="cuda").to(getattr(torch, dtype))

    typed_refusals(gemm_epi._CtypesCalls(gemm_epi.load_library()), tensor)
    typed_refusals(gemm_epi._bind_calls(), tensor)
