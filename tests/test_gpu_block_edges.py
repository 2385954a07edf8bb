"""Block-scaled products and the LayerNorm calls at their edges: activations of extreme values, every number of
K slices, plans on two streams and in two graphs, operands and results past 2^31 elements."""
import math

import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import HALF

pytestmark = pytest.mark.gpu
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("variant", [2, 3])
@pytest.mark.parametrize("epilog", ["GELU_BIAS", "RELU_BIAS", "RELU_AUX_BIAS"])
def test_activations_of_every_size(epilog, variant, blocks):
    """A of zeros: the pre-activations are the bias, from 2^-126 to the largest bf16 of both signs, infinities and
    NaN, each of which stays in its own place."""
    m, n, k = 40, 1032, 144
    p = ref.product_problem(m, n, k, blocks, seed=1, device="cuda")
    p["A"].zero_()
    exponents = torch.arange(-126, 128, device="cuda")
    x = torch.cat([2.0 ** exponents, torch.tensor([3.3895e38], device="cuda"), torch.linspace(0.02, 12, 255, device="cuda")])
    x = torch.cat([x, -x, torch.tensor([0.0, float("inf"), float("-inf"), float("nan")], device="cuda")])
    x = x[torch.randperm(x.numel(), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")]
    p["bias"] = torch.cat([x, torch.zeros(n - x.numel(), device="cuda")]).to(BF16)
    D = torch.empty(m, n, dtype=BF16, device="cuda")
    aux = torch.empty(m, (n + 31) // 32, dtype=torch.int32, device="cuda") if epilog == "RELU_AUX_BIAS" else None
    with gemm_epi.Plan(m, n, k, "e4m3", epilog, SCALE_BLOCKS=blocks, VARIANT=variant) as plan:
        plan.execute(p["A"], p["B"], p["bias"], D, aux=aux, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    assert torch.equal(D.view(torch.int16), D[:1].view(torch.int16).expand(m, n))
    got, b = D[0].double(), p["bias"].double()
    if epilog == "GELU_BIAS":
        want = torch.where(b == -math.inf, 0.0, 0.5 * b * torch.special.erfc(-b / math.sqrt(2.0)))
        assert torch.equal(got.isnan(), b.isnan())
        assert got[b == math.inf].isinf().all() and (got[b == math.inf] > 0).all()
        fine = b.isfinite() | (b == -math.inf)
        # the approximation is within 3.1e-5 max(1, |x|), and a negative result of it no larger than |x| itself
        error = (3.1e-5 * b.abs().clamp(min=1.0)).minimum(torch.where(b < -9, 1e-8, math.inf))
        bound = HALF["bf16"] * (want.abs() + error) + error
        assert torch.all((got - want).abs()[fine] <= bound[fine])
    else:
        # (a NaN is not above 0)
        assert torch.equal(got, torch.where(b > 0, b, 0.0))


@pytest.mark.parametrize("variant", [2, 3])
@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("a,b", [(1e-27, 1e37), (1e37, 1e-27), (1e-3, 1e-27), (1e-27, 1e-3)])
def test_scales_of_opposite_extremes(a, b, blocks, variant):
    """The product of the two scales is formed first, whichever kernel runs: it has to be a normal number, a block's
    sum times either scale need not."""
    p = ref.product_problem(40, 264, 1040, blocks, seed=6, device="cuda")
    p["sa"] *= a
    p["sb"] *= b
    D = torch.empty(40, 264, dtype=BF16, device="cuda")
    with gemm_epi.Plan(40, 264, 1040, "e4m3", "NONE", SCALE_BLOCKS=blocks, VARIANT=variant) as plan:
        plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, blocks, "NONE")
    assert want.abs().max() < 3e38
    ref.check(D, want, error)


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("split", range(1, 9))
def test_every_split(split, tile, blocks):
    m, n, k = 70, 264, 2064
    p = ref.product_problem(m, n, k, blocks, seed=split, device="cuda")
    D = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
    again = torch.empty_like(D)
    with gemm_epi.Plan(m, n, k, "e4m3", "BIAS", SCALE_BLOCKS=blocks, VARIANT=2, TILE_N=tile, SPLIT_K=split) as plan:
        plan.execute(p["A"], p["B"], p["bias"], D, scales=(p["sa"], p["sb"]))
        plan.execute(p["A"], p["B"], p["bias"], again, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, blocks, "BIAS")
    ref.check(D, want, error)
    assert torch.equal(D, again)


def test_a_split_past_the_blocks_of_k():
    p = ref.product_problem(5, 136, 272, 1, seed=9, device="cuda")
    D = torch.full((5, 136), float("nan"), dtype=BF16, device="cuda")
    with gemm_epi.Plan(5, 136, 272, "e4m3", "NONE", SCALE_BLOCKS=1, VARIANT=2, SPLIT_K=8) as plan:
        assert "split_k=3(" in plan.describe()
        plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, 1, "NONE")
    ref.check(D, want, error)


@pytest.mark.parametrize("blocks", [1, 2])
def test_two_streams_at_once(blocks):
    """Calls of both kernels, the norm and the quantisation that run at the same time on two streams."""
    shapes = [(900, 784, 1040), (24, 1040, 4112)]
    problems = [ref.product_problem(m, n, k, blocks, seed=m, device="cuda") for m, n, k in shapes]
    plans = [gemm_epi.Plan(m, n, k, "e4m3", "GELU_BIAS", SCALE_BLOCKS=blocks, TILE_ORDER=2) for m, n, k in shapes]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()

    def alone(i, stream, times):
        p, (m, n, _) = problems[i], shapes[i]
        with torch.cuda.stream(stream):
            D = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(times)]
            gamma, beta = torch.ones(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
            out = []
            for d in D:
                plans[i].execute(p["A"], p["B"], p["bias"], d, scales=(p["sa"], p["sb"]), stream=stream)
                Y = torch.empty_like(d)
                gemm_epi.gemm_epi_layernorm_forward(m, n, "bf16", d, None, gamma, beta, 1e-5, None, Y, stream=stream)
                Q = torch.empty(m, n, dtype=E4M3, device="cuda")
                s = torch.empty((n + 127) // 128, m, device="cuda")
                gemm_epi.gemm_epi_e4m3_quantize(m, n, "bf16", "1X128", Y, Q, s, stream=stream)
                out += [d, Y, Q.view(torch.uint8), s]
        return out

    want = []
    for i in range(2):
        want.append(alone(i, streams[i], 1))
        torch.cuda.synchronize()
    got = [alone(i, streams[i], 20) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert plans[i].sync_status() == 0
        for j, v in enumerate(got[i]):
            assert torch.equal(v, want[i][j % len(want[i])])
        plans[i].free()
    for i in range(2):
        d, _, error = ref.product(problems[i], blocks, "GELU_BIAS")
        ref.check(want[i][0], d, error)


def test_one_plan_in_two_graphs():
    """Two graphs of one plan (and of one workspace) replayed in turn on a stream."""
    m, n, k = 1500, 528, 528
    p = ref.product_problem(m, n, k, 1, seed=3, device="cuda")
    D = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2)]
    dX = [torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(2)]
    stats, gamma = torch.ones(m, 2, device="cuda"), torch.ones(n, dtype=BF16, device="cuda")
    sums = torch.empty(2, 2, n, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_layernorm_workspace(m, n), dtype=torch.uint8, device="cuda")
    with gemm_epi.Plan(m, n, k, "e4m3", "BIAS", SCALE_BLOCKS=1, TILE_ORDER=2, GRID=4) as plan:
        graphs = []
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                plan.execute(p["A"], p["B"], p["bias"], D[i], scales=(p["sa"], p["sb"]))
                gemm_epi.gemm_epi_layernorm_backward(m, n, "bf16", p["R"], D[i], gamma, stats, None, dX[i], sums[i][0],
                                                     sums[i][1], ws)
        for i in (0, 1, 1, 0, 1):
            graphs[i].replay()
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, 1, "BIAS")
    ref.check(D[0], want, error)
    for pair in (D, dX, sums):
        assert torch.equal(pair[0], pair[1])


def _last(p, rows, cols, blocks):
    """The problem of the last rows of A and of B (whole tiles of 128 of them)."""
    m, n = p["A"].shape[0], p["B"].shape[0]
    i, j = m - rows, (n - cols) // 128 * 128
    sb = p["sb"][:, j:] if blocks == 2 else p["sb"][:, j // 128:]
    return {"A": p["A"][i:], "B": p["B"][j:], "sa": p["sa"][:, i:], "sb": sb.contiguous(),
            "bias": p["bias"][j:]}, i, j


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("m,n,k", [(33000, 136, 65552), (3, 33000, 65552), (262400, 8200, 16)])
def test_past_32_bits(m, n, k, blocks):
    """A, B or D of more than 2^31 elements: the last rows and columns."""
    kb = ref.up(k, 128) // 128
    g = torch.Generator(device="cuda").manual_seed(m)

    def bytes_of(rows):  # (no NaN: every code with its top bits below 0x78, both signs)
        v = torch.randint(0, 0x78, (rows, k), dtype=torch.uint8, generator=g, device="cuda")
        return v.bitwise_or_(torch.randint(0, 2, (rows, 1), dtype=torch.uint8, generator=g, device="cuda") * 128).view(E4M3)

    p = {"A": bytes_of(m), "B": bytes_of(n), "sa": torch.rand(kb, m, generator=g, device="cuda") / 4096,
         "sb": torch.rand(kb, n if blocks == 2 else ref.up(n, 128) // 128, generator=g, device="cuda") / 4096,
         "bias": torch.randn(n, generator=g, device="cuda").to(BF16)}
    D = torch.empty(m, n, dtype=BF16, device="cuda")
    with gemm_epi.Plan(m, n, k, "e4m3", "BIAS", SCALE_BLOCKS=blocks) as plan:
        plan.execute(p["A"], p["B"], p["bias"], D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    last, i, j = _last(p, min(m, 140), min(n, 140), blocks)
    want, _, error = ref.product(last, blocks, "BIAS")
    ref.check(D[i:, j:], want, error, what="last")


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("variant", [2, 3])
@pytest.mark.parametrize("n", [2 ** 31 - 120, 2 ** 31 - 8])
def test_the_largest_n(n, variant, blocks):
    """n up to the largest that a plan takes, where n + 127 passes 32 bits: columns of the first, the middle and the
    last tiles."""
    torch.cuda.empty_cache()
    m, k = 1, 16
    g = torch.Generator(device="cuda").manual_seed(n % 1000)
    B = torch.empty(n, k, dtype=torch.uint8, device="cuda")
    for at in range(0, n, 2 ** 26):  # (no NaN: every code with its top bits below 0x78)
        some = B[at:at + 2 ** 26]
        some.copy_(torch.randint(0, 0x78, some.shape, dtype=torch.uint8, generator=g, device="cuda"))
    p = {"A": torch.randn(m, k, generator=g, device="cuda").to(E4M3), "B": B.view(E4M3),
         "sa": torch.rand(1, m, generator=g, device="cuda") + 0.5,
         "sb": torch.rand(1, n if blocks == 2 else ref.up(n, 128) // 128, generator=g, device="cuda") + 0.5}
    D = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
    with gemm_epi.Plan(m, n, k, "e4m3", "NONE", SCALE_BLOCKS=blocks, VARIANT=variant) as plan:
        plan.execute(p["A"], p["B"], None, D, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    cols = 2 ** 20
    for first in (0, n // 2 // 128 * 128, (n - cols) // 128 * 128):
        last = first + cols if first + cols + 128 <= n else n
        sb = p["sb"][:, first:last] if blocks == 2 else p["sb"][:, first // 128:ref.up(last, 128) // 128]
        want, _, error = ref.product({"A": p["A"], "B": p["B"][first:last], "sa": p["sa"], "sb": sb.contiguous()},
                                     blocks, "NONE")
        ref.check(D[:, first:last], want, error, what=f"from column {first}")
    assert not D.isnan().any()


@pytest.mark.parametrize("t,d", [(131200, 16384), (2 ** 28 + 40, 8), (40000, 65536)])
def test_layernorm_past_32_bits(t, d):
    """More than 2^31 elements: the last rows, forward, to E4M3 and backward."""
    g = torch.Generator(device="cuda").manual_seed(d)
    rows = 64
    X = torch.zeros(t, d, dtype=BF16, device="cuda")
    tail = torch.randn(rows, d, generator=g, device="cuda").to(BF16)
    X[-rows:] = tail
    gamma = (torch.rand(d, generator=g, device="cuda") + 0.5).to(BF16)
    beta = torch.randn(d, generator=g, device="cuda").to(BF16)
    Y, stats = torch.empty_like(X), torch.empty(t, 2, device="cuda")
    gemm_epi.gemm_epi_layernorm_forward(t, d, "bf16", X, None, gamma, beta, 1e-5, None, Y, stats)
    y, _, _, error = ref.layernorm(tail, gamma, beta, 1e-5)
    ref.check(Y[-rows:], y, error, what="Y")
    assert torch.equal(Y[0], beta)
    Q, s = torch.empty(t, d, dtype=E4M3, device="cuda"), torch.empty(ref.up(d, 128) // 128, t, device="cuda")
    gemm_epi.gemm_epi_layernorm_e4m3(t, d, "bf16", X, None, gamma, beta, 1e-5, None, Q, s)
    wide = ref.spread(s[:, -rows:].contiguous(), "1X128", rows, d)
    ref.check_codes(Q[-rows:], y / wide, error / wide + 4 * 2.0 ** -24 * (y / wide).abs(), "Q")
    del Q, s
    dY = Y.zero_()
    dY[-rows:] = torch.randn(rows, d, generator=g, device="cuda").to(BF16)
    dX, dgamma, dbeta = torch.empty_like(X), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    ws = torch.empty(gemm_epi.gemm_epi_layernorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    gemm_epi.gemm_epi_layernorm_backward(t, d, "bf16", dY, X, gamma, stats, None, dX, dgamma, dbeta, ws)
    want = ref.layernorm_backward(dY[-rows:], tail, gamma, stats[-rows:].contiguous(), None)
    ref.check(dX[-rows:], want[0], want[3], what="dX")
    assert not dX[0].any()
    # (rows of zeros add nothing to the sums and to the sizes that bound their errors)
    assert torch.all((dgamma.double() - want[1]).abs() <= want[4])
    assert torch.all((dbeta.double() - want[2]).abs() <= want[5])


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("order", [1, 2])
@pytest.mark.parametrize("k", [16, 128, 144, 384, 512, 528, 640, 1040])
def test_one_pair_walks_every_tile(k, order, blocks):
    """15 tiles of one to nine blocks of k in turn: what is handed from tile to tile (accumulators, scales, the
    bias of three tiles, boxes of D) in both orders."""
    m, n = 520, 1032
    p = ref.product_problem(m, n, k, blocks, seed=k, device="cuda")
    for epilog in ("BIAS", "GELU_BIAS"):
        D = torch.full((m, n), float("nan"), dtype=BF16, device="cuda")
        with gemm_epi.Plan(m, n, k, "e4m3", epilog, SCALE_BLOCKS=blocks, VARIANT=3, GRID=2, TILE_ORDER=order) as plan:
            for _ in range(2):
                plan.execute(p["A"], p["B"], p["bias"], D, scales=(p["sa"], p["sb"]))
            assert plan.sync_status() == 0
        want, _, error = ref.product(p, blocks, epilog)
        ref.check(D, want, error)
