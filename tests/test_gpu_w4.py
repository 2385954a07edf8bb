"""Products with 4-bit weights and group scales, and the weights written out, against 64 bits."""
import pytest
import torch

import sublayer_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import TD

pytestmark = pytest.mark.gpu

EPILOGS = ["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS", "TANH_BIAS", "BIAS_RESIDUAL"]
# (m, n, k): one to 64 rows around every multiple of 8, n and k that end inside a tile
SHAPES = [(1, 8, 32), (1, 264, 96), (2, 520, 1024), (3, 40, 2080), (7, 72, 4096), (8, 136, 160),
          (9, 1000, 512), (15, 24, 8192), (16, 256, 256), (17, 48, 1056), (31, 88, 640),
          (32, 64, 2048), (33, 200, 384), (48, 1024, 1152), (63, 16, 4160), (64, 328, 1024)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _run(p, group, dtype, epilog, stream=None, D=None):
    m, k = p["A"].shape
    n = p["W"].shape[0]
    g = {key: None if v is None else v.cuda() for key, v in p.items() if key != "q"}
    if D is None:
        D = torch.full((m, n), float("nan"), dtype=TD[dtype], device="cuda")
    gemm_epi.gemm_epi_w4_matmul(m, n, k, group, dtype, epilog, g["A"], g["W"], g["scales"], g["zeros"],
                                None if epilog == "NONE" else g["bias"],
                                g["R"] if epilog == "BIAS_RESIDUAL" else None, D, stream)
    return D


def _check(p, group, dtype, epilog, what=""):
    D = _run(p, group, dtype, epilog)
    want, error = ref.w4_matmul(p, group, epilog)
    ref.check_16(D, want, dtype, error, f"D {what}")


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_matmul(m, n, k, group, dtype):
    k = -(-k // group) * group
    epilog = EPILOGS[(m + n // 8 + group // 32) % len(EPILOGS)]
    _check(ref.w4_problem(m, n, k, group, dtype, (m + group // 32) % 2 == 0, m + n + k), group, dtype, epilog)


@pytest.mark.parametrize("m,n,k", [(9, 4104, 4096), (16, 12296, 1152), (13, 1536, 8320), (24, 4232, 4096),
                                   (48, 19600, 672), (64, 1160, 12320), (3, 16392, 1056), (8, 5000, 4224)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_larger_weights(m, n, k, group):
    # weights large enough for the other choices of kernel and of k's split, with more tiles of
    # columns than SMs among them
    k = -(-k // group) * group
    dtype, epilog = ("bf16", "GELU_BIAS") if group == 64 else ("f16", "BIAS_RESIDUAL")
    _check(ref.w4_problem(m, n, k, group, dtype, group != 64, m + n), group, dtype, epilog)


@pytest.mark.parametrize("m,n,k,group", [(1, 5128, 4224, 128), (4, 2056, 10368, 128), (2, 264, 81920, 128),
                                         (3, 21856, 1024, 128), (1, 40, 600064, 128), (3, 4104, 15424, 64),
                                         (4, 512, 122944, 64)])
@pytest.mark.parametrize("dtype,zeros", [("bf16", False), ("f16", True)])
def test_w4_few_rows_of_a_large_weight(m, n, k, group, dtype, zeros):
    _check(ref.w4_problem(m, n, k, group, dtype, zeros, m + n), group, dtype, "BIAS_RESIDUAL" if zeros else "TANH_BIAS")


def _integer_problem(m, n, k, group, dtype, zeros, seed):
    """Integer activations, weights and scales whose sums fp32 holds exactly in any order, and a residual
    that takes each sum down to what its rounding to 16 bits left: D is a small whole number, exactly,
    and one wrong, missing or doubled term shows in it."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (n, k), generator=g, dtype=torch.uint8)
    z = torch.randint(0, 16, (k // group, n), generator=g).to(torch.uint8) if zeros else None
    scales = torch.randint(1, 3, (k // group, n), generator=g).to(TD[dtype])
    A = torch.randint(-1, 2, (m, k), generator=g).to(TD[dtype])
    B = ref.w4_weight(q, scales, z, group)
    # every partial sum is a whole number below 2^24
    assert (A.double().abs() @ B.abs()).max() < 2 ** 24
    total = A.double() @ B
    R = (-total).to(TD[dtype])
    want = total + R.double()
    assert torch.equal(want.to(TD[dtype]).double(), want)
    return dict(q=q, W=ref.w4_pack(q), scales=scales, zeros=z, A=A, bias=torch.zeros(n, dtype=TD[dtype]), R=R), want


@pytest.mark.parametrize("m,n,k,group", [(1, 40, 600064, 128), (2, 264, 98432, 128), (4, 264, 81920, 128),
                                         (1, 104, 604992, 64), (4, 512, 122944, 64)])
@pytest.mark.parametrize("dtype,zeros", [("bf16", False), ("f16", True)])
def test_w4_stretches_of_k_are_exact(m, n, k, group, dtype, zeros):
    """k of several stretches of shared memory in each block of the streaming kernel (100 KB hold 36
    times 1024 values of k for one row with groups of 128, 8 for four rows), the last one shorter."""
    p, want = _integer_problem(m, n, k, group, dtype, zeros, m + n)
    D = torch.full((m + 1, n), 7.0, dtype=TD[dtype], device="cuda")
    _run(p, group, dtype, "BIAS_RESIDUAL", D=D[:m])
    assert torch.equal(D[:m].double().cpu(), want) and (D[m:] == 7.0).all()


@pytest.mark.parametrize("m,n,k,group", [(1, 40, 600064, 128), (4, 264, 81920, 128), (4, 512, 122944, 64)])
@pytest.mark.parametrize("dtype,zeros", [("bf16", False), ("f16", True)])
def test_w4_stretches_of_k_within_the_sum_s_own_chain(m, n, k, group, dtype, zeros):
    p = ref.w4_problem(m, n, k, group, dtype, zeros, m + n)
    B, A = ref.w4_weight(p["q"], p["scales"], p["zeros"], group), p["A"].double()
    want = A @ B
    # the chain of a sum: the matrix instructions of one group (16 k each; they may truncate, a whole
    # step), a group's sum scaled and added for each of the warp's groups (an eighth of k or less), then
    # the eight warps and up to eight blocks
    error = (group / 16 + k / (8 * group) + 1 + 16) * 2 * ref.F32 * (A.abs() @ B.abs())
    assert error.mean() < 0.1 * want.abs().mean()  # (a bound that a wrong sum does not keep)
    ref.check_16(_run(p, group, dtype, "NONE"), want, dtype, error, "D")


def test_w4_eight_rows_of_the_largest_weights():
    _check(ref.w4_problem(6, 16392, 6144, 128, "bf16", True, 5), 128, "bf16", "GELU_BIAS")


def test_w4_few_rows_of_a_large_weight_exact_and_untouched():
    # integers as above at the larger sizes, and rows behind the last left as they were
    g = torch.Generator().manual_seed(3)
    m, n, k = 3, 1032, 21248
    for group in (128, 64):
        n = 1032 if group == 128 else 2968
        q = torch.full((n, k), 8)
        at = torch.randint(0, k, (n, 9), generator=g)
        q.scatter_(1, at, torch.randint(0, 16, (n, 9), generator=g))
        A = torch.randint(-2, 3, (m, k), generator=g).to(torch.bfloat16)
        p = dict(q=q, W=ref.w4_pack(q), scales=torch.ones(k // group, n, dtype=torch.bfloat16), zeros=None, A=A,
                 bias=None, R=None)
        D = torch.full((m + 2, n), 7.0, dtype=torch.bfloat16, device="cuda")
        _run(p, group, "bf16", "NONE", D=D[:m])
        want = A.double() @ ref.w4_weight(q, p["scales"], None, group)
        assert torch.equal(D[:m].double().cpu(), want) and (D[m:] == 7.0).all()


@pytest.mark.parametrize("epilog", EPILOGS)
@pytest.mark.parametrize("m", [1, 5, 12, 40])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_epilogs(epilog, m, zeros):
    for dtype in ("bf16", "f16"):
        _check(ref.w4_problem(m, 104, 768, 64, dtype, zeros, m), 64, dtype, epilog, epilog)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1, 11, 37])
def test_w4_integers_are_exact(group, dtype, m):
    # integer activations and unit scales: every sum is an integer that fp32 holds, and small
    # enough for the output type (a wrong or missing term shows as a whole number)
    g = torch.Generator().manual_seed(group + m)
    n, k = 72, 896
    q = torch.full((n, k), 8)
    z = torch.full((k // group, n), 8, dtype=torch.uint8)
    at = torch.randint(0, k, (n, 6), generator=g)
    q.scatter_(1, at, torch.randint(0, 16, (n, 6), generator=g))
    A = torch.randint(-2, 3, (m, k), generator=g).to(TD[dtype])
    p = dict(q=q, W=ref.w4_pack(q), scales=torch.ones(k // group, n, dtype=TD[dtype]), zeros=z, A=A,
             bias=None, R=None)
    want = A.double() @ ref.w4_weight(q, p["scales"], z, group)
    for zeros in (z, None):
        D = _run({**p, "zeros": zeros}, group, dtype, "NONE")
        assert torch.equal(D.double().cpu(), want)


def test_w4_every_position_and_value():
    # A picks out single rows of B: every nibble position, value, group and zero point
    n, group = 16, 32
    for dtype in ("bf16", "f16"):
        for k in (32, 128, 288, 512):
            q = (torch.arange(n * k).view(n, k) * 7 + torch.arange(n).view(n, 1)) % 16
            z = (torch.arange(k // group * n).view(-1, n) % 16).to(torch.uint8)
            scales = torch.pow(2.0, (torch.arange(k // group * n).view(-1, n) % 5 - 2).float()).to(TD[dtype])
            B = ref.w4_weight(q, scales, z, group)
            for k0 in range(0, k, 64):
                rows = min(64, k - k0)
                A = torch.zeros(rows, k, dtype=TD[dtype])
                A[torch.arange(rows), k0 + torch.arange(rows)] = 1
                p = dict(q=q, W=ref.w4_pack(q), scales=scales, zeros=z, A=A, bias=None, R=None)
                assert torch.equal(_run(p, group, dtype, "NONE").double().cpu(), B[k0:k0 + rows])


def test_w4_rows_do_not_mix():
    # a NaN or an infinity in one row of A reaches that row of D only; behind the last row
    # nothing is written
    p = ref.w4_problem(5, 64, 512, 64, "bf16", False, 3)
    clean = _run(p, 64, "bf16", "BIAS").cpu()
    p["A"][2, 100] = float("nan")
    p["A"][3, 7] = float("inf")
    D = torch.full((8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    _run(p, 64, "bf16", "BIAS", D=D[:5])
    D = D.cpu()
    assert D[2].isnan().all() and not D[3].isfinite().any()
    assert torch.equal(D[[0, 1, 4]], clean[[0, 1, 4]]) and (D[5:] == 7.0).all()


def test_w4_in_place_residual_and_repeatable():
    p = ref.w4_problem(3, 520, 2048, 128, "bf16", True, 5)
    first = _run(p, 128, "bf16", "BIAS_RESIDUAL")
    R = p["R"].cuda()
    g = {key: None if v is None else v.cuda() for key, v in p.items() if key != "q"}
    gemm_epi.gemm_epi_w4_matmul(3, 520, 2048, 128, "bf16", "BIAS_RESIDUAL", g["A"], g["W"], g["scales"],
                                g["zeros"], g["bias"], R, R)
    assert torch.equal(R, first) and torch.equal(_run(p, 128, "bf16", "BIAS_RESIDUAL"), first)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_w4_gelu_over_its_range(dtype):
    """k = 0: D = GELU(bias) = max(v, 0) - |v| Phi(-|v|), for every finite 16-bit value.  The tail's
    exponent, up to 13^2 / (2 ln 2) = 122, is rounded to fp32 twice: 2 * 122 * 2^-24 * ln 2 = 1.0e-5
    of the tail; fp32 roundings of the two terms; 1e-37 where the tail leaves fp32's range."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TD[dtype])
    bias = torch.where(bits.isfinite(), bits, torch.zeros_like(bits)).cuda()
    D = torch.full((2, 65536), float("nan"), dtype=TD[dtype], device="cuda")
    gemm_epi.gemm_epi_w4_matmul(2, 65536, 0, 128, dtype, "GELU_BIAS", None, None, None, None, bias, None, D)
    v = bias.double()
    # Phi(v) = erfc(-v / sqrt 2) / 2, accurate in relative terms for negative v as well
    want = v * 0.5 * torch.special.erfc(-v / 2.0 ** 0.5)
    assert torch.equal(D[0], D[1])
    tail = v.abs() * 0.5 * torch.special.erfc(v.abs() / 2.0 ** 0.5)
    error = (1.0e-5 + 4 * ref.F32) * tail + 2 * ref.F32 * v.clamp(min=0) + 1e-37
    ref.check_16(D[0].cpu(), want.cpu(), dtype, error.cpu(), "GELU")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m", [2, 12])
def test_w4_gelu_of_every_value(m, dtype):
    """k = 0: every 16-bit pattern, the far tail (below -13), infinities and NaN with it.  The tail's
    exponent, up to 15^2 / (2 ln 2) = 163, is rounded to fp32 twice: 2 * 163 * 2^-24 * ln 2 = 1.4e-5 of
    the tail; fp32 roundings of the two terms, and of the smallest numbers of fp32 (2^-149 each)."""
    bias = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(TD[dtype]).cuda()
    D = torch.full((m, 65536), 7.0, dtype=TD[dtype], device="cuda")
    gemm_epi.gemm_epi_w4_matmul(m, 65536, 0, 128, dtype, "GELU_BIAS", None, None, None, None, bias, None, D)
    v, D = bias.double().cpu(), D.cpu()
    assert torch.equal(D[:1].expand(m, -1).contiguous().view(torch.int16), D.view(torch.int16))
    D = D[0]
    assert D[v.isnan()].isnan().all() and (D[v == float("inf")] == float("inf")).all()
    assert (D[v < -15] == 0).all() and (D[v == float("-inf")] == 0).all()
    finite = v.isfinite()
    v, D = v[finite], D[finite]
    tail = v.abs() * 0.5 * torch.special.erfc(v.abs() / 2.0 ** 0.5)
    want = v.clamp(min=0) - tail
    error = (1.4e-5 + 4 * ref.F32) * tail + 2 * ref.F32 * v.clamp(min=0) + 4 * 2.0 ** -149
    ref.check_16(D, want, dtype, error, "GELU")


@pytest.mark.parametrize("m", [3, 12, 40])
def test_w4_k_zero_is_the_epilogue_alone(m):
    bias = torch.randn(64, generator=torch.Generator().manual_seed(1)).to(torch.float16)
    D = torch.full((m, 64), float("nan"), dtype=torch.float16, device="cuda")
    gemm_epi.gemm_epi_w4_matmul(m, 64, 0, 64, "f16", "RELU_BIAS", None, None, None, None, bias.cuda(), None, D)
    assert torch.equal(D.cpu(), bias.clamp(min=0).expand(m, -1))


@pytest.mark.parametrize("m", [2, 45])
def test_w4_in_a_graph_and_on_a_stream(m):
    p = ref.w4_problem(m, 264, 1024, 32, "f16", True, 6)
    want = _run(p, 32, "f16", "GELU_BIAS").cpu()
    g = {key: None if v is None else v.cuda() for key, v in p.items() if key != "q"}
    D = torch.zeros(m, 264, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()

    def call(stream=None):
        gemm_epi.gemm_epi_w4_matmul(m, 264, 1024, 32, "f16", "GELU_BIAS", g["A"], g["W"], g["scales"],
                                    g["zeros"], g["bias"], None, D, stream)
    with torch.cuda.graph(graph):
        call()
    g["A"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(D.cpu(), _run({**p, "A": -p["A"]}, 32, "f16", "GELU_BIAS").cpu())
    g["A"].mul_(-1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    side.synchronize()
    assert torch.equal(D.cpu(), want)


def test_w4_calls_on_two_streams_at_once():
    # the tcgen05 kernel takes all of an SM's tensor memory: calls that meet on the GPU, with
    # each other and with a plan's GEMM, wait their turn
    p = [ref.w4_problem(m, 1000, 2048, 64, "bf16", True, m) for m in (48, 5)]
    want = [_run(q, 64, "bf16", "BIAS").cpu() for q in p]
    gpu = [{key: v.cuda() for key, v in q.items() if v is not None and key != "q"} for q in p]
    D = [torch.zeros_like(w, device="cuda") for w in want]
    B = torch.randn(2048, 1000, device="cuda").to(torch.bfloat16)
    C, C0 = (torch.zeros(48, 1000, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    with gemm_epi.Plan(48, 1000, 2048, "bf16", "NONE") as plan:
        plan.execute(gpu[0]["A"], B, None, C0)
        streams = [torch.cuda.Stream() for _ in range(3)]
        torch.cuda.synchronize()
        for _ in range(20):
            for s, q, d in zip(streams, gpu, D):
                gemm_epi.gemm_epi_w4_matmul(q["A"].shape[0], 1000, 2048, 64, "bf16", "BIAS", q["A"], q["W"],
                                            q["scales"], q["zeros"], q["bias"], None, d, s)
            plan.execute(gpu[0]["A"], B, None, C, stream=streams[2])
        torch.cuda.synchronize()
        assert plan.sync_status() == 0
    assert all(torch.equal(d.cpu(), w) for d, w in zip(D, want)) and torch.equal(C, C0)


@pytest.mark.parametrize("n,k", [(8, 32), (40, 96), (64, 64), (72, 1056), (264, 384), (1000, 2048),
                                 (4104, 2912), (8200, 4128)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,zeros", [("bf16", True), ("f16", False)])
def test_w4_dequantize(n, k, group, dtype, zeros):
    k = -(-k // group) * group
    p = ref.w4_problem(1, n, k, group, dtype, zeros, n + k)
    B = torch.full((k + 1, n), 7.0, dtype=TD[dtype], device="cuda")
    gemm_epi.gemm_epi_w4_dequantize(n, k, group, dtype, p["W"].cuda(), p["scales"].cuda(),
                                    p["zeros"].cuda() if zeros else None, B)
    # (q - z) s is exact in fp32 (4 bits times 11 at most): one rounding, the same bits
    want = ref.w4_weight(p["q"], p["scales"], p["zeros"], group).to(TD[dtype])
    assert torch.equal(B[:k].cpu(), want) and (B[k:] == 7.0).all()


@pytest.mark.slow
def test_w4_offsets_past_32_bits():
    n, k, group, m = 65544, 65536 + 128, 128, 2       # 4.3e9 weights, B of 8.6 GB
    g = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(k // group, n, generator=g, device="cuda") / 256).to(torch.bfloat16)
    A = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
    D = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gemm_epi.gemm_epi_w4_matmul(m, n, k, group, "bf16", "NONE", A, W, scales, None, None, None, D)
    cols = torch.tensor([0, 7, 32768, n - 9, n - 1])
    w = W[cols.cuda()].cpu()
    q = torch.stack((w & 15, w >> 4), 2).view(len(cols), k)
    p = dict(q=q, scales=scales[:, cols.cuda()].cpu(), zeros=None, A=A.cpu())
    want, error = ref.w4_matmul(p, group, "NONE")
    ref.check_16(D[:, cols.cuda()], want, "bf16", error, "D")
    B = torch.empty(k, n, dtype=torch.bfloat16, device="cuda")
    gemm_epi.gemm_epi_w4_dequantize(n, k, group, "bf16", W, scales, None, B)
    want = ref.w4_weight(q, p["scales"], None, group).to(torch.bfloat16)
    assert torch.equal(B[:, cols.cuda()].cpu(), want)
