"""E4M3 codes with block scales (gemm_epi_e4m3_quantize) against the same in 64 bits."""
import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi
from sublayer_reference import TD

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _quantize(x, block, rows=True, transposed=True):
    r, c = x.shape
    rb, cb, ldt = ref.up(r, 128) // 128, ref.up(c, 128) // 128, ref.up(r, 16)
    square = block == "128X128"
    # (bytes and scales that no call writes, so that what it leaves out shows)
    Q = torch.full((r, c), 0x55, dtype=torch.uint8, device="cuda").view(E4M3) if rows else None
    s = torch.full((cb, rb if square else r), -1.0, device="cuda") if rows else None
    Qt = torch.full((c, ldt), 0x55, dtype=torch.uint8, device="cuda").view(E4M3) if transposed else None
    st = torch.full((rb, cb if square else c), -1.0, device="cuda") if transposed else None
    dtype = "bf16" if x.dtype == torch.bfloat16 else "f16"
    gemm_epi.gemm_epi_e4m3_quantize(r, c, dtype, block, x, Q, s, Qt, st)
    return Q, s, Qt, st


def _matrix(rows, cols, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows * cols)
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(2 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= torch.exp(torch.randn(1, cols, generator=g, device="cuda"))
    return x.clamp(-60000, 60000).to(TD[dtype])


@pytest.mark.parametrize("block", ["1X128", "128X128"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 144), (4, 128), (7, 2064), (16, 16), (17, 272), (127, 128),
                                       (128, 128), (129, 400), (255, 1040), (1000, 528), (2039, 16)])
def test_codes(rows, cols, dtype, block):
    x = _matrix(rows, cols, dtype)
    Q, s, Qt, st = _quantize(x, block)
    ref.check_quantized(x, block, Q, s, "rows")
    ref.check_quantized(x.t(), block, Qt[:, :rows], st, "transposed")
    assert not Qt[:, rows:].view(torch.uint8).any()
    if block == "128X128":
        assert torch.equal(Qt[:, :rows].view(torch.uint8), Q.view(torch.uint8).t()) and torch.equal(st, s.t())
    # each output alone has the same bits
    Q1, s1, _, _ = _quantize(x, block, transposed=False)
    _, _, Qt1, st1 = _quantize(x, block, rows=False)
    assert torch.equal(Q1.view(torch.uint8), Q.view(torch.uint8)) and torch.equal(s1, s)
    assert torch.equal(Qt1.view(torch.uint8), Qt.view(torch.uint8)) and torch.equal(st1, st)


@pytest.mark.parametrize("block", ["1X128", "128X128"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_pattern(dtype, block):
    """Each finite 16-bit pattern within the factor of 2^18 that E4M3 spans below 448, and zero blocks."""
    p = torch.arange(2 ** 16, device="cuda", dtype=torch.int32).to(torch.int16).view(TD[dtype])
    p = p[torch.isfinite(p)]
    p = p[p.abs().float().argsort()]
    x = torch.zeros(-(-p.numel() // 144) + 130, 144, dtype=TD[dtype], device="cuda")
    x.view(-1)[:p.numel()] = p
    Q, s, Qt, st = _quantize(x, block)
    ref.check_quantized(x, block, Q, s, "rows")
    ref.check_quantized(x.t(), block, Qt[:, :x.shape[0]], st, "transposed")
    assert s.min() == 0 and st.min() == 0 and torch.isfinite(s).all()


@pytest.mark.parametrize("block", ["1X128", "128X128"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nan_and_infinity(dtype, block):
    x = _matrix(300, 272, dtype)
    x[5, 7], x[200, 130] = float("nan"), float("-inf")
    clean = x.nan_to_num(0.0, 0.0, 0.0)
    Q, s, Qt, st = _quantize(x, block)
    Qc, sc, Qtc, stc = _quantize(clean, block)
    for q, scale, qc, scale_c, y in ((Q, s, Qc, sc, x), (Qt[:, :300], st, Qtc[:, :300], stc, x.t())):
        wide, wide_c = (ref.spread(v, block, *y.shape) for v in (scale, scale_c))
        assert torch.equal(wide.isnan().any(1).nonzero(), (y.isnan().any(1) if block == "1X128" else wide.isnan().any(1)).nonzero())
        at = tuple(y.isnan().nonzero()[0].tolist())
        assert wide[at].isnan() and q.float()[wide.isnan()].isnan().all()
        at = tuple(y.isinf().nonzero()[0].tolist())
        assert wide[at].isinf() and q.float()[at].isnan()
        rest = wide.isinf() & ~y.isinf()
        assert (q.float()[rest] == 0).all()
        fine = torch.isfinite(wide)  # blocks that hold neither keep theirs
        assert torch.equal(wide[fine], wide_c[fine])
        assert torch.equal(q.view(torch.uint8)[fine], qc.view(torch.uint8)[fine])
    assert not Qt[:, 300:].view(torch.uint8).any()  # also where the scale is NaN


@pytest.mark.parametrize("block", ["1X128", "128X128"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(300, 272), (128, 384), (1, 144), (257, 16)])
def test_which_blocks_a_nan_marks(rows, cols, dtype, block):
    """The blocks that hold a NaN, and no others, have a NaN scale; those that hold an infinity and no NaN an infinite
    one (corners of blocks and of the matrix among the places)."""
    x = _matrix(rows, cols, dtype)
    at = {(0, 0), (0, cols - 1), (rows - 1, 0), (rows - 1, cols - 1), (min(127, rows - 1), min(128, cols - 1)),
          (min(128, rows - 1), min(127, cols - 1)), (rows // 2, cols // 2)}
    for i, (r, c) in enumerate(sorted(at)):
        x[r, c] = float(("nan", "inf", "-inf")[i % 3])
    Q, s, Qt, st = _quantize(x, block)
    for scale, y in ((s, x), (st, x.t())):
        r, c = y.shape
        high = 128 if block == "128X128" else 1

        def blocks_with(mark):  # every element's block, by plain indexing
            out = torch.zeros(r, c, dtype=torch.bool, device="cuda")
            for i, j in mark.nonzero().tolist():
                i0, j0 = i // high * high, j // 128 * 128
                out[i0:i0 + high, j0:j0 + 128] = True
            return out

        nan, inf = blocks_with(y.isnan()), blocks_with(y.isinf())
        wide = ref.spread(scale, block, r, c)
        assert torch.equal(wide.isnan(), nan)
        assert torch.equal(wide.isinf(), inf & ~nan)


def test_rows_past_32_bits():
    """A matrix of more than 2^31 values: its last rows."""
    rows, cols = 2 ** 31 // 16384 + 130, 16384
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-200:] = _matrix(200, cols, "bf16")
    Q, s, Qt, st = _quantize(x, "1X128")
    tail, at = x[-200:], rows - 200
    ref.check_quantized(tail, "1X128", Q[at:], s[:, at:].contiguous(), "rows")
    first = at // 128 * 128
    ref.check_quantized(x[first:].t()[-256:], "1X128", Qt[-256:, first:rows], st[first // 128:, -256:].contiguous(), "transposed")


def test_on_another_stream_and_in_a_graph():
    x = _matrix(333, 528, "bf16")
    Q, s, Qt, st = _quantize(x, "1X128")
    out = [torch.empty_like(v) for v in (Q, s, Qt, st)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        gemm_epi.gemm_epi_e4m3_quantize(333, 528, "bf16", "1X128", x, *out)
    x.copy_(_matrix(333, 528, "bf16", seed=1))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for got, want in zip(out, _quantize(x, "1X128")):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))
