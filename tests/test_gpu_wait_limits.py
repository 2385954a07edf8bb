"""The device-side wait limit: what it counts, and what a call that ran into it leaves behind."""
import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class _Product:
    """A plan with its operands."""

    def __init__(self, m, n, k, dtype, epilog, seed=1, **options):
        blocks = options.get("SCALE_BLOCKS", 0)
        self.plan = gemm_epi.Plan(m, n, k, dtype, epilog, **options)
        self.bias = None
        if dtype == "e4m3":
            p = ref.product_problem(m, n, k, blocks or 1, seed, device="cuda")
            self.A, self.B, bias = p["A"], p["B"], p["bias"]
            self.scales = (p["sa"], p["sb"]) if blocks else (p["sa"][0, :1].clone(), p["sb"][0, :1].clone())
        else:
            g = torch.Generator(device="cuda").manual_seed(seed)
            self.A, self.B = (torch.randn(*s, generator=g, device="cuda").to(BF16) for s in ((m, k), (k, n)))
            bias, self.scales = torch.randn(n, generator=g, device="cuda").to(BF16), None
        if epilog != "NONE":
            self.bias = bias
        self.D = torch.empty(m, n, dtype=BF16, device="cuda")

    def __call__(self):
        self.plan.execute(self.A, self.B, self.bias, self.D, scales=self.scales)
        return self.D


@pytest.fixture(scope="module")
def long_product():
    """(a product on one CTA pair, which leaves room on the other SMs for what follows it, its milliseconds)"""
    long = _Product(256, 256, 2 ** 21, "e4m3", "NONE", SCALE_BLOCKS=1, VARIANT=3)
    long()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    long()
    end.record()
    assert long.plan.sync_status() == 0
    yield long, start.elapsed_time(end)
    long.plan.free()


@pytest.mark.parametrize("shape,dtype,options", [
    ((3, 264, 1040), "e4m3", dict(SCALE_BLOCKS=1, VARIANT=2)),
    ((3, 264, 1040), "e4m3", dict(SCALE_BLOCKS=2, VARIANT=2, SPLIT_K=1, B_READY=1)),
    ((300, 264, 1040), "e4m3", dict(SCALE_BLOCKS=1, VARIANT=3)),
    ((300, 264, 1040), "e4m3", dict(SCALE_BLOCKS=2, VARIANT=3, TILE_ORDER=2, GRID=2)),
    ((300, 264, 1040), "e4m3", dict()),
    ((300, 264, 1040), "e4m3", dict(TILE_ORDER=2, GRID=2)),
    ((300, 264, 1040), "bf16", dict(VARIANT=1)),
    ((300, 264, 4096), "bf16", dict(VARIANT=1, SPLIT_K=4)),
    ((30, 264, 1040), "bf16", dict(VARIANT=2, B_READY=1)),
    ((300, 264, 1040), "bf16", dict(VARIANT=3)),
    ((30, 264, 1040), "bf16", dict(VARIANT=5)),
])
def test_a_predecessor_that_outlasts_the_limit(long_product, shape, dtype, options):
    """The limit is for the kernel's own waits: a healthy predecessor on the stream may take longer than it."""
    long, ms = long_product
    limit_us = int(ms * 1000 / 4)
    assert limit_us > 500
    product = _Product(*shape, dtype, "BIAS", **options)
    want = product().clone()
    assert product.plan.sync_status() == 0
    product.plan.set_option("WAIT_LIMIT_US", limit_us)
    product.D.fill_(7)
    torch.cuda.synchronize()
    long()
    product()
    assert product.plan.sync_status() == 0
    assert torch.equal(product.D, want)
    product.plan.free()
    assert long.plan.sync_status() == 0


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("epilog", ["BIAS", "RELU_AUX_BIAS"])
@pytest.mark.parametrize("split", [1, 2, 5, 8])
def test_no_rows_of_a_cluster_that_gave_up(split, epilog, blocks):
    """K split over a cluster, one block of which gives up on a wait: nothing of its tile is stored, neither by it nor
    by the others, whose sums lack its part of k."""
    m, n, k = 40, 1032, 2064
    p = ref.product_problem(m, n, k, blocks, seed=split, device="cuda")
    D = torch.full((m, n), 7.0, dtype=BF16, device="cuda")
    aux = torch.full((m, (n + 31) // 32), -7, dtype=torch.int32, device="cuda") if epilog == "RELU_AUX_BIAS" else None
    with gemm_epi.Plan(m, n, k, "e4m3", epilog, SCALE_BLOCKS=blocks, VARIANT=2, SPLIT_K=split, WAIT_LIMIT_US=2000,
                       DEBUG_STALL=2) as plan:
        for _ in range(2):
            plan.execute(p["A"], p["B"], p["bias"], D, aux=aux, scales=(p["sa"], p["sb"]))
            assert plan.sync_status() == 8
            assert (D == 7).all() and (aux is None or (aux == -7).all())
        plan.set_option("DEBUG_STALL", 0)
        plan.set_option("WAIT_LIMIT_US", 0)
        plan.execute(p["A"], p["B"], p["bias"], D, aux=aux, scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
    want, _, error = ref.product(p, blocks, epilog)
    ref.check(D, want, error)
