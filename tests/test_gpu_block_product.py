"""E4M3 products with a scale for each block of 128 of k (plans with SCALE_BLOCKS) against the same
in 64 bits, on the CTA pairs and on the kernel for few rows of A."""
import numpy as np
import pytest
import torch

import block_reference as ref
from activation_epilogue_gb300 import gemm_epi

pytestmark = pytest.mark.gpu

EPILOGS = ["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS", "RELU_AUX_BIAS", "BIAS_RESIDUAL"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from activation_epilogue_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _run(p, blocks, epilog, layout="1N", stream=None, **opts):
    m, k = p["A"].shape
    n = p["B"].shape[0]
    D = torch.full((m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    aux = torch.full((m, (n + 31) // 32), -1, dtype=torch.int32, device="cuda") if epilog == "RELU_AUX_BIAS" else None
    bias = None if epilog == "NONE" else p["bias"] if layout == "1N" else p["bias_m"]
    with gemm_epi.Plan(m, n, k, "e4m3", epilog, layout, SCALE_BLOCKS=blocks, **opts) as plan:
        plan.execute(p["A"], p["B"], bias, D, aux=aux, residual=p["R"] if epilog == "BIAS_RESIDUAL" else None,
                     scales=(p["sa"], p["sb"]))
        assert plan.sync_status() == 0
        return D, aux, plan.describe()


def _check(p, blocks, epilog, layout="1N", **opts):
    D, aux, desc = _run(p, blocks, epilog, layout, **opts)
    want, pre, error = ref.product(p, blocks, epilog, layout)
    ref.check(D, want, error, what=desc)
    if aux is not None:
        n = D.shape[1]
        bits = np.unpackbits(aux.cpu().numpy().view(np.uint8), axis=1, bitorder="little")
        assert not bits[:, n:].any()
        wrong = torch.from_numpy(bits[:, :n].astype(bool)).cuda() != (pre > 0)
        assert not (wrong & (pre.abs() > error)).any()
    return desc


# one row to many, a column tile's edge, k below a block, at it and past it, several tiles a pair
SHAPES = [(1, 8, 16, {}), (1, 264, 128, {}), (5, 520, 272, {}), (16, 128, 1024, {}), (17, 136, 384, {}),
          (48, 1032, 2064, {}), (64, 256, 4112, {}), (100, 776, 400, {}), (128, 128, 128, {}),
          (129, 264, 1040, {}), (300, 520, 208, {"VARIANT": 3}), (600, 264, 1040, {"VARIANT": 3}),
          (1, 8, 16, {"VARIANT": 3}), (257, 1032, 528, {"VARIANT": 3, "GRID": 2}),
          (2304, 264, 128, {"VARIANT": 3, "GRID": 4, "TILE_ORDER": 2}),
          (1000, 776, 2320, {"VARIANT": 3, "GRID": 6, "TILE_ORDER": 1}),
          (300, 264, 1168, {"VARIANT": 2}), (200, 136, 1040, {"VARIANT": 2, "TILE_N": 16, "SPLIT_K": 3}),
          (33, 264, 1040, {"VARIANT": 2, "TILE_N": 32, "SPLIT_K": 8}),
          (70, 264, 4112, {"VARIANT": 2, "TILE_N": 64, "SPLIT_K": 1})]


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("m,n,k,opts", SHAPES)
def test_shapes(m, n, k, opts, blocks):
    p = ref.product_problem(m, n, k, blocks, seed=m + n + k, device="cuda")
    desc = _check(p, blocks, "BIAS", **opts)
    if "VARIANT" in opts:
        assert {2: "variant=block-swapped", 3: "variant=row-pair"}[opts["VARIANT"]] in desc


@pytest.mark.parametrize("blocks", [1, 2])
@pytest.mark.parametrize("layout", ["1N", "M1"])
@pytest.mark.parametrize("epilog", EPILOGS)
@pytest.mark.parametrize("m,n,k,opts", [(300, 520, 656, {"VARIANT": 3}), (37, 424, 1296, {})])
def test_epilogs(m, n, k, opts, epilog, layout, blocks):
    p = ref.product_problem(m, n, k, blocks, seed=len(epilog) + m, device="cuda")
    _check(p, blocks, epilog, layout, **opts)


@pytest.mark.parametrize("m,n,k,few", [  # for either kind of scales: whether the kernel for few rows of A is quicker
    (64, 4096, 512, (1, 1)), (64, 16384, 128, (1, 1)), (128, 4096, 512, (0, 0)), (512, 1024, 640, (0, 0)),
    (128, 4096, 768, (0, 1)), (128, 4096, 1024, (1, 1)), (256, 4096, 1024, (0, 1)), (256, 4096, 2048, (0, 1)),
    (256, 4096, 4096, (1, 1)), (512, 4096, 4096, (0, 1)), (768, 4096, 4096, (0, 0))])
def test_which_kernel(m, n, k, few):
    for blocks in (1, 2):
        with gemm_epi.Plan(m, n, k, "e4m3", "GELU_BIAS", SCALE_BLOCKS=blocks) as plan:
            assert ("variant=block-swapped" in plan.describe()) == bool(few[blocks - 1]), plan.describe()
