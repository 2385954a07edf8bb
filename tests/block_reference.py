"""Plain 64-bit implementations of the block-scaled E4M3 operators and the bounds that their kernels
are held to."""
from __future__ import annotations

import math

import torch

from sublayer_reference import F32, FLOOR, HALF

E4M3_MAX = 448.0
NOTHING = 2.0 ** -100  # a block without a value above it: scale 0, codes 0
BLOCKS = {1: "128X128", 2: "1X128"}  # what SCALE_BLOCKS says of B


def up(x: int, to: int) -> int:
    return -(-x // to) * to


def spread(scale: torch.Tensor, block: str, rows: int, k: int) -> torch.Tensor:
    """The scale of every element of a rows x k operand, in 64 bits."""
    s = scale.double().repeat_interleave(128, 0)[:k].t()
    return s.repeat_interleave(128, 0)[:rows] if block == "128X128" else s


def product_problem(m, n, k, blocks, seed, device="cpu"):
    """E4M3 codes of every size, and scales over a few powers of two."""
    g = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=device)

    kb = up(k, 128) // 128
    A = (normal(m, k) * 2 ** torch.randint(-3, 7, (m, 1), generator=g, device=device)).clamp(-448, 448)
    B = (normal(n, k) * 16).clamp(-448, 448)
    sa = torch.exp(normal(kb, m)) / 32
    sb = torch.exp(normal(kb, n if blocks == 2 else up(n, 128) // 128)) / (16 * math.sqrt(k))
    return {"A": A.to(torch.float8_e4m3fn), "B": B.to(torch.float8_e4m3fn), "sa": sa, "sb": sb,
            "bias": normal(n).to(torch.bfloat16), "bias_m": normal(m).to(torch.bfloat16),
            "R": normal(m, n).to(torch.bfloat16)}


def product(p, blocks: int, epilog: str, layout: str = "1N"):
    """(D, the pre-activation, a bound of the error of D before its rounding) in 64 bits.

    The products of two E4M3 values are exact in fp32.  A block's 128 of them are summed with at most
    one step of fp32 (2^-23 of the sum of their sizes) lost an addition; the blocks' sums, their two
    scales' product and the additions are roundings to fp32 (2^-24 of the sum of the sizes each), as
    are the bias and the residual.  GELU's approximation is within 3.1e-5 max(1, |x|), its slope at
    most 1.13."""
    m, k = p["A"].shape
    n = p["B"].shape[0]
    a = p["A"].double() * spread(p["sa"], "1X128", m, k)
    b = p["B"].double() * spread(p["sb"], BLOCKS[blocks], n, k)
    pre, size = a @ b.t(), a.abs() @ b.abs().t()
    if epilog != "NONE":
        bias = p["bias"].double()[None, :] if layout == "1N" else p["bias_m"].double()[:, None]
        pre, size = pre + bias, size + bias.abs()
    error = size * (128 * 2 * F32 + (up(k, 128) // 128 + 12) * F32)
    d = pre
    if epilog in ("RELU_BIAS", "RELU_AUX_BIAS"):
        d = pre.clamp(min=0)
    elif epilog == "GELU_BIAS":
        d = 0.5 * pre * torch.special.erfc(-pre / math.sqrt(2.0))
        error = 1.13 * error + 3.1e-5 * pre.abs().clamp(min=1.0)
    elif epilog == "BIAS_RESIDUAL":
        d = pre + p["R"].double()
        error = error + F32 * (pre.abs() + p["R"].double().abs())
    return d, pre, error


def check(got, want, error, dtype="bf16", what=""):
    """got (of a 16-bit type) is one rounding of a value within `error` of want."""
    got = got.double()
    bound = HALF[dtype] * (want.abs() + error) + error + FLOOR[dtype]
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / bound)[bad].nan_to_num(1e30).max()):.3g} of the bound, "
                           f"first at {bad.nonzero()[0].tolist()}")
