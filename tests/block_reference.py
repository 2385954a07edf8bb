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


# ---- quantisation ----------------------------------------------------------------------------

def tops(x: torch.Tensor, block: str) -> torch.Tensor:
    """The largest |x| of every block: [block of columns][row, or block of rows]."""
    rows, cols = x.shape
    high = 128 if block == "128X128" else 1
    x = torch.nn.functional.pad(x.double(), (0, up(cols, 128) - cols, 0, up(rows, high) - rows))
    return x.reshape(-1, high, up(cols, 128) // 128, 128).abs().amax((1, 3)).t()


def check_codes(codes: torch.Tensor, value: torch.Tensor, error: torch.Tensor, what: str):
    """codes are E4M3 roundings of quotients within `error` (absolute) of `value`: half a step is 2^-4 of
    the value, 2^-10 in the subnormal range."""
    v = value.clamp(-E4M3_MAX, E4M3_MAX)
    bound = (2.0 ** -4 * (v.abs() + error)).clamp(min=2.0 ** -10) + error
    bad = ~((codes.float().double() - v).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"


def check_quantized(x, block, codes, scale, what=""):
    """The codes and scales of a finite x: a scale is one fp32 division of a 16-bit value (2^-24), the
    reciprocal and the product add a rounding each."""
    top = tops(x, block)
    want = torch.where(top < NOTHING, 0.0, top / E4M3_MAX)
    assert torch.all((scale.double() - want).abs() <= F32 * want), what + " scale"
    rows, cols = x.shape
    s = spread(scale, block, rows, cols)
    q = torch.where(s > 0, x.double() / s, 0.0)
    check_codes(codes, q, 3 * F32 * q.abs(), what)


# ---- LayerNorm -------------------------------------------------------------------------------

def sum_error(n: int) -> float:
    """Relative error of an fp32 sum of n terms of one sign: no summation tree that splits n over at
    least a warp has a longer chain than n / 32 + 32 roundings."""
    return (n / 32 + 32) * F32


def layernorm(h, gamma, beta, eps):
    """(y, mean, rstd, a bound of the error of y before its rounding) in 64 bits of the rows of h.

    The kernels take the deviations u from a first mean m0, which is off by at most S mean|h| (S:
    sum_error), and what their mean says m0 lacks, itself off by S of the mean of |u|.  So u - more is
    three roundings of u and S mean|u| off, the variance S of itself, rstd half of that and four
    roundings."""
    h, gamma, beta = h.double(), gamma.double(), beta.double()
    mean = h.mean(1, keepdim=True)
    dev = h - mean
    rstd = 1.0 / torch.sqrt((dev * dev).mean(1, keepdim=True) + eps)
    xh = dev * rstd
    y = xh * gamma + beta
    S = sum_error(h.shape[1])
    lacks = S * h.abs().mean(1, keepdim=True)  # how far m0 may be off
    spread_ = dev.abs().mean(1, keepdim=True) + lacks
    e_dev = 4 * F32 * (dev.abs() + lacks) + S * spread_
    e_var = 2 * S * ((dev * dev).mean(1, keepdim=True) + lacks * lacks)
    rel = e_var * rstd * rstd + 8 * F32
    error = gamma.abs() * (rstd * e_dev + xh.abs() * rel) + 3 * F32 * (y.abs() + beta.abs())
    return y, mean[:, 0], rstd[:, 0], error


def layernorm_backward(dy, h, gamma, stats, dh):
    """(dx, dgamma, dbeta, bounds of their errors) in 64 bits, for the stats that are given."""
    dy, h, gamma = dy.double(), h.double(), gamma.double()
    mean, r = stats.double()[:, :1], stats.double()[:, 1:]
    g, xh = dy * gamma, (h - mean) * r
    m1, m2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - m1 - xh * m2)
    t, d = h.shape
    S = sum_error(d) + 6 * F32
    error = r * (6 * F32 * (g.abs() + m1.abs() + (xh * m2).abs()) +
                 S * (g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True)))
    if dh is not None:
        dx = dx + dh.double()
        error = error + F32 * dx.abs()
    chain = (t + 64) * F32  # no order of summation has a longer chain of roundings
    return (dx, (dy * xh).sum(0), dy.sum(0), error, chain * (dy * xh).abs().sum(0), chain * dy.abs().sum(0))
