"""Plain 64-bit implementations of the operators around the feed-forward block (RMS norm,
products with 4-bit weights, dropout) and the bounds their fp32 kernels are held to."""
from __future__ import annotations

import math

import numpy as np
import torch

TD = {"bf16": torch.bfloat16, "f16": torch.float16}
# half a step of each 16-bit type relative to the value, and half its smallest subnormal
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FLOOR = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25}
F32 = 2.0 ** -24            # half a step of fp32
E4M3_MAX = 448.0


# ---- RMS norm -------------------------------------------------------------------------------

def sum_error(n: int) -> float:
    """Relative error of an fp32 sum of n terms of one sign: no summation tree that splits n over
    at least a warp has a longer chain than n / 32 + 32 roundings."""
    return (n / 32 + 32) * F32


def rmsnorm(h: torch.Tensor, gamma: torch.Tensor, eps: float):
    """(y, rstd) in 64 bits of the rows of h (the stored, rounded H)."""
    h = h.double()
    rstd = 1.0 / torch.sqrt((h * h).mean(1) + eps)
    return h * rstd[:, None] * gamma.double(), rstd


def check_16(got: torch.Tensor, want: torch.Tensor, dtype: str, error, what: str):
    """got is one rounding of a value within `error` (absolute, >= 0) of want."""
    got = got.double().cpu()
    bound = HALF[dtype] * (want.abs() + error) + error + FLOOR[dtype]
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / bound)[bad].max()):.3g} of the bound")


def check_e4m3(codes: torch.Tensor, value: torch.Tensor, rel: float, what: str):
    """E4M3 codes against the quotients they round, each known to a relative error `rel`."""
    q = codes.float().double().cpu()
    v = value.clamp(-E4M3_MAX, E4M3_MAX)
    # half a step: 2^-4 of the value, 2^-10 in the subnormal range
    bound = torch.maximum(2.0 ** -4 * v.abs(), torch.full_like(v, 2.0 ** -10)) * (1 + rel) + rel * v.abs()
    bad = ~((q - v).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} codes off"


def rmsnorm_backward(dy, h, gamma, rstd, dh):
    """(dx, dgamma, the magnitude that rounding errors of dx scale with, that of dgamma)."""
    dy, h, gamma = dy.double(), h.double(), gamma.double()
    r = rstd.double()[:, None]
    g, xh = dy * gamma, h * r
    dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    size = (r * g).abs() + (r * xh).abs() * (g * xh).abs().mean(1, keepdim=True)
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    return dx, (dy * xh).sum(0), size, (dy * xh).abs().sum(0)


# ---- 4-bit weights --------------------------------------------------------------------------

def w4_pack(q: torch.Tensor) -> torch.Tensor:
    """n x k values 0..15 to n x k/2 bytes, two along k per byte, the lower half first."""
    q = q.to(torch.uint8)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()


def w4_weight(q, scales, zeros, group: int) -> torch.Tensor:
    """The weight as B (k x n) in 64 bits from q (n x k), scales and zeros (k/group x n)."""
    s = scales.double().repeat_interleave(group, 0)
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, 0)
    return (q.t().double() - z) * s


def w4_problem(m, n, k, group, dtype, zeros, seed, residual=False):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(0, 16, (n, k), generator=g)
    scales = ((0.5 + torch.rand(k // group, n, generator=g)) * 0.3 / math.sqrt(max(k, 1))).to(TD[dtype])
    z = torch.randint(0, 16, (k // group, n), generator=g).to(torch.uint8) if zeros else None
    A = torch.randn(m, k, generator=g).to(TD[dtype])
    bias = torch.randn(n, generator=g).to(TD[dtype])
    R = torch.randn(m, n, generator=g).to(TD[dtype])
    return dict(q=q, W=w4_pack(q), scales=scales, zeros=z, A=A, bias=bias, R=R)


def w4_matmul(p, group, epilog):
    """(D, bound on the fp32 error of D) in 64 bits."""
    B = w4_weight(p["q"], p["scales"], p["zeros"], group)
    A = p["A"].double()
    k = A.shape[1]
    d = A @ B
    # products are exact; every partial sum is one of at most k/16 + 64 fp32 additions along a
    # chain (16 terms per matrix instruction, which may truncate: a whole step, not half)
    error = (k / 16 + 64) * 2 * F32 * (A.abs() @ B.abs())
    if epilog != "NONE":
        d = d + p["bias"].double()
        error = error + F32 * d.abs()
    if epilog == "RELU_BIAS":
        d = d.clamp(min=0.0)
    elif epilog == "GELU_BIAS":
        # the slope of GELU is below 1.13; erfc itself a few steps
        error = 1.13 * error + 8 * F32 * d.abs()
        d = 0.5 * d * torch.special.erfc(-d / math.sqrt(2.0))
    elif epilog == "TANH_BIAS":
        d = torch.tanh(d)
        error = error + 4 * F32
    elif epilog == "BIAS_RESIDUAL":
        d = d + p["R"].double()
        error = error + F32 * d.abs()
    return d, error


# ---- dropout --------------------------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """Philox4x32 (Salmon et al., 2011) on arrays of four counter words and two key words."""
    mask, x, k = np.uint64(0xFFFFFFFF), [np.asarray(c, dtype=np.uint64) for c in counter], list(key)
    for _ in range(rounds):
        a, b = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64(k[0]), b & mask,
             (a >> np.uint64(32)) ^ x[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def dropout_keep(first: int, count: int, p: float, seed: int, offset: int) -> np.ndarray:
    """keep of elements first .. first + count - 1 (first a multiple of 8)."""
    assert first % 8 == 0
    with np.errstate(over="ignore"):
        block = np.arange((count + 7) // 8, dtype=np.uint64) + np.uint64((offset + first // 8) % 2 ** 64)
    zero = np.zeros_like(block)
    words = philox4x32([block & np.uint64(0xFFFFFFFF), block >> np.uint64(32), zero, zero],
                       [seed & 0xFFFFFFFF, seed >> 32])
    bits = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1)
    return bits.reshape(-1)[:count] >= dropped(p)


def dropped(p: float) -> int:
    return round(float(np.float32(p)) * 65536)


def dropout(x, r, keep, p):
    drop = dropped(p)
    y = torch.where(torch.from_numpy(keep), x.double() * (65536 / (65536 - drop) if drop < 65536 else 0.0), 0.0)
    return y if r is None else y + r.double()
