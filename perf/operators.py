"""Timed cases of the operators around the fused GEMMs of a transformer's feed-forward block.

Five operators, each as a user's program calls it:

  rmsnorm      H = X + R, Y = H * rstd * gamma per row, Y in 16 bits or in E4M3 with scales
  rmsnorm_bwd  its gradients: dX (shared by X and R) and dgamma
  w4           D = epi(A . W + bias) for a few rows of A, W in 4 bits with group scales
  w4_dequant   the same W written out as the 16-bit B of a GEMM plan (prompts)
  dropout      Y = R + keep * X / (1 - p), keep from a counter-based generator

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.
"""
import math

import numpy as np
import torch

own = False

BF16, F16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
EPS = 1e-6
E4M3_MAX = 448.0


def _td(case):
    return BF16 if case["dtype"] == "bf16" else F16


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # one new token's norm between two layers: nothing but latency
        dict(name="rmsnorm token", op="rmsnorm", t=1, d=4096, dtype="bf16", residual=True, out="16"),
        # an odd prompt, quantised for an 8-bit GEMM with a scale for each token
        dict(name="rmsnorm prompt e4m3 rows", op="rmsnorm", t=2039, d=4096, dtype="f16", residual=True,
             out="rows"),
        # a large batch, quantised with one scale for the whole tensor (the E4M3 plans' scale_a)
        dict(name="rmsnorm batch e4m3 tensor", op="rmsnorm", t=16384, d=8192, dtype="bf16",
             residual=True, out="tensor"),
        # training: a short sequence of a narrow model, and a full batch of a wide one
        dict(name="rmsnorm_bwd short", op="rmsnorm_bwd", t=333, d=1000, dtype="f16", dh=True),
        dict(name="rmsnorm_bwd batch", op="rmsnorm_bwd", t=16384, d=8192, dtype="bf16", dh=True),
        # decoding: the first and second product of a feed-forward block for one token, and a
        # served batch of 48 sequences
        dict(name="w4 token 1024x4096", op="w4", m=1, n=4096, k=1024, group=128, dtype="bf16",
             epilog="GELU_BIAS", zeros=False),
        dict(name="w4 token 16384x8192", op="w4", m=1, n=8192, k=16384, group=128, dtype="f16",
             epilog="BIAS_RESIDUAL", zeros=True),
        dict(name="w4 batch 48", op="w4", m=48, n=16384, k=8192, group=64, dtype="bf16",
             epilog="GELU_BIAS", zeros=False),
        # a prompt's weights written out for the 16-bit plans: a small and a large layer
        dict(name="w4_dequant 1024x4096", op="w4_dequant", n=4096, k=1024, group=32, dtype="f16",
             zeros=True),
        dict(name="w4_dequant 8192x16384", op="w4_dequant", n=16384, k=8192, group=128, dtype="bf16",
             zeros=False),
        # training: residual + dropout of a short sequence forward, and a full batch's backward
        dict(name="dropout short forward", op="dropout", count=333 * 1000, dtype="f16", residual=True,
             p=0.1),
        dict(name="dropout batch backward", op="dropout", count=16384 * 8192, dtype="bf16",
             residual=False, p=0.1),
    ]


MOST = 16384 * 8192  # elements of the largest listed activation or weight


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(["rmsnorm", "rmsnorm", "rmsnorm_bwd", "w4", "w4", "w4_dequant", "dropout"])
    dtype = rng.choice(["bf16", "f16"])
    if op in ("rmsnorm", "rmsnorm_bwd"):
        d = 8 * max(1, round(_log(rng, 64, 16384) / 8))
        t = max(1, round(_log(rng, 1, min(32768, MOST // d))))
        if op == "rmsnorm":
            return dict(op=op, t=t, d=d, dtype=dtype, residual=rng.random() < 0.7,
                        out=rng.choice(["16", "rows", "tensor", "given"]))
        return dict(op=op, t=t, d=d, dtype=dtype, dh=rng.random() < 0.7)
    if op in ("w4", "w4_dequant"):
        group = rng.choice([32, 64, 128])
        n = 8 * max(1, round(_log(rng, 256, 16384) / 8))
        k = group * max(1, round(_log(rng, 256, min(16384, MOST // n)) / group))
        while n * k > MOST:
            k -= group
        zeros = rng.random() < 0.5
        if op == "w4_dequant":
            return dict(op=op, n=n, k=k, group=group, dtype=dtype, zeros=zeros)
        return dict(op=op, m=round(_log(rng, 1, 48)), n=n, k=k, group=group, dtype=dtype,
                    epilog=rng.choice(["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS", "TANH_BIAS",
                                       "BIAS_RESIDUAL"]), zeros=zeros)
    return dict(op=op, count=round(_log(rng, 1000, MOST)), dtype=dtype, residual=rng.random() < 0.5,
                p=round(rng.uniform(0.02, 0.5), 3))


# ---- what a user's program holds before the call ---------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    td, op = _td(case), case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case=case, workspace=None)
    if op in ("rmsnorm", "rmsnorm_bwd"):
        t, d = case["t"], case["d"]
        # a residual stream: rows of different size, a few columns far above the others
        column = torch.exp(0.5 * normal(d)) * (1 + 20 * (torch.rand(d, generator=g, device="cuda") < 0.005))
        row = torch.exp(0.3 * normal(t, 1))
        s["gamma"] = (1 + 0.2 * normal(d)).to(td)
        if op == "rmsnorm":
            s["X"] = normal(t, d).to(td)
            s["R"] = (normal(t, d) * column * row).to(td) if case["residual"] else None
            s["H"] = torch.empty(t, d, dtype=td, device="cuda") if case["residual"] else None
            s["Y"] = torch.empty(t, d, dtype=td if case["out"] == "16" else E4M3, device="cuda")
            s["rstd"] = torch.empty(t, dtype=torch.float32, device="cuda")
            s["scale"] = (None if case["out"] == "16" else
                          torch.full((t if case["out"] == "rows" else 1,), 0.04, device="cuda"))
        else:
            s["H"] = (normal(t, d) * column * row).to(td)
            s["rstd"] = torch.rsqrt(s["H"].float().square().mean(1) + EPS)
            s["dY"] = (0.1 * normal(t, d)).to(td)
            s["dH"] = (0.1 * normal(t, d)).to(td) if case["dh"] else None
            s["dX"] = torch.empty(t, d, dtype=td, device="cuda")
            s["dgamma"] = torch.empty(d, dtype=torch.float32, device="cuda")
    elif op in ("w4", "w4_dequant"):
        n, k, group = case["n"], case["k"], case["group"]
        # a weight rounded to 4 bits in groups along k: values q - zero (8 where there are none)
        w = (normal(n, k // group, group) / math.sqrt(k))
        if case["zeros"]:
            lo, hi = w.amin(2), w.amax(2)
            scale = ((hi - lo) / 15).to(td)
            zero = torch.clamp(torch.round(-lo / scale.float()), 0, 15)
        else:
            scale = (w.abs().amax(2) / 7).to(td)
            zero = torch.full_like(scale, 8.0)
        q = torch.clamp(torch.round(w / scale.float()[:, :, None]) + zero.float()[:, :, None], 0, 15)
        q = q.to(torch.uint8).view(n, k // 2, 2)
        s["W"] = (q[:, :, 0] | (q[:, :, 1] << 4)).contiguous()              # n x k/2 bytes
        s["scales"] = scale.t().contiguous()                                # k/group x n
        s["zeros"] = zero.to(torch.uint8).t().contiguous() if case["zeros"] else None
        if op == "w4":
            m = case["m"]
            s["A"] = normal(m, k).to(td)
            s["bias"] = (0.1 * normal(n)).to(td) if case["epilog"] != "NONE" else None
            s["R"] = normal(m, n).to(td) if case["epilog"] == "BIAS_RESIDUAL" else None
            s["D"] = torch.empty(m, n, dtype=td, device="cuda")
        else:
            s["B"] = torch.empty(k, n, dtype=td, device="cuda")
    else:
        count = case["count"]
        s["X"] = normal(count).to(td)
        s["R"] = normal(count).to(td) if case["residual"] else None
        s["Y"] = torch.empty(count, dtype=td, device="cuda")
        # the generator's key and the counter this call starts at, as a training loop keeps them
        s["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) % 2 ** 63
        s["offset"] = (seed * 1000003 + 77) % 2 ** 40
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s, s["case"])


def _own(s, c):
    from activation_epilogue_gb300 import gemm_epi as ge
    op, dtype = c["op"], c["dtype"]
    if op == "rmsnorm":
        t, d = c["t"], c["d"]
        if c["out"] == "16":
            ge.gemm_epi_rmsnorm(t, d, dtype, s["X"], s["R"], s["gamma"], EPS, s["H"], s["Y"], s["rstd"])
            return _named(H=s["H"], Y=s["Y"], rstd=s["rstd"])
        mode = {"rows": "ROW", "tensor": "TENSOR", "given": "GIVEN"}[c["out"]]
        if mode == "TENSOR" and s["workspace"] is None:
            s["workspace"] = torch.empty(ge.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8,
                                         device="cuda")
        ge.gemm_epi_rmsnorm_e4m3(t, d, dtype, s["X"], s["R"], s["gamma"], EPS, s["H"], s["Y"], mode,
                                 s["scale"], s["rstd"], s["workspace"])
        return _named(H=s["H"], Q=s["Y"], rstd=s["rstd"], scale=None if mode == "GIVEN" else s["scale"])
    if op == "rmsnorm_bwd":
        t, d = c["t"], c["d"]
        if s["workspace"] is None:
            s["workspace"] = torch.empty(ge.gemm_epi_rmsnorm_workspace(t, d), dtype=torch.uint8,
                                         device="cuda")
        ge.gemm_epi_rmsnorm_backward(t, d, dtype, s["dY"], s["H"], s["gamma"], s["rstd"], s["dH"],
                                     s["dX"], s["dgamma"], s["workspace"])
        return _named(dX=s["dX"], dgamma=s["dgamma"])
    if op == "w4":
        ge.gemm_epi_w4_matmul(c["m"], c["n"], c["k"], c["group"], dtype, c["epilog"], s["A"], s["W"],
                              s["scales"], s["zeros"], s["bias"], s["R"], s["D"])
        return s["D"]
    if op == "w4_dequant":
        ge.gemm_epi_w4_dequantize(c["n"], c["k"], c["group"], dtype, s["W"], s["scales"], s["zeros"],
                                  s["B"])
        return s["B"]
    ge.gemm_epi_dropout(c["count"], dtype, s["X"], s["R"], c["p"], s["seed"], s["offset"], s["Y"])
    return s["Y"]


def _named(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _plain(s, c):
    td, op = _td(c), c["op"]
    if op == "rmsnorm":
        H = None
        x = s["X"].float()
        if c["residual"]:
            H = (x + s["R"].float()).to(td)
            x = H.float()
        rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        y = x * rstd * s["gamma"].float()
        if c["out"] == "16":
            return _named(H=H, Y=y.to(td), rstd=rstd.view(-1))
        scale = {"rows": lambda: y.abs().amax(1) / E4M3_MAX,
                 "tensor": lambda: y.abs().amax().view(1) / E4M3_MAX,
                 "given": lambda: s["scale"]}[c["out"]]()
        q = torch.clamp(y / scale.view(-1, 1), -E4M3_MAX, E4M3_MAX).to(E4M3)
        return _named(H=H, Q=q, rstd=rstd.view(-1), scale=None if c["out"] == "given" else scale)
    if op == "rmsnorm_bwd":
        h, dy, r = s["H"].float(), s["dY"].float(), s["rstd"].view(-1, 1)
        xh = h * r
        dyg = dy * s["gamma"].float()
        dx = r * (dyg - xh * (dyg * xh).mean(1, keepdim=True))
        if c["dh"]:
            dx = dx + s["dH"].float()
        return _named(dX=dx.to(td), dgamma=(dy * xh).sum(0))
    if op in ("w4", "w4_dequant"):
        w = _weight(s, c)
        if op == "w4_dequant":
            return w.to(td).t().contiguous()
        d = s["A"].float() @ w.t()
        e = c["epilog"]
        if e != "NONE":
            d = d + s["bias"].float()
        if e == "RELU_BIAS":
            d = torch.clamp(d, min=0.0)
        elif e == "GELU_BIAS":
            d = 0.5 * d * (1.0 + torch.erf(d / math.sqrt(2.0)))
        elif e == "TANH_BIAS":
            d = torch.tanh(d)
        elif e == "BIAS_RESIDUAL":
            d = d + s["R"].float()
        return d.to(td)
    keep = _random16(c["count"], s["seed"], s["offset"]) >= round(c["p"] * 65536)
    y = torch.where(keep, s["X"].float() * (65536.0 / (65536 - round(c["p"] * 65536))), 0.0)
    if c["residual"]:
        y = y + s["R"].float()
    return y.to(td)


def _weight(s, c):
    """The weight in 32 bits, n x k: (q - zero) * scale."""
    n, k, group = c["n"], c["k"], c["group"]
    q = torch.stack((s["W"] & 15, s["W"] >> 4), 2).view(n, k // group, group).float()
    zero = s["zeros"].t().float()[:, :, None] if c["zeros"] else 8.0
    return ((q - zero) * s["scales"].t().float()[:, :, None]).view(n, k)


def _mulhilo(a, m):
    """High and low 32 bits of a * m for 32-bit values held in int64 (a a tensor)."""
    lo = a * (m & 0xFFFF)                      # below 2^48
    hi = a * (m >> 16)                         # below 2^48
    mid = (lo >> 16) + (hi & 0xFFFFFFFF)       # bits 16 .. of the product, without hi's top
    return ((mid >> 16) + ((hi >> 32) << 16)) & 0xFFFFFFFF, ((mid << 16) | (lo & 0xFFFF)) & 0xFFFFFFFF


def _random16(count, seed, offset):
    """16 random bits for each element: Philox4x32-10 (Salmon et al., "Parallel random numbers: as
    easy as 1, 2, 3", 2011) with key `seed` and counter offset + element / 8; element e takes half
    e % 2 of word (e % 8) / 2."""
    b = torch.arange((count + 7) // 8, device="cuda", dtype=torch.int64) + offset
    x0, x1, x2, x3 = b & 0xFFFFFFFF, (b >> 32) & 0xFFFFFFFF, torch.zeros_like(b), torch.zeros_like(b)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(x0, 0xD2511F53)
        h1, l1 = _mulhilo(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    words = torch.stack((x0, x1, x2, x3), 1)
    return torch.stack((words & 0xFFFF, words >> 16), 2).view(-1)[:count]


# ---- the definition in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rmsnorm":
        return _exact_rmsnorm(s, case)
    if op == "rmsnorm_bwd":
        # the gradient of sum(dY * Y) + sum(dH * H) by the product rule on Y = gamma h / rms
        h, dy, gamma = s["H"].double(), s["dY"].double(), s["gamma"].double()
        rstd = s["rstd"].double()
        dot = torch.einsum("td,td,d->t", dy, h, gamma)
        dx = torch.einsum("td,d,t->td", dy, gamma, rstd)
        dx -= h * (dot * rstd ** 3 / case["d"])[:, None]
        if case["dh"]:
            dx += s["dH"].double()
        return dict(dX=dx, dgamma=torch.einsum("td,td,t->d", dy, h, rstd))
    if op in ("w4", "w4_dequant"):
        n, k, group = case["n"], case["k"], case["group"]
        w = torch.empty(n, k, dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["W"] % 16).double()
        w[:, 1::2] = (s["W"] // 16).double()
        w -= s["zeros"].repeat_interleave(group, 0).t().double() if case["zeros"] else 8.0
        w *= s["scales"].repeat_interleave(group, 0).t().double()
        if op == "w4_dequant":
            return w.t().contiguous()
        d = torch.mm(w, s["A"].double().t()).t()
        if s["bias"] is not None:
            d = d + s["bias"].double()[None, :]
        e = case["epilog"]
        if e == "GELU_BIAS":
            d = d * torch.special.ndtr(d)
        elif e == "RELU_BIAS":
            d = d * (d > 0)
        elif e == "TANH_BIAS":
            d = 1.0 - 2.0 / (torch.exp(2.0 * d) + 1.0)
        elif e == "BIAS_RESIDUAL":
            d = d + s["R"].double()
        return d.contiguous()
    return _exact_dropout(s, case)


def _exact_rmsnorm(s, case):
    td = _td(case)
    h = s["X"].double()
    if case["residual"]:
        h = h + s["R"].double()
    hq = h.to(td).double()  # the norm is of the stored (16-bit) H
    rstd = (hq.pow(2).sum(1) / case["d"] + EPS).pow(-0.5)
    y = hq.mul(rstd[:, None]).mul(s["gamma"].double())
    H = h if case["residual"] else None
    if case["out"] == "16":
        return _named(H=H, Y=y, rstd=rstd)
    if case["out"] == "given":
        scale = s["scale"].double()
    else:
        top = torch.linalg.vector_norm(y, float("inf"), 1)
        scale = top / E4M3_MAX if case["out"] == "rows" else top.max().reshape(1) / E4M3_MAX
    q = (y / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return _named(H=H, Q=q, rstd=rstd, scale=None if case["out"] == "given" else scale)


def _exact_dropout(s, case):
    u32, u64 = np.uint64(0xFFFFFFFF), np.uint64
    count = case["count"]
    block = np.arange((count + 7) // 8, dtype=np.uint64) + u64(s["offset"])
    ctr = [block & u32, block >> u64(32), np.zeros_like(block), np.zeros_like(block)]
    key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
    for _ in range(10):
        a, b = ctr[0] * u64(0xD2511F53), ctr[2] * u64(0xCD9E8D57)
        ctr = [(b >> u64(32)) ^ ctr[1] ^ u64(key[0]), b & u32, (a >> u64(32)) ^ ctr[3] ^ u64(key[1]), a & u32]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    bits = np.empty((block.size, 8), dtype=np.uint16)
    for w in range(4):
        bits[:, 2 * w] = ctr[w] & u64(0xFFFF)
        bits[:, 2 * w + 1] = ctr[w] >> u64(16)
    drop = round(case["p"] * 65536)
    keep = torch.from_numpy(bits.reshape(-1)[:count] >= drop).cuda()
    y = s["X"].double() * 65536 / (65536 - drop) * keep
    return y + s["R"].double() if case["residual"] else y


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rmsnorm":
        e = case["t"] * case["d"]
        out = 2 if case["out"] == "16" else 1
        move = 2 + (4 if case["residual"] else 0) + out
        scales = {"16": 0, "rows": 4 * case["t"], "tensor": 4, "given": 4}[case["out"]]
        return dict(bytes=e * move + 2 * case["d"] + 4 * case["t"] + scales, flops=5 * e)
    if op == "rmsnorm_bwd":
        e = case["t"] * case["d"]
        return dict(bytes=e * (8 if case["dh"] else 6) + 6 * case["d"] + 4 * case["t"], flops=9 * e)
    if op in ("w4", "w4_dequant"):
        n, k, groups = case["n"], case["k"], case["k"] // case["group"]
        weight = n * k // 2 + n * groups * (3 if case["zeros"] else 2)
        if op == "w4_dequant":
            return dict(bytes=weight + 2 * n * k, flops=2 * n * k)
        m, e = case["m"], case["epilog"]
        more = (2 * n if e != "NONE" else 0) + (2 * m * n if e == "BIAS_RESIDUAL" else 0)
        return dict(bytes=weight + 2 * m * (n + k) + more, flops=2 * m * n * k)
    return dict(bytes=case["count"] * (6 if case["residual"] else 4), flops=2 * case["count"])
