"""Timed cases of the operators of a pre-norm layer in block-scaled 8 bits, forward and backward.

Four operators, each as a user's program calls it:

  quantize       Q = E4M3(X / scale), a scale for each 1 x 128 or 128 x 128 block of X, row-major
                 and / or transposed in one pass
  product        D = epi(A . B^T + bias) for E4M3 A and B with a scale for each 128 of k and row of A,
                 and for each 128 of k and 128 rows (or one row) of B
  layernorm      H = X + R, Y = (H - mean) * rstd * gamma + beta, Y in 16 bits or block-scaled E4M3
  layernorm_bwd  its gradients: dX (shared by X and R), dgamma and dbeta

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with
``own`` true it makes the library's calls.
"""
import math

import torch

own = False

BF16, F16, E4M3 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
EPS = 1e-5
E4M3_MAX = 448.0
NOTHING = 2.0 ** -100  # a block without a value above it has scale 0 and codes 0


def _td(case):
    return BF16 if case["dtype"] == "bf16" else F16


def _up(x, to):
    return -(-x // to) * to


# ---- the cases ------------------------------------------------------------------------------

def listed():
    return [
        # the hidden activation of one new token, ahead of the second product: nothing but latency
        dict(name="quantize token", op="quantize", rows=1, cols=16384, dtype="bf16", block="1X128",
             out="rows"),
        # an odd short sequence in training: along the columns for one product, along the tokens for
        # the weight's gradient
        dict(name="quantize short both", op="quantize", rows=2039, cols=4096, dtype="f16", block="1X128",
             out="both"),
        # a large layer's weight after an update: for the forward product and for the input's gradient
        dict(name="quantize weight both", op="quantize", rows=16384, cols=8192, dtype="bf16",
             block="128X128", out="both"),
        # decoding: the second product of a feed-forward block for one token, and the first one for a
        # served batch of 48 sequences
        dict(name="product token", op="product", m=1, n=8192, k=16384, blocks=1, epilog="BIAS_RESIDUAL"),
        dict(name="product batch 48", op="product", m=48, n=16384, k=8192, blocks=1, epilog="GELU_BIAS"),
        # an odd prompt through a small layer, and a full training batch through a large one
        dict(name="product prompt", op="product", m=2039, n=4096, k=1024, blocks=1, epilog="GELU_BIAS"),
        dict(name="product training", op="product", m=16384, n=8192, k=8192, blocks=1, epilog="NONE"),
        # a weight's gradient: both operands scaled along the tokens, a few of them in the last block
        dict(name="product weight gradient", op="product", m=4096, n=8192, k=2064, blocks=2, epilog="NONE"),
        # one new token's norm between two layers, and a training batch's, quantised for the product
        dict(name="layernorm token", op="layernorm", t=1, d=4096, dtype="bf16", residual=True, out="16"),
        dict(name="layernorm batch e4m3", op="layernorm", t=16384, d=8192, dtype="bf16", residual=True,
             out="e4m3"),
        # training: a short sequence of a narrow model, and a full batch of a wide one
        dict(name="layernorm_bwd short", op="layernorm_bwd", t=333, d=1000, dtype="f16", dh=True),
        dict(name="layernorm_bwd batch", op="layernorm_bwd", t=16384, d=8192, dtype="bf16", dh=True),
    ]


MOST = 16384 * 8192          # elements of the largest listed activation or weight
MOST_PRODUCT = MOST * 8192   # and of the largest listed product


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "product", "product", "product", "layernorm", "layernorm",
                     "layernorm_bwd"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "quantize":
        cols = 16 * max(1, round(_log(rng, 64, 16384) / 16))
        return dict(op=op, rows=round(_log(rng, 1, min(32768, MOST // cols))), cols=cols, dtype=dtype,
                    block=rng.choice(["1X128", "1X128", "128X128"]), out=rng.choice(["rows", "transposed", "both"]))
    if op == "product":
        n = 8 * max(1, round(_log(rng, 256, 16384) / 8))
        k = 16 * max(1, round(_log(rng, 256, min(16384, MOST // n)) / 16))
        while n * k > MOST:
            k -= 16
        most = min(16384, MOST // n, MOST // k, MOST_PRODUCT // (n * k))
        m = round(_log(rng, 1, 64)) if rng.random() < 0.4 else round(_log(rng, 64, most))
        return dict(op=op, m=m, n=n, k=k, blocks=rng.choice([1, 1, 2]),
                    epilog=rng.choice(["NONE", "BIAS", "RELU_BIAS", "GELU_BIAS", "BIAS_RESIDUAL"]))
    d = 8 * max(1, round(_log(rng, 64, 16384) / 8))
    t = round(_log(rng, 1, min(32768, MOST // d)))
    if op == "layernorm":
        return dict(op=op, t=t, d=d, dtype=dtype, residual=rng.random() < 0.7, out=rng.choice(["16", "e4m3"]))
    return dict(op=op, t=t, d=d, dtype=dtype, dh=rng.random() < 0.7)


# ---- what a user's program holds before the call ---------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def stream(t, d):
        # a residual stream: rows of different size and mean, a few columns far above the others
        column = torch.exp(0.5 * normal(d)) * (1 + 20 * (torch.rand(d, generator=g, device="cuda") < 0.005))
        return normal(t, d).mul_(column).add_(0.3 * normal(d)).mul_(torch.exp(0.3 * normal(t, 1)))

    s = dict(case=case, plan=None, workspace=None)
    if op == "quantize":
        td, rows, cols = _td(case), case["rows"], case["cols"]
        s["X"] = stream(rows, cols).to(td)
        kb, rb, ldt = -(-cols // 128), -(-rows // 128), _up(rows, 16)
        by_block = case["block"] == "128X128"
        if case["out"] != "transposed":
            s["Q"] = torch.empty(rows, cols, dtype=E4M3, device="cuda")
            s["scale"] = torch.empty(kb, rb if by_block else rows, device="cuda")
        if case["out"] != "rows":
            s["Qt"] = torch.empty(cols, ldt, dtype=E4M3, device="cuda")
            s["scale_t"] = torch.empty(rb, kb if by_block else cols, device="cuda")
    elif op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # operands as the quantiser leaves them: A row by row, B a weight in 128 x 128 blocks, or,
        # for a gradient, row by row
        s["A"], s["scale_a"] = _quantized(stream(m, k), "1X128")
        s["B"], s["scale_b"] = _quantized(normal(n, k) * (torch.exp(0.5 * normal(n, 1)) / math.sqrt(k)),
                                          "128X128" if case["blocks"] == 1 else "1X128")
        s["bias"] = (0.1 * normal(n)).to(BF16) if case["epilog"] != "NONE" else None
        s["R"] = normal(m, n).to(BF16) if case["epilog"] == "BIAS_RESIDUAL" else None
        s["D"] = torch.empty(m, n, dtype=BF16, device="cuda")
    else:
        td, t, d = _td(case), case["t"], case["d"]
        s["gamma"] = (1 + 0.2 * normal(d)).to(td)
        if op == "layernorm":
            s["beta"] = (0.1 * normal(d)).to(td)
            s["X"] = normal(t, d).to(td)
            s["R"] = stream(t, d).to(td) if case["residual"] else None
            s["H"] = torch.empty(t, d, dtype=td, device="cuda") if case["residual"] else None
            s["Y"] = torch.empty(t, d, dtype=td if case["out"] == "16" else E4M3, device="cuda")
            s["scale"] = torch.empty(-(-d // 128), t, device="cuda") if case["out"] == "e4m3" else None
            s["stats"] = torch.empty(t, 2, device="cuda")
        else:
            s["H"] = stream(t, d).to(td)
            h = s["H"].double()
            mean = h.mean(1, keepdim=True)
            rstd = ((h - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
            s["stats"] = torch.cat((mean, rstd), 1).float()
            s["dY"] = (0.1 * normal(t, d)).to(td)
            s["dH"] = (0.1 * normal(t, d)).to(td) if case["dh"] else None
            s["dX"] = torch.empty(t, d, dtype=td, device="cuda")
            s["dgamma"] = torch.empty(d, device="cuda")
            s["dbeta"] = torch.empty(d, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s, s["case"])


def _own(s, c):
    from activation_epilogue_gb300 import gemm_epi as ge
    op = c["op"]
    if op == "quantize":
        ge.gemm_epi_e4m3_quantize(c["rows"], c["cols"], c["dtype"], c["block"], s["X"], s.get("Q"),
                                  s.get("scale"), s.get("Qt"), s.get("scale_t"))
        return _named(Q=s.get("Q"), scale=s.get("scale"), Qt=s.get("Qt"), scale_t=s.get("scale_t"))
    if op == "product":
        if s["plan"] is None:
            s["plan"] = ge.Plan(c["m"], c["n"], c["k"], "e4m3", c["epilog"], SCALE_BLOCKS=c["blocks"])
        s["plan"].execute(s["A"], s["B"], s["bias"], s["D"], residual=s["R"],
                          scales=(s["scale_a"], s["scale_b"]))
        return s["D"]
    t, d, dtype = c["t"], c["d"], c["dtype"]
    if op == "layernorm":
        if c["out"] == "16":
            ge.gemm_epi_layernorm_forward(t, d, dtype, s["X"], s["R"], s["gamma"], s["beta"], EPS, s["H"],
                                          s["Y"], s["stats"])
            return _named(H=s["H"], Y=s["Y"], stats=s["stats"])
        ge.gemm_epi_layernorm_e4m3(t, d, dtype, s["X"], s["R"], s["gamma"], s["beta"], EPS, s["H"], s["Y"],
                                   s["scale"], s["stats"])
        return _named(H=s["H"], Q=s["Y"], scale=s["scale"], stats=s["stats"])
    if s["workspace"] is None:
        s["workspace"] = torch.empty(ge.gemm_epi_layernorm_workspace(t, d), dtype=torch.uint8, device="cuda")
    ge.gemm_epi_layernorm_backward(t, d, dtype, s["dY"], s["H"], s["gamma"], s["stats"], s["dH"], s["dX"],
                                   s["dgamma"], s["dbeta"], s["workspace"])
    return _named(dX=s["dX"], dgamma=s["dgamma"], dbeta=s["dbeta"])


def _named(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _quantized(x, block):
    """Codes and scales of a matrix in 32 bits; the scales as [block along the columns][row or block of rows]."""
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // 128)
    high = 128 if block == "128X128" else 1
    x = torch.nn.functional.pad(x, (0, kb * 128 - cols, 0, _up(rows, high) - rows))
    x = x.reshape(-1, high, kb, 128)
    scale = x.abs().amax((1, 3)) / E4M3_MAX
    scale = torch.where(scale < NOTHING / E4M3_MAX, 0.0, scale)
    q = torch.where(scale[:, None, :, None] > 0, x / scale[:, None, :, None], 0.0)
    q = torch.clamp(q, -E4M3_MAX, E4M3_MAX).reshape(-1, kb * 128)[:rows, :cols].to(E4M3)
    return q.contiguous(), scale.t().contiguous()


def _spread(scale, block, rows, k):
    """A scale for every element of a rows x k operand."""
    s = scale.repeat_interleave(128, 0)[:k].t()
    return s.repeat_interleave(128, 0)[:rows] if block == "128X128" else s


def _plain(s, c):
    op = c["op"]
    if op == "quantize":
        x = s["X"].float()
        out = {}
        if c["out"] != "transposed":
            out["Q"], out["scale"] = _quantized(x, c["block"])
        if c["out"] != "rows":
            q, out["scale_t"] = _quantized(x.t(), c["block"])
            out["Qt"] = torch.zeros_like(s["Qt"])
            out["Qt"][:, :c["rows"]] = q
        return _named(Q=out.get("Q"), scale=out.get("scale"), Qt=out.get("Qt"), scale_t=out.get("scale_t"))
    if op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        a = s["A"].float() * _spread(s["scale_a"], "1X128", m, k)
        b = s["B"].float() * _spread(s["scale_b"], "128X128" if c["blocks"] == 1 else "1X128", n, k)
        d = a @ b.t()
        e = c["epilog"]
        if e != "NONE":
            d = d + s["bias"].float()
        if e == "RELU_BIAS":
            d = torch.clamp(d, min=0.0)
        elif e == "GELU_BIAS":
            d = 0.5 * d * (1.0 + torch.erf(d / math.sqrt(2.0)))
        elif e == "BIAS_RESIDUAL":
            d = d + s["R"].float()
        return d.to(BF16)
    td = _td(c)
    if op == "layernorm":
        H = None
        x = s["X"].float()
        if c["residual"]:
            H = (x + s["R"].float()).to(td)
            x = H.float()
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
        y = x * rstd * s["gamma"].float() + s["beta"].float()
        stats = torch.cat((mean, rstd), 1)
        if c["out"] == "16":
            return _named(H=H, Y=y.to(td), stats=stats)
        q, scale = _quantized(y, "1X128")
        return _named(H=H, Q=q, scale=scale, stats=stats)
    dy = s["dY"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xh = (s["H"].float() - mean) * rstd
    g = dy * s["gamma"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if c["dh"]:
        dx = dx + s["dH"].float()
    return _named(dX=dx.to(td), dgamma=(dy * xh).sum(0), dbeta=dy.sum(0))


# ---- the definition in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x = s["X"].double()
        out = {}
        if case["out"] != "transposed":
            out["Q"], out["scale"] = _exact_codes(x, case["block"] == "128X128")
        if case["out"] != "rows":
            q, out["scale_t"] = _exact_codes(x.t(), case["block"] == "128X128")
            out["Qt"] = torch.cat((q, q.new_zeros(q.shape[0], _up(case["rows"], 16) - case["rows"])), 1)
        return _named(Q=out.get("Q"), scale=out.get("scale"), Qt=out.get("Qt"), scale_t=out.get("scale_t"))
    if op == "product":
        d = torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
        for b in range(s["scale_a"].shape[0]):  # block by block of k, as the scales are given
            k = slice(128 * b, min(128 * b + 128, case["k"]))
            sb = s["scale_b"][b].double()
            if case["blocks"] == 1:
                sb = sb[torch.arange(case["n"], device="cuda") // 128]
            a = s["A"][:, k].double().mul_(s["scale_a"][b].double()[:, None])
            d.addmm_(a, s["B"][:, k].double().mul_(sb[:, None]).t())
        if s["bias"] is not None:
            d += s["bias"].double()[None, :]
        e = case["epilog"]
        if e == "GELU_BIAS":
            d = d * torch.special.ndtr(d)
        elif e == "RELU_BIAS":
            d = d * (d > 0)
        elif e == "BIAS_RESIDUAL":
            d = d + s["R"].double()
        return d
    h = s["X"].double() + (s["R"].double() if case["residual"] else 0.0) if op == "layernorm" else s["H"].double()
    if op == "layernorm":
        hq = h.to(_td(case)).double()  # the norm is of the stored (16-bit) H
        var, mean = torch.var_mean(hq, 1, correction=0, keepdim=True)
        rstd = (var + EPS).pow(-0.5)
        y = torch.addcmul(s["beta"].double(), (hq - mean).mul(rstd), s["gamma"].double())
        stats, H = torch.cat((mean, rstd), 1), h if case["residual"] else None
        if case["out"] == "16":
            return _named(H=H, Y=y, stats=stats)
        q, scale = _exact_codes(y, False)
        return _named(H=H, Q=q, scale=scale, stats=stats)
    # the gradient of sum(dY * Y) + sum(dH * H) through y = gamma (h - mean) rstd + beta, with the
    # projections onto the constant and onto h written out
    dy, gamma = s["dY"].double(), s["gamma"].double()
    mean, rstd = s["stats"][:, 0].double(), s["stats"][:, 1].double()
    c = h - mean[:, None]
    along_one = torch.einsum("td,d->t", dy, gamma) / case["d"]
    along_h = torch.einsum("td,td,d->t", dy, c, gamma) / case["d"]
    dx = torch.einsum("td,d,t->td", dy, gamma, rstd)
    dx -= (along_one * rstd)[:, None]
    dx -= c * (along_h * rstd ** 3)[:, None]
    if case["dh"]:
        dx += s["dH"].double()
    return dict(dX=dx, dgamma=torch.einsum("td,td,t->d", dy, c, rstd), dbeta=dy.sum(0))


def _exact_codes(x, square):
    """What the codes stand for before they are rounded, and the scales."""
    rows, cols = x.shape
    kb = -(-cols // 128)
    q = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    scales = []
    for b in range(kb):
        part = x[:, 128 * b:128 * b + 128]
        top = torch.linalg.vector_norm(part, float("inf"), 1)
        if square:
            top = torch.stack([t.max() for t in top.split(128)])
        scale = top / E4M3_MAX
        scales.append(scale)
        wide = scale.repeat_interleave(128)[:rows] if square else scale
        q[:, 128 * b:128 * b + 128] = part / wide.clamp(min=NOTHING / E4M3_MAX)[:, None]
    return q, torch.stack(scales)


# ---- what a pass cannot do without ------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        kb, rb = -(-cols // 128), -(-rows // 128)
        square = case["block"] == "128X128"
        move = 2 * rows * cols
        if case["out"] != "transposed":
            move += rows * cols + 4 * kb * (rb if square else rows)
        if case["out"] != "rows":
            move += cols * _up(rows, 16) + 4 * rb * (kb if square else cols)
        return dict(bytes=move, flops=2 * rows * cols)
    if op == "product":
        m, n, k, e = case["m"], case["n"], case["k"], case["epilog"]
        kb = -(-k // 128)
        scales = 4 * kb * (m + (-(-n // 128) if case["blocks"] == 1 else n))
        more = (2 * n if e != "NONE" else 0) + (2 * m * n if e == "BIAS_RESIDUAL" else 0)
        return dict(bytes=(m + n) * k + scales + 2 * m * n + more, flops=2 * m * n * k)
    t, d = case["t"], case["d"]
    e = t * d
    if op == "layernorm":
        move = 2 + (4 if case["residual"] else 0) + (2 if case["out"] == "16" else 1)
        scales = 4 * t * (-(-d // 128)) if case["out"] == "e4m3" else 0
        return dict(bytes=e * move + 4 * d + 8 * t + scales, flops=8 * e)
    return dict(bytes=e * (8 if case["dh"] else 6) + 10 * d + 8 * t, flops=13 * e)
