"""Cases of the normalisation, 8-bit linear and grouped linear operators.

`own = False` computes an operator in plain torch (32 bits, 64 next to a rounding border);
`own = True` makes the calls of the package's public entry points on the same state.

Kinds of case:
  norm     RMS norm of the residual stream: forward (bf16 or 8-bit output) or forward + backward
  fp8      linear with an 8-bit weight (one scale per 128 x 128) and 8-bit rows (one per 1 x 128)
  grouped  linears of a mixture of experts on rows sorted by expert, bf16 or 8 bit
"""
import math
import random

import torch

own = False

EPS = 1e-6
F8 = torch.float8_e4m3fn
FLOOR = 2.0 ** -100      # the block quantizer's smallest maximum


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decoded token through a 4096-wide block's norm: latency counts
        dict(name="norm token", kind="norm", mode="fp8", rows=1, hidden=4096, residual=True),
        # a long prompt's norm whose output feeds 8-bit linears
        dict(name="norm prompt fp8", kind="norm", mode="fp8", rows=8192, hidden=4096, residual=True),
        # a training step's norm, forward and backward, with an odd row count
        dict(name="norm step", kind="norm", mode="step", rows=4099, hidden=5120, residual=True),
        # one token through a square 8-bit linear, its row quantized in the call
        dict(name="fp8 token", kind="fp8", mode="fwd", rows=1, out=4096, inp=4096, rows_in_8bit=False),
        # a serving batch of odd size through an up projection
        dict(name="fp8 batch", kind="fp8", mode="fwd", rows=77, out=11008, inp=4096, rows_in_8bit=True),
        # a prompt through an up projection, rows already in 8 bit from the norm
        dict(name="fp8 prompt", kind="fp8", mode="fwd", rows=8192, out=11008, inp=4096, rows_in_8bit=True),
        # the gradient of the rows through a frozen 8-bit weight, a ragged token count
        dict(name="fp8 dx", kind="fp8", mode="bwd", rows=4100, out=5120, inp=5120, rows_in_8bit=False),
        # a decode step of a mixture of experts: few rows for each of many experts
        dict(name="experts fp8 decode", kind="grouped", mode="fwd", dtype="fp8", rows=128, experts=32, out=2048, inp=4096),
        # a prompt through the experts' up projections in 8 bit
        dict(name="experts fp8 prompt", kind="grouped", mode="fwd", dtype="fp8", rows=16384, experts=8, out=11008, inp=4096),
        # odd and small: a step over few rows, sizes that are no multiple of a tile
        dict(name="experts bf16 odd step", kind="grouped", mode="step", dtype="bf16", rows=333, experts=5, out=528, inp=272),
        # a training step of bf16 experts: output, gradients of rows and weights
        dict(name="experts bf16 step", kind="grouped", mode="step", dtype="bf16", rows=8209, experts=16, out=1408, inp=2048),
        # many narrow experts in bf16, forward
        dict(name="experts bf16 prompt", kind="grouped", mode="fwd", dtype="bf16", rows=16384, experts=64, out=1024, inp=2048),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(("norm", "fp8", "grouped"))
    if kind == "norm":
        return dict(kind=kind, mode=rng.choice(("bf16", "fp8", "step")), rows=_log(rng, 1, 8192), hidden=_log(rng, 256, 8192, 16),
                    residual=rng.random() < 0.7)
    if kind == "fp8":
        return dict(kind=kind, mode=rng.choice(("fwd", "fwd", "bwd")), rows=_log(rng, 1, 8192), out=_log(rng, 256, 11008, 16),
                    inp=_log(rng, 256, 5120, 16), rows_in_8bit=rng.random() < 0.5)
    dtype = rng.choice(("bf16", "fp8"))
    return dict(kind=kind, mode=rng.choice(("fwd", "step")) if dtype == "bf16" else rng.choice(("fwd", "bwd")), dtype=dtype,
                rows=_log(rng, 1, 16384), experts=_log(rng, 2, 64), out=_log(rng, 256, 2048, 16), inp=_log(rng, 256, 4096, 16))


# ------------------------------------------------------------------ inputs

def _sizes(case):
    """Rows of each expert: skewed, with every seventh expert empty; the same for every seed up to their order."""
    E, M = case["experts"], case["rows"]
    r = random.Random(E * 1000003 + M)
    w = [0.0 if e % 7 == 6 else math.exp(0.5 * r.gauss(0, 1)) for e in range(E)]
    n = [0] * E
    for e in r.choices(range(E), weights=w, k=M):
        n[e] += 1
    return n


def _randn(g, shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _hidden(g, rows, cols):
    """Activations: normal, with a few channels that are 20 times larger."""
    ch = torch.ones(cols, device="cuda")
    ch[torch.randperm(cols, generator=g, device="cuda")[: max(1, cols // 256)]] = 20.0
    return torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32).mul_(ch).to(torch.bfloat16)


def _rows_to_blocks(x, nb):
    pad = nb * 128 - x.shape[-1]
    return torch.nn.functional.pad(x, (0, pad)).view(*x.shape[:-1], nb, 128)


def _quantize_rows(x):
    """(codes, scales) of the rows of x in 32 bits: a scale for each 128 values, the quotient in 64 bits."""
    cols, nb = x.shape[-1], (x.shape[-1] + 127) // 128
    b = _rows_to_blocks(x.float(), nb)
    a = b.abs().amax(-1, keepdim=True).clamp_min(FLOOR)
    q = (b.double() * 448 / a.double()).float().clamp_(-448, 448).to(F8)
    return q.flatten(-2)[..., :cols].contiguous(), torch.div(a, torch.full_like(a, 448)).squeeze(-1)


def _quantize_weight(W):
    """(codes, scales) of a weight [..., out, in] with a scale for each 128 x 128 block."""
    o, i = W.shape[-2:]
    no, ni = (o + 127) // 128, (i + 127) // 128
    b = torch.nn.functional.pad(W.float(), (0, ni * 128 - i, 0, no * 128 - o))
    b = b.view(*W.shape[:-2], no, 128, ni, 128)
    a = b.abs().amax((-3, -1), keepdim=True).clamp_min(FLOOR)
    q = (b * (448 / a)).clamp_(-448, 448).to(F8).view(*W.shape[:-2], no * 128, ni * 128)
    return q[..., :o, :i].contiguous(), torch.div(a, torch.full_like(a, 448)).squeeze(-1).squeeze(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["kind"] == "norm":
        M, H = case["rows"], case["hidden"]
        s["x"] = _hidden(g, M, H)
        s["r"] = _hidden(g, M, H) if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        if case["mode"] == "step":
            s["dy"] = _randn(g, (M, H))
            s["dh"] = _randn(g, (M, H))
        return s
    M, o, i = case["rows"], case["out"], case["inp"]
    shape = (o, i) if case["kind"] == "fp8" else (case["experts"], o, i)
    W = _randn(g, shape, 0.02)
    eight = case["kind"] == "fp8" or case["dtype"] == "fp8"
    if eight:
        s["q"], s["scale"] = _quantize_weight(W)
    else:
        s["W"] = W
    fwd, step = case["mode"] in ("fwd", "step"), case["mode"] == "step"
    if fwd:
        s["x"] = _hidden(g, M, i)
    if not fwd or step:
        s["dy"] = _randn(g, (M, o))
    if case["kind"] == "fp8":
        if case["rows_in_8bit"]:
            s["rows8"] = _quantize_rows(s.pop("x" if fwd else "dy"))
        return s
    n = _sizes(case)
    k = seed % len(n)
    n = n[k:] + n[:k]
    at = [sum(n[:e]) for e in range(len(n) + 1)]
    s["offsets"] = torch.tensor(at, dtype=torch.int32, device="cuda")
    s["cap"] = max(n)
    e = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    s["slot"] = (e * s["cap"] + torch.arange(M) - torch.tensor(at)[e]).cuda()
    return s


# ------------------------------------------------------------------ plain forms

def _dequantize_rows(q, scale):
    return (_rows_to_blocks(q.float(), scale.shape[-1]) * scale[..., None]).flatten(-2)[..., : q.shape[-1]]


def _dequantize_weight(q, scale):
    o, i = q.shape[-2:]
    up = scale.repeat_interleave(128, -2).repeat_interleave(128, -1)
    return q.float() * up[..., :o, :i]


def _plain_norm(s):
    x, w = s["x"], s["w"].float()
    h = x if s["r"] is None else (x.float() + s["r"].float()).to(x.dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS)
    y = hf * rstd * w
    if s["mode"] == "fp8":
        q, scale = _quantize_rows(y)
        return {"q": q, "scale": scale, "h": h, "rstd": rstd[:, 0]}
    out = {"y": y.to(x.dtype), "h": h, "rstd": rstd[:, 0]}
    if s["mode"] == "step":
        dy = s["dy"].float()
        xhat = hf * rstd
        gr = dy * w
        dx = s["dh"].float() + rstd * (gr - xhat * (gr * xhat).mean(-1, keepdim=True))
        out["dx"] = dx.to(x.dtype)
        out["dw"] = (dy * xhat).sum(0, dtype=torch.float64).float()
    return out


def _plain_fp8(s):
    W = _dequantize_weight(s["q"], s["scale"])
    fwd = s["mode"] == "fwd"
    q, scale = s["rows8"] if s["rows_in_8bit"] else _quantize_rows(s["x" if fwd else "dy"])
    return (_dequantize_rows(q, scale) @ (W.t() if fwd else W)).to(torch.bfloat16)


def _pad(s, x):
    """The experts' rows as one batch [E, cap, cols] of 32-bit values, zero past each expert's last row."""
    p = torch.zeros((s["experts"] * s["cap"], x.shape[1]), device=x.device)
    p[s["slot"]] = x.float()
    return p.view(s["experts"], s["cap"], -1)


def _plain_grouped(s):
    eight = s["dtype"] == "fp8"
    W = _dequantize_weight(s["q"], s["scale"]) if eight else s["W"].float()

    def rows(x):
        return _pad(s, _dequantize_rows(*_quantize_rows(x)) if eight else x)

    def back(p):
        return p.flatten(0, 1)[s["slot"]].to(torch.bfloat16)

    out = {}
    if s["mode"] != "bwd":
        x = rows(s["x"])
        out["y"] = back(torch.bmm(x, W.transpose(1, 2)))
    if s["mode"] != "fwd":
        dy = rows(s["dy"])
        out["dx"] = back(torch.bmm(dy, W))
    if s["mode"] == "step":
        out["dw"] = torch.bmm(dy.transpose(1, 2), x)
    return out


# ------------------------------------------------------------------ one pass

def _own(s):
    from quantized_lora_fine_b200 import api
    if s["kind"] == "norm":
        y, h, rstd = api.rms_norm_fwd(s["x"], s["w"], EPS, residual=s["r"], fp8=s["mode"] == "fp8")
        if s["mode"] == "fp8":
            return {"q": y.codes, "scale": y.scale, "h": h, "rstd": rstd}
        out = {"y": y, "h": h, "rstd": rstd}
        if s["mode"] == "step":
            out["dx"], out["dw"] = api.rms_norm_bwd(s["dy"], h, rstd, s["w"], dh=s["dh"])
        return out
    if s["kind"] == "fp8":
        w = api.FP8Weight(s["q"], s["scale"])
        if s["mode"] == "fwd":
            return api.fp8_linear_fwd(w, api.FP8Rows(*s["rows8"]) if s["rows_in_8bit"] else s["x"])
        return api.fp8_linear_bwd(w, api.FP8Rows(*s["rows8"]) if s["rows_in_8bit"] else s["dy"])
    W = api.FP8Weight(s["q"], s["scale"]) if s["dtype"] == "fp8" else s["W"]
    out = {}
    if s["mode"] != "bwd":
        out["y"] = api.grouped_linear_fwd(W, s["x"], s["offsets"])
    if s["mode"] == "bwd":
        out["dx"], _ = api.grouped_linear_bwd(W, None, s["dy"], s["offsets"], need_dW=False)
    if s["mode"] == "step":
        out["dx"], out["dw"] = api.grouped_linear_bwd(W, s["x"], s["dy"], s["offsets"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "fp8": _plain_fp8, "grouped": _plain_grouped}[state["kind"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    M = case["rows"]
    if case["kind"] == "norm":
        H = case["hidden"]
        n, nb = M * H, M * ((H + 127) // 128)
        b = n * 2 * (3 if case["residual"] else 1) + H * 2 + M * 4      # x (, r and h), w, rstd
        b += n + nb * 4 if case["mode"] == "fp8" else n * 2
        f = 6 * n
        if case["mode"] == "step":
            b += n * 6 + H * 4                                          # dy, dh, dx, dw
            f += 10 * n
        return {"bytes": b, "flops": f}
    o, i = case["out"], case["inp"]
    if case["kind"] == "fp8":
        k, n = (i, o) if case["mode"] == "fwd" else (o, i)
        rows = M * k + M * ((k + 127) // 128) * 4 if case["rows_in_8bit"] else 2 * M * k
        return {"bytes": rows + o * i + ((o + 127) // 128) * ((i + 127) // 128) * 4 + 2 * M * n, "flops": 2 * M * o * i}
    live = sum(1 for v in _sizes(case) if v)
    wb = o * i if case["dtype"] == "fp8" else 2 * o * i
    b = live * wb + 2 * M * (i + o) + (case["experts"] + 1) * 4
    f = 2 * M * o * i
    if case["mode"] == "step":
        b += 2 * M * (o + i) + case["experts"] * o * i * 4
        f *= 3
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even (|v| <= 448): 3 bits behind the leading one, spacing 2^-9 below 2^-6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _block_max(v, dims):
    """Largest magnitude of each block of 128 along the given dims, spread back over the block's elements."""
    a = v.abs()
    for d in dims:
        n = a.shape[d]
        parts = [p.amax(d, keepdim=True).expand_as(p) for p in a.split(128, d)]
        a = torch.cat(parts, d) if n else a
    return a.clamp_min(FLOOR)


def _rows64(x):
    """(codes, value of each element's scale) of rows in 64 bits."""
    a = _block_max(x, (-1,))
    return _e4m3(x * 448 / a), a / 448


def _weight64(s):
    """The weight that the stored codes and scales stand for."""
    W = s["q"].double()
    o, i = W.shape[-2:]
    ro = torch.arange(o, device=W.device) // 128
    ri = torch.arange(i, device=W.device) // 128
    return W * s["scale"].double()[..., ro, :][..., ri]


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "norm":
        x = s["x"].double()
        h = s["x"] if s["r"] is None else (x + s["r"].double()).to(torch.bfloat16)
        z = h.double()
        rstd = 1 / torch.sqrt((z * z).sum(-1) / z.shape[-1] + EPS)
        w = s["w"].double()
        n = z * rstd[:, None]
        y = n * w
        if case["mode"] == "fp8":
            q, sc = _rows64(y)
            return {"q": q, "scale": sc[:, ::128].contiguous(), "h": h.double(), "rstd": rstd}
        out = {"y": y, "h": h.double(), "rstd": rstd}
        if case["mode"] == "step":
            dy = s["dy"].double()
            t = (dy * w * n).sum(-1, keepdim=True) / z.shape[-1]
            out["dx"] = s["dh"].double() + (dy * w - n * t) * rstd[:, None]
            out["dw"] = (dy * n).sum(0)
        return out
    eight = case["kind"] == "fp8" or case["dtype"] == "fp8"
    W = _weight64(s) if eight else s["W"].double()

    def value(name):
        if case["kind"] == "fp8" and case["rows_in_8bit"]:
            q, sc = s["rows8"]
            c = torch.arange(q.shape[1], device=q.device) // 128
            return q.double() * sc.double()[:, c]
        if not eight:
            return s[name].double()
        q, sc = _rows64(s[name].double())
        return q * sc

    if case["kind"] == "fp8":
        return torch.mm(value("x"), W.t()) if case["mode"] == "fwd" else torch.mm(value("dy"), W)
    at = s["offsets"].tolist()
    spans = list(zip(at[:-1], at[1:]))
    out = {}
    if case["mode"] != "bwd":
        x = value("x")
        out["y"] = torch.cat([x[a:b] @ W[e].t() for e, (a, b) in enumerate(spans)])
    if case["mode"] != "fwd":
        dy = value("dy")
        out["dx"] = torch.cat([dy[a:b] @ W[e] for e, (a, b) in enumerate(spans)])
    if case["mode"] == "step":
        out["dw"] = torch.stack([dy[a:b].t() @ x[a:b] for a, b in spans])
    return out
