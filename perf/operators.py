"""The layer operators around the Muon step, as they are measured: each case once in plain torch, once through the library.

Three operators of a transformer block whose weight matrices the library's optimizer updates:

- ``rms_norm`` / ``rms_norm_q8`` / ``rms_norm_backward``: s = x + residual, y = w s / sqrt(mean(s^2) + eps), in 16 or 32
  bits or as int8 with one scale a row, and its gradients;
- ``gated_ffn`` / ``gated_ffn_backward``: h = act(x Wg^T) * (x Wu^T) and its gradients;
- ``i8_matmul``: (a b^T) of int8 operands times a scale for each row of a (token) and each row of b (channel).

The sizes 4096, 1024 and 14336 are the Llama layer's of the repository's own configurations; the others are generic.
"""

import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of a decoding step through the pre-FFN norm: nothing but latency
        dict(name="norm_1x4096", op="norm", dtype="bf16", rows=1, cols=4096, residual=True),
        # the norm of a training micro-batch of 8192 tokens, with the residual stream's addition
        dict(name="norm_8192x4096", op="norm", dtype="bf16", rows=8192, cols=4096, residual=True),
        # the norm of a ragged prompt that feeds an int8 projection
        dict(name="norm_q8_2047x4096", op="norm_q8", dtype="fp16", rows=2047, cols=4096, residual=True),
        # the norm's gradients in that training micro-batch (input, residual stream and weight)
        dict(name="norm_bwd_8192x4096", op="norm_bwd", dtype="bf16", rows=8192, cols=4096, residual=True),
        # the same of a small model of odd width in fp32, no residual
        dict(name="norm_bwd_777x1001", op="norm_bwd", dtype="fp32", rows=777, cols=1001, residual=False),
        # one token through an int8 up projection: the weights are read once
        dict(name="i8_1x14336x4096", op="i8", dtype="bf16", m=1, n=14336, k=4096),
        # a ragged batch of decoding streams through the down projection
        dict(name="i8_77x4096x14336", op="i8", dtype="fp16", m=77, n=4096, k=14336),
        # a long prompt through the up projection
        dict(name="i8_8192x14336x4096", op="i8", dtype="bf16", m=8192, n=14336, k=4096),
        # a few decoding streams through the gated block's 16-bit weights
        dict(name="ffn_4x4096x14336", op="ffn", dtype="bf16", t=4, d=4096, h=14336, act="silu", save=False),
        # the training forward of a micro-batch, pre-activations kept for the backward pass
        dict(name="ffn_4096x4096x14336", op="ffn", dtype="bf16", t=4096, d=4096, h=14336, act="silu", save=True),
        # the gradients of a small model of odd sizes
        dict(name="ffn_bwd_513x1000x2730", op="ffn_bwd", dtype="fp16", t=513, d=1000, h=2730, act="gelu_tanh"),
        # the gradients of the micro-batch
        dict(name="ffn_bwd_8192x4096x14336", op="ffn_bwd", dtype="bf16", t=8192, d=4096, h=14336, act="silu"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A matrix width: mostly a multiple of 64 or 8, sometimes any number."""
    v = _log(rng, lo, hi)
    step = rng.choice([64, 64, 8, 1])
    return max(step, v // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm_q8", "norm_bwd", "i8", "i8", "ffn", "ffn", "ffn_bwd"])
    if op in ("norm", "norm_q8", "norm_bwd"):
        # (the values an int8 output stands for come back in 16 bits: a value at a rounding border may fall to either side)
        dtype = rng.choice(["bf16", "fp16"] if op == "norm_q8" else ["bf16", "fp16", "fp32"])
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, 16384), cols=_width(rng, 64, 8192), residual=rng.random() < 0.5)
    if op == "i8":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, dtype=dtype, m=_log(rng, 1, 8192), n=_width(rng, 64, 14336), k=_width(rng, 64, 14336))
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice(["silu", "gelu", "gelu_tanh"])
    t, d, h = _log(rng, 1, 8192), _width(rng, 64, 4096), _width(rng, 64, 14336)
    if op == "ffn":
        return dict(op=op, dtype=dtype, t=t, d=d, h=h, act=act, save=rng.random() < 0.5)
    return dict(op=op, dtype=dtype, t=t, d=d, h=h, act=act)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case, "dt": dt}
    if op in ("norm", "norm_q8", "norm_bwd"):
        shape = (case["rows"], case["cols"])
        # activations with a few heavy channels, as a residual stream has them
        heavy = 1.0 + 8.0 * (torch.rand(case["cols"], generator=g, device="cuda") < 0.01).float()
        s["x"] = (torch.randn(shape, generator=g, device="cuda") * heavy).to(dt)
        s["w"] = (1.0 + 0.2 * torch.randn(case["cols"], generator=g, device="cuda")).to(dt)
        s["r"] = _normal(g, shape, 1.0, dt) if case["residual"] else None
        if op == "norm_bwd":  # x stands for the stored sum, r for the gradient that reaches it past the norm
            s["dy"] = _normal(g, shape, 1e-2, dt)
            s["r"] = _normal(g, shape, 1e-2, dt) if case["residual"] else None
    elif op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        # rows quantised to their largest magnitude: the rest lies around zero
        s["a"] = (torch.randn((m, k), generator=g, device="cuda") * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["b"] = (torch.randn((n, k), generator=g, device="cuda") * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["sa"] = 0.01 + 0.04 * torch.rand(m, generator=g, device="cuda")
        s["sb"] = (0.5 + torch.rand(n, generator=g, device="cuda")) * (0.02 / math.sqrt(k))
    else:
        t, d, h = case["t"], case["d"], case["h"]
        s["x"] = _normal(g, (t, d), 1.0, dt)
        s["wg"] = _normal(g, (h, d), 1.0 / math.sqrt(d), dt)
        s["wu"] = _normal(g, (h, d), 1.0 / math.sqrt(d), dt)
        if op == "ffn_bwd":  # the pre-activations that the forward pass kept, and the gradient of h
            s["gate"] = s["x"] @ s["wg"].T
            s["up"] = s["x"] @ s["wu"].T
            s["dh"] = _normal(g, (t, h), 1.0 / math.sqrt(h), dt)
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits (quantised values in 64)

def _act(g, act):
    """The activation and its derivative at g."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_norm(s, wide):
    """y in `wide`, and the sum in the inputs' type: the norm is that of the stored sum."""
    if s["r"] is None:
        z, stored = s["x"].to(wide), None
    else:
        stored = (s["x"].float() + s["r"].float()).to(s["dt"])
        z = stored.to(wide)
    y = z * torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS) * s["w"].to(wide)
    return y, stored


def _plain_quantised(y, stored, dt):
    scale = y.abs().amax(dim=1, keepdim=True) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale)))
    out = [(q * scale).to(dt), scale[:, 0].float()]
    return out if stored is None else out + [stored]


def _plain_norm_bwd(s, wide):
    z, w = s["x"].to(wide), s["w"].to(wide)
    rstd = torch.rsqrt((z * z).mean(dim=1, keepdim=True) + EPS)
    n = z * rstd
    dy = s["dy"].to(wide)
    dn = dy * w
    dz = rstd * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    if s["r"] is not None:
        dz = dz + s["r"].to(wide)
    return dz, (dy * n).sum(dim=0)


def _plain(s):
    case, dt = s["case"], s["dt"]
    op = case["op"]
    if op == "norm":
        y, stored = _plain_norm(s, torch.float32)
        return [y.to(dt)] if stored is None else [y.to(dt), stored]
    if op == "norm_q8":
        y, stored = _plain_norm(s, torch.float64)
        return _plain_quantised(y, stored, dt)
    if op == "norm_bwd":
        dz, dw = _plain_norm_bwd(s, torch.float32)
        return [dz.to(dt), dw.to(dt)]
    if op == "i8":
        acc = s["a"].float() @ s["b"].float().T
        return [(acc * s["sa"][:, None] * s["sb"]).to(dt)]
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    if op == "ffn":
        g, u = x @ wg.T, x @ wu.T
        h = (_act(g, case["act"])[0] * u).to(dt)
        return [h, g.to(dt), u.to(dt)] if case["save"] else [h]
    a, da = _act(s["gate"].float(), case["act"])
    dh = s["dh"].float()
    dg, du = dh * s["up"].float() * da, dh * a
    return [(dg @ wg + du @ wu).to(dt), (dg.T @ x).to(dt), (du.T @ x).to(dt)]


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import newton_schulz_msign_b200 as msb

    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        out = msb.rms_norm(s["x"], s["w"], s["r"], eps=EPS)
        return [out] if s["r"] is None else list(out)
    if op == "norm_q8":
        out = msb.rms_norm_q8(s["x"], s["w"], s["r"], eps=EPS)
        q, scale = out[0], out[1]
        # the values that the int8 output stands for, read back in one pass
        back = torch.empty(q.shape, dtype=s["dt"], device=q.device)
        torch.mul(q, scale[:, None], out=back)
        return [back, scale] if s["r"] is None else [back, scale, out[2]]
    if op == "norm_bwd":
        return list(msb.rms_norm_backward(s["dy"], s["x"], s["w"], dsum=s["r"], eps=EPS))
    if op == "i8":
        return [msb.i8_matmul(s["a"], s["sa"], s["b"], s["sb"], out_dtype=s["dt"])]
    if op == "ffn":
        out = msb.gated_ffn(s["x"], s["wg"], s["wu"], activation=case["act"], save=case["save"])
        return list(out) if case["save"] else [out]
    return list(msb.gated_ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], s["gate"], s["up"], activation=case["act"]))


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    op, es = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op in ("norm", "norm_q8", "norm_bwd"):
        e, c = case["rows"] * case["cols"], case["cols"]
        if op == "norm":  # x and w in, y out; the residual in and the sum out
            return {"bytes": es * (2 * e + c + (2 * e if case["residual"] else 0)), "flops": 5 * e}
        if op == "norm_q8":
            return {"bytes": es * (e + c + (2 * e if case["residual"] else 0)) + e + 4 * case["rows"], "flops": 8 * e}
        return {"bytes": es * (3 * e + 2 * c + (e if case["residual"] else 0)), "flops": 12 * e}
    if op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + n) + es * m * n, "flops": 2 * m * n * k}
    t, d, h = case["t"], case["d"], case["h"]
    if op == "ffn":
        return {"bytes": 2 * (t * d + 2 * h * d + t * h * (3 if case["save"] else 1)), "flops": 4 * t * d * h}
    # in: dh, gate, up, x, both weights; out: dx and both weights' gradients
    return {"bytes": 2 * (3 * t * h + 2 * t * d + 4 * h * d), "flops": 8 * t * d * h}


# ---------------------------------------------------------------- definitions in 64 bits, apart from the forms above

def _exact_act(g, act):
    """act(g) and act'(g) from their definitions, in 64 bits."""
    if act == "silu":
        e = torch.exp(-g.abs())
        sig = torch.where(g >= 0, 1.0 / (1.0 + e), e / (1.0 + e))
        return g * sig, sig + g * e / ((1.0 + e) * (1.0 + e))
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        pdf = torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
        return g * cdf, cdf + g * pdf
    b = math.sqrt(2.0 / math.pi)
    z = b * (g + 0.044715 * g**3)
    dz = b * (1.0 + 0.134145 * g**2)
    sig = torch.sigmoid(2.0 * z)  # (1 + tanh z) / 2
    return g * sig, sig + g * 2.0 * sig * torch.sigmoid(-2.0 * z) * dz


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_q8", "norm_bwd"):
        x, w = s["x"].double(), s["w"].double()
        if op == "norm_bwd":
            var = x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS
            dy = s["dy"].double()
            t = dy * w
            dz = t / var.sqrt() - x * ((t * x).sum(1, keepdim=True) / (x.shape[1] * var.pow(1.5)))
            return [dz + s["r"].double() if case["residual"] else dz, (dy * x / var.sqrt()).sum(0)]
        stored = None
        if case["residual"]:
            stored = x + s["r"].double()
            x = stored.to(s["dt"]).double()
        y = x * w / (x.pow(2).sum(1, keepdim=True) / x.shape[1] + EPS).sqrt()
        if op == "norm":
            return [y] if stored is None else [y, stored]
        step = y.abs().max(1).values / 127
        out = [torch.round(y / step[:, None]) * step[:, None], step]
        return out if stored is None else out + [stored]
    if op == "i8":
        return [torch.matmul(s["a"].double(), s["b"].double().T) * torch.outer(s["sa"].double(), s["sb"].double())]
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    if op == "ffn":
        g, u = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
        h = _exact_act(g, case["act"])[0] * u
        return [h, g, u] if case["save"] else [h]
    g, dh = s["gate"].double(), s["dh"].double()
    a, da = _exact_act(g, case["act"])
    du = dh * a
    dg = dh * s["up"].double() * da
    return [torch.matmul(dg, wg) + torch.matmul(du, wu), torch.matmul(dg.T, x), torch.matmul(du.T, x)]
