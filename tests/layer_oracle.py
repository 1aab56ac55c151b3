"""The layer operators in 64 bits on the CPU or GPU, with the bounds that their tests use.

u is half a step of the output type.  fp32 sums: a sum of n terms in any
order is off by at most n 2^-24 of the sum of magnitudes; the tensor cores'
fp32 accumulation by up to 2^-22 of it per 16-wide step."""

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -149}


def act(g, name):
    """act(g), act'(g) in 64 bits."""
    if name == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * torch.sigmoid(-g)
    if name == "gelu":
        c = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    p = torch.sigmoid(2 * k * (g + 0.044715 * g ** 3))
    q = torch.sigmoid(-2 * k * (g + 0.044715 * g ** 3))
    return g * p, p + 2 * g * p * q * k * (1 + 0.134145 * g ** 2)


def rms(s, w, eps):
    s = s.double()
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def rms_backward(dy, s, w, dsum, eps):
    """dx, dw and the sums of magnitudes that their errors scale with."""
    s, dy = s.double(), dy.double()
    rstd = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    n = s * rstd
    g = dy if w is None else dy * w.double()
    dx = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    mag = rstd * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if dsum is not None:
        dx, mag = dx + dsum.double(), mag + dsum.double().abs()
    return dx, (dy * n).sum(0), mag, (dy * n).abs().sum(0)


def acc_error(k):
    """Relative error of a tensor-core sum over k, of the sum of magnitudes."""
    return (k / 16 + 16) * 2.0 ** -22


def ffn(x, wg, wu, name):
    """h, gate, up and bounds of the errors of each before its rounding."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.T, x @ wu.T
    e = acc_error(x.shape[-1])
    eg, eu = e * (x.abs() @ wg.abs().T), e * (x.abs() @ wu.abs().T)
    a = act(g, name)[0]
    # |act'| <= 1.13 for all three; the device's exp and quotient are within 2^-14 at these arguments
    eh = 1.2 * eg * (u.abs() + eu) + a.abs() * eu + 2.0 ** -14 * (a * u).abs()
    return a * u, g, u, eh, eg, eu


def ffn_backward(dh, x, wg, wu, gate, up, name):
    """dx, dwg, dwu, the sums of magnitudes of their products, and of the factors that dg and du meet."""
    dh, x, wg, wu, gate, up = (t.double() for t in (dh, x, wg, wu, gate, up))
    a, da = act(gate, name)
    dg, du = dh * up * da, dh * a
    # act' crosses zero: its error is 2^-21 in absolute terms there
    mg, mu = (dh * up).abs() * (da.abs() + 2.0 ** -10), du.abs()
    fx = x.abs().sum(0)
    return ((dg @ wg + du @ wu, dg.T @ x, du.T @ x), (mg @ wg.abs() + mu @ wu.abs(), mg.T @ x.abs(), mu.T @ x.abs()),
            (wg.abs().sum(0) + wu.abs().sum(0), fx, fx))


def worst(got, want, bound):
    """max of |got - want| / bound; at most 1 where the bound holds (nan counts as infinitely far)."""
    off = (got.double() - want).abs()
    d = torch.where(off == 0, torch.zeros_like(off), off / bound)  # no difference is within a bound of 0 too
    return float(torch.nan_to_num(d, nan=math.inf).max()) if d.numel() else 0.0
