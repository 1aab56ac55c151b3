"""Calls of the layer operators that the documentation allows beside the plain
ones: keywords in any order on another stream, rows off 16-byte boundaries
called twice, values outside the finite numbers.  Bounds as in
test_gpu_layers.py."""

import pytest
import torch

import layer_oracle as L
import newton_schulz_msign_b200 as msb

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def randn(shape, seed, dtype, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


# ---------------------------------------------------------------- streams

STREAM_CALLS = {
    "norm": lambda x, w, h, q, one, **kw: msb.rms_norm(eps=1e-5, x=x, **kw),
    "norm, None first": lambda x, w, h, q, one, **kw: msb.rms_norm(weight=None, x=x, **kw),
    "norm, by position": lambda x, w, h, q, one, **kw: msb.rms_norm(x, **kw),
    "norm to int8": lambda x, w, h, q, one, **kw: msb.rms_norm_q8(scale_out=None, x=x, **kw),
    "norm gradients": lambda x, w, h, q, one, **kw: msb.rms_norm_backward(eps=1e-5, s=x, dy=x, **kw),
    "int8 product": lambda x, w, h, q, one, **kw: msb.i8_matmul(out_dtype=FP32, b=q, a=q, a_scale=one, b_scale=one, **kw),
    "gated block": lambda x, w, h, q, one, **kw: msb.gated_ffn(activation="gelu", x=x, w_gate=w, w_up=w, **kw),
    "gated gradients": lambda x, w, h, q, one, **kw: msb.gated_ffn_backward(
        activation="gelu", dh=h, x=x, w_gate=w, w_up=w, gate=h, up=h, **kw),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", list(STREAM_CALLS))
def test_a_call_on_a_stream_comes_after_what_that_stream_does(name, raw):
    # the inputs are written at the end of some 20 ms of products on the side stream: a call on any other reads zeros
    call = STREAM_CALLS[name]
    new = [randn((64, 128), 1, BF16), randn((96, 128), 2, BF16, 0.1), randn((64, 96), 3, BF16),
           randn((64, 128), 4, FP32, 40.0).clamp(-127, 127).to(torch.int8), randn((64,), 5, FP32).abs() + 0.1]
    want = call(*new)
    work = torch.ones((8192, 8192), device="cuda", dtype=BF16)
    torch.matmul(work, work)
    now = [torch.zeros_like(t) for t in new]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(25):
            torch.matmul(work, work)
        for a, b in zip(now, new):
            a.copy_(b)
    got = call(*now, stream=side.cuda_stream if raw else side)
    side.synchronize()
    for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
        assert a is None and b is None or torch.equal(a, b)


# ---------------------------------------------------------------- rows off 16-byte boundaries

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("cols", [257, 1001, 2046])
@pytest.mark.parametrize("rows", [1, 2, 3])
def test_norm_gradients_whose_row_is_its_edges(dtype, cols, rows):
    # everything but the few elements before the first and behind the last 16-byte boundary is zero, in launches where
    # each row is the first or the last of its matrix: what the statistic sees is stored by single lanes
    edge = 16 // dtype.itemsize - 1
    s, dy, w = randn((rows, cols), 10, dtype), randn((rows, cols), 11, dtype), randn((cols,), 12, dtype)
    s[:, edge:-edge] = 0
    dy[:, edge:-edge] = 0
    for _ in range(20):
        dx, dw = msb.rms_norm_backward(dy, s, w, eps=1e-5)
        wx, ww, mx, mw = L.rms_backward(dy, s, w, None, 1e-5)
        assert L.worst(dx, wx, wx.abs() * L.U[dtype] + mx * 200 * 2.0 ** -24 + L.TINY[dtype]) <= 1
        assert L.worst(dw, ww, ww.abs() * L.U[dtype] + mw * 200 * 2.0 ** -24 + L.TINY[dtype]) <= 1
    msb.sync_status()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 3.0])
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_no_result_depends_on_what_lies_between_rows(fill, pad):
    # rows whose neighbours' bytes are read with them, in every operator that does so
    def apart(t, value):
        big = torch.full((t.shape[0], t.shape[1] + pad), value, device="cuda").to(t.dtype)
        big[:, :t.shape[1]] = t
        return big[:, :t.shape[1]]

    x, dy, ds = (randn((37, 1001), s, BF16) for s in (20, 21, 22))
    w, wg, wu = randn((1001,), 23, BF16), randn((50, 1001), 24, BF16, 0.03), randn((50, 1001), 25, BF16, 0.03)
    q, b = (randn((n, 1001), 26 + n, FP32, 40.0).clamp(-127, 127).to(torch.int8) for n in (37, 50))
    one = torch.ones(50, device="cuda")

    def run(value):
        lay = lambda t: apart(t, value if t.is_floating_point() else 77)  # noqa: E731
        z = lay(torch.zeros_like(x))
        out = [*msb.rms_norm(lay(x), w, lay(ds)), *msb.rms_norm_q8(lay(x), w, lay(ds))]
        out += msb.rms_norm_backward(lay(dy), lay(x), w, dsum=lay(ds), dx_out=z)
        out += [*msb.gated_ffn(lay(x), lay(wg), lay(wu), save=True), msb.i8_matmul(lay(q), one[:37], lay(b), one)]
        return [t.clone() for t in out]

    for a, c in zip(run(0.0), run(fill)):
        assert torch.equal(a, c)


# ---------------------------------------------------------------- values outside the finite numbers

@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("h", [64, 101])
def test_a_nan_gate_reaches_its_gradients(dtype, act, h):
    # a NaN gate makes dg NaN whatever the activation: dx of its token and dWg of its unit, and nothing else of them
    t, d = 40, 64
    x, wg, wu = randn((t, d), 30, dtype), randn((h, d), 31, dtype, 0.1), randn((h, d), 32, dtype, 0.1)
    gate, up, dh = randn((t, h), 33, dtype), randn((t, h), 34, dtype), randn((t, h), 35, dtype)
    gate[3, 7] = float("nan")
    dx, dwg, dwu = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act)
    for g, i in ((dx, 3), (dwg, 7), (dwu, 7)):
        keep = [j for j in range(g.shape[0]) if j != i]
        assert bool(torch.isnan(g[i]).all()) and bool(torch.isfinite(g[keep]).all())


# ---------------------------------------------------------------- the longest rows

@pytest.mark.parametrize("cols,lead", [(2 ** 28, 0), (2 ** 28 - 3, 1)])
def test_sums_of_very_long_rows(cols, lead):
    # 2^20 terms a thread, added in runs: 1024 terms, 1024 runs and 13 joins of halved weight (the root), and five more
    # operations.  (One sum all along is off by several times this bound.)
    rel = ((1024 + 1024 + 13) / 2 + 5) * 2.0 ** -24
    x = randn((cols + lead,), 40, BF16)[lead:]
    dy = randn((cols + lead,), 41, BF16)[lead:]
    y, scale = msb.rms_norm(x), msb.rms_norm_q8(x)[1]
    dx = msb.rms_norm_backward(dy, x)[0]
    part = 2 ** 26
    ss = sum(float((x[i:i + part].double() ** 2).sum()) for i in range(0, cols, part))
    dot = sum(float((x[i:i + part].double() * dy[i:i + part].double()).sum()) for i in range(0, cols, part))
    mag = sum(float((x[i:i + part].double() * dy[i:i + part].double()).abs().sum()) for i in range(0, cols, part))
    rstd = (ss / cols + 1e-6) ** -0.5
    amax = float(x.abs().max()) * rstd
    assert abs(float(scale) - amax / 127) <= amax / 127 * rel
    for i in range(0, cols, part):
        z, g = x[i:i + part].double(), dy[i:i + part].double()
        want = z * rstd
        assert L.worst(y[i:i + part], want, want.abs() * (L.U[BF16] + rel) + L.TINY[BF16]) <= 1
        m = rstd / cols
        want = rstd * (g - z * rstd * (dot * m))
        bound = rstd * (g.abs() + z.abs() * rstd * mag * m) * 2 * rel
        assert L.worst(dx[i:i + part], want, want.abs() * L.U[BF16] + bound + L.TINY[BF16]) <= 1


# ---------------------------------------------------------------- the same call twice

# (lead, pad, apart) as in test_gpu_layers.py
OFF = [(0, 0, 0), (1, 0, 1), (3, 0, 0), (5, 1, 0), (7, 2, 3), (2, 5, 0)]


def inside(shape, dtype, lead, pad, seed=None):
    """Rows ``pad`` elements apart, ``lead`` elements into a larger buffer."""
    rows, cols = shape
    big = torch.zeros(lead + rows * (cols + pad), device="cuda", dtype=dtype)
    v = big.as_strided(shape, (cols + pad, 1), lead)
    if seed is not None:
        v.copy_(randn(shape, seed, dtype))
    return v


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(41, 257), (600, 1003), (2500, 1003), (5, 2046), (700, 4607), (3, 16381), (300, 20001)])
@pytest.mark.parametrize("lead,pad,apart", OFF)
def test_norm_gradients_off_boundaries_repeat_their_bits(dtype, rows, cols, lead, pad, apart):
    # every layout, with outputs of the inputs' layout, so that both calls take the same kernel and the same blocks
    s, ds = inside((rows, cols), dtype, lead, pad, 50), inside((rows, cols), dtype, lead, pad, 51) if rows % 2 else None
    dy, w = inside((rows, cols), dtype, lead + apart, pad, 52), randn((cols,), 53, dtype)
    busy = torch.ones((2048, 2048), device="cuda", dtype=BF16)
    side = torch.cuda.Stream()
    first = None
    for i in range(4):
        if i % 2:  # beside other work, which changes the order in which blocks run
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.matmul(busy, busy)
        dx = inside((rows, cols), dtype, lead, pad)
        _, dw = msb.rms_norm_backward(dy, s, w, dsum=ds, dx_out=dx)
        if first is None:
            first = (dx, dw)
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
    torch.cuda.synchronize()
    wx, ww, mx, mw = L.rms_backward(dy, s, w, ds, 1e-6)
    serial = 200 + (rows + 99) // 100
    assert L.worst(first[0], wx, wx.abs() * L.U[dtype] + mx * serial * 2.0 ** -24 + L.TINY[dtype]) <= 1
    assert L.worst(first[1], ww, ww.abs() * L.U[dtype] + mw * serial * 2.0 ** -24 + L.TINY[dtype]) <= 1


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("t", [3, 300])
def test_the_activations_tails(act, t):
    # gates down to where the activation leaves bf16's normal numbers, one a hidden unit, times an up of 2^100 that
    # brings it back: x holds one feature for the gate and one for up
    h = 256
    # (act_of and its derivative are 1e-37 there; below it they go under the type's smallest normal)
    last = {"silu": -88.5, "gelu": -12.5, "gelu_tanh": -9.8}[act]
    g = torch.linspace(0.5 * last, last, h, device="cuda").to(BF16)
    wg, wu = torch.zeros((h, 64), device="cuda", dtype=BF16), torch.zeros((h, 64), device="cuda", dtype=BF16)
    wg[:, 0], wu[:, 1] = g, 2.0 ** 50
    x = torch.zeros((t, 64), device="cuda", dtype=BF16)
    x[:, 0], x[:, 1] = 1.0, 2.0 ** 50
    out, gate, up = msb.gated_ffn(x, wg, wu, activation=act, save=True)
    assert bool((gate == g).all()) and bool((up == 2.0 ** 100).all())
    a, da = L.act(g.double(), act)
    # The exponent's argument (at most 90, from up to six fp32 operations: 2^-21.5 relative) is off by 2^-15 and so is
    # the exponential, relative to itself; gelu's erfc is closer.  Below 2^-126 fp32 steps by 2^-149.
    bound = a.abs() * 2.0 ** 100 * (L.U[BF16] + 2.0 ** -14) + 2.0 ** (100 - 149) * g.double().abs()
    assert L.worst(out, (a * 2.0 ** 100).expand_as(out), bound.expand_as(out)) <= 1
    dh = torch.ones_like(out)
    dx, dwg, dwu = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, grad_dtype=FP32)
    # dWg[:, 0] = t dg: the derivative is p (1 + ...) with the same exponential, dg rounded once
    bound = da.abs() * 2.0 ** 100 * (L.U[BF16] + 2.0 ** -13) + 2.0 ** (100 - 149) * 4 * g.double().abs() ** 2
    assert L.worst(dwg[:, 0] / t, da * 2.0 ** 100, bound) <= 1
