"""The layer operators on the GPU against their definitions in 64 bits: RMS
norm (also int8), the gated feed-forward block and the int8 product, and a run
of them up to the Muon step.  The bounds are derived in layer_oracle.py and
beside each check."""

import math

import pytest
import torch

import layer_oracle as L
import newton_schulz_msign_b200 as msb

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(shape, seed, dtype, std=1.0):
    return (torch.randn(shape, generator=gen(seed), device="cuda") * std).to(dtype)


def view(t, pad, lead=0):
    """The same values as a view into a larger tensor: rows ``pad`` elements further apart, ``lead`` elements in."""
    big = torch.full((t.shape[0], t.shape[1] + pad + lead), 3.0, device="cuda").to(t.dtype)
    v = big[:, lead:lead + t.shape[1]]
    v.copy_(t)
    return v


# ---------------------------------------------------------------- rms_norm

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (2, 100), (257, 256), (9, 1024), (4, 1032), (33, 4096), (3, 5000), (2, 8192),
               (2, 16384), (2, 40000), (700, 1001)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm(dtype, shape, residual):
    x = randn(shape, 1, dtype)
    w = randn(shape[1:], 2, FP32 if shape[0] % 2 else dtype)
    r = randn(shape, 3, dtype) if residual else None
    out = msb.rms_norm(x, w, r, eps=1e-5)
    msb.sync_status()
    s = x
    if residual:
        out, s = out
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
    want = L.rms(s, w, 1e-5)
    # fp32: the sum of squares of up to 160 terms a thread and 11 joins, halved by the root, and five more operations
    bound = want.abs() * (L.U[dtype] + 100 * 2.0 ** -24) + L.TINY[dtype]
    assert L.worst(out, want, bound) <= 1


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_rms_norm_q8(dtype, shape, residual):
    x = randn(shape, 4, dtype)
    w = randn(shape[1:], 5, dtype if shape[0] % 2 else FP32)
    r = randn(shape, 6, dtype) if residual else None
    got = msb.rms_norm_q8(x, w, r)
    msb.sync_status()
    q, scale = got[0], got[1]
    s = x
    if residual:
        s = got[2]
        assert torch.equal(s, (x.float() + r.float()).to(dtype))
    y = L.rms(s, w, 1e-6)
    amax = y.abs().amax(1)
    rel = 110 * 2.0 ** -24
    assert L.worst(scale, amax / 127, amax / 127 * rel) <= 1
    assert q.dtype == torch.int8 and int(q.abs().max()) == 127
    # the nearest step, up to the fp32 error of y / scale (127 steps at most, both sides of the quotient)
    assert L.worst(q, y / (amax / 127)[:, None], torch.tensor(0.5 + 127 * 2 * rel, device="cuda")) <= 1


@pytest.mark.parametrize("dtype,tiny,big", [(BF16, 1e-38, 1e18), (FP16, 6e-8, 6e4), (FP32, 1e-40, 1e18)])
@pytest.mark.parametrize("cols", [64, 77, 4096])
def test_rms_norm_q8_at_the_ends_of_the_range(dtype, tiny, big, cols):
    # rows of the smallest and largest magnitudes whose squares fp32 holds or loses, and weights that make y tiny or huge
    x = randn((6, cols), 400 + cols, FP32)
    x[0] = torch.where(x[0] > 0, tiny, -tiny)
    x[1] = torch.where(x[1] > 0, big, -big)
    x = x.to(dtype)
    for scale in (1.0, 1e-38, 1e-30, 1e30):
        w = randn((cols,), 500, FP32) * scale
        q, s = msb.rms_norm_q8(x, w, eps=1e-6)
        y = L.rms(x, w, 1e-6)
        amax = y.abs().amax(1)
        # fp32 flushes nothing here, but its subnormals carry fewer digits: 2^-149 absolute in y and in the scale
        ok = amax / 127 > 2.0 ** -126
        rel = 110 * 2.0 ** -24
        assert L.worst(s[ok], (amax / 127)[ok], (amax / 127 * rel)[ok]) <= 1
        assert int(q.abs().max()) <= 127 and bool((q[ok].abs().amax(1) == 127).all())
        assert L.worst(q[ok], (y / (amax / 127)[:, None])[ok], torch.tensor(0.5 + 127 * 2 * rel, device="cuda")) <= 1
        assert bool(torch.isfinite(s).all())


@pytest.mark.parametrize("cols", [64, 77, 1024, 4096, 16384])
def test_rms_norm_of_rows_whose_squares_leave_fp32(cols):
    x = randn((7, cols), 600, FP32) * torch.tensor([1e18, 1e30, 1e-25, 1.0, 1e-38, 3e19, 1e37], device="cuda")[:, None]
    x[1, 3] = 1e-30
    w, dy = randn((cols,), 601, FP32), randn((7, cols), 602, FP32)
    y = msb.rms_norm(x, w, eps=0.0)
    want = L.rms(x, w, 0.0)
    # as the ordinary rows, and 2^-149 absolute of rstd where the row is near the type's end (1e37: 2e-8 of rstd)
    assert L.worst(y, want, want.abs() * (2.0 ** -24 + 400 * 2.0 ** -24) + 2.0 ** -126) <= 1
    dx, dw = msb.rms_norm_backward(dy, x, w, eps=0.0)
    wx, ww, mx, mw = L.rms_backward(dy, x, w, None, 0.0)
    for i in range(7):
        if float(mx[i].max()) < 1e38:
            assert L.worst(dx[i], wx[i], mx[i] * 400 * 2.0 ** -24 + 2.0 ** -126) <= 1, i
    assert L.worst(dw, ww, mw * 400 * 2.0 ** -24) <= 1
    one = msb.rms_norm(x[:1].to(BF16), w, eps=1e-6)
    want = L.rms(x[:1].to(BF16), w, 1e-6)
    assert L.worst(one, want, want.abs() * (L.U[BF16] + 100 * 2.0 ** -24)) <= 1


def test_rms_norm_without_weight_and_in_place():
    for cols in (512, 1003):
        x, r = randn((6, cols), 7, BF16), randn((6, cols), 8, BF16)
        s = (x.float() + r.float()).to(BF16)
        want = L.rms(s, None, 1e-6)
        bound = want.abs() * (L.U[BF16] + 2.0 ** -17)
        r2 = r.clone()
        y, s2 = msb.rms_norm(x, None, r2, sum_out=r2)  # the residual stream updated in place
        assert s2 is r2 and torch.equal(r2, s)
        assert L.worst(y, want, bound) <= 1
        x2 = x.clone()
        y, s2 = msb.rms_norm(x2, None, r, sum_out=x2)
        assert torch.equal(x2, s) and L.worst(y, want, bound) <= 1
        x3 = x.clone()
        y, s2 = msb.rms_norm(x3, None, r, out=x3)  # y over x, the sum elsewhere
        assert y is x3 and torch.equal(s2, s) and L.worst(x3, want, bound) <= 1


@pytest.mark.parametrize("pad,lead", [(8, 8), (3, 1)])
def test_rms_norm_strided_rows(pad, lead):
    x, r = randn((37, 640), 9, FP16), randn((37, 640), 10, FP16)
    xv, rv = view(x, pad, lead), view(r, pad, 0)
    out, s = view(torch.zeros_like(x), pad, lead), view(torch.zeros_like(x), 0, lead)
    msb.rms_norm(xv, None, rv, out=out, sum_out=s)
    want_y, want_s = msb.rms_norm(x, None, r)
    # another thread layout may join the sums in another order: one step of the type apart at most
    assert torch.equal(s, want_s)
    assert L.worst(out, want_y.double(), want_y.double().abs() * 2 * L.U[FP16] + 2.0 ** -24) <= 1
    base = out._base
    assert bool((base[:, lead + 640:] == 3).all()) and bool((base[:, :lead] == 3).all())


def test_rms_norm_rows_that_hold_nothing_finite():
    x = randn((5, 4096), 11, BF16)
    x[1, 17] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 0
    y = msb.rms_norm(x)
    assert bool(torch.isfinite(y[[0, 4]]).all()) and bool(torch.isnan(y[1]).all()) and not bool(torch.isfinite(y[2, 5]))
    assert bool((y[3] == 0).all())
    q, scale = msb.rms_norm_q8(x)
    assert bool(torch.isnan(scale[1])) and not bool(torch.isfinite(scale[2]))
    assert float(scale[3]) == 0 and bool((q[1:4] == 0).all())
    back = q.float() * scale[:, None]
    assert bool(torch.isnan(back[1:3]).all()) and bool(torch.isfinite(back[[0, 3, 4]]).all())
    b = torch.ones((40, 4096), dtype=torch.int8, device="cuda")
    out = msb.i8_matmul(q, scale, b, torch.ones(40, device="cuda"))
    assert bool(torch.isnan(out[1:3]).all()) and bool(torch.isfinite(out[[0, 3, 4]]).all())


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", NORM_SHAPES + [(3000, 64), (1500, 520)])
@pytest.mark.parametrize("dsum", [False, True])
def test_rms_norm_backward(dtype, shape, dsum):
    s, dy = randn(shape, 12, dtype), randn(shape, 13, dtype)
    w = randn(shape[1:], 14, dtype if shape[0] % 2 else FP32)
    ds = randn(shape, 15, dtype) if dsum else None
    dx, dw = msb.rms_norm_backward(dy, s, w, dsum=ds, eps=1e-5)
    msb.sync_status()
    wx, ww, mx, mw = L.rms_backward(dy, s, w, ds, 1e-5)
    serial = 200 + math.ceil(shape[0] / 100)  # terms a thread adds one after another, and the joins
    assert L.worst(dx, wx, wx.abs() * L.U[dtype] + mx * serial * 2.0 ** -24 + L.TINY[dtype]) <= 1
    assert dw.dtype == w.dtype
    assert L.worst(dw, ww, ww.abs() * L.U[w.dtype] + mw * serial * 2.0 ** -24 + L.TINY[w.dtype]) <= 1
    again = msb.rms_norm_backward(dy, s, w, dsum=ds, eps=1e-5)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # no order of blocks shows
    nx, nw = msb.rms_norm_backward(dy, s, None, dsum=ds, eps=1e-5)
    wx, _, mx, _ = L.rms_backward(dy, s, None, ds, 1e-5)
    assert nw is None and L.worst(nx, wx, wx.abs() * L.U[dtype] + mx * serial * 2.0 ** -24 + L.TINY[dtype]) <= 1


def test_rms_norm_backward_against_differences():
    s, w, dy, v = (randn((6, 776), i, FP32) for i in (16, 17, 18, 19))
    w, vw = w[0].contiguous(), randn((776,), 20, FP32)
    dx, dw = msb.rms_norm_backward(dy, s, w)
    h = 1e-6
    f = lambda s_, w_: float((L.rms(s_, w_, 1e-6) * dy.double()).sum())  # noqa: E731
    d = (f(s.double() + h * v.double(), w) - f(s.double() - h * v.double(), w)) / (2 * h)
    # 64-bit differences are good to h^2 and 1e-16 / h; the gradient to fp32
    assert abs(float((dx.double() * v.double()).sum()) - d) <= 1e-5 * float((dx.double() * v.double()).abs().sum())
    d = (f(s, w.double() + h * vw.double()) - f(s, w.double() - h * vw.double())) / (2 * h)
    assert abs(float((dw.double() * vw.double()).sum()) - d) <= 1e-5 * float((dw.double() * vw.double()).abs().sum())


def inside(t, lead, pad, tail, fill):
    """The same values as rows ``pad`` elements apart, ``lead`` elements into a larger buffer of ``fill`` that goes on
    for ``tail`` elements behind the last row; and that buffer."""
    rows, cols = t.shape
    big = torch.full((lead + rows * (cols + pad) - pad + tail,), fill, device="cuda").to(t.dtype)
    v = big.as_strided((rows, cols), (cols + pad, 1), lead)
    v.copy_(t)
    return v, big


def untouched(v, big, fill):
    """Whether the buffer around a view from ``inside`` still holds its fill."""
    around = torch.ones_like(big, dtype=torch.bool)
    around.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
    return bool((big[around] == fill).all())


# Rows off 16-byte boundaries: every matrix in the same phase (x_lead = lead), with rows that start in all phases or in
# one, first and last rows whose neighbours belong to nobody; and one matrix apart from the others.
OFF = [(0, 0, 0), (1, 0, 1), (3, 0, 0), (5, 1, 0), (7, 2, 3), (2, 5, 0)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 257), (41, 257), (19, 1001), (600, 1003), (5, 2046), (7, 4099), (3, 16383), (2, 20001)])
@pytest.mark.parametrize("lead,pad,apart", OFF)
def test_rms_norm_off_boundaries(dtype, rows, cols, lead, pad, apart):
    nan = float("nan")
    x, _ = inside(randn((rows, cols), 40, dtype), lead + apart, pad, 0, nan)
    r, _ = inside(randn((rows, cols), 41, dtype), lead, pad, 0, nan)
    w = randn((cols,), 42, dtype if rows % 2 else FP32)
    y, yb = inside(torch.zeros_like(x), lead, pad, 40, 3)
    s, sb = inside(torch.zeros_like(x), lead, pad, 40, 3)
    msb.rms_norm(x, w, r, eps=1e-5, out=y, sum_out=s)
    q, qb = inside(torch.zeros((rows, cols), dtype=torch.int8, device="cuda"), lead, pad, 40, 3)
    _, scale, s8 = msb.rms_norm_q8(x, w, r, eps=1e-5, out=q)
    msb.sync_status()
    want_s = (x.float() + r.float()).to(dtype)
    assert torch.equal(s, want_s) and torch.equal(s8, want_s)
    want = L.rms(want_s, w, 1e-5)
    # (the bounds of test_rms_norm and test_rms_norm_q8)
    assert L.worst(y, want, want.abs() * (L.U[dtype] + 100 * 2.0 ** -24) + L.TINY[dtype]) <= 1
    amax, rel = want.abs().amax(1), 110 * 2.0 ** -24
    assert L.worst(scale, amax / 127, amax / 127 * rel) <= 1
    assert L.worst(q, want / (amax / 127)[:, None], torch.tensor(0.5 + 127 * 2 * rel, device="cuda")) <= 1
    assert untouched(y, yb, 3) and untouched(s, sb, 3) and untouched(q, qb, 3)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("rows,cols", [(1, 257), (41, 257), (19, 1001), (2500, 1003), (5, 2046), (7, 4099), (700, 4607),
                                       (3, 16381), (2, 20001)])
@pytest.mark.parametrize("lead,pad,apart", OFF)
def test_rms_norm_backward_off_boundaries(dtype, rows, cols, lead, pad, apart):
    nan = float("nan")
    s, _ = inside(randn((rows, cols), 43, dtype), lead, pad, 0, nan)
    dy, _ = inside(randn((rows, cols), 44, dtype), lead + apart, pad, 0, nan)
    ds = inside(randn((rows, cols), 45, dtype), lead, pad, 0, nan)[0] if rows % 2 else None
    w = randn((cols,), 46, dtype if rows % 2 else FP32)
    dx, xb = inside(torch.zeros_like(s), lead, pad, 40, 3)
    _, dw = msb.rms_norm_backward(dy, s, w, dsum=ds, eps=1e-5, dx_out=dx)
    msb.sync_status()
    wx, ww, mx, mw = L.rms_backward(dy, s, w, ds, 1e-5)
    serial = 200 + math.ceil(rows / 100)  # (see test_rms_norm_backward)
    assert L.worst(dx, wx, wx.abs() * L.U[dtype] + mx * serial * 2.0 ** -24 + L.TINY[dtype]) <= 1
    assert L.worst(dw, ww, ww.abs() * L.U[w.dtype] + mw * serial * 2.0 ** -24 + L.TINY[w.dtype]) <= 1
    assert untouched(dx, xb, 3)
    again = msb.rms_norm_backward(dy, s, w, dsum=ds, eps=1e-5)
    assert torch.equal(again[1], dw) or apart or lead or pad  # (rows elsewhere may lie in other blocks)


def test_rms_norm_off_boundaries_at_the_ends_of_the_range():
    # squares beyond fp32, an infinity and a NaN, in rows whose neighbours share their 16 bytes
    x = randn((24, 1001), 47, FP32)
    x[3] *= 1e25
    x[8] *= 1e-25
    x[11, 1000] = float("inf")
    x[14, 0] = float("nan")
    x[20] = 0.0
    dy = randn((24, 1001), 48, FP32)
    y = msb.rms_norm(x, eps=0.0)
    dx, _ = msb.rms_norm_backward(dy, x, eps=0.0)
    msb.sync_status()
    ok = [i for i in range(24) if i not in (11, 14, 20)]
    want = L.rms(x, None, 0.0)[ok]
    assert L.worst(y[ok], want, want.abs() * (L.U[FP32] + 100 * 2.0 ** -24) + L.TINY[FP32]) <= 1
    wx, _, mx, _ = L.rms_backward(dy, x, None, None, 0.0)
    assert L.worst(dx[ok], wx[ok], wx[ok].abs() * L.U[FP32] + mx[ok] * 201 * 2.0 ** -24 + L.TINY[FP32]) <= 1
    for i in (11, 14, 20):
        assert not bool(torch.isfinite(y[i]).all())
    assert bool(torch.isnan(dx[14]).all()) and bool(torch.isnan(dx[20]).all())


# ---------------------------------------------------------------- i8_matmul

def i8(shape, seed):
    return torch.randint(-128, 128, shape, generator=gen(seed), device="cuda", dtype=torch.int8)


def i8_check(a, sa, b, sb, dtype, got):
    want = (a.double() @ b.double().T) * sa.double()[:, None] * sb.double()
    # the integer sum is exact: its conversion and two products in fp32, then the type's rounding
    assert L.worst(got, want, want.abs() * (L.U[dtype] + 3 * 2.0 ** -24) + L.TINY[dtype]) <= 1


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 128, 128), (1, 4096, 1024), (3, 130, 16), (16, 64, 4096), (17, 200, 300),
                                   (64, 1000, 144), (65, 96, 2000), (77, 384, 1024), (200, 333, 513), (256, 512, 640),
                                   (257, 512, 640), (300, 77, 129), (513, 1100, 256), (1000, 260, 4099)])
def test_i8_matmul(dtype, m, n, k):
    a, b = i8((m, k), m + k), i8((n, k), n + k + 1)
    sa = torch.rand(m, generator=gen(3), device="cuda") * 1e-2
    sb = torch.rand(n, generator=gen(4), device="cuda") * 1e-2
    got = msb.i8_matmul(a, sa, b, sb, out_dtype=dtype)
    msb.sync_status()
    i8_check(a, sa, b, sb, dtype, got)


@pytest.mark.parametrize("m", [5, 300])
def test_i8_matmul_extremes_are_exact(m):
    # the largest sums of each sign, over the longest K: every value of the type is a factor
    k = 2 ** 17 - 1
    a = torch.full((m, k), -128, dtype=torch.int8, device="cuda")
    b = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    b[1] = 127
    b[2, ::2] = 127
    one = torch.ones(m, device="cuda"), torch.ones(3, device="cuda")
    got = msb.i8_matmul(a, one[0], b, one[1], out_dtype=FP32)
    want = (a.double() @ b.double().T).float()
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 9, 150, 400])
@pytest.mark.parametrize("pad,lead", [(16, 16), (5, 3)])
def test_i8_matmul_strided(m, pad, lead):
    n, k = 150, 272
    a, b = i8((m, k), 5), i8((n, k), 6)
    sa, sb = torch.rand(m, generator=gen(7), device="cuda"), torch.rand(n, generator=gen(8), device="cuda")
    out = view(torch.zeros((m, n), device="cuda", dtype=BF16), pad, lead)
    msb.i8_matmul(view(a, pad, lead), sa, view(b, pad, lead), sb, out=out)
    assert torch.equal(out, msb.i8_matmul(a, sa, b, sb))
    assert bool((out._base[:, lead + n:] == 3).all()) and bool((out._base[:, :lead] == 3).all())


def test_i8_matmul_empty():
    a, b = i8((4, 0), 1), i8((6, 0), 1)
    out = msb.i8_matmul(a, torch.ones(4, device="cuda"), b, torch.ones(6, device="cuda"))
    assert out.shape == (4, 6) and bool((out == 0).all())
    assert msb.i8_matmul(i8((0, 8), 1), torch.ones(0, device="cuda"), i8((6, 8), 1), torch.ones(6, device="cuda")).shape == (0, 6)


# ---------------------------------------------------------------- gated_ffn

FFN_SHAPES = [(1, 8, 1), (1, 64, 64), (1, 4096, 1024), (4, 1000, 333), (16, 64, 128), (17, 72, 200), (63, 136, 100),
              (100, 1001, 130), (256, 256, 320), (257, 128, 256), (300, 1000, 344), (513, 1003, 129), (700, 2048, 1024)]
ACTS = ["silu", "gelu", "gelu_tanh"]


def ffn_inputs(t, d, h, dtype, seed):
    return (randn((t, d), seed, dtype), randn((h, d), seed + 1, dtype, d ** -0.5), randn((h, d), seed + 2, dtype, d ** -0.5))


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,d,h", FFN_SHAPES)
def test_gated_ffn(dtype, act, t, d, h):
    x, wg, wu = ffn_inputs(t, d, h, dtype, 20)
    out, gate, up = msb.gated_ffn(x, wg, wu, activation=act, save=True)
    alone = msb.gated_ffn(x, wg, wu, activation=act)
    msb.sync_status()
    wh, g, u, eh, eg, eu = L.ffn(x, wg, wu, act)
    tiny = L.TINY[dtype]
    assert L.worst(out, wh, wh.abs() * L.U[dtype] + eh * (1 + L.U[dtype]) + tiny) <= 1
    assert L.worst(gate, g, g.abs() * L.U[dtype] + eg * (1 + L.U[dtype]) + tiny) <= 1
    assert L.worst(up, u, u.abs() * L.U[dtype] + eu * (1 + L.U[dtype]) + tiny) <= 1
    assert torch.equal(out, alone)


def ffn_grad_check(got, want, mags, facs, dtype, types, ks):
    for g, w, m, f, ty, k in zip(got, want, mags, facs, types, ks):
        # dg and du are rounded once (u), their activation is good to 2^-14, then the sum and the output's rounding.
        # Below the type's normal numbers dg and du are off by up to half of TINY in absolute terms instead (fp16: a
        # gate's tail of 1e-5 times dh is there), each times the operand that it meets: f sums those
        e = m * (L.U[dtype] + 2.0 ** -13 + L.acc_error(k)) + f * L.TINY[dtype] + L.TINY[ty]
        assert g.dtype == ty
        assert L.worst(g, w, w.abs() * L.U[ty] + e) <= 1
        # and as a whole: independent roundings of the operands and of the result
        assert float((g.double() - w).norm()) <= 2 * L.U[dtype] * float(w.norm()) + L.TINY[dtype] * float(f.norm()) * math.sqrt(g.shape[0])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("t,d,h", FFN_SHAPES)
def test_gated_ffn_backward(dtype, act, t, d, h):
    x, wg, wu = ffn_inputs(t, d, h, dtype, 30)
    gate, up, dh = randn((t, h), 33, dtype), randn((t, h), 34, dtype), randn((t, h), 35, dtype)
    grad = FP32 if t % 2 else dtype
    got = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, grad_dtype=grad)
    msb.sync_status()
    want, mags, facs = L.ffn_backward(dh, x, wg, wu, gate, up, act)
    ffn_grad_check(got, want, mags, facs, dtype, (dtype, grad, grad), (2 * h, t, t))
    again = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, grad_dtype=grad)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    dx, n1, n2 = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, need_dw=False)
    assert n1 is None and n2 is None and torch.equal(dx, got[0])
    n0, g1, g2 = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, grad_dtype=grad, need_dx=False)
    assert n0 is None and torch.equal(g1, got[1]) and torch.equal(g2, got[2])


@pytest.mark.parametrize("t", [3, 300])
@pytest.mark.parametrize("pad,lead", [(8, 8), (3, 1)])
def test_gated_ffn_strided(t, pad, lead):
    d, h = 200, 144
    x, wg, wu = ffn_inputs(t, d, h, BF16, 40)
    both = torch.cat([wg, wu])  # one matrix whose halves are the two projections
    wv = view(both, pad, lead)
    outs = [view(torch.zeros((t, h), device="cuda", dtype=BF16), pad, lead) for _ in range(3)]
    msb.gated_ffn(view(x, pad, lead), wv[:h], wv[h:], out=outs[0], gate_out=outs[1], up_out=outs[2])
    want = msb.gated_ffn(x, wg, wu, save=True)
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
        assert bool((o._base[:, lead + h:] == 3).all()) and bool((o._base[:, :lead] == 3).all())
    dh = randn((t, h), 43, BF16)
    dws = view(torch.zeros((2 * h, d), device="cuda", dtype=BF16), pad, lead)
    dx = view(torch.zeros((t, d), device="cuda", dtype=BF16), pad, lead)
    msb.gated_ffn_backward(view(dh, pad, lead), view(x, pad, lead), wv[:h], wv[h:], outs[1], outs[2], dx_out=dx,
                           dw_gate_out=dws[:h], dw_up_out=dws[h:])
    want = msb.gated_ffn_backward(dh, x, wg, wu, want[1], want[2])
    assert torch.equal(dx, want[0]) and torch.equal(dws[:h], want[1]) and torch.equal(dws[h:], want[2])
    for o, n in ((dx, d), (dws, d)):
        assert bool((o._base[:, lead + n:] == 3).all()) and bool((o._base[:, :lead] == 3).all())


def test_gated_ffn_large_pre_activations():
    # gates far outside exp's range on both sides: no NaN, the limits of the activations and of their derivatives
    d, h = 64, 64
    for act in ACTS:
        x = torch.ones((2, d), device="cuda", dtype=BF16)
        x[1] = -1
        wg = torch.full((h, d), 1e4, device="cuda", dtype=BF16)
        wu = torch.full((h, d), 0.5, device="cuda", dtype=BF16)
        out, gate, up = msb.gated_ffn(x, wg, wu, activation=act, save=True)
        assert torch.equal(out[0].float(), (gate[0].float() * 32).to(BF16).float()) and bool((out[1] == 0).all())
        dh = torch.ones_like(out)
        dx, dwg, dwu = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act)
        # row 0: act' = 1, row 1: 0, so dWg = up_0 x_0 and dWu = act(gate_0) x_0
        assert bool((dwg == 32).all()) and torch.equal(dwu[:, 0], gate[0])


def test_gated_ffn_nonfinite_tokens_stay_in_their_rows():
    for t in (5, 300):
        x, wg, wu = ffn_inputs(t, 128, 96, BF16, 50)
        clean = msb.gated_ffn(x, wg, wu)
        x[3, 7] = float("nan")
        out = msb.gated_ffn(x, wg, wu)
        keep = [i for i in range(t) if i != 3]
        assert bool(torch.isnan(out[3]).all()) and torch.equal(out[keep], clean[keep])


def test_gated_ffn_empty():
    z = lambda *s: torch.zeros(s, device="cuda", dtype=BF16)  # noqa: E731
    out, gate, up = msb.gated_ffn(z(4, 0), z(6, 0), z(6, 0), save=True)
    assert out.shape == (4, 6) and not bool(out.any() or gate.any() or up.any())
    assert msb.gated_ffn(z(0, 8), z(6, 8), z(6, 8)).shape == (0, 6)
    dwg, dwu = torch.ones((6, 8), device="cuda", dtype=BF16), torch.ones((6, 8), device="cuda", dtype=BF16)
    msb.gated_ffn_backward(z(0, 6), z(0, 8), z(6, 8), z(6, 8), z(0, 6), z(0, 6), dw_gate_out=dwg, dw_up_out=dwu)
    assert not bool(dwg.any() or dwu.any())
    dw = torch.ones(8, device="cuda")
    msb.rms_norm_backward(z(0, 8), z(0, 8), torch.ones(8, device="cuda"), dw_out=dw)
    assert not bool(dw.any())


def test_gated_ffn_gradients_against_differences():
    t, d, h = 260, 96, 80
    x, wg, wu = ffn_inputs(t, d, h, FP16, 60)
    dh = randn((t, h), 63, FP16)
    for act in ACTS:
        _, gate, up = msb.gated_ffn(x, wg, wu, activation=act, save=True)
        grads = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, activation=act, grad_dtype=FP32)
        f = lambda a, b, c: float((L.act(a @ b.T, act)[0] * (a @ c.T) * dh.double()).sum())  # noqa: E731
        args = [x.double(), wg.double(), wu.double()]
        for i, g in enumerate(grads):
            v = randn(tuple(g.shape), 70 + i, FP32).double()
            up_, dn = list(args), list(args)
            up_[i], dn[i] = args[i] + 1e-6 * v, args[i] - 1e-6 * v
            diff = (f(*up_) - f(*dn)) / 2e-6
            # the kept gate and up and the operands dg and du are rounded to fp16: 4 u of what is summed
            assert abs(float((g.double() * v).sum()) - diff) <= 4 * L.U[FP16] * float((g.double() * v).abs().sum())


# ---------------------------------------------------------------- together

def layer_step(x, r, w, wg, wu, mom, dh):
    y, s = msb.rms_norm(x, w, r)
    h, gate, up = msb.gated_ffn(y, wg, wu, save=True)
    dy, dwg, dwu = msb.gated_ffn_backward(dh, y, wg, wu, gate, up)
    dx, dw = msb.rms_norm_backward(dy, s, w)
    msb.muon_step([wg, wu], mom, [dwg, dwu])
    return h, dx, dw


def test_a_training_step_of_the_block():
    t, d, h = 300, 256, 512
    x, r, w = randn((t, d), 80, BF16), randn((t, d), 81, BF16), randn((d,), 82, FP32)
    wg, wu = randn((h, d), 83, BF16, d ** -0.5), randn((h, d), 84, BF16, d ** -0.5)
    dh = randn((t, h), 85, BF16)
    mom = [torch.zeros((h, d), device="cuda") for _ in range(2)]
    w0 = [wg.clone(), wu.clone()]
    out, dx, dw = layer_step(x, r, w, wg, wu, mom, dh)
    msb.sync_status()
    # the same chain in 64 bits from the inputs
    s = (x.float() + r.float()).to(BF16).double()
    y = L.rms(s, w, 1e-6)
    want = L.act(y @ w0[0].double().T, "silu")[0] * (y @ w0[1].double().T)
    u = L.U[BF16]
    assert float((out.double() - want).norm()) <= 4 * u * float(want.norm())  # y, then h: two roundings, gate and up apart
    g, up = y @ w0[0].double().T, y @ w0[1].double().T
    (wy, wdg, wdu), _, _ = L.ffn_backward(dh, y, w0[0], w0[1], g, up, "silu")
    wx, ww, _, _ = L.rms_backward(wy, s, w, None, 1e-6)
    for got, ref in ((dx, wx), (dw, ww)):
        assert float((got.double() - ref).norm()) <= 8 * u * float(ref.norm())  # eight roundings on the way
    for m, ref in zip(mom, (wdg, wdu)):
        assert float((m.double() - ref).norm()) <= 8 * u * float(ref.norm())
    assert all(not torch.equal(a, b) for a, b in zip((wg, wu), w0))


def test_the_int8_path_of_a_projection():
    t, d, n = 70, 1024, 640
    x, r, w = randn((t, d), 86, FP16), randn((t, d), 87, FP16), randn((d,), 88, FP16)
    weight = randn((n, d), 89, FP32, d ** -0.5)
    sb = weight.abs().amax(1) / 127
    b = torch.round(weight / sb[:, None]).to(torch.int8)
    q, scale, s = msb.rms_norm_q8(x, w, r)
    out = msb.i8_matmul(q, scale, b, sb, out_dtype=FP16)
    msb.sync_status()
    i8_check(q, scale, b, sb, FP16, out)
    want = L.rms(s, w, 1e-6) @ weight.double().T
    # each factor is off by up to half a step of max / 127: its variance is a twelfth of a step squared
    y = L.rms(s, w, 1e-6)
    rel = math.sqrt(float(((y.abs().amax(1) / 127) ** 2 / 12 / (y * y).mean(1)).mean() + (sb.double() ** 2 / 12 / (weight.double() ** 2).mean(1)).mean()))
    assert float((out.double() - want).norm()) <= 1.5 * rel * float(want.norm())


def test_two_streams_and_a_captured_graph():
    t, d, h = 64, 256, 320
    sets = []
    for i in range(2):
        x, wg, wu = ffn_inputs(t + 250 * i, d, h, BF16, 90 + 10 * i)
        w, dh = randn((d,), 95 + 10 * i, FP32), randn((t + 250 * i, h), 96 + 10 * i, BF16)
        sets.append((x, wg, wu, w, dh))

    def run(x, wg, wu, w, dh):
        y, _ = msb.rms_norm(x, w, x)
        out, gate, up = msb.gated_ffn(y, wg, wu, save=True)
        dy, dwg, dwu = msb.gated_ffn_backward(dh, y, wg, wu, gate, up)
        dx, dw = msb.rms_norm_backward(dy, x, w)
        q, sc = msb.rms_norm_q8(y)
        z = msb.i8_matmul(q, sc, q, sc)
        return [out, dy, dwg, dwu, dx, dw, z]

    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = []
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            got.append([run(*s) for _ in range(3)][-1])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = run(*s)
        graphs.append((g, o))
    for _ in range(2):
        for g, o in graphs:
            for v in o:
                v.zero_()
            g.replay()
    torch.cuda.synchronize()
    for a, (_, b) in zip(want, graphs):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    msb.sync_status()


def test_explicit_streams_and_more_dims():
    x, wg, wu = ffn_inputs(24, 64, 96, BF16, 200)
    w, dh = randn((64,), 203, BF16), randn((24, 96), 204, BF16)
    q, b = i8((24, 64), 205), i8((40, 64), 206)
    sa, sb = torch.rand(24, device="cuda"), torch.rand(40, device="cuda")

    def run(v, **kw):
        """The operators on inputs whose leading dims are those of v(tensor)."""
        y, s = msb.rms_norm(v(x), w, v(x), **kw)
        qq, sc, _ = msb.rms_norm_q8(x=v(x), weight=w, residual=v(x), **kw)
        dx, dw = msb.rms_norm_backward(v(x), v(x), w, dsum=v(x), **kw)
        z = msb.i8_matmul(v(q), v(sa), b, sb, **kw)
        h, g, u = msb.gated_ffn(v(x), wg, wu, save=True, **kw)
        return [y, s, qq, sc, dx, dw, z, h, g, u, *msb.gated_ffn_backward(v(dh), v(x), wg, wu, g, u, **kw)]

    want = run(lambda t: t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        got = run(lambda t: t, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for shape in ((2, 3, 4), (4, 6)):
        got = run(lambda t: t.view(shape + t.shape[1:]))
        assert got[0].shape == shape + (64,) and got[3].shape == shape and got[6].shape == shape + (40,)
        assert all(torch.equal(a, c.view(a.shape)) for a, c in zip(want, got))
    # a single row without a leading dim
    y, dw = msb.rms_norm(x[3], w), msb.rms_norm_backward(x[3], x[3], w)[1]
    assert y.shape == (64,) and dw.shape == (64,)
    q1, s1 = msb.rms_norm_q8(x[3], w, scale_out=torch.empty((), device="cuda"))
    assert s1.shape == () and msb.i8_matmul(q1, s1, b, sb).shape == (40,)
    assert torch.equal(msb.gated_ffn(x[3], wg, wu), msb.gated_ffn(x[3:4], wg, wu)[0])


def test_rows_beyond_32_bit_offsets():
    # three rows 2^30 elements apart (the last at 2^31), and the same rows side by side
    big = torch.empty(2 ** 31 + 4096, dtype=BF16, device="cuda")
    far = lambda off, n: torch.as_strided(big, (3, n), (2 ** 30, 1), off)  # noqa: E731
    x, dh = randn((3, 64), 210, BF16), randn((3, 96), 211, BF16)
    wg, wu = randn((96, 64), 212, BF16, 0.1), randn((96, 64), 213, BF16, 0.1)
    xf, df = far(0, 64), far(64, 96)
    xf.copy_(x), df.copy_(dh)
    w = randn((64,), 214, FP32)
    y, s = msb.rms_norm(x, w, x)
    yf, sf = msb.rms_norm(xf, w, xf, out=far(256, 64), sum_out=far(320, 64))
    assert torch.equal(y, yf) and torch.equal(s, sf)
    assert torch.equal(msb.rms_norm_backward(x, x, w)[0], msb.rms_norm_backward(xf, xf, w, dx_out=far(384, 64))[0])
    h, g, u = msb.gated_ffn(x, wg, wu, save=True)
    hf, gf, uf = msb.gated_ffn(xf, wg, wu, out=far(512, 96), gate_out=far(640, 96), up_out=far(768, 96))
    assert torch.equal(h, hf) and torch.equal(g, gf) and torch.equal(u, uf)
    a = msb.gated_ffn_backward(dh, x, wg, wu, g, u)
    c = msb.gated_ffn_backward(df, xf, wg, wu, gf, uf, dx_out=far(1024, 64))
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    # 600 rows through the kernels of many rows: out rows 2^22 elements apart
    x6 = randn((600, 64), 215, BF16)
    of = torch.as_strided(big, (512, 96), (2 ** 22, 1), 0)
    msb.gated_ffn(x6[:512], wg.repeat(64, 1)[:96], wu, out=of)
    assert torch.equal(of, msb.gated_ffn(x6[:512], wg, wu))
    wide = randn((96 * 70, 64), 216, BF16, 0.1)
    of = torch.as_strided(big, (512, 96 * 70), (2 ** 22, 1), 0)
    msb.gated_ffn(x6[:512], wide, wide, out=of)
    assert torch.equal(of, msb.gated_ffn(x6[:512], wide, wide))


def test_a_given_workspace_and_a_small_one():
    x, wg, wu = ffn_inputs(40, 73, 50, FP16, 220)  # rows that have to be copied
    need = msb.gated_ffn_workspace_size(x, wg, wu)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(msb.gated_ffn(x, wg, wu, workspace=ws), msb.gated_ffn(x, wg, wu))
    with pytest.raises(msb.MsignError):
        msb.gated_ffn(x, wg, wu, workspace=ws[: need - 256])
    a, b = i8((40, 73), 221), i8((50, 73), 222)
    ws = torch.empty(msb.i8_matmul_workspace_size(a, b), dtype=torch.uint8, device="cuda")
    one = torch.ones(50, device="cuda")
    assert torch.equal(msb.i8_matmul(a, one[:40], b, one, workspace=ws), msb.i8_matmul(a, one[:40], b, one))
    # a workspace that holds anything is fine: no call reads what an earlier one left
    dh, gate, up = (randn((40, 50), s, FP16) for s in (223, 224, 225))
    ws = torch.full((msb.gated_ffn_backward_workspace_size(x, wg, wu),), 255, dtype=torch.uint8, device="cuda")
    got = msb.gated_ffn_backward(dh, x, wg, wu, gate, up, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(got, msb.gated_ffn_backward(dh, x, wg, wu, gate, up)))
    s, dy, w = randn((40, 4096), 226, FP16), randn((40, 4096), 227, FP16), randn((4096,), 228, FP16)
    ws = torch.full((msb.rms_norm_backward_workspace_size(40, 4096),), 255, dtype=torch.uint8, device="cuda")
    got = msb.rms_norm_backward(dy, s, w, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(got, msb.rms_norm_backward(dy, s, w)))


def test_the_largest_tiles_and_many_splits():
    # shapes that reach every tile width and split of the few-row kernel, against the integer product
    one = torch.ones(4200, device="cuda")
    for m, n, k in ((1, 128, 8192), (16, 256, 4096), (30, 640, 2048), (64, 128, 16384), (65, 640, 4096), (100, 128, 9000),
                    (129, 300, 2048), (150, 1000, 4096), (208, 512, 6000), (256, 256, 512), (300, 640, 2048),
                    (450, 1000, 1024), (1500, 128, 300), (2500, 256, 4096)):
        a, b = i8((m, k), m), i8((n, k), n)
        got = msb.i8_matmul(a, one[:m], b, one[:n], out_dtype=FP32)
        assert torch.equal(got, (a.double() @ b.double().T).float()), (m, n, k)


@pytest.mark.parametrize("t,d,h", [(4000, 256, 256), (2100, 300, 200), (2048, 1000, 512), (200, 3000, 96), (1, 512, 8192)])
def test_gated_ffn_backward_long_and_wide(t, d, h):
    # long sums of the weight gradients (the split form), and outputs much wider than they are high
    x, wg, wu = ffn_inputs(t, d, h, BF16, 230)
    gate, up, dh = randn((t, h), 233, BF16), randn((t, h), 234, BF16), randn((t, h), 235, BF16)
    got = msb.gated_ffn_backward(dh, x, wg, wu, gate, up)
    want, mags, facs = L.ffn_backward(dh, x, wg, wu, gate, up, "silu")
    ffn_grad_check(got, want, mags, facs, BF16, (BF16, BF16, BF16), (2 * h, t, t))


@pytest.mark.parametrize("t", [5, 300])
def test_rows_behind_the_last_stay(t):
    # outputs that are the first rows of larger tensors, in every kernel's range
    def room(shape, dtype=BF16):
        big = torch.full((shape[0] + 40, shape[1]), 5.0, device="cuda").to(dtype)
        return big, big[:shape[0]]

    x, wg, wu = ffn_inputs(t, 136, 264, BF16, 300)
    dh, w = randn((t, 264), 303, BF16), randn((136,), 304, FP32)
    bigs = []

    def new(*shape, dtype=BF16):
        big, v = room(shape, dtype)
        bigs.append((big, shape[0]))
        return v

    s = new(t, 136)
    msb.rms_norm(x, w, x, out=new(t, 136), sum_out=s)
    msb.rms_norm_q8(x, w, out=new(t, 136, dtype=torch.int8))
    msb.rms_norm_backward(x, s, w, dx_out=new(t, 136))
    g, u = new(t, 264), new(t, 264)
    msb.gated_ffn(x, wg, wu, out=new(t, 264), gate_out=g, up_out=u)
    msb.gated_ffn_backward(dh, x, wg, wu, g, u, dx_out=new(t, 136), dw_gate_out=new(264, 136), dw_up_out=new(264, 136))
    q = i8((t, 136), 305)
    one = torch.ones(t, device="cuda")
    for dtype in (BF16, FP32):
        msb.i8_matmul(q, one, q, one, out=new(t, t, dtype=dtype))
    msb.sync_status()
    for big, rows in bigs:
        assert bool((big[rows:] == 5).all()) and not bool((big[:rows] == 5).all())
