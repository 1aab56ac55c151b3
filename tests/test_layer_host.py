"""Refusals and host-side queries of the layer operators: no call here reaches
a device, so these run without a GPU."""

import ctypes

import pytest
import torch

import newton_schulz_msign_b200 as msb
from newton_schulz_msign_b200 import _lib, build

B, H, F = _lib.BF16, _lib.FP16, _lib.FP32
BAD, UNS, WS, OK = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE, _lib.OK
P = 1 << 20  # an address that no refused call touches


def at(i):
    """Another such address."""
    return P + (i << 16)



@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def norm(lib, x=P, r=None, w=at(1), y=at(2), s=None, io=B, wd=B, rows=4, cols=64, xs=0, rs=0, ys=0, ss=0, eps=1e-6):
    return lib.rms_norm(x, r, w, y, s, io, wd, rows, cols, xs, rs, ys, ss, eps, None)


@pytest.mark.parametrize("kw,status", [
    (dict(io=7), BAD), (dict(wd=-1), BAD), (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(eps=-1e-6), BAD),
    (dict(eps=float("nan")), BAD), (dict(eps=float("inf")), BAD), (dict(xs=63), BAD), (dict(rs=-1), BAD), (dict(ys=1), BAD),
    (dict(ss=63), BAD), (dict(s=P), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(wd=H), UNS), (dict(io=F, wd=B), UNS),
    (dict(rows=2 ** 30 + 1), UNS), (dict(cols=2 ** 30 + 1), UNS), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(rows=0, x=None, y=None), OK), (dict(r=at(3), s=at(2)), BAD), (dict(w=at(2)), BAD), (dict(r=at(3), s=at(1)), BAD)])
def test_rms_norm_statuses(lib, kw, status):
    assert norm(lib, **kw) == status


def test_rms_norm_q8_statuses(lib):
    call = lambda scale=at(3), rows=4, q=at(2): lib.rms_norm_q8(P, None, at(1), q, scale, None, B, B, rows, 64, 0, 0, 0, 0, 1e-6, None)  # noqa: E731
    assert call(scale=None) == BAD and call(q=None) == BAD and call(rows=0, scale=None) == OK and call(q=P) == BAD


def test_rms_norm_backward_statuses(lib):
    need = lib.rms_norm_backward_workspace_size(4, 64)
    assert need > 4 * 64 * 4 and lib.rms_norm_backward_workspace_size(0, 64) == 0
    # the partial sums do not grow with the rows beyond a fixed number of blocks
    assert lib.rms_norm_backward_workspace_size(10 ** 6, 64) < 4 * 10 ** 6 + 2 ** 20

    def call(dy=P, s=at(1), w=at(2), ds=None, dx=at(3), dw=at(4), io=B, wd=B, rows=4, cols=64, st=(0, 0, 0, 0), eps=1e-6, ws=P, wsb=need):
        return lib.rms_norm_backward(dy, s, w, ds, dx, dw, io, wd, rows, cols, *st, eps, ws, wsb, None)

    assert call(dy=None) == BAD and call(s=None) == BAD and call(dx=None) == BAD and call(io=9) == BAD
    assert call(eps=-1.0) == BAD and call(rows=-2) == BAD and call(wd=H) == UNS and call(rows=2 ** 31) == UNS
    for i in range(4):
        assert call(st=tuple(32 if j == i else 0 for j in range(4))) == BAD
    assert call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=P + 16) == WS
    assert call(cols=0) == OK and call(rows=0, dw=None) == OK
    assert call(dx=P) == BAD and call(dx=at(1)) == BAD and call(ds=at(5), dx=at(5)) == BAD and call(dw=at(2)) == BAD and call(dw=at(3)) == BAD


def test_i8_matmul_statuses(lib):
    size = lambda m=4, n=64, k=64, a=P, sa=0, b=P, sb=0: lib.i8_matmul_workspace_size(m, n, k, a, sa, b, sb)  # noqa: E731
    assert size() == 0 and size(k=0) == 0
    assert size(k=65) >= 80 * (4 + 64) and size(m=1, n=1, k=65) == 0  # one row needs no stride
    assert size(a=P + 1) >= 4 * 64 and size(b=P + 8) >= 64 * 64 and size(sb=72) >= 64 * 64 and size(sb=80) == 0

    def call(a=P, sa=P, b=P, sb=P, out=P, dt=B, m=4, n=64, k=64, st=(0, 0, 0), ws=None, wsb=0):
        return lib.i8_matmul(a, sa, b, sb, out, dt, m, n, k, *st, ws, wsb, None)

    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(dt=5), dict(m=-1), dict(n=-1),
               dict(k=-1), dict(st=(63, 0, 0)), dict(st=(0, 63, 0)), dict(st=(0, 0, 63)), dict(st=(-64, 0, 0))):
        assert call(**kw) == BAD, kw
    assert call(m=2 ** 30, n=2 ** 30, k=16) == UNS  # more tiles than the kernels count
    assert call(k=2 ** 17) == UNS and call(m=2 ** 30 + 1) == UNS and call(n=2 ** 30 + 1) == UNS
    assert call(k=65) == WS and call(k=65, ws=P, wsb=size(k=65) - 1) == WS and call(k=65, ws=P + 128, wsb=1 << 20) == WS
    assert call(m=0) == OK and call(n=0, out=None) == OK


def ffn_args(lib, **kw):
    d = dict(x=P, wg=at(1), wu=at(2), out=at(3), g=None, u=None, dt=B, act=0, t=4, d=64, h=64, st=(0, 0, 0, 0), ws=None, wsb=0)
    d.update(kw)
    return lib.gated_ffn(d["x"], d["wg"], d["wu"], d["out"], d["g"], d["u"], d["dt"], d["act"], d["t"], d["d"], d["h"],
                         *d["st"], d["ws"], d["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(wg=None), BAD), (dict(wu=None), BAD), (dict(out=None), BAD), (dict(g=P), BAD), (dict(u=P), BAD),
    (dict(dt=3), BAD), (dict(act=3), BAD), (dict(act=-1), BAD), (dict(t=-1), BAD), (dict(d=-1), BAD), (dict(h=-1), BAD),
    (dict(st=(63, 0, 0, 0)), BAD), (dict(st=(0, 63, 0, 0)), BAD), (dict(st=(0, 0, 63, 0)), BAD), (dict(st=(0, 0, 0, 63)), BAD),
    (dict(dt=F), UNS), (dict(t=2 ** 30 + 1), UNS), (dict(d=2 ** 30 + 1), UNS), (dict(h=2 ** 30 + 1), UNS), (dict(t=2 ** 30, h=2 ** 30), UNS),
    (dict(d=65), WS), (dict(x=P + 2), WS), (dict(wu=P + 8), WS),
    (dict(out=P), BAD), (dict(out=at(1)), BAD), (dict(g=at(3), u=at(4)), BAD), (dict(g=at(4), u=at(4)), BAD), (dict(st=(65, 0, 0, 0)), WS), (dict(st=(0, 68, 0, 0)), WS),
    (dict(t=0), OK), (dict(h=0, out=None), OK)])
def test_gated_ffn_statuses(lib, kw, status):
    assert ffn_args(lib, **kw) == status


def test_gated_ffn_backward_statuses(lib):
    need = lib.gated_ffn_backward_workspace_size(4, 64, 64, P, 0, P, P, 0)
    assert need >= 4 * 4 * 64  # dg and du
    assert lib.gated_ffn_backward_workspace_size(4, 65, 64, P, 0, P, P, 0) >= need + 2 * 72 * (4 + 128)
    assert lib.gated_ffn_backward_workspace_size(0, 64, 64, P, 0, P, P, 0) == 0

    def call(dh=P, x=at(1), wg=at(2), wu=at(3), g=at(4), u=at(5), dx=at(6), dg=at(7), du=at(8), dt=B, gd=B, act=0, t=4, d=64, h=64, st=(0,) * 6, ws=P, wsb=need):
        return lib.gated_ffn_backward(dh, x, wg, wu, g, u, dx, dg, du, dt, gd, act, t, d, h, *st, ws, wsb, None)

    for kw in (dict(dh=None), dict(x=None), dict(wg=None), dict(wu=None), dict(g=None), dict(u=None), dict(dg=None),
               dict(du=None), dict(dx=None, dg=None, du=None), dict(dt=4), dict(gd=4), dict(act=9), dict(t=-1)):
        assert call(**kw) == BAD, kw
    for i in range(6):
        assert call(st=tuple(32 if j == i else 0 for j in range(6))) == BAD
    assert call(dt=F) == UNS and call(gd=H) == UNS and call(h=2 ** 30 + 1) == UNS
    assert call(ws=None) == WS and call(wsb=need - 1) == WS and call(ws=P + 64) == WS
    for kw in (dict(dx=P), dict(dx=at(1)), dict(dg=at(2)), dict(du=at(7)), dict(dg=at(6)), dict(du=at(5))):
        assert call(**kw) == BAD, kw
    assert call(d=0) == OK and call(t=0, dx=None, dg=P, du=P, h=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    q = torch.zeros(4, 64, dtype=torch.int8)
    for f in (lambda: msb.rms_norm(x), lambda: msb.rms_norm_q8(x), lambda: msb.rms_norm_backward(x, x),
              lambda: msb.gated_ffn(x, w, w), lambda: msb.gated_ffn_backward(x, x, w, w, x, x),
              lambda: msb.i8_matmul(q, torch.ones(4), q, torch.ones(4))):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()
    with pytest.raises(TypeError):
        msb.i8_matmul(x, torch.ones(4), q, torch.ones(4))
    with pytest.raises(TypeError):
        msb.rms_norm(x.double())
    with pytest.raises(ValueError, match="activation"):
        msb.gated_ffn(x, w, w, activation="relu")


@pytest.mark.parametrize("make,want", [
    (lambda: torch.empty(2, 3, 8), (6, 8, 0)), (lambda: torch.empty(8), (1, 8, 0)), (lambda: torch.empty(4, 20)[:, :8], (4, 8, 20)),
    (lambda: torch.empty(2, 3, 20)[..., 4:12], (6, 8, 20)), (lambda: torch.empty(6, 8)[::2], (3, 8, 16)),
    (lambda: torch.empty(5, 1), (5, 1, 0)), (lambda: torch.empty(1, 30)[:, :7], (1, 7, 0)), (lambda: torch.empty(0, 8), (0, 8, 0)),
    (lambda: torch.empty(8, 4).T, None), (lambda: torch.empty(1, 8).expand(3, 8), None),
    (lambda: torch.empty(4, 6, 8)[:, :3], None)])
def test_row_layouts(make, want):
    class OnDevice:  # the layout of a host tensor, as if it lay on a device
        def __init__(self, t):
            self.t, self.is_cuda, self.shape = t, True, t.shape

        def dim(self):
            return self.t.dim()

        def stride(self, d):
            return self.t.stride(d)

        def is_contiguous(self):
            return self.t.is_contiguous()

    t = OnDevice(make())
    if want is None:
        with pytest.raises(ValueError):
            msb._rows_layout(t, "t")
    else:
        assert msb._rows_layout(t, "t") == want
