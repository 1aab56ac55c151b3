"""How the layer operators' binding and C entry points take their arguments,
without a GPU: streams by keyword, buffers that share memory, addresses, and
the launch plans of the widest rows."""

import contextlib
import os
import re
import shutil
import subprocess
import sys

import pytest
import torch

import newton_schulz_msign_b200 as msb
from newton_schulz_msign_b200 import _lib, build


CSRC = os.path.join(os.path.dirname(msb.__file__), "csrc")


class Placed(torch.Tensor):
    """A host tensor that says that it lies on a device."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


def placed(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(Placed)


class Reached(Exception):
    pass


def stream_calls():
    x, w, v = placed(4, 8), placed(6, 8), placed(8)
    q, one = placed(4, 8, dtype=torch.int8), placed(4, dtype=torch.float32)
    return {
        "norm, a number first": (msb.rms_norm, (), dict(eps=1e-5, x=x)),
        "norm, None first": (msb.rms_norm, (), dict(weight=None, x=x)),
        "norm, a weight first": (msb.rms_norm, (), dict(weight=v, x=x)),
        "norm, by position": (msb.rms_norm, (x, v), dict(eps=1e-5)),
        "norm to int8, an output first": (msb.rms_norm_q8, (), dict(scale_out=None, eps=1e-6, x=x)),
        "norm gradients, a number first": (msb.rms_norm_backward, (), dict(eps=1e-5, s=x, dy=x)),
        "int8 product, a type first": (msb.i8_matmul, (), dict(out_dtype=torch.float32, b=q, a=q, a_scale=one, b_scale=one)),
        "gated block, a name first": (msb.gated_ffn, (), dict(activation="gelu", x=x, w_gate=w, w_up=w)),
        "gated block, a flag first": (msb.gated_ffn, (), dict(save=True, w_gate=w, w_up=w, x=x)),
        "gradients, a flag first": (msb.gated_ffn_backward, (), dict(need_dx=False, x=x, dh=x, w_gate=w, w_up=w, gate=x, up=x)),
    }


@pytest.mark.parametrize("name", list(stream_calls()))
def test_the_stream_is_entered_whatever_argument_comes_first(monkeypatch, name):
    entered = []

    class Stream:
        device = torch.device("cuda", 0)

    @contextlib.contextmanager
    def enter(stream):
        entered.append(stream)
        yield
        entered.pop()

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", enter)
    op, args, kwargs = stream_calls()[name]
    stream = Stream()
    seen = []

    def reached_in(*a, **kw):
        seen.append(list(entered))
        raise Reached

    monkeypatch.setattr(msb, "_dtype_code", reached_in)
    monkeypatch.setattr(msb, "_rows_layout", reached_in)
    with pytest.raises(Reached):
        op(*args, stream=stream, **kwargs)
    assert seen == [[stream]]


def test_a_stream_without_a_device_tensor_is_refused():
    for f in (lambda: msb.rms_norm(eps=1e-5, x=torch.zeros(4, 8), stream=5), lambda: msb.rms_norm(torch.zeros(4, 8), stream=5),
              lambda: msb.rms_norm(weight=None, stream=5)):
        with pytest.raises(ValueError, match="x must be a CUDA tensor"):
            f()


def test_edge_elements_are_published_in_order():
    # The lanes of a warp store a row's edge elements, one lane arrives on the barrier that the readers wait for: between
    # the two every path needs a barrier of the warp that orders memory (shuffles and reductions order none).  No run
    # shows it, since one warp's stores happen to land in order.
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "norm_sm100.cuh")).read())
    fill = text[text.index("const auto fill = "):]
    stores = [m.end() for m in re.finditer(r"d\[c\] = src\[c\];", fill)]
    arrive = fill.index("mbar_arrive_expect_tx", stores[-1])
    assert len(stores) == 2 and "__syncwarp();" in fill[stores[-1]:arrive]


# ---------------------------------------------------------------- launch plans

PIECES, ELEMS, LOOP, LOOP_SUMS = range(4)
RING_BYTES, DW_PARTS = 232448 - 2048, 592


@pytest.fixture(scope="module")
def norm_plans(tmp_path_factory):
    """The plans of a list of (rows, cols, bytes of an element, whole pieces, shifted pieces, elements an access)."""
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("plan") / "norm_plan")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c", "norm_plan.cpp")
    subprocess.run([compiler, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-static-libubsan", "-I", CSRC, src, "-o", exe], check=True)

    def plans(cases):
        run = subprocess.run([exe], input="\n".join(" ".join(str(int(v)) for v in c) for c in cases), capture_output=True,
                             text=True, timeout=60)
        assert run.returncode == 0, run.stderr
        return [tuple(int(v) for v in line.split()) for line in run.stdout.splitlines()]

    return plans


def reaches(cols, es):
    """How rows of this width may be reached: whole pieces, shifted pieces, elements by two and one."""
    if cols % (16 // es) == 0:
        yield 1, 0, 2
    if cols >= 32 * (16 // es):
        yield 0, 1, 1 + (cols % 2 == 0)
    yield 0, 0, 1 + (cols % 2 == 0)


@pytest.mark.parametrize("es", [2, 4])
def test_the_widest_rows_take_the_loop(norm_plans, es):
    # rows of 2^31 and 2^32 bytes: their size does not fit 32 bits
    cases = [(rows, cols, es) + by for cols in (2 ** 28, 2 ** 29 - 8, 2 ** 29, 2 ** 29 + 1, 2 ** 30 - 8, 2 ** 30 - 6, 2 ** 30 - 1, 2 ** 30)
             for rows in (1, 3) for by in reaches(cols, es)]
    for c, p in zip(cases, norm_plans(cases)):
        assert p[0] == LOOP and p[4] == LOOP and p[2:4] == p[6:8] == (256, 1), (c, p)


@pytest.mark.parametrize("es", [2, 4])
def test_every_plan_holds_its_rows(norm_plans, es):
    widths = sorted({w for n in (1, 8, 32, 64, 101, 128, 256, 257, 500, 1000, 1024, 2048, 2730, 3000, 4096, 6144, 8192, 10240, 12000,
                                 16384, 20000, 32768, 40000, 10 ** 6) for w in (n - 1, n, n + 1, n + 8) if w > 0})
    cases = [(rows, cols, es) + by for cols in widths for rows in (1, 2, 7, 64, 777, 1184, 1185, 8192, 10 ** 6) for by in reaches(cols, es)]
    plans = norm_plans(cases)
    assert len(plans) == len(cases)
    for c, p in zip(cases, plans):
        rows, cols, _, vec, shift, pair = c
        # the 16-byte units that a row can touch, in bytes
        row = (cols * es + 31 - es) // 16 * 16 if shift else cols * es
        form, vpt, x, y = p[:4]
        assert x % 32 == 0 and x * y <= 1024 and (y == 1 or x == 32), (c, p)
        assert {PIECES: x * vpt * 16 >= row, ELEMS: x * 8 * pair >= cols, LOOP: (x, y) == (256, 1)}[form], (c, p)
        form, vpt, x, y, full, slot, stages, parts = p[4:]
        if form == PIECES:
            assert x * vpt * 16 >= row and x * y <= (256 if vpt <= 2 else 512) and x % 32 == 0, (c, p)
            assert slot == 3 * y * row and 2 <= stages <= 8 and stages * slot <= RING_BYTES, (c, p)
            assert 1 <= parts <= min(rows, DW_PARTS) and y * cols * 4 <= stages * slot, (c, p)
            # whole blocks where the plan says so, and one phase a thread where rows are shifted
            assert not full or (rows % y == 0 and x * vpt * 16 == row)
            assert not shift or parts * y >= rows or parts * y % (16 // es) == 0, (c, p)
        elif form == ELEMS:
            assert x * 8 * pair >= cols and x * y <= 512, (c, p)
        elif form == LOOP_SUMS:
            assert cols <= 12000 and 1 <= parts <= min(rows, DW_PARTS), (c, p)


# ---------------------------------------------------------------- buffers that share memory

B, H, F = _lib.BF16, _lib.FP16, _lib.FP32
BAD, OK = _lib.ERR_INVALID_ARG, _lib.OK


def at(i):
    """An address that no refused call touches."""
    return (1 << 20) + (i << 16)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


@pytest.mark.parametrize("out", [0, 1, 2, 3])
def test_i8_matmul_refuses_an_input_as_its_output(lib, out):
    # (fp32 out of the operands' size in bytes fits either of them)
    assert lib.i8_matmul(at(0), at(1), at(2), at(3), at(out), F, 4, 64, 256, 0, 0, 0, None, 0, None) == BAD


@pytest.mark.parametrize("scale", [0, 1, 2, 3, 4])
def test_rms_norm_q8_refuses_another_buffer_as_its_scales(lib, scale):
    assert lib.rms_norm_q8(at(0), at(1), at(2), at(3), at(scale), at(4), F, F, 4, 64, 0, 0, 0, 0, 1e-6, None) == BAD


IN_PLACE = [  # over which input, with which strides (x, residual, y, sum)
    (dict(y=0), (0, 0, 72, 0)), (dict(y=0), (72, 0, 0, 0)), (dict(y=1), (0, 80, 72, 0)), (dict(y=1), (72, 0, 72, 0)),
    (dict(s=0), (0, 0, 0, 72)), (dict(s=0), (80, 0, 0, 72)), (dict(s=1), (0, 72, 0, 0)), (dict(s=1), (72, 0, 0, 72))]


def in_place_status(lib, outs, strides, rows, q8=False):
    y, s = at(outs.get("y", 3)), at(outs.get("s", 4))
    if q8:
        return lib.rms_norm_q8(at(0), at(1), at(2), y, at(5), s, B, B, rows, 64, *strides, 1e-6, None)
    return lib.rms_norm(at(0), at(1), at(2), y, s, B, B, rows, 64, *strides, 1e-6, None)


@pytest.mark.parametrize("outs,strides", IN_PLACE)
def test_rms_norm_in_place_needs_the_inputs_row_stride(lib, outs, strides):
    assert in_place_status(lib, outs, strides, 4) == BAD
    if "s" in outs:
        assert in_place_status(lib, outs, strides, 4, q8=True) == BAD


BIG = 1 << 24  # bytes enough for any of these workspaces


@pytest.mark.parametrize("ws", range(6))
def test_a_workspace_at_another_buffer_is_refused(lib, ws):
    # (where the call needs one: rows of 65 elements have to be copied)
    assert lib.rms_norm_backward(*(at(i) for i in range(6)), B, B, 4, 64, 0, 0, 0, 0, 1e-6, at(ws), BIG, None) == BAD
    if ws < 5:
        assert lib.i8_matmul(*(at(i) for i in range(5)), B, 4, 64, 65, 0, 0, 0, at(ws), BIG, None) == BAD
    assert lib.gated_ffn(*(at(i) for i in range(6)), B, 0, 4, 65, 64, 0, 0, 0, 0, at(ws), BIG, None) == BAD
    for i in (0, 3):  # any of the nine
        assert lib.gated_ffn_backward(*(at(j) for j in range(9)), B, B, 0, 4, 64, 64, 0, 0, 0, 0, 0, 0, at(ws + i), BIG, None) == BAD


# ---------------------------------------------------------------- addresses between elements

def norm_at(lib, i, off, io=B, wd=F, q8=False):
    """The norm with its i-th buffer (x, residual, weight, y, sum, scales) `off` bytes further on."""
    p = [at(j) + (off if j == i else 0) for j in range(6)]
    if q8:
        return lib.rms_norm_q8(p[0], p[1], p[2], p[3], p[5], p[4], io, wd, 4, 64, 0, 0, 0, 0, 1e-6, None)
    return lib.rms_norm(*p[:5], io, wd, 4, 64, 0, 0, 0, 0, 1e-6, None)


@pytest.mark.parametrize("i", range(5))
def test_rms_norm_refuses_addresses_between_elements(lib, i):
    assert norm_at(lib, i, 1) == BAD and norm_at(lib, i, 2, io=F) == BAD
    if i != 3:
        assert norm_at(lib, i, 1, q8=True) == BAD
    if i == 2:  # the weight's own type counts
        assert norm_at(lib, i, 2) == BAD
    assert norm_at(lib, 5, 2, q8=True) == BAD


@pytest.mark.parametrize("i", range(6))
def test_rms_norm_backward_refuses_addresses_between_elements(lib, i):
    p = [at(j) + (1 if j == i else 0) for j in range(6)]  # dy, s, w, dsum, dx, dw
    size = lib.rms_norm_backward_workspace_size(4, 64)
    assert lib.rms_norm_backward(*p, B, B, 4, 64, 0, 0, 0, 0, 1e-6, at(6), size, None) == BAD


@pytest.mark.parametrize("i,off", [(1, 2), (3, 2), (4, 1)])
def test_i8_matmul_refuses_addresses_between_elements(lib, i, off):
    p = [at(j) + (off if j == i else 0) for j in range(5)]
    assert lib.i8_matmul(*p, B, 4, 64, 256, 0, 0, 0, None, 0, None) == BAD


@pytest.mark.parametrize("i", range(9))
def test_gated_ffn_refuses_addresses_between_elements(lib, i):
    p = [at(j) + (1 if j == i else 0) for j in range(9)]
    big = 1 << 20
    if i < 6:  # x, the weights, out, gate, up
        assert lib.gated_ffn(*p[:6], B, 0, 4, 64, 64, 0, 0, 0, 0, at(9), big, None) == BAD
    # dh, x, the weights, gate, up, dx, the weights' gradients
    assert lib.gated_ffn_backward(*p, B, B, 0, 4, 64, 64, 0, 0, 0, 0, 0, 0, at(9), big, None) == BAD


# ---------------------------------------------------------------- the package

@pytest.mark.parametrize("flags", [[], ["-O"], ["-OO"]])
def test_the_package_imports_without_docstrings(flags):
    root = os.path.dirname(os.path.dirname(msb.__file__))
    run = subprocess.run([sys.executable, *flags, "-c", "import newton_schulz_msign_b200 as m; m.rms_norm, m.gated_ffn"],
                         cwd=root, capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr


def test_the_current_stream_without_torchs_own_lookup(monkeypatch):
    class Current:
        cuda_stream = 1234

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Current())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(msb, "_torch_module", None)
    monkeypatch.setattr(msb, "_raw_stream", None, raising=False)

    class On:
        def get_device(self):
            return 0

    assert msb._call(lambda *a: a, On(), "x") == ("x", 1234)
