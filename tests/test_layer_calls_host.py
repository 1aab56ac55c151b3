"""How the layer operators' binding and C entry points take their arguments,
without a GPU: streams by keyword, buffers that share memory, addresses, and
the launch plans of the widest rows."""

import contextlib
import os
import re

import pytest
import torch

import newton_schulz_msign_b200 as msb


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
