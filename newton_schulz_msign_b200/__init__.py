"""B200 (sm_100a) Newton-Schulz msign: thin PyTorch binding of the C ABI.

Each function marshals tensors into the pointer/size arguments of the C entry
point of the same name (include/msign_b200.h) and enqueues it on the current
CUDA stream.  Every step of the computation runs in the library's kernels;
PyTorch only supplies device memory and the stream.  There is no CPU path:
calling these without the built library or without a CUDA tensor raises.
"""

from __future__ import annotations

import ctypes
import functools
import inspect
import math

from . import _lib
from ._lib import BF16, FP16, FP32, MsignError, check, make_coeffs

__all__ = [
    "MsignError", "msign_ns", "msign_ns_workspace_size", "msign_ns_route", "msign_ns_host",
    "msign_ns_host_workspace_size", "msign_ns_noalloc", "msign_ns_noalloc_max_bytes",
    "gram_xxt", "gram_xxt_workspace_size", "gram_ns",
    "gram_ns_workspace_size", "muon_step", "muon_step_workspace_size", "muon_step_route", "mousse_inv_root",
    "mousse_direction",
    "rms_norm", "rms_norm_q8", "rms_norm_backward", "rms_norm_backward_workspace_size",
    "i8_matmul", "i8_matmul_workspace_size",
    "gated_ffn", "gated_ffn_workspace_size", "gated_ffn_backward", "gated_ffn_backward_workspace_size",
    "sync_status", "selftest_timeout", "set_chaining", "library_path",
]


def library_path() -> str:
    return _lib.LIB_PATH


_torch_module = None
_dtype_codes = {}
_raw_stream = None


def _torch():
    """torch, imported on first use."""
    global _torch_module, _raw_stream
    if _torch_module is None:
        import torch

        _dtype_codes.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
        # The current stream's handle on a device.  torch's own lookup without a Stream object takes 0.07 us, the public
        # form 1.3 of a small call's 11; a torch that has none takes the public one.
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch_module = torch
    return _torch_module


def _dtype_code(t) -> int:
    _torch()
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _compute_code(name) -> int:
    return {"bf16": BF16, "fp16": FP16, "fp32": FP32}[name]


def _stream(stream, device=None) -> int:
    """The raw cudaStream_t: the given stream, else the current stream of
    ``device`` (of the current device when None)."""
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _need_cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _batch_layout(t, name):
    """(batch, rows, cols, stride) of a CUDA tensor whose last two dims are a
    dense row-major matrix and whose leading dims step through memory with
    one stride (any view of that form, e.g. ``big[:, 0]``); stride 0 means
    back to back."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dim() < 2:
        raise ValueError(f"{name} needs at least two dims")
    rows, cols = t.shape[-2], t.shape[-1]
    if rows * cols == 0:  # empty matrices have no layout to check
        return math.prod(t.shape[:-2]), rows, cols, 0
    if (cols > 1 and t.stride(-1) != 1) or (rows > 1 and t.stride(-2) != cols):
        raise ValueError(f"{name}: each matrix (the last two dims) must be dense row-major")
    lead = [(t.shape[d], t.stride(d)) for d in range(t.dim() - 2) if t.shape[d] != 1]
    batch = math.prod(sz for sz, _ in lead)
    if batch <= 1:
        return batch, rows, cols, 0
    stride = lead[-1][1]
    for (sz_o, st_o), (sz_i, st_i) in zip(lead[:-1], lead[1:]):
        if st_o != st_i * sz_i:
            raise ValueError(f"{name}: the batch dims must step through memory with one stride")
    if stride < rows * cols:
        raise ValueError(f"{name}: matrices of the batch overlap (stride {stride} < {rows * cols})")
    return batch, rows, cols, (0 if stride == rows * cols else stride)


def _same_device(t, device, name):
    """The C side works on the current device: every tensor of a call must
    live on the device the call runs on."""
    if t is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")


def _workspace(nbytes, device, workspace):
    torch = _torch()
    if workspace is not None:
        _same_device(workspace, device, "workspace")
    if nbytes == 0:
        return workspace, (0 if workspace is None else workspace.numel() * workspace.element_size())
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def _ptr(t):
    return None if t is None else t.data_ptr()


def sync_status(stream=None, device=None) -> None:
    """Waits for the stream (default: the current stream of ``device``, or of
    the current device) and raises MsignError if a kernel's bounded wait on
    that device ran out."""
    torch = _torch()
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        check(_lib.lib().msign_sync_status(_stream(stream, device)), "msign_sync_status")


# ---------------------------------------------------------------- msign_ns

def msign_ns_workspace_size(batch: int, rows: int, cols: int, compute: str = "bf16") -> int:
    return int(_lib.lib().msign_ns_workspace_size(batch, rows, cols, _compute_code(compute)))


_METHODS = {"standard": 0, "auto": 1}


def msign_ns_route(batch: int, rows: int, cols: int, compute: str = "bf16", *, method: str = "auto", coeffs=None,
                   improved_init=False) -> str:
    """The iteration ``msign_ns`` runs for these arguments: "standard" or "gram" (host only)."""
    c, keep = make_coeffs(coeffs, None, 1 if improved_init else 0, _METHODS[method])
    r = _lib.lib().msign_ns_route(batch, rows, cols, _compute_code(compute), ctypes.byref(c) if c is not None else None)
    del keep
    if r < 0:
        check(-r, "msign_ns_route")
    return "gram" if r == 1 else "standard"


def msign_ns(x, out=None, *, compute: str = "bf16", coeffs=None, eps=None, improved_init=False, method="standard",
             workspace=None, stream=None):
    """Newton-Schulz msign of the last two dims of ``x`` (bf16/fp16/fp32 CUDA tensor).

    ``x`` and ``out`` may be batched views whose matrices are dense but not
    back to back (e.g. ``big[:, 0]``): their batch strides are passed on.
    ``improved_init``: the sharper step-0 normalisation (msign_coeffs.init = 1).
    ``method``: "standard" (standard NS) or "auto" (Gram NS where ``msign_ns_route``
    picks it, msign_coeffs.method = 1)."""
    torch = _torch()
    batch, rows, cols, in_stride = _batch_layout(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(out, x.device, "out")
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    _, _, _, out_stride = _batch_layout(out, "out")
    with torch.cuda.device(x.device):
        ws, wsb = _workspace(msign_ns_workspace_size(batch, rows, cols, compute), x.device, workspace)
        c, keep = make_coeffs(coeffs, eps, 1 if improved_init else 0, _METHODS[method])
        st = _lib.lib().msign_ns(x.data_ptr(), out.data_ptr(), _dtype_code(x), _compute_code(compute), batch, rows,
                                 cols, in_stride, out_stride, ctypes.byref(c) if c is not None else None, _ptr(ws),
                                 wsb, _stream(stream, x.device))
        del keep
    check(st, "msign_ns")
    return out


def msign_ns_host_workspace_size(batch: int, rows: int, cols: int, io: str = "bf16", compute: str = "bf16") -> int:
    return int(_lib.lib().msign_ns_host_workspace_size(batch, rows, cols, _compute_code(io), _compute_code(compute)))


def msign_ns_host(x, out=None, *, compute: str = "bf16", coeffs=None, eps=None, improved_init=False,
                  method="standard", workspace=None, stream=None, device=None):
    """msign_ns of HOST matrices (``x``: a CPU tensor, dense, bf16/fp16/fp32;
    page-locked for asynchronous copies): the call enqueues the copy in, the
    iteration and the copy out on ``stream`` (default: the current stream of
    ``device``, default the current device) and returns ``out`` (a CPU
    tensor, page-locked when allocated here) BEFORE the result is there:
    synchronize the stream before reading it.  ``workspace``: a device uint8
    tensor of at least msign_ns_host_workspace_size() bytes."""
    torch = _torch()
    if x.is_cuda or out is not None and out.is_cuda:
        raise ValueError("msign_ns_host takes host (CPU) tensors; use msign_ns for device tensors")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if x.dim() < 2:
        raise ValueError("x needs at least two dims")
    rows, cols = x.shape[-2], x.shape[-1]
    batch = x.numel() // max(rows * cols, 1) if rows * cols else 0
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype).pin_memory()
    if out.shape != x.shape or out.dtype != x.dtype or not out.is_contiguous():
        raise ValueError("out must be a contiguous CPU tensor matching x in shape and dtype")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    io = _dtype_code(x)
    with torch.cuda.device(dev):
        need = int(_lib.lib().msign_ns_host_workspace_size(batch, rows, cols, io, _compute_code(compute)))
        ws, wsb = _workspace(need, dev, workspace)
        c, keep = make_coeffs(coeffs, eps, 1 if improved_init else 0, _METHODS[method])
        st = _lib.lib().msign_ns_host(x.data_ptr(), out.data_ptr(), io, _compute_code(compute), batch, rows, cols,
                                      ctypes.byref(c) if c is not None else None, _ptr(ws), wsb, _stream(stream, dev))
        del keep
    check(st, "msign_ns_host")
    return out


def msign_ns_noalloc_max_bytes() -> int:
    """Size of the scratch array built into the library (the largest
    msign_ns_workspace_size() that msign_ns_noalloc accepts)."""
    return int(_lib.lib().msign_ns_noalloc_max_bytes())


def msign_ns_noalloc(x, out, *, coeffs=None, eps=None, improved_init=False, method="standard", stream=None):
    """msign_ns (bf16 arithmetic) in the library's built-in scratch array: no
    workspace and no device allocation.  ``x`` and ``out`` are the caller's
    dense CUDA tensors of one shape and dtype.  Calls on one device share the
    scratch array: order them on one stream.  Raises MsignError with status
    ERR_WORKSPACE, before anything is enqueued, when the problem needs more
    than msign_ns_noalloc_max_bytes() of workspace."""
    torch = _torch()
    _need_cuda(x, "x")
    _need_cuda(out, "out")
    _same_device(out, x.device, "out")
    if x.dim() < 2:
        raise ValueError("x needs at least two dims")
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    rows, cols = x.shape[-2], x.shape[-1]
    batch = math.prod(x.shape[:-2])
    c, keep = make_coeffs(coeffs, eps, 1 if improved_init else 0, _METHODS[method])
    with torch.cuda.device(x.device):
        st = _lib.lib().msign_ns_noalloc(x.data_ptr(), out.data_ptr(), _dtype_code(x), batch, rows, cols,
                                         ctypes.byref(c) if c is not None else None, _stream(stream, x.device))
    del keep
    check(st, "msign_ns_noalloc")
    return out


# ---------------------------------------------------------------- gram_xxt

def gram_xxt_workspace_size(x) -> int:
    n, m = x.shape[-2], x.shape[-1]
    batch = math.prod(x.shape[:-2])
    return int(_lib.lib().gram_xxt_workspace_size(batch, n, m, _dtype_code(x), x.data_ptr()))


def gram_xxt(x, out=None, *, out_dtype=None, workspace=None, stream=None):
    """A = X X^T over the last two dims of ``x`` (bf16 or fp16), exactly symmetric."""
    torch = _torch()
    _need_cuda(x, "x")
    n, m = x.shape[-2], x.shape[-1]
    batch = math.prod(x.shape[:-2])
    if out is None:
        out = torch.empty(*x.shape[:-2], n, n, dtype=out_dtype or x.dtype, device=x.device)
    _need_cuda(out, "out")
    _same_device(out, x.device, "out")
    if tuple(out.shape) != tuple(x.shape[:-2]) + (n, n):
        raise ValueError("out must be (..., n, n)")
    with torch.cuda.device(x.device):
        ws, wsb = _workspace(gram_xxt_workspace_size(x), x.device, workspace)
        st = _lib.lib().gram_xxt(x.data_ptr(), _dtype_code(x), out.data_ptr(), _dtype_code(out), batch, n, m,
                                 _ptr(ws), wsb, _stream(stream, x.device))
    check(st, "gram_xxt")
    return out


# ---------------------------------------------------------------- gram_ns

def gram_ns_workspace_size(batch: int, rows: int, cols: int) -> int:
    return int(_lib.lib().gram_ns_workspace_size(batch, rows, cols))


def gram_ns(x, out=None, *, coeffs=None, eps=None, restart_after=(2,), workspace=None, stream=None):
    """Stabilized Gram Newton-Schulz (fp16 inner iteration) of the last two dims of ``x``
    (batched views with one batch stride accepted, as for ``msign_ns``)."""
    torch = _torch()
    batch, rows, cols, in_stride = _batch_layout(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(out, x.device, "out")
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must match x in shape and dtype")
    _, _, _, out_stride = _batch_layout(out, "out")
    c, keep = make_coeffs(coeffs, eps)
    if restart_after is None:
        rbuf, nr = None, -1
    else:
        r = [int(v) for v in restart_after]
        rbuf, nr = (ctypes.c_int * max(1, len(r)))(*r), len(r)
    with torch.cuda.device(x.device):
        ws, wsb = _workspace(gram_ns_workspace_size(batch, rows, cols), x.device, workspace)
        st = _lib.lib().gram_ns(x.data_ptr(), out.data_ptr(), _dtype_code(x), batch, rows, cols, in_stride,
                                out_stride, ctypes.byref(c) if c is not None else None,
                                ctypes.cast(rbuf, ctypes.POINTER(ctypes.c_int)) if rbuf is not None else None, nr,
                                _ptr(ws), wsb, _stream(stream, x.device))
    del keep
    check(st, "gram_ns")
    return out


# ---------------------------------------------------------------- muon_step

def _i64_array(vals):
    return (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])


def muon_step_route(rows: int, cols: int, *, coeffs=None, improved_init=False, method="auto") -> str:
    """The iteration ``muon_step`` runs for one rows x cols matrix: "standard" or "gram" (host only)."""
    c, keep = make_coeffs(coeffs, None, 1 if improved_init else 0, _METHODS[method])
    r = _lib.lib().muon_step_route(rows, cols, ctypes.byref(c) if c is not None else None)
    del keep
    if r < 0:
        check(-r, "muon_step_route")
    return "gram" if r == 1 else "standard"


def muon_step_workspace_size(shapes) -> int:
    rows = _i64_array([s[0] for s in shapes])
    cols = _i64_array([s[1] for s in shapes])
    return int(_lib.lib().muon_step_workspace_size(len(shapes), rows, cols))


def muon_step(weights, momenta, grads, *, momentum: float = 0.95, lr: float = 0.02, coeffs=None, eps=None,
              improved_init=False, method="standard", workspace=None, stream=None):
    """In-place Muon update of lists of weights (bf16/fp32), fp32 momenta and grads (bf16/fp32).

    ``method="auto"``: the matrices ``muon_step_route`` gives to Gram NS take it
    (msign_coeffs.method = 1)."""
    torch = _torch()
    num = len(weights)
    if not (len(momenta) == num and len(grads) == num):
        raise ValueError("weights, momenta and grads must have the same length")
    if num == 0:
        return
    device = weights[0].device
    for w, m, g in zip(weights, momenta, grads):
        for t, nm in ((w, "weight"), (m, "momentum"), (g, "grad")):
            _need_cuda(t, nm)
            _same_device(t, device, nm)
        if w.dim() != 2 or w.shape != m.shape or w.shape != g.shape:
            raise ValueError("each weight, momentum and grad must be the same 2-D shape")
        if m.dtype != torch.float32:
            raise TypeError("momenta must be float32")
    wdt = {_dtype_code(w) for w in weights}
    gdt = {_dtype_code(g) for g in grads}
    if len(wdt) != 1 or len(gdt) != 1:
        raise TypeError("all weights (and all grads) must share one dtype")
    shapes = [tuple(w.shape) for w in weights]
    W = (ctypes.c_void_p * num)(*[w.data_ptr() for w in weights])
    M = (ctypes.c_void_p * num)(*[m.data_ptr() for m in momenta])
    G = (ctypes.c_void_p * num)(*[g.data_ptr() for g in grads])
    rows = _i64_array([s[0] for s in shapes])
    cols = _i64_array([s[1] for s in shapes])
    c, keep = make_coeffs(coeffs, eps, 1 if improved_init else 0, _METHODS[method])
    with torch.cuda.device(device):
        ws, wsb = _workspace(muon_step_workspace_size(shapes), device, workspace)
        st = _lib.lib().muon_step(num, W, M, G, rows, cols, wdt.pop(), gdt.pop(), float(momentum), float(lr),
                                  ctypes.byref(c) if c is not None else None, _ptr(ws), wsb,
                                  _stream(stream, device))
    del keep
    check(st, "muon_step")


# ---------------------------------------------------------------- Mousse

def mousse_inv_root(a, out=None, *, eps: float = 0.0, iters: int = 0, workspace=None, stream=None):
    """(A + eps I)^(-1/4) of symmetric positive semidefinite fp32 matrices (the
    last two dims of ``a``), exactly symmetric, by the coupled Newton
    iteration in fp32-accurate arithmetic (``iters`` 0: the library default)."""
    torch = _torch()
    _need_cuda(a, "a")
    if a.dtype != torch.float32 or a.dim() < 2 or a.shape[-1] != a.shape[-2]:
        raise ValueError("a must be float32 (..., n, n)")
    n = a.shape[-1]
    batch = math.prod(a.shape[:-2])
    if out is None:
        out = torch.empty_like(a)
    _need_cuda(out, "out")
    _same_device(out, a.device, "out")
    if out.shape != a.shape or out.dtype != torch.float32:
        raise ValueError("out must match a")
    with torch.cuda.device(a.device):
        ws, wsb = _workspace(int(_lib.lib().mousse_inv_root_workspace_size(batch, n)), a.device, workspace)
        st = _lib.lib().mousse_inv_root(a.data_ptr(), out.data_ptr(), batch, n, float(eps), int(iters), _ptr(ws), wsb,
                                        _stream(stream, a.device))
    check(st, "mousse_inv_root")
    return out


def mousse_direction(g, l_root, r_root, out=None, *, coeffs=None, eps=None, improved_init=False, workspace=None,
                     stream=None):
    """L^(-1/4) msign(L^(-1/4) G R^(-1/4)) R^(-1/4) of the last two dims of ``g``,
    given ``l_root`` = L^(-1/4) (..., rows, rows) and ``r_root`` = R^(-1/4)
    (..., cols, cols) as float32 (e.g. from ``mousse_inv_root``)."""
    torch = _torch()
    for t, nm in ((g, "g"), (l_root, "l_root"), (r_root, "r_root")):
        _need_cuda(t, nm)
        _same_device(t, g.device, nm)
    if g.dim() < 2:
        raise ValueError("g needs at least two dims")
    rows, cols = g.shape[-2], g.shape[-1]
    lead = tuple(g.shape[:-2])
    if (l_root.dtype != torch.float32 or r_root.dtype != torch.float32 or tuple(l_root.shape) != lead + (rows, rows)
            or tuple(r_root.shape) != lead + (cols, cols)):
        raise ValueError("l_root and r_root must be float32 (..., rows, rows) and (..., cols, cols)")
    batch = math.prod(lead)
    if out is None:
        out = torch.empty_like(g)
    _need_cuda(out, "out")
    _same_device(out, g.device, "out")
    if out.shape != g.shape or out.dtype != g.dtype:
        raise ValueError("out must match g")
    c, keep = make_coeffs(coeffs, eps, 1 if improved_init else 0, 0)
    with torch.cuda.device(g.device):
        ws, wsb = _workspace(int(_lib.lib().mousse_direction_workspace_size(batch, rows, cols)), g.device, workspace)
        st = _lib.lib().mousse_direction(g.data_ptr(), out.data_ptr(), _dtype_code(g), batch, rows, cols,
                                         l_root.data_ptr(), r_root.data_ptr(),
                                         ctypes.byref(c) if c is not None else None, _ptr(ws), wsb,
                                         _stream(stream, g.device))
    del keep
    check(st, "mousse_direction")
    return out


# ---------------------------------------------------------------- layer operators
#
# Like every call of this library they are not recorded by autograd: outputs
# carry no graph, and gradients come of the *_backward calls.

def _rows_layout(t, name, cols=None):
    """(rows, cols, stride) of a CUDA tensor whose last dim is dense and whose
    leading dims step through memory with one row stride (any view of that
    form, e.g. ``big[:, :n]``); stride 0 means back to back."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} needs at least one dim")
    width = shape[-1]
    if cols is not None and width != cols:
        raise ValueError(f"{name} must have {cols} columns, has {width}")
    rows = math.prod(shape[:-1])
    if rows * width == 0 or t.is_contiguous():
        return rows, width, 0
    if width > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: each row (the last dim) must be dense")
    lead = [(shape[d], t.stride(d)) for d in range(len(shape) - 1) if shape[d] != 1]
    if not lead:
        return rows, width, 0
    for (sz_o, st_o), (sz_i, st_i) in zip(lead[:-1], lead[1:]):
        if st_o != st_i * sz_i:
            raise ValueError(f"{name}: the leading dims must step through memory with one row stride")
    stride = lead[-1][1]
    if stride < width:
        raise ValueError(f"{name}: rows overlap (stride {stride} < {width})")
    return rows, width, (0 if stride == width else stride)


def _on(t, index, name):
    """t lies on the device that the call runs on."""
    if t.get_device() != index:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{index}")


def _operand(t, index, name, shape, dtype):
    """The row stride of an input that must have this shape, dtype and device."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} of {dtype}")
    _on(t, index, name)
    return 0 if t.is_contiguous() else _rows_layout(t, name)[2]


def _like(t, ref, name, shape=None, dtype=None):
    """The given output, checked, or a new one: like ``ref`` but for shape and
    dtype; and its row stride."""
    if t is None:
        torch = _torch()
        if shape is not None:
            return ref.new_empty(shape, dtype=dtype or ref.dtype), 0
        if not ref.is_contiguous():
            return torch.empty(ref.shape, dtype=dtype or ref.dtype, device=ref.device), 0
        return (torch.empty_like(ref) if dtype is None else torch.empty_like(ref, dtype=dtype)), 0
    shape = ref.shape if shape is None else shape
    dtype = ref.dtype if dtype is None else dtype
    _on(t, ref.get_device(), name)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{name} must be {tuple(shape)} of {dtype}")
    return t, _rows_layout(t, name)[2]


def _on_stream(op):
    """Runs the operator with its ``stream`` argument (a torch stream or a raw
    handle) as the current stream, so that the outputs and the workspace that
    it allocates belong to that stream too.  The device is that of the
    operator's first parameter, by position or by name."""
    first = next(iter(inspect.signature(op).parameters))

    @functools.wraps(op)
    def call(*args, stream=None, **kwargs):
        if stream is None:
            return op(*args, **kwargs)
        torch = _torch()
        t = args[0] if args else kwargs.get(first)
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{first} must be a CUDA tensor (there is no CPU path)")
        device = t.device
        if not isinstance(stream, torch.cuda.Stream):
            # (handle 0 would make ExternalStream take a new stream)
            stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the call runs on {device}")
        with torch.cuda.stream(stream):
            return op(*args, **kwargs)
    # (python -OO leaves no docstring to add to)
    if op.__doc__:
        call.__doc__ = op.__doc__ + (
            "\n\n    Autograd does not record the call: the outputs carry no graph."
            "\n    ``stream``: the stream to run on, for the outputs too (default: the current one).")
    return call


def _call(fn, t, *args):
    """The status of an entry point called on t's device, with that device's
    current stream as its last argument."""
    torch = _torch()
    index = t.get_device()
    stream = _raw_stream(index)
    if torch.cuda.current_device() == index:
        return fn(*args, stream)
    with torch.cuda.device(index):
        return fn(*args, stream)


def _call_with_workspace(fn, size_fn, size_args, plain, t, workspace, *args):
    """_call with a workspace (pointer and bytes) behind args.  Where the width
    looks ``plain``, the usual case, the entry point is called without asking
    for a size; it refuses before it enqueues anything where it needs one."""
    ws = workspace
    if ws is not None:
        _on(ws, t.get_device(), "workspace")
        return _call(fn, t, *args, ws.data_ptr(), ws.numel() * ws.element_size())
    st = _call(fn, t, *args, None, 0) if plain else _lib.ERR_WORKSPACE
    if st == _lib.ERR_WORKSPACE:
        ws, wsb = _workspace(size_fn(*size_args), t.device, None)
        st = _call(fn, t, *args, _ptr(ws), wsb)
    return st


def _norm_weight(weight, x, index):
    """(dtype code, pointer) of a norm's weight."""
    if weight is None:
        return _dtype_codes[x.dtype], None
    _on(weight, index, "weight")
    if weight.dim() != 1 or weight.shape[0] != x.shape[-1]:
        raise ValueError(f"weight must have shape ({x.shape[-1]},)")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    if weight.dtype != x.dtype and weight.dtype != _torch().float32:
        raise TypeError("weight must be of the input's dtype or float32")
    return _dtype_codes[weight.dtype], weight.data_ptr()


def _norm_inputs(x, residual, sum_out, index):
    """(rows, cols, x stride, residual stride, sum, its stride)"""
    rows, cols, xs = _rows_layout(x, "x")
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
        return rows, cols, xs, 0, None, 0
    rs = _operand(residual, index, "residual", x.shape, x.dtype)
    return (rows, cols, xs, rs) + _like(sum_out, x, "sum_out")


@_on_stream
def rms_norm(x, weight=None, residual=None, *, eps: float = 1e-6, out=None, sum_out=None):
    """RMS norm of the last dim of ``x`` (bf16/fp16/fp32), after adding ``residual`` if one is given.

    Returns y = s * weight / sqrt(mean(s^2) + eps), or (y, s) with the sum
    s = x + residual (rounded to x's dtype) when there is a residual.
    ``weight``: of x's dtype or float32, None for ones.  ``sum_out`` may be
    ``x`` or ``residual`` itself, and so may ``out`` where ``sum_out`` is not."""
    code, index = _dtype_code(x), x.get_device()
    rows, cols, xs, rs, s, ss = _norm_inputs(x, residual, sum_out, index)
    wdt, wp = _norm_weight(weight, x, index)
    y, ys = _like(out, x, "out")
    check(_call(_lib.lib().rms_norm, x, x.data_ptr(), _ptr(residual), wp, y.data_ptr(), _ptr(s), code, wdt, rows,
                cols, xs, rs, ys, ss, eps), "rms_norm")
    return y if residual is None else (y, s)


@_on_stream
def rms_norm_q8(x, weight=None, residual=None, *, eps: float = 1e-6, out=None, scale_out=None, sum_out=None):
    """``rms_norm`` with y quantised to int8, one float32 scale a row (max|y| / 127): returns
    (q, scale), or (q, scale, s) when there is a residual.  q * scale[..., None] is what it stands for."""
    torch = _torch()
    code, index = _dtype_code(x), x.get_device()
    rows, cols, xs, rs, s, ss = _norm_inputs(x, residual, sum_out, index)
    wdt, wp = _norm_weight(weight, x, index)
    q, qs = _like(out, x, "out", dtype=torch.int8)
    if scale_out is None:
        scale = x.new_empty(x.shape[:-1], dtype=torch.float32)
    else:
        scale = scale_out
        _on(scale, index, "scale_out")
        if scale.shape != x.shape[:-1] or scale.dtype != torch.float32 or not scale.is_contiguous():
            raise ValueError(f"scale_out must be contiguous float32 of shape {tuple(x.shape[:-1])}")
    check(_call(_lib.lib().rms_norm_q8, x, x.data_ptr(), _ptr(residual), wp, q.data_ptr(), scale.data_ptr(),
                _ptr(s), code, wdt, rows, cols, xs, rs, qs, ss, eps), "rms_norm_q8")
    return (q, scale) if residual is None else (q, scale, s)


def rms_norm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(_lib.lib().rms_norm_backward_workspace_size(rows, cols))


@_on_stream
def rms_norm_backward(dy, s, weight=None, *, dsum=None, eps: float = 1e-6, dx_out=None, dw_out=None, workspace=None):
    """Gradients of ``rms_norm``: (dx, dw) from ``dy`` and ``s``, the sum that it returned (x without a residual).

    ``dsum``: the gradient that reaches s past the norm, added to dx.  dx is
    the gradient of x and of the residual alike; dw is None without a weight."""
    code, index = _dtype_code(s), s.get_device()
    rows, cols, zs = _rows_layout(s, "s")
    sdy = _operand(dy, index, "dy", s.shape, s.dtype)
    sds = 0 if dsum is None else _operand(dsum, index, "dsum", s.shape, s.dtype)
    wdt, wp = _norm_weight(weight, s, index)
    dx, dxs = _like(dx_out, s, "dx_out")
    L = _lib.lib()
    dw, ws, wsb = None, None, 0
    if weight is not None:
        dw = _torch().empty_like(weight) if dw_out is None else _like(dw_out, weight, "dw_out")[0]
        ws, wsb = _workspace(L.rms_norm_backward_workspace_size(rows, cols), s.device, workspace)
    elif dw_out is not None:
        raise ValueError("dw_out needs a weight")
    check(_call(L.rms_norm_backward, s, dy.data_ptr(), s.data_ptr(), wp, _ptr(dsum), dx.data_ptr(), _ptr(dw), code,
                wdt, rows, cols, sdy, zs, sds, dxs, eps, _ptr(ws), wsb), "rms_norm_backward")
    return dx, dw


def i8_matmul_workspace_size(a, b) -> int:
    m, k, sa = _rows_layout(a, "a")
    n, _, sb = _rows_layout(b, "b")
    return int(_lib.lib().i8_matmul_workspace_size(m, n, k, a.data_ptr(), sa, b.data_ptr(), sb))


@_on_stream
def i8_matmul(a, a_scale, b, b_scale, *, out=None, out_dtype=None, workspace=None):
    """(a b^T) of int8 ``a`` (..., k) and ``b`` (n, k), times float32 ``a_scale`` (...) for each row of a (token)
    and ``b_scale`` (n,) for each row of b (output channel).

    The integer sums are exact.  ``out_dtype``: bf16 (default), fp16 or
    float32, or that of ``out``.  ``a`` and ``a_scale`` are what
    ``rms_norm_q8`` returns."""
    torch = _torch()
    if a.dtype != torch.int8 or b.dtype != torch.int8:
        raise TypeError("a and b must be int8")
    if b.dim() != 2:
        raise ValueError("b must be (n, k)")
    index = a.get_device()
    m, k, sa = _rows_layout(a, "a")
    n, _, sb = _rows_layout(b, "b", k)
    _on(b, index, "b")
    for t, nm, shape in ((a_scale, "a_scale", a.shape[:-1]), (b_scale, "b_scale", b.shape[:1])):
        _on(t, index, nm)
        if t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{nm} must be contiguous float32 of shape {tuple(shape)}")
    if out_dtype is None:
        out_dtype = torch.bfloat16 if out is None else out.dtype
    out, so = _like(out, a, "out", shape=a.shape[:-1] + (n,), dtype=out_dtype)
    code, L = _dtype_code(out), _lib.lib()
    pa, pb = a.data_ptr(), b.data_ptr()
    check(_call_with_workspace(L.i8_matmul, L.i8_matmul_workspace_size, (m, n, k, pa, sa, pb, sb), k % 16 == 0, a,
                               workspace, pa, a_scale.data_ptr(), pb, b_scale.data_ptr(), out.data_ptr(), code, m, n, k,
                               sa, sb, so), "i8_matmul")
    return out


_ACTIVATIONS = {"silu": _lib.SILU, "gelu": _lib.GELU, "gelu_tanh": _lib.GELU_TANH}


def _activation_code(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(_ACTIVATIONS)}, not {name!r}")
    return _ACTIVATIONS[name]


def _ffn_inputs(x, w_gate, w_up):
    """(tokens, d, h, x stride, weight stride) of a gated block's inputs."""
    t, d, xs = _rows_layout(x, "x")
    shape = w_gate.shape
    if len(shape) != 2 or shape[1] != d:
        raise ValueError(f"w_gate must be (h, {d})")
    h, index = shape[0], x.get_device()
    sg = _operand(w_gate, index, "w_gate", shape, x.dtype)
    su = _operand(w_up, index, "w_up", shape, x.dtype)
    if sg != su and h > 1 and (sg or d) != (su or d):
        raise ValueError("w_gate and w_up must have one row stride")
    return t, d, h, xs, sg


def gated_ffn_workspace_size(x, w_gate, w_up) -> int:
    t, d, h, xs, ws = _ffn_inputs(x, w_gate, w_up)
    return int(_lib.lib().gated_ffn_workspace_size(t, d, h, x.data_ptr(), xs, w_gate.data_ptr(), w_up.data_ptr(), ws))


@_on_stream
def gated_ffn(x, w_gate, w_up, *, activation: str = "silu", save: bool = False, out=None, gate_out=None, up_out=None,
              workspace=None):
    """act(x w_gate^T) * (x w_up^T) of ``x`` (..., d) and weights (h, d), bf16 or fp16, in one kernel.

    ``activation``: "silu", "gelu" or "gelu_tanh".  With ``save`` (or
    ``gate_out`` and ``up_out``) returns (out, gate, up), what
    ``gated_ffn_backward`` takes; else out."""
    code, act = _dtype_code(x), _activation_code(activation)
    t, d, h, xs, sw = _ffn_inputs(x, w_gate, w_up)
    shape = x.shape[:-1] + (h,)
    if (gate_out is None) != (up_out is None):
        raise ValueError("gate_out and up_out go together")
    out, so = _like(out, x, "out", shape=shape)
    gate = up = None
    sp = 0
    if save or gate_out is not None:
        save = True
        gate, sp = _like(gate_out, x, "gate_out", shape=shape)
        up, su = _like(up_out, x, "up_out", shape=shape)
        if (sp or h) != (su or h):
            raise ValueError("gate_out and up_out must have one row stride")
    L = _lib.lib()
    px, pg, pu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    check(_call_with_workspace(L.gated_ffn, L.gated_ffn_workspace_size, (t, d, h, px, xs, pg, pu, sw), d % 8 == 0, x,
                               workspace, px, pg, pu, out.data_ptr(), _ptr(gate), _ptr(up), code, act, t, d, h, xs, sw, so, sp),
          "gated_ffn")
    return (out, gate, up) if save else out


def gated_ffn_backward_workspace_size(x, w_gate, w_up) -> int:
    t, d, h, xs, ws = _ffn_inputs(x, w_gate, w_up)
    return int(_lib.lib().gated_ffn_backward_workspace_size(t, d, h, x.data_ptr(), xs, w_gate.data_ptr(),
                                                            w_up.data_ptr(), ws))


@_on_stream
def gated_ffn_backward(dh, x, w_gate, w_up, gate, up, *, activation: str = "silu", grad_dtype=None, need_dx=True,
                       need_dw=True, dx_out=None, dw_gate_out=None, dw_up_out=None, workspace=None):
    """Gradients of ``gated_ffn``: (dx, dw_gate, dw_up) from ``dh`` and the kept ``gate`` and ``up``.

    ``grad_dtype``: of the weight gradients, x's dtype (default) or float32;
    either is what ``muon_step`` takes as grads (fp16 blocks: float32).  The
    gradients of gate and up are held in x's dtype on the way: in fp16 scale
    ``dh`` so that dh * up and dh * act(gate) stay below 65504.
    ``need_dx`` / ``need_dw`` False leaves that part out (None in its place)."""
    torch = _torch()
    code, act = _dtype_code(x), _activation_code(activation)
    t, d, h, xs, sw = _ffn_inputs(x, w_gate, w_up)
    if not need_dx and not need_dw:
        raise ValueError("at least one of need_dx and need_dw")
    shape, index = x.shape[:-1] + (h,), x.get_device()
    sdh = _operand(dh, index, "dh", shape, x.dtype)
    sp, su = _operand(gate, index, "gate", shape, x.dtype), _operand(up, index, "up", shape, x.dtype)
    if sp != su and (sp or h) != (su or h):
        raise ValueError("gate and up must have one row stride")
    if grad_dtype is None:
        grad_dtype = x.dtype if dw_gate_out is None else dw_gate_out.dtype
    if grad_dtype not in (x.dtype, torch.float32):
        raise TypeError("grad_dtype must be x's dtype or float32")
    dx = dwg = dwu = None
    sdx = sdw = 0
    if need_dx:
        dx, sdx = _like(dx_out, x, "dx_out")
    if need_dw:
        other = None if grad_dtype == x.dtype else grad_dtype
        dwg, sdw = _like(dw_gate_out, w_gate, "dw_gate_out", dtype=other)
        dwu, su = _like(dw_up_out, w_up, "dw_up_out", dtype=other)
        if (sdw or d) != (su or d):
            raise ValueError("dw_gate_out and dw_up_out must have one row stride")
    L = _lib.lib()
    px, pg, pu = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr()
    ws, wsb = _workspace(L.gated_ffn_backward_workspace_size(t, d, h, px, xs, pg, pu, sw), x.device, workspace)
    check(_call(L.gated_ffn_backward, x, dh.data_ptr(), px, pg, pu, gate.data_ptr(), up.data_ptr(), _ptr(dx),
                _ptr(dwg), _ptr(dwu), code, _dtype_codes[grad_dtype], act, t, d, h, sdh, xs, sw, sp, sdx, sdw, _ptr(ws),
                wsb), "gated_ffn_backward")
    return dx, dwg, dwu


# ---------------------------------------------------------------- launch records

PROFILE_KINDS = {"gemm": 0, "norm": 1, "ingest": 2, "elementwise": 3}


def selftest_timeout(limit_ns: int = 50_000_000, stream=None) -> None:
    """Makes the library's bounded waits expire on purpose (see
    msign_selftest_timeout): the next sync_status() raises MsignError with
    status ERR_TIMEOUT, and the GPU context stays usable."""
    check(_lib.lib().msign_selftest_timeout(int(limit_ns), _stream(stream)), "msign_selftest_timeout")


def set_chaining(enable: bool) -> bool:
    """Diagnostics (msign_set_chaining): False runs each product of a
    standard-route iteration step as a launch of its own, for profiling the
    phases apart; True (the default) chains them.  Returns the previous
    setting."""
    return bool(_lib.lib().msign_set_chaining(1 if enable else 0))


def profile_enable(enable: bool = True) -> None:
    check(_lib.lib().msign_profile_enable(1 if enable else 0), "msign_profile_enable")


def profile_reset() -> None:
    check(_lib.lib().msign_profile_reset(), "msign_profile_reset")


def profile_read(kind: str) -> dict:
    """{'launches', 'ms', 'flops', 'bytes'} summed over the recorded launches of one kind."""
    n = ctypes.c_int()
    ms, fl, by = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    check(_lib.lib().msign_profile_read(PROFILE_KINDS[kind], ctypes.byref(n), ctypes.byref(ms), ctypes.byref(fl),
                                        ctypes.byref(by)), "msign_profile_read")
    return {"launches": n.value, "ms": ms.value, "flops": fl.value, "bytes": by.value}
