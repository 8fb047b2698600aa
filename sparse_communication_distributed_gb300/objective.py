"""Python binding of the training-objective calls of libscape (argument
marshalling only; the operators are defined in ``include/scape.h``).

Tensors are torch CUDA tensors on the current device.  Logits are 2-D with
unit column stride (a view of wider rows is fine); every other input is
contiguous.  Results are new tensors, allocated on the stream that the call
runs on (``stream``: None for the current one, a torch stream or a raw handle),
unless ``grad`` says where the gradient goes.  Inputs are borrowed until the
work enqueued on that stream has finished.  A wrong type, shape or device
raises ``ValueError``; an error of the library raises ``ScapeError``.

The calls build no autograd graph: results of inputs that require a gradient
do not.  ``distill_loss_grad`` and ``route_backward`` are the gradients, and
``examples/distill_moe.py`` wraps them in two ``torch.autograd.Function``s.
"""
from __future__ import annotations

import ctypes

from .scape import SCAPE_OK, DistillArgs, RouteArgs, ScapeError, load_library

BF16, F16, F32 = 0, 1, 2

# Set by the first call: torch and the library are not needed to import the package.
torch = None
_lib = None
_codes: dict = {}


def _load() -> None:
    global torch, _lib, _codes
    import torch as t
    _codes = {t.bfloat16: BF16, t.float16: F16, t.float32: F32}
    torch = t
    _lib = load_library()


def _stream_context(stream):
    """Context in which ``stream`` is the current stream."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _code(x, name: str) -> int:
    code = _codes.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, not {x.dtype}")
    return code


def _rows(x, name: str = "logits") -> int:
    """Checks a 2-D tensor of rows; returns its row stride in elements."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D, not of shape {tuple(x.shape)}")
    if not x.is_cuda or x.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device, not {x.device}")
    rows, n = x.shape
    s0, s1 = x.stride()
    if s1 != 1 and n > 1:
        raise ValueError(f"{name} must have contiguous rows (column stride 1, not {s1})")
    return s0 if rows > 1 else max(n, 1)


def _arg(x, name: str, dtypes, shape, device) -> int | None:
    """Address of an optional contiguous input, checked."""
    if x is None:
        return None
    if x.dtype in dtypes and x.shape == shape and x.device == device and x.is_contiguous():
        return x.data_ptr()
    raise ValueError(f"{name} must be contiguous, of type {' or '.join(map(str, dtypes))} and shape "
                     f"{shape} on {device}, not {x.dtype} {tuple(x.shape)} with strides "
                     f"{x.stride()} on {x.device}")


def _count(k: int) -> int:
    """Checks that k is what a C int holds (ctypes would cut it down); returns
    the entries of a row that results have."""
    if not -2 ** 31 <= k < 2 ** 31:
        raise ValueError(f"k={k} does not fit 32 bits")
    return max(k, 0)


def _check(rc: int) -> None:
    if rc != SCAPE_OK:
        raise ScapeError(rc, _lib.scape_last_error(None).decode())


def topk_logits(logits, k: int, temperature: float = 1.0, stream=None):
    """scape_topk_logits: (idx int32 [rows, k], vals [rows, k], lse float32
    [rows]) of the k largest logits of every row."""
    if _lib is None:
        _load()
    if stream is not None:
        with _stream_context(stream):
            return topk_logits(logits, k, temperature)
    stride = _rows(logits)
    rows, vocab = logits.shape
    dev, n = logits.device, _count(k)
    code = _code(logits, "logits")
    idx = torch.empty((rows, n), dtype=torch.int32, device=dev)
    vals = torch.empty((rows, n), dtype=logits.dtype, device=dev)
    lse = torch.empty(rows, dtype=torch.float32, device=dev)
    _check(_lib.scape_topk_logits(logits.data_ptr(), code, rows, vocab, stride, k, temperature,
                                  idx.data_ptr(), vals.data_ptr(), lse.data_ptr(),
                                  torch._C._cuda_getCurrentRawStream(dev.index)))
    return idx, vals, lse


def _distill(logits, idx, vals, teacher_lse, labels, row_weight, temperature, kd_weight, ce_weight,
             bad_count, with_grad, grad, stream):
    if _lib is None:
        _load()
    if stream is not None:
        with _stream_context(stream):
            return _distill(logits, idx, vals, teacher_lse, labels, row_weight, temperature,
                            kd_weight, ce_weight, bad_count, with_grad, grad, None)
    stride = _rows(logits)
    rows, vocab = logits.shape
    dev = logits.device
    code = _code(logits, "logits")
    k = vcode = 0
    p_idx = p_vals = None
    if idx is not None:
        if vals is None or idx.dim() != 2:
            raise ValueError("idx must be 2-D and come with vals")
        k = idx.shape[1]
        vcode = _code(vals, "vals")
        p_idx = _arg(idx, "idx", (torch.int32,), (rows, k), dev)
        p_vals = _arg(vals, "vals", (vals.dtype,), (rows, k), dev)
    f32 = (torch.float32,)
    p_lse = _arg(teacher_lse, "teacher_lse", f32, (rows,), dev)
    p_lab = _arg(labels, "labels", (torch.int64,), (rows,), dev)
    p_w = _arg(row_weight, "row_weight", f32, (rows,), dev)
    p_bad = _arg(bad_count, "bad_count", (torch.int32,), (1,), dev)
    gstride = 0
    if grad is not None:
        if grad.shape != logits.shape or grad.dtype != logits.dtype:
            raise ValueError("grad must have the shape and type of the logits")
        gstride = _rows(grad, "grad")
    loss = torch.empty(rows, dtype=torch.float32, device=dev)
    if with_grad and grad is None:
        grad = torch.empty((rows, vocab), dtype=logits.dtype, device=dev)
        gstride = max(vocab, 1)
    args = DistillArgs(logits.data_ptr(), code, k, rows, vocab, stride, p_idx, p_vals, vcode,
                       temperature, kd_weight, ce_weight, p_lse, p_lab, p_w, loss.data_ptr(),
                       grad.data_ptr() if with_grad else None, gstride, p_bad)
    _check(_lib.scape_distill_loss(ctypes.byref(args),
                                   torch._C._cuda_getCurrentRawStream(dev.index)))
    return loss, grad


def distill_loss(logits, idx, vals, *, teacher_lse=None, labels=None, row_weight=None,
                 temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                 bad_count=None, stream=None):
    """scape_distill_loss without a gradient: the loss of every row (float32
    [rows]).  ``idx`` and ``vals`` may be None (cross entropy alone)."""
    return _distill(logits, idx, vals, teacher_lse, labels, row_weight, temperature, kd_weight,
                    ce_weight, bad_count, False, None, stream)[0]


def distill_loss_grad(logits, idx, vals, *, teacher_lse=None, labels=None, row_weight=None,
                      temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                      bad_count=None, grad=None, stream=None):
    """scape_distill_loss: (loss [rows], gradient of the logits in their type).
    ``grad=logits`` overwrites the logits by their gradient.  ``row_weight``
    carries what comes from above (a mean's 1/rows, padding, an upstream
    gradient of each row's loss)."""
    return _distill(logits, idx, vals, teacher_lse, labels, row_weight, temperature, kd_weight,
                    ce_weight, bad_count, True, grad, stream)


def _route_args(logits, k, renormalize, cu_tokens, valid):
    stride = _rows(logits)
    tokens, experts = logits.shape
    dev = logits.device
    groups = 1
    if cu_tokens is not None:
        if cu_tokens.dim() != 1 or cu_tokens.shape[0] < 2:
            raise ValueError("cu_tokens must be 1-D with at least 2 entries")
        groups = cu_tokens.shape[0] - 1
    return RouteArgs(logits.data_ptr(), _code(logits, "logits"), k, tokens, experts,
                     1 if renormalize else 0, stride,
                     _arg(cu_tokens, "cu_tokens", (torch.int32,), (groups + 1,), dev), groups,
                     _arg(valid, "valid", (torch.bool, torch.uint8), (tokens,), dev))


def route(logits, k: int, *, renormalize: bool = True, cu_tokens=None, valid=None, stream=None):
    """scape_route: (idx int32 [tokens, k], weights float32 [tokens, k], counts
    int32 [groups, experts], live int32 [groups + 2], losses float32 [2] =
    balance, z)."""
    if _lib is None:
        _load()
    if stream is not None:
        with _stream_context(stream):
            return route(logits, k, renormalize=renormalize, cu_tokens=cu_tokens, valid=valid)
    n = _count(k)
    args = _route_args(logits, k, renormalize, cu_tokens, valid)
    tokens, experts = logits.shape
    groups, dev = args.n_groups, logits.device
    need = ctypes.c_uint64()
    ref = ctypes.byref(args)
    _check(_lib.scape_route_workspace(ref, ctypes.byref(need)))
    nbytes = need.value
    i32, f32, empty = torch.int32, torch.float32, torch.empty
    idx = empty((tokens, n), dtype=i32, device=dev)
    weights = empty((tokens, n), dtype=f32, device=dev)
    counts = empty((groups, experts), dtype=i32, device=dev)
    live = empty(groups + 2, dtype=i32, device=dev)
    losses = empty(2, dtype=f32, device=dev)
    ws = empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check(_lib.scape_route(ref, idx.data_ptr(), weights.data_ptr(), counts.data_ptr(),
                            live.data_ptr(), losses.data_ptr(),
                            None if ws is None else ws.data_ptr(), nbytes,
                            torch._C._cuda_getCurrentRawStream(dev.index)))
    return idx, weights, counts, live, losses


def route_backward(logits, idx, counts, live, *, d_weights=None, d_losses=None,
                   renormalize: bool = True, cu_tokens=None, stream=None):
    """scape_route_backward: the gradient of the logits, in their type."""
    if _lib is None:
        _load()
    if stream is not None:
        with _stream_context(stream):
            return route_backward(logits, idx, counts, live, d_weights=d_weights,
                                  d_losses=d_losses, renormalize=renormalize, cu_tokens=cu_tokens)
    if idx.dim() != 2:
        raise ValueError("idx must be 2-D")
    k = idx.shape[1]
    args = _route_args(logits, k, renormalize, cu_tokens, None)
    tokens, experts = logits.shape
    groups, dev = args.n_groups, logits.device
    i32, f32 = (torch.int32,), (torch.float32,)
    p_idx = _arg(idx, "idx", i32, (tokens, k), dev)
    p_counts = _arg(counts, "counts", i32, (groups, experts), dev)
    p_live = _arg(live, "live", i32, (groups + 2,), dev)
    p_dw = _arg(d_weights, "d_weights", f32, (tokens, k), dev)
    p_dl = _arg(d_losses, "d_losses", f32, (2,), dev)
    grad = torch.empty((tokens, experts), dtype=logits.dtype, device=dev)
    _check(_lib.scape_route_backward(ctypes.byref(args), p_idx, p_counts, p_live, p_dw, p_dl,
                                     grad.data_ptr(), max(experts, 1),
                                     torch._C._cuda_getCurrentRawStream(dev.index)))
    return grad
