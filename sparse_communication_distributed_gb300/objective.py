"""Python binding of the training-objective calls of libscape (argument
marshalling only; the operators are defined in ``include/scape.h``).

Tensors are torch CUDA tensors on the current device.  Logits are 2-D with
unit column stride (a view of wider rows is fine); every other input is
contiguous.  Results are new tensors, allocated on the stream that the call
runs on, unless ``grad`` says where the gradient goes.  Inputs are borrowed
until the work enqueued on ``stream`` has finished.  A wrong type, shape or
device raises ``ValueError``; an error of the library raises ``ScapeError``.
"""
from __future__ import annotations

import contextlib
import ctypes

from .scape import SCAPE_OK, DistillArgs, RouteArgs, ScapeError, _stream_handle, load_library

BF16, F16, F32 = 0, 1, 2


def _torch():
    import torch
    return torch


def _dtype(x, name: str) -> int:
    torch = _torch()
    code = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}.get(x.dtype)
    if code is None:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, not {x.dtype}")
    return code


def _logits(x, name: str = "logits") -> int:
    """Checks a 2-D tensor of rows; returns its row stride in elements."""
    if x.dim() != 2:
        raise ValueError(f"{name} must be 2-D, not of shape {tuple(x.shape)}")
    if not x.is_cuda or x.device.index != _torch().cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device, not {x.device}")
    rows, n = x.shape
    if n > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows (column stride 1, not {x.stride(1)})")
    return x.stride(0) if rows > 1 else max(n, 1)


def _arg(x, name: str, dtypes, shape, device) -> int | None:
    """Address of an optional contiguous input, checked."""
    if x is None:
        return None
    if x.dtype not in dtypes:
        raise ValueError(f"{name} must be of type {' or '.join(map(str, dtypes))}, not {x.dtype}")
    if tuple(x.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(x.shape)}")
    if x.device != device:
        raise ValueError(f"{name} must be on {device}, not {x.device}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return x.data_ptr()


def _on(stream):
    """Context in which results are allocated: the stream that writes them."""
    if stream is None:
        return contextlib.nullcontext()
    torch = _torch()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _check(lib, rc: int) -> None:
    if rc != SCAPE_OK:
        raise ScapeError(rc, lib.scape_last_error(None).decode())


def topk_logits(logits, k: int, temperature: float = 1.0, stream=None):
    """scape_topk_logits: (idx int32 [rows, k], vals [rows, k], lse float32
    [rows]) of the k largest logits of every row."""
    torch = _torch()
    lib = load_library()
    stride = _logits(logits)
    rows, vocab = logits.shape
    dt = _dtype(logits, "logits")
    n = max(k, 0)
    with _on(stream):
        idx = torch.empty(rows, n, dtype=torch.int32, device=logits.device)
        vals = torch.empty(rows, n, dtype=logits.dtype, device=logits.device)
        lse = torch.empty(rows, dtype=torch.float32, device=logits.device)
        _check(lib, lib.scape_topk_logits(logits.data_ptr(), dt, rows, vocab, stride, k,
                                          temperature, idx.data_ptr(), vals.data_ptr(),
                                          lse.data_ptr(), _stream_handle(stream)))
    return idx, vals, lse


def _distill(logits, idx, vals, teacher_lse, labels, row_weight, temperature, kd_weight, ce_weight,
             bad_count, with_grad, grad, stream):
    torch = _torch()
    lib = load_library()
    stride = _logits(logits)
    rows, vocab = logits.shape
    dev = logits.device
    dt = _dtype(logits, "logits")
    k = vdt = 0
    if idx is not None:
        if vals is None or idx.dim() != 2:
            raise ValueError("idx must be 2-D and come with vals")
        k = idx.shape[1]
        vdt = _dtype(vals, "vals")
    f32 = (torch.float32,)
    ptrs = (_arg(idx, "idx", (torch.int32,), (rows, k), dev),
            _arg(vals, "vals", () if vals is None else (vals.dtype,), (rows, k), dev))
    side = (_arg(teacher_lse, "teacher_lse", f32, (rows,), dev),
            _arg(labels, "labels", (torch.int64,), (rows,), dev),
            _arg(row_weight, "row_weight", f32, (rows,), dev))
    bad = _arg(bad_count, "bad_count", (torch.int32,), (1,), dev)
    gstride = 0
    if grad is not None:
        if tuple(grad.shape) != (rows, vocab) or grad.dtype != logits.dtype:
            raise ValueError("grad must have the shape and type of the logits")
        gstride = _logits(grad, "grad")
    with _on(stream):
        loss = torch.empty(rows, dtype=torch.float32, device=dev)
        if with_grad and grad is None:
            grad = torch.empty(rows, vocab, dtype=logits.dtype, device=dev)
            gstride = max(vocab, 1)
        args = DistillArgs(logits.data_ptr(), dt, k, rows, vocab, stride, *ptrs, vdt, temperature,
                           kd_weight, ce_weight, *side, loss.data_ptr(),
                           grad.data_ptr() if with_grad else None, gstride, bad)
        _check(lib, lib.scape_distill_loss(ctypes.byref(args), _stream_handle(stream)))
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
    torch = _torch()
    stride = _logits(logits)
    tokens, experts = logits.shape
    groups = 1
    if cu_tokens is not None:
        if cu_tokens.dim() != 1 or cu_tokens.numel() < 2:
            raise ValueError("cu_tokens must be 1-D with at least 2 entries")
        groups = cu_tokens.numel() - 1
    return RouteArgs(logits.data_ptr(), _dtype(logits, "logits"), k, tokens, experts,
                     1 if renormalize else 0, stride,
                     _arg(cu_tokens, "cu_tokens", (torch.int32,), (groups + 1,), logits.device),
                     groups, _arg(valid, "valid", (torch.bool, torch.uint8), (tokens,),
                                  logits.device))


def route(logits, k: int, *, renormalize: bool = True, cu_tokens=None, valid=None, stream=None):
    """scape_route: (idx int32 [tokens, k], weights float32 [tokens, k], counts
    int32 [groups, experts], live int32 [groups + 2], losses float32 [2] =
    balance, z)."""
    torch = _torch()
    lib = load_library()
    args = _route_args(logits, k, renormalize, cu_tokens, valid)
    n, experts, groups, dev = max(k, 0), logits.shape[1], args.n_groups, logits.device
    need = ctypes.c_uint64()
    _check(lib, lib.scape_route_workspace(ctypes.byref(args), ctypes.byref(need)))
    with _on(stream):
        idx = torch.empty(args.tokens, n, dtype=torch.int32, device=dev)
        weights = torch.empty(args.tokens, n, dtype=torch.float32, device=dev)
        counts = torch.empty(groups, experts, dtype=torch.int32, device=dev)
        live = torch.empty(groups + 2, dtype=torch.int32, device=dev)
        losses = torch.empty(2, dtype=torch.float32, device=dev)
        ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
        _check(lib, lib.scape_route(ctypes.byref(args), idx.data_ptr(), weights.data_ptr(),
                                    counts.data_ptr(), live.data_ptr(), losses.data_ptr(),
                                    ws.data_ptr(), need.value, _stream_handle(stream)))
    return idx, weights, counts, live, losses


def route_backward(logits, idx, counts, live, *, d_weights=None, d_losses=None,
                   renormalize: bool = True, cu_tokens=None, stream=None):
    """scape_route_backward: the gradient of the logits, in their type."""
    torch = _torch()
    lib = load_library()
    if idx.dim() != 2:
        raise ValueError("idx must be 2-D")
    k = idx.shape[1]
    args = _route_args(logits, k, renormalize, cu_tokens, None)
    tokens, experts, dev = args.tokens, args.experts, logits.device
    i32, f32 = (torch.int32,), (torch.float32,)
    fwd = (_arg(idx, "idx", i32, (tokens, k), dev),
           _arg(counts, "counts", i32, (args.n_groups, experts), dev),
           _arg(live, "live", i32, (args.n_groups + 2,), dev),
           _arg(d_weights, "d_weights", f32, (tokens, k), dev),
           _arg(d_losses, "d_losses", f32, (2,), dev))
    with _on(stream):
        grad = torch.empty(tokens, experts, dtype=logits.dtype, device=dev)
        _check(lib, lib.scape_route_backward(ctypes.byref(args), *fwd, grad.data_ptr(),
                                             max(experts, 1), _stream_handle(stream)))
    return grad
