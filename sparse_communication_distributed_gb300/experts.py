"""Python binding of the experts' rows of libscape (argument marshalling only;
the operators are defined in ``include/scape.h``): between ``route`` and the
experts' matrix products, and back.

Conventions as in ``objective``: CUDA tensors on the current device, new tensors
as results, no autograd graph.  The gradient of ``expert_dispatch`` is
``expert_combine`` of the rows' gradient without weights, that of
``expert_combine`` is ``expert_combine_backward``.
"""
from __future__ import annotations

import ctypes

from . import objective as _o


def _int32(x, name: str, dim: int, dev):
    if x.dtype is _o.torch.int32 and x.dim() == dim and x.is_contiguous() and x.device == dev:
        return x.data_ptr()
    raise ValueError(f"{name} must be contiguous, int32 and {dim}-D on {dev}, not {x.dtype} of shape "
                     f"{tuple(x.shape)} with strides {x.stride()} on {x.device}")


def _contiguous(x, name: str):
    _o._rows(x, name)
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous, not of strides {x.stride()}")
    return x.data_ptr()


def _raw(dev):
    return _o.torch._C._cuda_getCurrentRawStream(dev.index)


def expert_plan(idx, experts: int, *, align: int = 1, bad_count=None, stream=None):
    """scape_expert_plan: (offsets int32 [experts + 1], slots int32 [tokens, k],
    source int32 [capacity]) of the router's choices ``idx`` [tokens, k]."""
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return expert_plan(idx, experts, align=align, bad_count=bad_count)
    t, lib = _o.torch, _o._lib
    _o._rows(idx, "idx")
    (tokens, k), dev = idx.shape, idx.device
    p_idx = _int32(idx, "idx", 2, dev)
    p_bad = _o._arg(bad_count, "bad_count", (t.int32,), (1,), dev)
    _o._count(experts)
    _o._count(align)
    room, need = ctypes.c_uint64(), ctypes.c_uint64()
    _o._check(lib.scape_expert_plan_sizes(tokens, k, experts, align, ctypes.byref(room),
                                          ctypes.byref(need)))
    offsets = t.empty(experts + 1, dtype=t.int32, device=dev)
    slots = t.empty((tokens, k), dtype=t.int32, device=dev)
    source = t.empty(room.value, dtype=t.int32, device=dev)
    ws = t.empty(need.value, dtype=t.uint8, device=dev) if need.value else None
    _o._check(lib.scape_expert_plan(p_idx, tokens, k, experts, align, offsets.data_ptr(),
                                    slots.data_ptr(), source.data_ptr(), p_bad,
                                    None if ws is None else ws.data_ptr(), need.value, _raw(dev)))
    return offsets, slots, source


def expert_dispatch(x, slots, source, *, stream=None):
    """scape_expert_dispatch: the rows [capacity, dim] by expert of the tokens'
    rows ``x`` [tokens, dim] (any row stride)."""
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return expert_dispatch(x, slots, source)
    stride = _o._rows(x, "x")
    code = _o._code(x, "x")
    (tokens, dim), dev = x.shape, x.device
    p_slots, p_source = _int32(slots, "slots", 2, dev), _int32(source, "source", 1, dev)
    if slots.shape[0] != tokens:
        raise ValueError(f"slots must have {tokens} rows, not {slots.shape[0]}")
    rows = source.shape[0]
    out = _o.torch.empty((rows, dim), dtype=x.dtype, device=dev)
    _o._check(_o._lib.scape_expert_dispatch(x.data_ptr(), code, tokens, dim, stride, slots.shape[1],
                                            p_slots, p_source, rows, out.data_ptr(), _raw(dev)))
    return out


def expert_combine(y, slots, weights=None, *, stream=None):
    """scape_expert_combine: the tokens' rows [tokens, dim] summed from the
    experts' rows ``y`` [rows, dim] with ``weights`` float32 [tokens, k]
    (None: all 1)."""
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return expert_combine(y, slots, weights)
    p_y = _contiguous(y, "y")
    code = _o._code(y, "y")
    (rows, dim), dev = y.shape, y.device
    p_slots = _int32(slots, "slots", 2, dev)
    tokens, k = slots.shape
    p_w = _o._arg(weights, "weights", (_o.torch.float32,), (tokens, k), dev)
    out = _o.torch.empty((tokens, dim), dtype=y.dtype, device=dev)
    _o._check(_o._lib.scape_expert_combine(p_y, code, rows, dim, p_slots, p_w, tokens, k,
                                           out.data_ptr(), _raw(dev)))
    return out


def expert_combine_backward(d_out, y, slots, source, weights, *, stream=None):
    """scape_expert_combine_backward: (d_y [rows, dim], d_weights float32
    [tokens, k])."""
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return expert_combine_backward(d_out, y, slots, source, weights)
    t = _o.torch
    p_y = _contiguous(y, "y")
    code = _o._code(y, "y")
    (rows, dim), dev = y.shape, y.device
    p_slots, p_source = _int32(slots, "slots", 2, dev), _int32(source, "source", 1, dev)
    tokens, k = slots.shape
    if source.shape[0] != rows:
        raise ValueError(f"source must have {rows} entries, not {source.shape[0]}")
    if weights is None or d_out is None:
        raise ValueError("d_out and weights are required")
    p_g = _o._arg(d_out, "d_out", (y.dtype,), (tokens, dim), dev)
    p_w = _o._arg(weights, "weights", (t.float32,), (tokens, k), dev)
    d_y = t.empty((rows, dim), dtype=y.dtype, device=dev)
    d_w = t.empty((tokens, k), dtype=t.float32, device=dev)
    _o._check(_o._lib.scape_expert_combine_backward(p_g, p_y, code, rows, dim, p_slots, p_source,
                                                    p_w, tokens, k, d_y.data_ptr(), d_w.data_ptr(),
                                                    _raw(dev)))
    return d_y, d_w
