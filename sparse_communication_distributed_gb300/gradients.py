"""Python binding of the gradients' norms of libscape (argument marshalling
only; the operators are defined in ``include/scape.h``): between the backward
pass and ``Scape.step``.

``grads`` is one worker's list of tensors, or a list of such lists, one for each
worker.  Tensors are contiguous CUDA tensors on the current device, each bf16,
fp16 or fp32, of any size.
"""
from __future__ import annotations

import ctypes
from array import array
from collections.abc import Iterable

from . import objective as _o
from .scape import GradsArgs


def _flat(grads, name: str):
    """(tensors of all workers, first tensor of each worker and the end)."""
    if isinstance(grads, _o.torch.Tensor):
        raise ValueError(f"{name} must be a list of tensors or of lists of them, not a tensor")
    grads = list(grads)
    if grads and not isinstance(grads[0], _o.torch.Tensor):
        first, flat = [0], []
        for worker in grads:
            if isinstance(worker, _o.torch.Tensor):
                raise ValueError(f"{name} must not mix tensors and lists")
            if not isinstance(worker, Iterable):  # (a parameter without a gradient, say)
                raise ValueError(f"{name} must hold tensors or lists of them, not {type(worker).__name__}")
            flat.extend(worker)
            first.append(len(flat))
        return flat, first
    return grads, [0, len(grads)]


def _describe(flat, name: str, dev):
    """Arrays of the tensors' addresses, sizes and types, checked.  (Lists have
    hundreds of tensors: each is gone through by calls that stay in C.)"""
    t, codes = _o.torch.Tensor, _o._codes
    try:
        contiguous = all(map(t.is_contiguous, flat))
    except TypeError:
        bad = next(x for x in flat if not isinstance(x, t))
        raise ValueError(f"{name} must hold tensors, not {type(bad).__name__}") from None
    if not contiguous:
        raise ValueError(f"{name} must hold contiguous tensors")
    where = set(map(t.get_device, flat))
    if where - {dev}:
        raise ValueError(f"{name} must be on the current CUDA device ({dev}), not on {sorted(where)} (-1: CPU)")
    dtypes = [x.dtype for x in flat]
    try:
        types = {d: codes[d] for d in set(dtypes)}
    except KeyError as e:
        raise ValueError(f"{name} must hold bfloat16, float16 or float32, not {e.args[0]}") from None
    if len(types) == 1:
        types = bytes(types.values()) * len(flat)
    else:
        types = bytes([types[d] for d in dtypes])
    return array("Q", map(t.data_ptr, flat)), array("Q", map(t.numel, flat)), types


def _run(grads, max_norm, out, clip: bool, stream):
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return _run(grads, max_norm, out, clip, None)
    torch, lib = _o.torch, _o._lib
    dev = torch.cuda.current_device()
    flat, first = _flat(grads, "grads")
    ptrs, numel, types = _describe(flat, "grads", dev)
    first = array("Q", first)
    groups = len(first) - 1
    args = GradsArgs(ptrs.buffer_info()[0], numel.buffer_info()[0], ctypes.cast(types, ctypes.c_void_p),
                     len(flat), groups, first.buffer_info()[0])
    need = ctypes.c_uint64()
    _o._check(lib.scape_grad_workspace(ctypes.byref(args), ctypes.byref(need)))
    norms = torch.empty(groups, dtype=torch.float32, device=dev)
    ws = torch.empty(need.value, dtype=torch.uint8, device=dev)
    raw = torch._C._cuda_getCurrentRawStream(dev)
    if not clip:
        _o._check(lib.scape_grad_norm(ctypes.byref(args), norms.data_ptr(), ws.data_ptr(), need.value, raw))
        return norms
    optrs = otypes = None
    if out is not None:
        oflat, _ = _flat(out, "out")
        optrs, onumel, otypes = _describe(oflat, "out", dev)
        if onumel != numel:
            raise ValueError("out must hold one tensor of the same size for each of grads")
    _o._check(lib.scape_clip_grads(ctypes.byref(args), max_norm,
                                   None if optrs is None else optrs.buffer_info()[0], otypes,
                                   norms.data_ptr(), ws.data_ptr(), need.value, raw))
    return norms


def grad_norm(grads, *, stream=None):
    """scape_grad_norm: the norm of every worker's gradients (float32
    [workers])."""
    return _run(grads, 0.0, None, False, stream)


def clip_grads(grads, max_norm: float, *, out=None, stream=None):
    """scape_clip_grads: scales every worker's gradients to a norm of at most
    ``max_norm``, in place or into ``out`` (nested like ``grads``, tensors of the
    same sizes and any of the types: views of the flat buffers that
    ``Scape.step`` takes).  Returns the norms before (float32 [workers])."""
    return _run(grads, max_norm, out, True, stream)
