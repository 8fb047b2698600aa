"""Python binding of the gradients' norms of libscape (argument marshalling
only; the operators are defined in ``include/scape.h``): between the backward
pass and ``Scape.step``.

``grads`` is one worker's list of tensors, or a list of such lists, one for each
worker.  Tensors are contiguous CUDA tensors on the current device, each bf16,
fp16 or fp32, of any size.
"""
from __future__ import annotations

import ctypes

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
            flat.extend(worker)
            first.append(len(flat))
        return flat, first
    return grads, [0, len(grads)]


def _describe(flat, name: str, dev):
    """Arrays of the tensors' addresses, sizes and types, checked."""
    t = _o.torch.Tensor
    codes, n = _o._codes, len(flat)
    for x in flat:
        if not isinstance(x, t):
            raise ValueError(f"{name} must hold tensors, not {type(x).__name__}")
    if not all(map(t.is_contiguous, flat)):
        raise ValueError(f"{name} must hold contiguous tensors")
    where = set(map(t.get_device, flat))
    if where - {dev}:
        raise ValueError(f"{name} must be on the current CUDA device ({dev}), not on {sorted(where)} (-1: CPU)")
    try:
        types = bytes([codes[x.dtype] for x in flat])
    except KeyError as e:
        raise ValueError(f"{name} must hold bfloat16, float16 or float32, not {e.args[0]}") from None
    numel = list(map(t.numel, flat))
    return (ctypes.c_uint64 * n)(*map(t.data_ptr, flat)), numel, (ctypes.c_uint64 * n)(*numel), types


def _run(grads, max_norm, out, clip: bool, stream):
    if _o._lib is None:
        _o._load()
    if stream is not None:
        with _o._stream_context(stream):
            return _run(grads, max_norm, out, clip, None)
    torch, lib = _o.torch, _o._lib
    dev = torch.cuda.current_device()
    flat, first = _flat(grads, "grads")
    ptrs, sizes, numel, types = _describe(flat, "grads", dev)
    groups = len(first) - 1
    first = (ctypes.c_uint64 * (groups + 1))(*first)
    args = GradsArgs(ctypes.addressof(ptrs), ctypes.addressof(numel), ctypes.cast(types, ctypes.c_void_p),
                     len(flat), groups, ctypes.addressof(first))
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
        optrs, osizes, _, otypes = _describe(oflat, "out", dev)
        if osizes != sizes:
            raise ValueError("out must hold one tensor of the same size for each of grads")
    _o._check(lib.scape_clip_grads(ctypes.byref(args), max_norm,
                                   None if optrs is None else ctypes.addressof(optrs), otypes,
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
