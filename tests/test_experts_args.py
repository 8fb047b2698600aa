"""Argument errors of the calls for experts' rows and gradients' norms without a
GPU: each is found before anything touches the pointers or CUDA."""
import ctypes
import os

import pytest

from sparse_communication_distributed_gb300 import build, scape

P = 1 << 20  # a placeholder address, aligned


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(scape.LIB_PATH):
        build.build()
    return scape.load_library()


def says(lib, rc, what):
    assert rc == scape.SCAPE_EINVAL
    assert what in lib.scape_last_error(None).decode(), lib.scape_last_error(None).decode()


def sizes(lib, tokens, k, experts, align):
    room, need = ctypes.c_uint64(), ctypes.c_uint64()
    rc = lib.scape_expert_plan_sizes(tokens, k, experts, align, ctypes.byref(room), ctypes.byref(need))
    return rc, room.value, need.value


def test_plan_sizes(lib):
    assert sizes(lib, 0, 2, 8, 128) == (0, 0, 0)
    assert sizes(lib, 1, 2, 8, 128) == (0, 2 + 2 * 127, 0)       # no more segments than choices
    assert sizes(lib, 1000, 2, 8, 16) == (0, 2000 + 8 * 15, 0)   # one chunk of choices: no workspace
    rc, room, need = sizes(lib, 10000, 8, 64, 1)
    assert rc == 0 and room == 80000 and need > 0


@pytest.mark.parametrize("change,what", [
    (dict(experts=0), "experts"), (dict(experts=1025), "experts"), (dict(k=0), "k=0"), (dict(k=33), "k=33"),
    (dict(align=0), "align"), (dict(align=65537), "align"), (dict(tokens=1 << 31), "tokens"),
    (dict(tokens=1 << 30, k=2), "rows"), (dict(idx=None), "idx"), (dict(offsets=None), "offsets"),
    (dict(idx=P + 2), "aligned"), (dict(ws=None), "workspace"), (dict(ws=P + 4), "workspace"),
    (dict(ws_bytes=0), "workspace"),
])
def test_plan_rejects(lib, change, what):
    a = dict(idx=P, tokens=10000, k=2, experts=8, align=1, offsets=P, ws=P, ws_bytes=1 << 30)
    a.update(change)
    says(lib, lib.scape_expert_plan(a["idx"], a["tokens"], a["k"], a["experts"], a["align"], a["offsets"], P, P, None,
                                    a["ws"], a["ws_bytes"], None), what)


@pytest.mark.parametrize("change,what", [
    (dict(dtype=3), "dtype"), (dict(k=0), "k=0"), (dict(dim=0), "dim"), (dict(dim=1 << 24), "dim"),
    (dict(rows=1 << 31), "rows"), (dict(tokens=1 << 31), "tokens"), (dict(stride=63), "row_stride"),
    (dict(x=None), "x"), (dict(slots=None), "slots"), (dict(source=None), "source"), (dict(out=None), "out"),
    (dict(x=P + 1), "aligned"), (dict(out=P + (1 << 24) + 1), "aligned"), (dict(out=P + 128), "overlap"),
])
def test_dispatch_rejects(lib, change, what):
    a = dict(x=P, dtype=0, tokens=100, dim=64, stride=64, k=2, slots=P, source=P, rows=200, out=P + (1 << 24))
    a.update(change)
    says(lib, lib.scape_expert_dispatch(a["x"], a["dtype"], a["tokens"], a["dim"], a["stride"], a["k"], a["slots"],
                                        a["source"], a["rows"], a["out"], None), what)


@pytest.mark.parametrize("change,what", [
    (dict(dtype=-1), "dtype"), (dict(k=33), "k=33"), (dict(dim=0), "dim"), (dict(y=None), "y"), (dict(slots=None), "slots"),
    (dict(out=None), "out"), (dict(w=P + 2), "aligned"), (dict(y=P + 1), "aligned"), (dict(out=P + 256), "overlap"),
])
def test_combine_rejects(lib, change, what):
    a = dict(y=P, dtype=1, rows=200, dim=64, slots=P, w=P, tokens=100, k=2, out=P + (1 << 24))
    a.update(change)
    says(lib, lib.scape_expert_combine(a["y"], a["dtype"], a["rows"], a["dim"], a["slots"], a["w"], a["tokens"], a["k"],
                                       a["out"], None), what)
    if "w" not in change:
        says(lib, lib.scape_expert_combine_backward(P + (1 << 26), a["y"], a["dtype"], a["rows"], a["dim"], a["slots"], P, P,
                                                    a["tokens"], a["k"], a["out"], P, None), what)


def grads(numel=(100, 28), ptrs=(P, P + 4096), dtypes=b"\0\0", groups=1, first=None, drop=()):
    n = len(numel)
    keep = [(ctypes.c_uint64 * n)(*ptrs), (ctypes.c_uint64 * n)(*numel), dtypes,
            None if first is None else (ctypes.c_uint64 * len(first))(*first)]
    a = scape.GradsArgs(ctypes.addressof(keep[0]), ctypes.addressof(keep[1]), ctypes.cast(dtypes, ctypes.c_void_p), n,
                        groups, None if first is None else ctypes.addressof(keep[3]))
    for f in drop:
        setattr(a, f, None)
    a.keep = keep
    return a


@pytest.mark.parametrize("change,what", [
    (dict(groups=0), "n_groups"), (dict(groups=65), "n_groups"), (dict(groups=2), "first_tensor"),
    (dict(groups=1, first=(0, 1)), "first_tensor"), (dict(groups=2, first=(0, 3, 2)), "ascend"),
    (dict(numel=(1 << 40, 1)), "numel"), (dict(drop=("numel",)), "numel"), (dict(drop=("grads",)), "grads"),
    (dict(drop=("dtypes",)), "dtypes"), (dict(dtypes=b"\0\3"), "dtype"), (dict(ptrs=(P, 0)), "NULL"),
    (dict(ptrs=(P, P + 4097)), "aligned"),
])
def test_grads_reject(lib, change, what):
    a = grads(**change)
    says(lib, lib.scape_grad_norm(ctypes.byref(a), P, P, 1 << 30, None), what)
    says(lib, lib.scape_clip_grads(ctypes.byref(a), 1.0, None, None, P, P, 1 << 30, None), what)


def test_grads_reject_buffers(lib):
    a = grads()
    need = ctypes.c_uint64()
    assert lib.scape_grad_workspace(ctypes.byref(a), ctypes.byref(need)) == 0 and need.value > 0
    says(lib, lib.scape_grad_workspace(ctypes.byref(a), None), "bytes")
    says(lib, lib.scape_grad_workspace(None, ctypes.byref(need)), "grads")
    ref = ctypes.byref(a)
    says(lib, lib.scape_grad_norm(ref, None, P, 1 << 30, None), "norms")
    says(lib, lib.scape_grad_norm(ref, P + 2, P, 1 << 30, None), "norms")
    says(lib, lib.scape_grad_norm(ref, P, None, 1 << 30, None), "workspace")
    need = ctypes.c_uint64()
    lib.scape_grad_workspace(ref, ctypes.byref(need))
    says(lib, lib.scape_grad_norm(ref, P, P, need.value - 1, None), "workspace")
    for bad in (0.0, -1.0, float("nan")):
        says(lib, lib.scape_clip_grads(ref, bad, None, None, P, P, 1 << 30, None), "max_norm")


@pytest.mark.parametrize("ptrs,out,types,what", [
    ((P, P), None, b"\0\0", "overlap"),                           # the same tensor twice, in place
    ((P, P + 100), None, b"\0\0", "overlap"),                     # two views of the same elements, in place
    ((P, P + 4096), (P + 8192, P + 8194), b"\0\0", "overlap"),    # results over one another
    ((P, P + 4096), (P + 2, P + 8192), b"\0\0", "overlap"),       # a result over its own tensor, shifted
    ((P, P + 4096), (P, P + 8192), b"\2\2", "overlap"),           # ... in another type
    ((P, P + 4096), (P + 4096, P), b"\0\0", "overlap"),           # ... over the other one
    ((P, P + 4096), (P + 8192, 0), b"\0\0", "NULL"),
    ((P, P + 4096), (P + 8193, P + 16384), b"\0\0", "aligned"),
    ((P, P + 4096), (P + 8192, P + 16384), b"\0\7", "dtype"),
    ((P, P + 4096), (P + 8192, P + 16384), None, "out_dtypes"),
])
def test_clip_rejects_overlap(lib, ptrs, out, types, what):
    a = grads(ptrs=ptrs)
    arr = None if out is None else (ctypes.c_uint64 * 2)(*out)
    says(lib, lib.scape_clip_grads(ctypes.byref(a), 1.0, None if arr is None else ctypes.addressof(arr), types, P, P,
                                   1 << 30, None), what)


@pytest.mark.parametrize("worker", [None, 1.0])
def test_a_parameter_without_a_gradient(worker):
    torch = pytest.importorskip("torch")
    from sparse_communication_distributed_gb300 import gradients, objective
    objective._load()
    for grads in ([worker], [[torch.zeros(3)], worker]):
        with pytest.raises(ValueError, match=type(worker).__name__):
            gradients._flat(grads, "grads")
    with pytest.raises(ValueError, match=type(worker).__name__):
        gradients._describe([torch.zeros(3), worker], "grads", -1)
