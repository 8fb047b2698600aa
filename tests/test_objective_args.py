"""Argument errors of the training-objective calls without a GPU: each is found
before anything touches the pointers or CUDA."""
import ctypes
import os

import pytest

from sparse_communication_distributed_gb300 import build, scape

P = 1 << 20  # a placeholder address, aligned
BIG = 1 << 32


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(scape.LIB_PATH):
        build.build()
    return scape.load_library()


def says(lib, rc, what):
    assert rc == scape.SCAPE_EINVAL
    assert what in lib.scape_last_error(None).decode(), lib.scape_last_error(None).decode()


@pytest.mark.parametrize("change,what", [
    (dict(dtype=3), "dtype"), (dict(vocab=0), "vocab"), (dict(vocab=1 << 31, stride=1 << 31), "vocab"),
    (dict(k=0), "k=0"), (dict(k=1025), "k=1025"), (dict(k=51, vocab=50), "k=51"), (dict(stride=99), "row_stride"),
    (dict(tau=0.0), "temperature"), (dict(tau=float("nan")), "temperature"), (dict(tau=float("inf")), "temperature"),
    (dict(tau=1e-45), "temperature"), (dict(rows=1 << 31), "rows"), (dict(stride=BIG), "row_stride"),
    (dict(x=None), "logits"), (dict(idx=None), "idx"), (dict(x=P + 1), "aligned"), (dict(idx=P + 2), "aligned"),
])
def test_topk_rejects(lib, change, what):
    a = dict(x=P, dtype=0, rows=2, vocab=100, stride=100, k=5, tau=1.0, idx=P)
    a.update(change)
    says(lib, lib.scape_topk_logits(a["x"], a["dtype"], a["rows"], a["vocab"], a["stride"], a["k"], a["tau"], a["idx"],
                                    P, P, None), what)


@pytest.mark.parametrize("change,what", [
    (dict(dtype=-1), "dtype"), (dict(vals_dtype=9), "vals_dtype"), (dict(vocab=0), "vocab"), (dict(k=-1), "k=-1"),
    (dict(k=1025), "k=1025"), (dict(row_stride=99), "row_stride"), (dict(grad_stride=99), "grad_stride"),
    (dict(rows=1 << 31), "rows"), (dict(grad_stride=BIG), "strides"), (dict(temperature=0.0), "temperature"),
    (dict(temperature=float("inf")), "temperature"), (dict(kd_weight=float("nan")), "kd_weight"),
    (dict(ce_weight=float("inf")), "ce_weight"), (dict(loss=None, grad=None), "loss or grad"), (dict(logits=None), "logits"),
    (dict(idx=None), "idx"), (dict(vals=None), "vals"), (dict(labels=P + 4), "aligned"), (dict(grad=P + 1), "aligned"),
    (dict(grad=P, grad_stride=128), "in-place"),
])
def test_distill_rejects(lib, change, what):
    a = dict(logits=P, dtype=0, k=5, rows=2, vocab=100, row_stride=100, idx=2 * P, vals=2 * P, vals_dtype=2,
             temperature=1.0, kd_weight=1.0, ce_weight=0.0, loss=2 * P, grad=2 * P, grad_stride=100)
    a.update(change)
    says(lib, lib.scape_distill_loss(ctypes.byref(scape.DistillArgs(**a)), None), what)


def test_null_arguments(lib):
    says(lib, lib.scape_distill_loss(None, None), "args")
    says(lib, lib.scape_route(None, P, P, P, P, P, P, 1 << 20, None), "args")
    says(lib, lib.scape_route_workspace(None, ctypes.byref(ctypes.c_uint64())), "args")
    says(lib, lib.scape_route_workspace(ctypes.byref(scape.RouteArgs()), None), "bytes")


def route_args(**change):
    a = dict(logits=P, dtype=0, k=2, tokens=100, experts=16, renormalize=1, row_stride=16, cu_tokens=None, n_groups=1,
             valid=None)
    a.update(change)
    return ctypes.byref(scape.RouteArgs(**a))


@pytest.mark.parametrize("change,what", [
    (dict(dtype=3), "dtype"), (dict(experts=0), "experts"), (dict(experts=1025, row_stride=1025), "experts"),
    (dict(k=0), "k=0"), (dict(k=17), "k=17"), (dict(k=33, experts=64, row_stride=64), "k=33"),
    (dict(tokens=1 << 31), "tokens"), (dict(row_stride=15), "row_stride"), (dict(n_groups=0), "n_groups"),
    (dict(n_groups=1 << 27, cu_tokens=P), "n_groups"), (dict(n_groups=2), "cu_tokens"), (dict(logits=None), "logits"),
    (dict(logits=P + 1), "aligned"),
])
def test_route_rejects(lib, change, what):
    says(lib, lib.scape_route(route_args(**change), P, P, P, P, P, P, 1 << 30, None), what)
    says(lib, lib.scape_route_backward(route_args(**change), P, P, P, P, P, 2 * P, 1 << 20, None), what)


def test_route_rejects_buffers(lib):
    need = ctypes.c_uint64()
    assert lib.scape_route_workspace(route_args(), ctypes.byref(need)) == 0 and need.value == 0  # a few tokens: none
    many = dict(tokens=100000)
    assert lib.scape_route_workspace(route_args(**many), ctypes.byref(need)) == 0 and need.value > 0
    says(lib, lib.scape_route(route_args(**many), P, P, P, P, P, P, need.value - 1, None), "workspace")
    says(lib, lib.scape_route(route_args(**many), P, P, P, P, P, P + 4, need.value, None), "workspace")
    says(lib, lib.scape_route(route_args(**many), P, P, P, P, P, None, need.value, None), "workspace")
    says(lib, lib.scape_route(route_args(), None, P, P, P, P, P, need.value, None), "idx")
    says(lib, lib.scape_route(route_args(), P, P, P + 2, P, P, P, need.value, None), "aligned")
    says(lib, lib.scape_route_backward(route_args(), P, P, P, P, P, 2 * P, 15, None), "grad_stride")
    says(lib, lib.scape_route_backward(route_args(), P, P, P, P, P, P, 16, None), "logits")
    says(lib, lib.scape_route_backward(route_args(), P, None, P, P, P, 2 * P, 16, None), "counts")
