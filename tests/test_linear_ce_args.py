"""Argument errors of scape_linear_ce without a GPU: each is found before anything
touches the pointers or CUDA."""
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


@pytest.mark.parametrize("change,what", [
    (dict(dtype=2), "dtype=2"), (dict(dtype=7), "dtype=7"), (dict(rows=1 << 24), "rows"), (dict(vocab=0), "vocab"),
    (dict(vocab=1 << 24), "vocab"), (dict(dim=0), "dim"), (dict(dim=60, hidden_stride=64), "dim"), (dict(dim=65544), "dim"),
    (dict(hidden_stride=56), "hidden"), (dict(hidden_stride=68), "hidden"), (dict(weight_stride=1 << 32), "weight"),
    (dict(hidden=P + 8), "hidden"), (dict(weight=P + 2), "weight"), (dict(hidden=None), "hidden"), (dict(weight=None), "weight"),
    (dict(labels=None), "labels"), (dict(loss=None), "loss"), (dict(labels=P + 4), "aligned"), (dict(row_weight=P + 1), "aligned"),
    (dict(d_hidden=None), "together"), (dict(d_weight=None), "together"), (dict(d_hidden=P * 5 + 8), "d_hidden"),
    (dict(d_weight_stride=63), "d_weight"), (dict(d_hidden=P), "overlap"), (dict(d_weight=2 * P), "overlap"),
    (dict(d_weight=4 * P + 64), "overlap"), (dict(ws=None), "workspace"), (dict(ws=6 * P + 16), "workspace"),
    (dict(ws_bytes=0), "workspace"),
])
def test_linear_ce_rejects(lib, change, what):
    a = dict(hidden=P, weight=2 * P, dtype=0, rows=100, vocab=200, dim=64, hidden_stride=64, weight_stride=64, labels=3 * P,
             row_weight=None, loss=3 * P, d_hidden=4 * P, d_hidden_stride=64, d_weight=5 * P, d_weight_stride=64,
             bad_count=None, ws=6 * P, ws_bytes=1 << 40)
    a.update(change)
    ws, size = a.pop("ws"), a.pop("ws_bytes")
    says(lib, lib.scape_linear_ce(ctypes.byref(scape.LinearCeArgs(**a)), ws, size, None), what)


def test_linear_ce_workspace(lib):
    need = ctypes.c_uint64()
    says(lib, lib.scape_linear_ce_workspace(None, ctypes.byref(need)), "args")
    says(lib, lib.scape_linear_ce(None, P, 1 << 40, None), "args")
    a = scape.LinearCeArgs(dtype=1, rows=8192, vocab=131072, dim=4096)
    says(lib, lib.scape_linear_ce_workspace(ctypes.byref(a), None), "bytes")
    assert lib.scape_linear_ce_workspace(ctypes.byref(a), ctypes.byref(need)) == 0
    loss_alone = need.value
    a.d_hidden = a.d_weight = P
    assert lib.scape_linear_ce_workspace(ctypes.byref(a), ctypes.byref(need)) == 0
    logits = 8192 * 131072 * 2
    # the hidden states' copy, 4 bytes for 64 logits, row scalars; for gradients a piece of G, sums in parts and those of d_hidden
    assert loss_alone < 8192 * 4096 * 2 + logits / 32 + 8192 * 64
    assert need.value < loss_alone + (1 << 30) + (80 << 20) + 8192 * 4096 * 4 + 4096


@pytest.mark.parametrize("rows,taken", [(0, 64), (1, 64), (16, 64), (64, 64), (65, 128), (128, 128), (129, 256), (256, 256), (257, 512)])
@pytest.mark.parametrize("vocab", [1000, 32000, 1000003])
def test_linear_ce_workspace_of_few_rows(lib, rows, taken, vocab):
    # the bound that the header gives: rows rounded up to 64 (more than 128: to 256), 4 bytes for every 64 logits (up to
    # 128 rows: for every 8) and the last tile's, the hidden states, 28 bytes a row, some of every buffer for its alignment
    need = ctypes.c_uint64()
    a = scape.LinearCeArgs(dtype=0, rows=rows, vocab=vocab, dim=2048)
    assert lib.scape_linear_ce_workspace(ctypes.byref(a), ctypes.byref(need)) == 0
    words = vocab + 256
    loss_alone = taken * (words // (16 if rows > 128 else 2) + 2048 * 2 + 28) + 9 * 256
    assert need.value <= loss_alone
    a.d_hidden = a.d_weight = P
    assert lib.scape_linear_ce_workspace(ctypes.byref(a), ctypes.byref(need)) == 0
    sums = max(taken, 128) * 2048 * 4 if taken * words * 2 > 512 << 20 else 0  # (several pieces)
    assert need.value <= loss_alone + taken * words * 2 + (80 << 20) + sums + 1024
