"""A wait of linear cross entropy's products that runs out, in the debug build: the
hook SCAPE_TEST_LOST_WAIT lets the first CTA wait for a barrier that nobody arrives at,
with its copies under way.  The kernels return, every loss and gradient is NaN, and the
next call is right."""
import os
import time

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from sparse_communication_distributed_gb300 import build as pkg_build  # noqa: E402
from sparse_communication_distributed_gb300 import objective  # noqa: E402
from sparse_communication_distributed_gb300.scape import DEBUG_LIB_PATH, load_library  # noqa: E402

pytestmark = pytest.mark.gpu
LOSS, GRAD, BACK = 1, 2, 3


@pytest.fixture
def debug_lib(monkeypatch):
    if not os.path.exists(DEBUG_LIB_PATH):
        pkg_build.build(debug_checks=True)
    objective._load()
    monkeypatch.setattr(objective, "_lib", load_library(DEBUG_LIB_PATH))


def inputs(T, D, V, dtype):
    gen = torch.Generator(device="cuda").manual_seed(T)
    H = torch.randn(T, D, generator=gen, device="cuda").to(dtype)
    W = (torch.randn(V, D, generator=gen, device="cuda") / 8).to(dtype)
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    y[1::5] = -100
    return H, W, y


def equal(a, b):
    return all(bool(torch.equal(x, y)) for x, y in zip(a, b))


# one row of tiles and pairs of CTAs; copies all issued before the wait and more of them to come; three pieces
@pytest.mark.parametrize("T,D,V", [(40, 64, 1000), (100, 2048, 5000), (300, 64, 1000), (700, 2048, 3001), (20000, 64, 30001)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_wait_that_runs_out(T, D, V, dtype, debug_lib, monkeypatch):
    H, W, y = inputs(T, D, V, dtype)
    want = pkg.linear_ce_grad(H, W, y)
    torch.cuda.synchronize()
    for job in (LOSS, GRAD, BACK):
        if job == GRAD and T < 20000:
            continue  # (nothing is recomputed)
        monkeypatch.setenv("SCAPE_TEST_LOST_WAIT", str(job))
        began = time.monotonic()
        got = pkg.linear_ce_grad(H, W, y)
        torch.cuda.synchronize()
        assert time.monotonic() - began < 20.0
        assert all(bool(x.isnan().all()) for x in got)
        if job == LOSS:
            assert bool(pkg.linear_ce(H, W, y)[y >= 0].isnan().all())
        monkeypatch.delenv("SCAPE_TEST_LOST_WAIT")
        again = pkg.linear_ce_grad(H, W, y)
        torch.cuda.synchronize()
        assert equal(again, want)


def test_the_debug_build_gives_the_same_bits(debug_lib, monkeypatch):
    H, W, y = inputs(500, 136, 3001, torch.bfloat16)
    want = pkg.linear_ce_grad(H, W, y)
    monkeypatch.undo()
    assert equal(pkg.linear_ce_grad(H, W, y), want)
