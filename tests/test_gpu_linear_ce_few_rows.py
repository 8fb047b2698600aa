"""Linear cross entropy of few rows, whose buffers are as small as their rows allow:
a vocabulary that has several pieces all the same, and a workspace of exactly the size
that is asked for, with guards around it."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from objective_ref import ROUND  # noqa: E402
from sparse_communication_distributed_gb300 import scape  # noqa: E402

pytestmark = pytest.mark.gpu


def inputs(T, D, V, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    H = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, D, generator=gen, device="cuda") / math.sqrt(D)).bfloat16()
    return H, W, torch.randint(V, (T,), generator=gen, device="cuda")


@pytest.mark.parametrize("T,V", [(128, 2200003), (64, 4300003), (5, 4300003)])
def test_several_pieces_of_millions_of_words(T, V):
    # narrow tiles of words that lie in two pieces: nothing is kept, each piece is worked out again
    H, W, y = inputs(T, 8, V)
    y[0], y[1], y[2] = V - 1, V // 2, V // 2 + 1
    loss, dh, dw = pkg.linear_ce_grad(H, W, y)
    w, h = W.double(), H.double()
    G = h @ w.T
    lse = torch.logsumexp(G, 1, keepdim=True)
    assert float((loss[:, None].double() - (lse - G.gather(1, y[:, None]))).abs().max()) <= 1e-5
    G = torch.exp(G.sub_(lse))
    G.scatter_add_(1, y[:, None], torch.full((T, 1), -1.0, dtype=G.dtype, device="cuda"))
    for got, want in ((dh, G @ w), (dw, G.T @ h)):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * ROUND["bf16"]


@pytest.mark.parametrize("T", [1, 8, 17, 63, 64, 65, 100, 128, 129])
@pytest.mark.parametrize("V", [70, 5003])
@pytest.mark.parametrize("masked", [False, True])
def test_nothing_beside_the_workspace(T, V, masked):
    H, W, y = inputs(T, 72, V, seed=T)
    if masked:
        y[:T // 2] = -100
    want = pkg.linear_ce_grad(H, W, y)
    lib = scape.load_library()
    loss, dh, dw = torch.empty(T, device="cuda"), torch.empty_like(H), torch.empty_like(W)
    args = scape.LinearCeArgs(H.data_ptr(), W.data_ptr(), 0, T, V, 72, 72, 72, y.data_ptr(), None, loss.data_ptr(),
                              dh.data_ptr(), 72, dw.data_ptr(), 72, None)
    need = ctypes.c_uint64()
    assert lib.scape_linear_ce_workspace(ctypes.byref(args), ctypes.byref(need)) == 0
    buf = torch.full((need.value + 2 * 65536,), 0xA5, dtype=torch.uint8, device="cuda")
    at = buf.data_ptr() + 65536
    assert at % 256 == 0
    # (what the workspace held before does not matter: NaN in every type)
    buf[65536:65536 + need.value] = 0xFF
    assert lib.scape_linear_ce(ctypes.byref(args), at, need.value, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert bool(buf[:65536].eq(0xA5).all()) and bool(buf[65536 + need.value:].eq(0xA5).all())
    assert all(bool(torch.equal(a, b)) for a, b in zip((loss, dh, dw), want))
