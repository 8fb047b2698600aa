"""Linear cross entropy and its gradients against the definition in 64 bits: both
types, odd sizes, strided views, rows without a term, one row and many pieces.

Bounds, U = 2^-24.  Products of 16-bit numbers are exact in fp32; the tensor cores
add them up in fp32, at least eight at a time, each such addition off by at most
2^-23 of the sum of magnitudes so far.  So a logit of D products is off by
  dl = (D / 8) 2^-23 sum_d |h_d W_d|,
a loss by w (2 dl + the bound of a log-sum-exp + roundings of its logits), a
probability by the factor 2 dl + that bound, an entry of G by p times this, its
rounding (half a step) and, for fp16, half the least step at the scale 2^14 of the
largest weight.  The exponentials are rounded to fp16 first, times 2^15 and against
the largest of their 128 words, so p carries half a step of that type and half its
least step, 2^-25, times 2^-15 of the largest p.  A gradient of n terms carries the terms' errors, n / 8 additions
and its own rounding.  These bounds hold whatever the signs; roundings of random
sign give a far smaller norm of the error, which is held to 2 half steps besides
(one of G, one of the result; equal parts of random sign would be sqrt(2 / 3))."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from objective_ref import ROUND, TINY, U, lse_tol  # noqa: E402
from sparse_communication_distributed_gb300 import ScapeError  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def inputs(T, D, V, dtype, seed=0, pad=0, scale=1.0, masked=0.0, weights=True):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def place(x):
        wide = torch.full((x.shape[0], D + 2 * pad), float("nan"), dtype=DT[dtype], device="cuda")
        wide[:, pad:pad + D] = x.to(DT[dtype])
        return wide[:, pad:pad + D] if pad else wide

    H, W = place(rand(T, D)), place(rand(V, D) * (scale / math.sqrt(D)))
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    y[torch.rand(T, generator=gen, device="cuda") < masked / 2] = -100
    w = None
    if weights:
        w = torch.rand(T, generator=gen, device="cuda") * 2 / T
        w[torch.rand(T, generator=gen, device="cuda") < masked / 2] = 0.0
    return H, W, y, w


def check(H, W, y, w, dtype, grad=True, norms=True):
    """One call with and one without gradients against 64 bits."""
    T, D = H.shape
    V = W.shape[0]
    if grad:
        loss, dh, dw = pkg.linear_ce_grad(H, W, y, row_weight=w)
        assert torch.equal(loss, pkg.linear_ce(H, W, y, row_weight=w))
    else:
        loss = pkg.linear_ce(H, W, y, row_weight=w)
    ww = torch.ones(T, device="cuda") if w is None else w
    on = (y >= 0) & (y < V) & (ww != 0)
    assert loss[~on].eq(0).all()
    at = torch.nonzero(on).squeeze(1)
    h, wt, k = H[at].double(), W.double(), ww[at].double()[:, None]
    x = h @ wt.T
    dl = (D / 8) * 2.0 ** -23 * (h.abs() @ wt.abs().T)
    lse = torch.logsumexp(x, 1, keepdim=True)
    ly = x.gather(1, y[at, None])
    ref = k * (lse - ly)
    dmax = dl.amax(1, keepdim=True) if at.numel() else dl
    tol_l = 2 * lse_tol(V) + 4 * U * (lse.abs() + ly.abs() + x.amax(1, keepdim=True).abs() if at.numel() else 0)
    if at.numel():
        off = (loss[at, None].double() - ref).abs() - (k.abs() * (2 * dmax + tol_l) + U * ref.abs())
        assert off.max().item() <= 0, off.max().item()
    if not grad:
        return
    p = torch.softmax(x, 1)
    G = p.clone()
    G.scatter_add_(1, y[at, None], torch.full_like(ly, -1.0))
    G *= k
    top = float(k.abs().max()) if at.numel() else 1.0
    eG = k.abs() * p * (2 * dl + tol_l + 8 * U) if at.numel() else G
    if at.numel():
        eG = eG + k.abs() * (ROUND["f16"] * p + 2.0 ** -40 * p.amax(1, keepdim=True))
    eG = eG + ROUND[dtype] * G.abs() + (top * 2.0 ** -14 * 2.0 ** -25 if dtype == "f16" else 0.0)
    assert dh[~on].eq(0).all()
    for got, a, b, ea, n in ((dh[at], G, wt, eG, V), (dw, G.T, h, eG.T, max(1, at.numel()))):
        want, size = a @ b, a.abs() @ b.abs()
        bound = (1 + 2 * ROUND[dtype]) * (ea @ b.abs()) + (n / 8 + 4) * 2.0 ** -23 * size
        bound = bound + ROUND[dtype] * (want.abs() + bound) + TINY[dtype]
        off = (got.double() - want).abs() - bound
        assert off.numel() == 0 or off.max().item() <= 0, off.max().item()
        if norms and float(want.abs().max() if want.numel() else 0) > 1e-3 * (1 if dtype == "f16" else 0):
            rel = float((got.double() - want).norm() / want.norm())
            assert rel <= 2 * ROUND[dtype], rel


SIZES = [(1, 8, 1), (1, 64, 5), (3, 72, 300), (2, 8, 257), (128, 64, 256), (129, 128, 257), (200, 136, 1000), (257, 1024, 1003),
         (64, 2048, 5000), (1000, 256, 4999), (300, 520, 20011), (16, 2048, 32000), (511, 1280, 777), (1, 4096, 50257)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,D,V", SIZES)
def test_sizes(T, D, V, dtype):
    H, W, y, w = inputs(T, D, V, dtype, seed=T + V, masked=0.3 if T > 3 else 0.0)
    if dtype == "f16" and w is not None:
        w *= T  # (loss scaling: the gradients stay above fp16's denormals)
    check(H, W, y, w, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_views_of_wider_rows(dtype):
    # what lies beside the rows is NaN
    H, W, y, w = inputs(150, 200, 700, dtype, pad=8, masked=0.2, weights=False)
    check(H, W, y, w, dtype)


def test_several_pieces_of_the_vocabulary():
    H, W, y, w = inputs(8200, 64, 33003, "bf16", masked=0.1)
    check(H, W, y, w, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pieces_that_are_worked_out_again(dtype):
    # more logits than exponentials are kept of (1 GB): three pieces, the last one recomputed
    H, W, y, w = inputs(20000, 64, 30001, dtype, masked=0.05)
    check(H, W, y, w * (8192.0 if dtype == "f16" else 1.0), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [3, 128])
def test_a_few_rows_of_a_million_words(T, dtype):
    # two pieces, and narrow tiles of words that lie in both: nothing is kept
    H, W, y, w = inputs(T, 8, 1100003, dtype, weights=False)
    y[0], y[1], y[2] = 1100002, 550143, 550144
    check(H, W, y, w, dtype)


def test_many_rows():
    H, W, y, w = inputs(300001, 64, 1000, "bf16", masked=0.3)
    check(H, W, y, w, "bf16")


def test_the_widest_rows():
    H, W, y, w = inputs(150, 65536, 300, "bf16", masked=0.1)
    check(H, W, y, w, "bf16")


@pytest.mark.parametrize("T", [127, 128, 129, 255, 256, 257])
def test_around_the_tiles_of_rows(T):
    for V in (255, 256, 257, 513):
        H, W, y, w = inputs(T, 64, V, "bf16", seed=V, weights=False)
        y[-1], y[0] = V - 1, 0
        check(H, W, y, w, "bf16")


def test_labels_beyond_32_bits_are_counted():
    H, W, y, w = inputs(50, 64, 100, "bf16")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    y[3], y[4], y[5] = 2 ** 32 + 5, 2 ** 62, -2 ** 40
    loss = pkg.linear_ce(H, W, y, row_weight=w, bad_count=bad)
    assert int(bad) == 2 and loss[3:6].eq(0).all() and (loss[6:] > 0).all()


def test_many_tiles_of_every_product():
    H, W, y, w = inputs(5000, 1288, 9001, "bf16", masked=0.05)
    check(H, W, y, w, "bf16")


@pytest.mark.parametrize("scale", [0.0, 30.0, 3000.0])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_flat_and_sharp_rows(scale, dtype):
    # all logits 0 (the loss is ln V); one word nearly certain; one word certain, and a wrong label
    H, W, y, w = inputs(140, 128, 3000, dtype, scale=scale, weights=False)
    with torch.no_grad():
        y[:70] = (H[:70].double() @ W.double().T).argmax(1)
    check(H, W, y, w, dtype, norms=scale != 3000.0)
    if scale == 0.0:
        got = pkg.linear_ce(H, W, y)
        assert (got.double() - math.log(3000)).abs().max().item() <= 2 * lse_tol(3000, math.log(3000))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_row_weights_of_any_size(dtype):
    H, W, y, _ = inputs(300, 64, 500, dtype)
    w = torch.ones(300, device="cuda")
    w[::3] = -0.5
    check(H, W, y, w * 16, dtype)
    # far from 1: the gradients scale by the same power of two, exactly
    _, dh, dw = pkg.linear_ce_grad(H, W, y, row_weight=w)
    for s in (2.0 ** -10, 2.0 ** 3) if dtype == "f16" else (2.0 ** -60, 2.0 ** 60):
        _, eh, ew = pkg.linear_ce_grad(H, W, y, row_weight=w * s)
        for a, b in ((dh, eh), (dw, ew)):
            a, b = a.double(), b.double()
            # exactly, as long as neither side is among the type's denormals; those are off by half their step
            # (fp16: 2^-25), on the unscaled side times s
            small = torch.minimum(a.abs(), a.abs() * s) < (2.0 ** -14 if dtype == "f16" else 2.0 ** -120)
            assert torch.equal(a[~small] * s, b[~small])
            assert (a * s - b).abs().max().item() <= (1 + s) * TINY[dtype]


def test_a_wide_range_of_row_weights_in_fp16():
    # weights down to 2^-10 of the largest, flat rows: entries of G far below fp16's range without the scaling
    H, W, y, _ = inputs(256, 64, 30000, "f16", scale=0.1)
    w = 2.0 ** -torch.randint(0, 11, (256,), device="cuda").float()
    check(H, W, y, w, "f16")


def test_rows_without_a_term_are_not_read():
    H, W, y, w = inputs(400, 64, 300, "bf16", masked=0.0)
    y[7], y[9], w[11] = -1, -100, 0.0
    w[13], y[15] = 0.0, 300
    want = pkg.linear_ce_grad(H, W, y, row_weight=w)
    H2 = H.clone()
    for r in (7, 9, 11, 13, 15):
        H2[r] = float("nan")
    bad = torch.full((1,), 3, dtype=torch.int32, device="cuda")
    got = pkg.linear_ce_grad(H2, W, y, row_weight=w, bad_count=bad)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and int(bad) == 4
    for r in (7, 9, 11, 13, 15):
        assert float(got[0][r]) == 0 and got[1][r].eq(0).all()
    # the rows that are left, alone
    keep = [r for r in range(400) if r not in (7, 9, 11, 13, 15)]
    alone = pkg.linear_ce_grad(H[keep], W, y[keep], row_weight=w[keep])
    assert torch.equal(alone[0], got[0][keep]) and torch.equal(alone[1], got[1][keep]) and torch.equal(alone[2], got[2])


@pytest.mark.parametrize("T", [0, 1, 300])
def test_no_row_has_a_term(T):
    H, W, y, _ = inputs(T, 64, 500, "bf16")
    y.fill_(-100)
    loss, dh, dw = pkg.linear_ce_grad(H, W, y)
    assert loss.shape == (T,) and loss.eq(0).all() and dh.shape == (T, 64) and dh.eq(0).all()
    assert dw.shape == (500, 64) and dw.eq(0).all()
    assert pkg.linear_ce(H, W, y).eq(0).all()


def test_nan_stays_in_its_row():
    H, W, y, w = inputs(300, 64, 500, "bf16")
    want = pkg.linear_ce_grad(H, W, y, row_weight=w)
    H[20, 3], H[21, 5] = float("nan"), float("inf")
    loss, dh, dw = pkg.linear_ce_grad(H, W, y, row_weight=w)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[20:22] = False
    assert torch.isnan(loss[20:22]).all() and torch.equal(loss[rest], want[0][rest])
    assert torch.isnan(dh[20]).all() and torch.equal(dh[rest], want[1][rest])
    assert torch.isnan(dw[:, 3]).all()


def test_gradient_against_differences():
    # along a direction v: (f(x + s v) - f(x - s v)) / 2 s is off by s^2 / 6 of the third derivative, at most
    # 2 a^3 for a change of the logits by at most a; and by the losses' own errors over s
    T, D, V = 40, 64, 100
    H, W, y, _ = inputs(T, D, V, "f16", scale=1.0)
    H, W = (H.double() * 64).round().div(64).half(), (W.double() * 256).round().div(256).half()
    loss, dh, dw = pkg.linear_ce_grad(H, W, y)
    for which, grad in (("h", dh), ("w", dw)):
        v = torch.randint(-1, 2, grad.shape, device="cuda", dtype=torch.int32).half()
        s = 2.0 ** -6
        up, down = ((H + s * v, W), (H - s * v, W)) if which == "h" else ((H, W + s * v), (H, W - s * v))
        diff = (pkg.linear_ce(*up, y).double().sum() - pkg.linear_ce(*down, y).double().sum()) / (2 * s)
        a = (v.double() @ W.double().T if which == "h" else H.double() @ v.double().T).abs().amax(1)
        size = (grad.double() * v.double()).abs().sum()
        tol = float((s * s / 3 * a ** 3).sum() + T * 1e-5 / s + 2 * ROUND["f16"] * size * 2)
        assert abs(float(diff) - float((grad.double() * v.double()).sum())) <= tol


def test_past_32_bit_offsets():
    # the last words' rows start 4.8e9 elements into the buffer
    V, D, stride = 257, 64, 18_750_000
    buf = torch.zeros((V - 1) * stride + D, dtype=torch.bfloat16, device="cuda")
    W = torch.as_strided(buf, (V, D), (stride, 1))
    H, W0, y, w = inputs(130, D, V, "bf16")
    W.copy_(W0)
    want = pkg.linear_ce_grad(H, W0, y, row_weight=w)
    got = pkg.linear_ce_grad(H, W, y, row_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_repeats_streams_and_graphs():
    H, W, y, w = inputs(700, 256, 3001, "bf16", masked=0.2)
    want = pkg.linear_ce_grad(H, W, y, row_weight=w)
    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [pkg.linear_ce_grad(H, W, y, row_weight=w, stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graphs, held = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(pkg.linear_ce_grad(H, W, y, row_weight=w))
        graphs.append(g)
    H.copy_(H.flip(0))
    y[5] = -100
    want = pkg.linear_ce_grad(H, W, y, row_weight=w)
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for h in held:
        assert all(torch.equal(a, b) for a, b in zip(want, h))


def test_refusals():
    H, W, y, w = inputs(10, 64, 50, "bf16")
    with pytest.raises(ScapeError, match="bf16 or fp16"):
        pkg.linear_ce(H.float(), W.float(), y)
    with pytest.raises(ValueError, match="weight"):
        pkg.linear_ce(H, W.half(), y)
    with pytest.raises(ValueError, match="weight"):
        pkg.linear_ce(H, W[:, :32], y)
    with pytest.raises(ValueError, match="labels"):
        pkg.linear_ce(H, W, y.int())
    with pytest.raises(ValueError, match="labels"):
        pkg.linear_ce(H, W, None)
    with pytest.raises(ValueError, match="row_weight"):
        pkg.linear_ce(H, W, y, row_weight=w[:5])
    with pytest.raises(ScapeError, match="multiple of 8"):
        pkg.linear_ce(H[:, :60].contiguous(), W[:, :60].contiguous(), y)
    with pytest.raises(ScapeError, match="aligned"):
        pkg.linear_ce(torch.zeros(641, dtype=torch.bfloat16, device="cuda")[1:].view(10, 64), W, y)
    with pytest.raises(ScapeError, match="stride"):
        pkg.linear_ce(torch.zeros(10, 68, dtype=torch.bfloat16, device="cuda")[:, :64], W, y)
    with pytest.raises(ValueError, match="column stride"):
        pkg.linear_ce(H.T.contiguous().T, W, y)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.linear_ce(H.cpu(), W, y)
    with pytest.raises(ScapeError, match="vocab"):
        pkg.linear_ce(H, W[:0], y)
