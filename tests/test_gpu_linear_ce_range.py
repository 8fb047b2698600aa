"""Linear cross entropy's gradients word by word, where the logits of a row lie far
apart: a word that is no row's label gets a gradient of nothing but small
probabilities, which a norm over all words does not see.

Bounds as in test_gpu_linear_ce.py, but without its absolute share of a row's largest
probability.  What is kept of a probability for the gradient is right to 2^-9 of itself
(bf16; fp16: to 2^-11) as far down as the type of G holds it: bf16 to fp32's least
normal number, fp16 to half its least step, 2^-25, at the largest weight's 2^14."""
import math

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from objective_ref import ROUND, TINY, U, lse_tol  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
KEPT = {"bf16": 2.0 ** -9, "f16": 2.0 ** -11}


def peaked(T, D, V, dtype, span, seed=0):
    """Hidden states along one direction, words spread along it: in every stretch of
    words some logits are next to the row's largest and some "span" nats below it.
    Labels are among the likely words."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    u = torch.full((D,), 1 / math.sqrt(D), device="cuda")
    a = torch.rand(V, generator=gen, device="cuda") * -span
    H = (8 * u + 0.25 * rand(T, D)).to(DT[dtype])
    W = (a[:, None] / 8 * u + 0.02 * rand(V, D)).to(DT[dtype])
    likely = torch.nonzero(a > -span / 20).squeeze(1)
    y = likely[torch.randint(likely.numel(), (T,), generator=gen, device="cuda")]
    return H, W, y


def check_words(H, W, y, dtype):
    (T, D), V = H.shape, W.shape[0]
    _, _, dw = pkg.linear_ce_grad(H, W, y)
    word = torch.ones(V, dtype=torch.bool, device="cuda")
    word[y] = False
    h, wt = H.double(), W.double()
    x = h @ wt.T
    lse = torch.logsumexp(x, 1, keepdim=True)
    tol = 2 * lse_tol(V) + 4 * U * (lse.abs() + x.abs().amax(1, keepdim=True)) + 8 * U
    p = torch.exp(x - lse)[:, word]
    # (logits far from the largest carry roundings of the distance in fp32, too)
    eG = p * (2 * (D / 8) * 2.0 ** -23 * (h.abs() @ wt[word].abs().T) + tol + KEPT[dtype] + ROUND[dtype])
    if dtype == "f16":
        eG += 2.0 ** -39
    want, size = p.T @ h, p.T @ h.abs()
    bound = (1 + 2 * ROUND[dtype]) * (eG.T @ h.abs()) + (T / 8 + 4) * 2.0 ** -23 * size
    bound += ROUND[dtype] * (want.abs() + bound) + TINY[dtype]
    off = (dw[word].double() - want).abs() - bound
    assert off.max().item() <= 0, (off.max().item(), int((off > 0).any(1).sum()), int(word.sum()))
    if dtype == "bf16":
        rel = (dw[word].double() - want).norm(dim=1) / want.norm(dim=1)
        assert rel.max().item() <= 2 * ROUND[dtype], rel.max().item()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("span", [12.0, 24.0, 40.0, 70.0])
@pytest.mark.parametrize("T", [1, 100, 140])
def test_words_far_below_the_likely_ones(T, span, dtype):
    check_words(*peaked(T, 64, 2003, dtype, span, seed=T), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_words_far_below_in_kept_and_recomputed_pieces(dtype):
    # three pieces of the vocabulary, two kept and one worked out again: the same bounds for all words
    check_words(*peaked(20000, 64, 30001, dtype, 40.0), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [128, 300])
def test_what_is_kept_adds_little_to_the_rounding_of_g(T, dtype):
    # Roundings of random sign: a step s makes s^2 / 12.  Those of G and of the result are counted from the exact numbers; what
    # is kept may add (2^-13)^2 / 3 of a probability (fp16, logits within 2^12 of the largest; bf16 (2^-11)^2 / 3), a
    # quarter of a half step, and a tenth is left for the sample
    gen = torch.Generator(device="cuda").manual_seed(T)
    D, V = 128, 2000
    H = torch.randn(T, D, generator=gen, device="cuda").to(DT[dtype])
    W = (torch.randn(V, D, generator=gen, device="cuda") * 0.75 / math.sqrt(D)).to(DT[dtype])
    y = torch.randint(64, (T,), generator=gen, device="cuda")
    _, _, dw = pkg.linear_ce_grad(H, W, y)
    h = H.double()
    p = torch.softmax(h @ W.double().T, 1)[:, 64:]
    want = p.T @ h
    bits, least = (7, -133) if dtype == "bf16" else (10, -24)

    def step(x, scale):
        return 2.0 ** torch.floor(torch.log2(x.abs() * scale)).clamp(min=least + bits).sub(bits) / scale

    kept = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -13) * p
    scale = 2.0 ** 14 if dtype == "f16" else 1.0
    expect = ((step(p, scale) ** 2 / 12 + kept ** 2 / 3).T @ h ** 2 + step(want, 1.0) ** 2 / 12).sum()
    got = (dw[64:].double() - want).square().sum()
    assert float(got) <= 1.1 * float(expect), float(got / expect)


def counted(x, bits, least, scale=1.0):
    """Squares that roundings to "bits" bits behind the leading one add, on average."""
    step = 2.0 ** torch.floor(torch.log2(x.abs() * scale)).clamp(min=least + bits).sub(bits) / scale
    return step.nan_to_num(0.0) ** 2 / 12


def test_sums_over_a_large_vocabulary():
    # Words with a common direction: a row's sum over the words before its label comes is as large as the result and what
    # follows is added to it, 2000 additions one behind the other.  Cut off at 512 of them, and 2^-24 each on average, they may add
    # a tenth to the roundings that are counted from the exact numbers: G's (not the label's, which is given back) and the result's
    gen = torch.Generator(device="cuda").manual_seed(0)
    T, D, V = 4096, 1280, 32000
    u = torch.nn.functional.normalize(torch.randn(D, generator=gen, device="cuda"), dim=0)
    W = torch.randn(V, D, generator=gen, device="cuda") * 0.02
    W -= torch.log1p(torch.arange(V, device="cuda"))[torch.randperm(V, generator=gen, device="cuda")][:, None] / 8 * u
    H, W = (torch.randn(T, D, generator=gen, device="cuda") + 8 * u).half(), W.half()
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    _, dh, _ = pkg.linear_ce_grad(H, W, y)
    w = W.double()
    got = expect = 0.0
    for r in range(0, T, 1024):
        p = torch.softmax(H[r:r + 1024].double() @ w.T, 1)
        at = y[r:r + 1024, None]
        off = (counted(p, 10, -24, 2.0 ** 14) + (2.0 ** -13 * p) ** 2 / 3).scatter(1, at, 0.0)
        p.scatter_add_(1, at, torch.full(at.shape, -1.0, dtype=p.dtype, device="cuda"))
        want = p @ w
        got += float((dh[r:r + 1024].double() - want).square().sum())
        expect += float((off @ w ** 2).sum() + counted(want, 10, -24).sum())
    assert got <= 1.21 * expect, got / expect


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sums_over_many_rows(dtype):
    # Rows sorted by label: a word's sum is as large as all its labels together when the other rows come, 12500 additions.
    # 512 of them, cut off by 2^-23 at most, make 2^-14 of the sum of magnitudes.  The probabilities of a word are nearly
    # the same in all rows here, and equal numbers are rounded alike: the errors of G add up, by half a step of each at
    # most, and not by their squares
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, D, V = 200000, 64, 1000
    H = (torch.randn(T, D, generator=gen, device="cuda") + 4).to(DT[dtype])
    W = (torch.randn(V, D, generator=gen, device="cuda") * 0.02).to(DT[dtype])
    y = torch.randint(V, (T,), generator=gen, device="cuda").sort().values
    weight = torch.full((T,), 2.0 ** -8, device="cuda")
    _, _, dw = pkg.linear_ce_grad(H, W, y, row_weight=weight)
    bits, least, scale = (7, -133, 1.0) if dtype == "bf16" else (10, -24, 2.0 ** 14)
    want, size, off = (torch.zeros(V, D, dtype=torch.float64, device="cuda") for _ in range(3))
    for r in range(0, T, 20000):
        h = H[r:r + 20000].double()
        G = torch.softmax(h @ W.double().T, 1)
        kept = (2.0 ** -11 if dtype == "bf16" else 2.0 ** -13) * G
        G.scatter_add_(1, y[r:r + 20000, None], torch.full((h.shape[0], 1), -1.0, dtype=G.dtype, device="cuda"))
        off += ((3 * counted(G, bits, least, scale)).sqrt() + kept).T @ h.abs()
        want += G.T @ h
        size += G.abs().T @ h.abs()
    want, size, off = want / 256, size / 256, off / 256
    err = (dw.double() - want).norm()
    assert float(err) <= float((off + (3 * counted(want, bits, least)).sqrt()).norm() + 2.0 ** -14 * size.norm())


def test_sums_over_millions_of_rows():
    # 250000 additions one behind the other.  Against the sum of G as it is rounded, in 64 bits: what is kept of the
    # probabilities adds 2^-13 of them, chains of 512 additions 2^-14 of the magnitudes, the result's rounding 2^-11
    gen = torch.Generator(device="cuda").manual_seed(2)
    T, D, V = 4000000, 16, 256
    H = (torch.randn(T, D, generator=gen, device="cuda") + 4).half()
    W = (torch.randn(V, D, generator=gen, device="cuda") * 0.3).half()
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    _, _, dw = pkg.linear_ce_grad(H, W, y, row_weight=torch.full((T,), 2.0 ** -12, device="cuda"))
    want, size, kept = (torch.zeros(V, D, dtype=torch.float64, device="cuda") for _ in range(3))
    for r in range(0, T, 100000):
        h = H[r:r + 100000].double()
        p = torch.softmax(h @ W.double().T, 1)
        kept += p.T @ h.abs()
        G = p.scatter_add_(1, y[r:r + 100000, None], torch.full((h.shape[0], 1), -1.0, dtype=p.dtype, device="cuda"))
        G = (G * 2 ** 14).half().double() / 2 ** 26
        want += G.T @ h
        size += G.abs().T @ h.abs()
    err = (dw.double() - want).norm()
    bound = 2.0 ** -11 * want.norm() + 2.0 ** -14 * size.norm() + 2.0 ** -13 * kept.norm() / 4096
    assert float(err) <= float(bound), (float(err), float(bound), float(want.norm()))


@pytest.mark.parametrize("T,D,V", [(300, 8, 600003), (64, 16, 600003), (9000, 256, 3000), (8193, 520, 9001), (20000, 264, 20001)])
def test_chains_in_parts_and_in_whole_tiles(T, D, V):
    # parts of a sum that are chains themselves, rows just above a chain, both products in chains: against 64 bits, bf16
    gen = torch.Generator(device="cuda").manual_seed(T)
    H = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, D, generator=gen, device="cuda") / math.sqrt(D)).bfloat16()
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    y[::7] = -100
    _, dh, dw = pkg.linear_ce_grad(H, W, y)
    w, rh, rw = W.double(), [], torch.zeros(V, D, dtype=torch.float64, device="cuda")
    step = max(1, (1 << 28) // V)
    for r in range(0, T, step):
        h, at = H[r:r + step].double(), y[r:r + step]
        G = torch.softmax(h @ w.T, 1)
        G.scatter_add_(1, at.clamp(min=0)[:, None], torch.full((h.shape[0], 1), -1.0, dtype=G.dtype, device="cuda"))
        G[at < 0] = 0.0
        rh.append(G @ w)
        rw += G.T @ h
    for got, want in ((dh, torch.cat(rh)), (dw, rw)):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * ROUND["bf16"]
    again = pkg.linear_ce_grad(H, W, y)
    assert bool(torch.equal(again[1], dh)) and bool(torch.equal(again[2], dw))


@pytest.mark.parametrize("exponent", [90, 97, 98, 100, 120, 127])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_row_weights_near_the_end_of_32_bits(exponent, dtype):
    # what is exactly 0 stays 0, and nothing becomes NaN: the gradient itself may be beyond the type
    gen = torch.Generator(device="cuda").manual_seed(exponent)
    T, D, V = 130, 64, 500
    H, W = (torch.randn(n, D, generator=gen, device="cuda").to(DT[dtype]) for n in (T, V))
    H[:, 5], W[:, 9] = 0.0, 0.0
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    w = torch.full((T,), 2.0 ** exponent, device="cuda")
    _, dh, dw = pkg.linear_ce_grad(H, W, y, row_weight=w)
    assert not dh.isnan().any() and not dw.isnan().any()
    assert dh[:, 9].eq(0).all() and dw[:, 5].eq(0).all()
    if dtype == "bf16":
        # the gradients scale by the power of two, exactly, as far as they are within the type
        _, eh, ew = pkg.linear_ce_grad(H, W, y)
        for a, b in ((dh, eh), (dw, ew)):
            want = b.double() * 2.0 ** exponent
            ok = (want.abs() < 3e38) & (b.abs() > 2.0 ** -100)
            assert torch.equal(a.double()[ok], want[ok])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [1344, 4096, 16384])
@pytest.mark.parametrize("T", [100, 300])
def test_losses_of_long_rows(T, D, dtype):
    # Labels with a logit of about -16, to which products of one sign add up; all other words are next to 0.  The tensor cores add
    # eight products at a time at least and cut off 2^-23 of the sum so far at most.  In chains of 1024 products, each of which
    # makes 1024 / D of the logit and is half of it on average, that is 128 2^-23 / 2 of the logit whatever D is; one
    # rounding more a chain
    gen = torch.Generator(device="cuda").manual_seed(T)
    V = 2000
    H = (4 + 0.25 * torch.randn(T, D, generator=gen, device="cuda")).to(DT[dtype])
    W = 1e-4 * torch.randn(V, D, generator=gen, device="cuda")
    W[:50] = -16 / (4 * D) * (1 + 0.1 * torch.rand(50, D, generator=gen, device="cuda"))
    W = W.to(DT[dtype])
    y = torch.randint(50, (T,), generator=gen, device="cuda")
    loss = pkg.linear_ce(H, W, y)
    x = H.double() @ W.double().T
    label = x.gather(1, y[:, None])
    want = (torch.logsumexp(x, 1, keepdim=True) - label).squeeze(1)
    others, most = float(x[:, 50:].abs().max()), float(label.abs().max())
    rms = float((loss.double() - want).square().mean().sqrt())
    assert rms <= U * (128 * (most + 2 * others) + D / 1024 * most + 2 * 24) + lse_tol(V), rms


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_rows_in_kept_and_recomputed_pieces(dtype):
    # three pieces, the last one worked out again; dim in two chains
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, D, V = 20000, 1344, 30001
    H = (torch.randn(T, D, generator=gen, device="cuda") + 0.5).to(DT[dtype])
    W = (torch.randn(V, D, generator=gen, device="cuda") / math.sqrt(D)).to(DT[dtype])
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    loss, dh, dw = pkg.linear_ce_grad(H, W, y)
    w, rh, rw = W.double(), [], torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for r in range(0, T, 4000):
        h, at = H[r:r + 4000].double(), y[r:r + 4000, None]
        x = h @ w.T
        lse = torch.logsumexp(x, 1, keepdim=True)
        off = (loss[r:r + 4000, None].double() - (lse - x.gather(1, at))).abs()
        # (logits of up to 6, 128 additions a chain)
        assert float(off.max()) <= 2 * 128 * 2.0 ** -23 * float(x.abs().max()) + 2 * lse_tol(V)
        G = x.sub_(lse).exp_()
        G.scatter_add_(1, at, torch.full(at.shape, -1.0, dtype=G.dtype, device="cuda"))
        rh.append(G @ w)
        rw += G.T @ h
    for got, want in ((dh, torch.cat(rh)), (dw, rw)):
        assert float((got.double() - want).norm() / want.norm()) <= 2 * ROUND[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,D", [(1, 8), (100, 4096), (33, 24), (300, 2048), (700, 40)])
def test_certain_labels_lose_nothing(T, D, dtype):
    # what is taken from a logit is in the maximum as well: the loss of a certain label is 0, not below
    gen = torch.Generator(device="cuda").manual_seed(D)
    V = 600
    H = (1 + torch.rand(T, D, generator=gen, device="cuda")).to(DT[dtype])
    W = torch.zeros(V, D, device="cuda", dtype=DT[dtype])
    y = torch.randint(V // 2, (T,), generator=gen, device="cuda")
    W[:V // 2] = 0.1 * torch.randn(V // 2, D, generator=gen, device="cuda").to(DT[dtype])
    W[V // 2] = 300 / D
    y[::2] = V // 2
    loss = pkg.linear_ce(H, W, y)
    x = H.double() @ W.double().T
    want = torch.logsumexp(x, 1) - x.gather(1, y[:, None]).squeeze(1)
    assert bool((loss >= 0).all())
    sure = want < 1e-20
    assert bool(sure[::2].any()) and bool(loss[sure].eq(0).all())
    # (the likeliest word's logit, of products of one sign, eight of which are added at least: D / 8 additions that cut off 2^-23
    # of it at most; where it is not the label's, this is in the loss)
    assert float(((loss - want).abs() - D / 8 * 2.0 ** -23 * x.amax(1) - 1e-6 * want - U * 600).max()) <= 0
