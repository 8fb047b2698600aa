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
