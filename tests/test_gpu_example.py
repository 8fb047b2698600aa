"""The example that runs the objective's operators and the optimizer together:
the student learns, and the balance loss keeps every expert in use."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_moe.py")


def load():
    spec = importlib.util.spec_from_file_location("distill_moe", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns():
    ex = load()
    losses, counts = ex.train(40, 2, log=None)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) / 5 < 0.8 * losses[0]
    assert counts.shape == (3, ex.EXPERTS) and int(counts.sum()) == 512 * ex.TOP
    assert int((counts.sum(0) > 0).sum()) == ex.EXPERTS


def test_example_gradients_against_autograd():
    # the student's gradients through the library against plain differentiable torch of the same objective
    ex = load()
    gen = torch.Generator(device="cuda").manual_seed(3)
    p = {k: (torch.randn(s, generator=gen, device="cuda") * 0.3).requires_grad_(True) for k, s in ex.SHAPES.items()}
    T = 64
    x = torch.randint(ex.VOCAB, (T,), generator=gen, device="cuda")
    z = torch.randn(T, ex.VOCAB, generator=gen, device="cuda") * 3
    labels = torch.randint(ex.VOCAB, (T,), generator=gen, device="cuda")
    cu = torch.tensor([0, 10, T], dtype=torch.int32, device="cuda")
    idx, vals, lse = ex.scape.topk_logits(z, 32, temperature=ex.TAU)
    logits, counts, aux = ex.student(p, x, cu)
    loss = ex.Distill.apply(logits, idx, vals, lse, labels)
    (loss + aux[0] + aux[1]).backward()

    q = {k: v.detach().double().requires_grad_(True) for k, v in p.items()}
    h = q["emb"][x]
    r = h @ q["router"]
    probs = torch.softmax(r, 1)
    top = r.topk(ex.TOP, 1)
    w = torch.softmax(top.values, 1)
    y = torch.zeros_like(h)
    for e in range(ex.EXPERTS):
        at, slot = torch.nonzero(top.indices == e, as_tuple=True)
        out = torch.nn.functional.gelu(h[at] @ q["w1"][e]) @ q["w2"][e]
        y = y.index_add(0, at, out * w[at, slot, None])
    s = (h + y) @ q["head"]
    lp = torch.log_softmax(s / ex.TAU, 1)
    qi = torch.exp(vals.double() / ex.TAU - lse.double()[:, None])
    rest = torch.ones_like(s, dtype=torch.bool).scatter_(1, idx.long(), False)
    qr = 1 - qi.sum(1)
    kl = (qi * (qi.log() - lp.gather(1, idx.long()))).sum(1) + qr * (qr.log() - lp.masked_fill(~rest, -1e30).logsumexp(1))
    want = (ex.KD * ex.TAU ** 2 * kl + ex.CE * torch.nn.functional.cross_entropy(s, labels, reduction="none")).mean()
    bal = 0.0
    for g, (a, b) in enumerate(((0, 10), (10, T))):
        f = counts[g].double() * ex.EXPERTS / (ex.TOP * (b - a))
        bal = bal + (f * probs[a:b].mean(0)).sum() / 2
    (want + bal + (r.logsumexp(1) ** 2).mean()).backward()
    # fp32 products of up to 1003 terms: 1003 * 2^-24 of the sum of magnitudes, under 1e-3 of a gradient's size
    assert abs(loss.item() - want.item()) < 1e-4 * abs(want.item())
    for k in p:
        off = (p[k].grad.double() - q[k].grad).norm() / q[k].grad.norm()
        assert off < 1e-3, (k, float(off))
