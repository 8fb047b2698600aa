"""The training-objective operators where a mask leaves little or nothing, where
it is a large finite number instead of -inf, and where logits are infinite.

References are objective_ref's on logits shifted by the row's largest, which
changes neither a softmax nor a loss: a row masked at -1e30 throughout is then a
row of zeros, and the bounds do not grow with the mask's size.  A word that is
more than 1e6 below the row's largest has a probability of 0 in any arithmetic
and stands as -inf."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import objective_ref as ref  # noqa: E402
import sparse_communication_distributed_gb300 as pkg  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")


def cuda(x, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DT[dtype]).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


# ---- top logits: fewer words than k are left --------------------------------------------------------


@pytest.mark.parametrize("R,V,k,dtype,left", [
    (1, 32000, 256, "bf16", 200), (1, 40000, 1024, "bf16", 700), (40, 50257, 1024, "bf16", 300), (700, 50257, 1024, "f16", 1000),
    (1000, 8100, 256, "bf16", 100), (1000, 8100, 200, "f16", 190), (3, 131075, 256, "f32", 255), (500, 4001, 250, "f32", 40),
    (2, 33000, 64, "bf16", 30), (900, 20000, 64, "bf16", 1)])
def test_topk_where_fewer_than_k_words_are_left(R, V, k, dtype, left):
    rng = np.random.default_rng(V + k)
    h = np.full((R, V), -INF, np.float32)
    for r in range(R):
        h[r, rng.choice(V, left, replace=False)] = rng.standard_normal(left) * 3
    x = cuda(h, dtype)
    idx, vals, lse = pkg.topk_logits(x, k)
    i = idx.cpu().numpy()
    assert all(np.unique(row).size == k for row in i)
    h = f64(x)
    for r in range(R):
        words = np.flatnonzero(h[r] > -INF)
        best = words[ref.topk(h[r, words], left)]
        masked = np.setdiff1d(np.arange(k), words, assume_unique=True)  # (the first k hold enough of them)
        masked = masked if masked.size >= k - left else np.setdiff1d(np.arange(2 * k), words)
        assert np.array_equal(i[r], np.concatenate([best, masked[:k - left]])), r
        L = ref.lse(h[r, words])
        assert abs(float(lse[r]) - L) <= ref.lse_tol(V, L) if r < 50 else True
    assert torch.equal(vals.cpu(), torch.gather(x.cpu(), 1, torch.from_numpy(i).long()))


# ---- masks that are large finite numbers ------------------------------------------------------------

LOWEST = {"bf16": -3.3895313892515355e38, "f16": -65504.0, "f32": -3.4028234663852886e38}


def masked(rng, R, V, dtype, where, value):
    """Logits of which the last 8 words, all but 40 words, or every word hold the mask's value."""
    h = (rng.standard_normal((R, V)) * 3).astype(np.float32)
    keep = np.ones((R, V), bool)
    if where == "tail":
        keep[:, -8:] = False
    elif where == "most":
        keep[:] = False
        for r in range(R):
            keep[r, rng.choice(V, 40, replace=False)] = True
    else:
        keep[:] = False
    low = LOWEST[dtype] if value == "lowest" else max(value, LOWEST[dtype])
    return cuda(np.where(keep, h, np.float32(low)), dtype), keep


def shifted(h):
    d = h - h.max(1, keepdims=True)
    return np.where(d < -1e6, -INF, d)


SIZES = [(3, 300), (400, 700), (2, 50257), (1, 140000)]
MASKS = ["lowest", -1e30, -1e10, -1e4]


@pytest.mark.parametrize("R,V", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("where", ["tail", "most", "whole"])
def test_topk_with_finite_masks(R, V, dtype, where):
    rng = np.random.default_rng(V)
    for value in MASKS:
        x, _ = masked(rng, R, V, dtype, where, value)
        h = f64(x)
        for tau in (1.0, 2.0, 1.7):
            idx, _, lse = pkg.topk_logits(x, 20, temperature=tau)
            got = f64(lse)
            for r in range(min(R, 5)):
                assert np.array_equal(idx[r].cpu().numpy(), ref.topk(h[r], 20))
                m = h[r].max()
                L = m / tau + ref.lse((h[r] - m) / tau)
                assert abs(got[r] - L) <= ref.lse_tol(V, L), (value, tau, r, got[r], L)
            assert np.isfinite(got).all()


# ---- distillation -----------------------------------------------------------------------------------


def check_distill(x, idx, vals, tl, y, tau, dtype, loss, grad, rows, kd=0.7, ce=0.4):
    """Rows of x against the shifted reference; a loss or gradient that is None is not looked at."""
    h, v = shifted(f64(x)), f64(vals)
    for r in rows:
        want, tol, wg, gtol = ref.distill(h[r], idx[r], v[r], None if tl is None else float(tl[r]), int(y[r]), 1.0, tau, kd, ce)
        if loss is not None:
            assert abs(float(loss[r]) - want) <= tol, (r, float(loss[r]), want, tol)
        if grad is not None:
            g = f64(grad[r])
            off = np.abs(g - wg) - (gtol + (np.abs(wg) + gtol) * ref.ROUND[dtype] + ref.TINY[dtype])
            assert off.max() <= 0, (r, int(off.argmax()), g[off.argmax()], wg[off.argmax()])


@pytest.mark.parametrize("V,k,tau", [(300, 64, 1.0), (50257, 200, 2.0), (140001, 400, 1.5), (900001, 64, 2.0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_with_teacher_entries_at_the_lowest_value(V, k, tau, dtype, tail):
    # a teacher whose own mask left it 20 words: the others of its k hold the type's lowest value, and q = 0; so
    # they do where the student's mask is -inf
    rng = np.random.default_rng(V)
    R = 3
    x = rng.standard_normal((R, V)).astype(np.float32) * 3
    idx = np.stack([rng.permutation(V)[:k] for _ in range(R)]).astype(np.int32)
    x[2, idx[2, 20:]] = -INF
    v = np.full((R, k), LOWEST[dtype], np.float32)
    v[:, :20] = rng.standard_normal((R, 20)) * 2
    vals, xt = cuda(v, dtype), cuda(x, dtype)
    tl = np.array([ref.lse(r[:20] / tau) + 0.1 for r in f64(vals)], np.float32) if tail else None
    y = np.full(R, -1)
    loss, grad = pkg.distill_loss_grad(xt, torch.from_numpy(idx).cuda(), vals, teacher_lse=None if tl is None else cuda(tl),
                                       temperature=tau, kd_weight=0.7)
    vals[:, 20:] = -INF  # what they count as
    check_distill(xt, idx, vals, tl, y, tau, dtype, loss, grad, range(R))


@pytest.mark.parametrize("V,k,tau", [(300, 40, 0.7), (50257, 200, 0.9), (140001, 400, 0.8), (900001, 64, 0.7)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("value", ["lowest", 2.0 ** 20])
def test_distill_with_teacher_entries_far_from_zero(V, k, tau, dtype, value):
    # entries that all hold the type's lowest value are equal (their quotient by a temperature below 1 is beyond fp32);
    # entries at 2^20 and a few eighths are those few eighths
    rng = np.random.default_rng(V)
    R = 2
    xt = cuda(rng.standard_normal((R, V)).astype(np.float32) * 3, dtype)
    idx = np.stack([rng.permutation(V)[:k] for _ in range(R)]).astype(np.int32)
    near = np.zeros((R, k)) if value == "lowest" else np.round(rng.standard_normal((R, k)) * 16) / 8
    vals = cuda(np.full((R, k), LOWEST[dtype]), dtype) if value == "lowest" else cuda(near + value)
    loss, grad = pkg.distill_loss_grad(xt, torch.from_numpy(idx).cuda(), vals, temperature=tau, kd_weight=0.7)
    check_distill(xt, idx, cuda(near), None, np.full(R, -1), tau, dtype, loss, grad, range(R))


def case_of(rng, x, keep, k, tau, tail):
    """k words of each row that are not masked (any words where all are) for a teacher, and a label among them or not."""
    R, V = x.shape
    idx = np.empty((R, k), np.int32)
    y = np.empty(R, np.int64)
    for r in range(R):
        words = np.flatnonzero(keep[r]) if keep[r].any() else np.arange(V)
        idx[r] = rng.choice(words, k, replace=False)
        y[r] = rng.choice(words)
    vals = cuda(rng.standard_normal((R, k)) * 2)
    tl = np.array([ref.lse(v / tau) + 0.3 for v in f64(vals)], np.float32) if tail else None
    return idx, vals, tl, y


def distill_masked(R, V, dtype, where, tail, labels):
    rng = np.random.default_rng(V)
    for value in MASKS:
        x, keep = masked(rng, R, V, dtype, where, value)
        for tau in (1.0, 2.0, 1.7):
            idx, vals, tl, y = case_of(rng, x, keep, 8, tau, tail)
            y = y if labels else np.full(R, -1)
            loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, teacher_lse=None if tl is None else cuda(tl),
                                               labels=torch.from_numpy(y).cuda(), temperature=tau, kd_weight=0.7, ce_weight=0.4)
            yield x, idx, vals, tl, y, tau, loss, grad


LONG = [(1, 900001, "bf16"), (1, 450001, "f32")]  # rows that do not fit on chip


@pytest.mark.parametrize("R,V,dtype", [(R, V, d) for R, V in SIZES for d in ("bf16", "f16", "f32")] + LONG)
@pytest.mark.parametrize("where", ["tail", "most", "whole"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_with_finite_masks(R, V, dtype, where, tail):
    for labels in (True, False):
        for x, idx, vals, tl, y, tau, loss, grad in distill_masked(R, V, dtype, where, tail, labels):
            check_distill(x, idx, vals, tl, y, tau, dtype, None if where == "whole" else loss, grad, range(min(R, 4)))
            assert bool(torch.isfinite(grad).all())


@pytest.mark.parametrize("dtype,V", [("bf16", 700), ("f32", 50257), ("f32", 450001)])
def test_distill_bucket_of_masked_words(dtype, V):
    # every word that is not listed is masked: the bucket's mass is exp(value / tau), the loss q_rest times its
    # distance, and the bucket's gradient - kd tau q_rest, spread evenly
    rng = np.random.default_rng(5)
    x = np.full((1, V), -1e10, np.float32)
    idx = rng.permutation(V)[:8].astype(np.int32)[None]
    x[0, idx[0]] = rng.standard_normal(8)
    xt = cuda(x, dtype)
    vals = cuda(rng.standard_normal((1, 8)))
    tau, tl = 2.0, np.array([ref.lse(f64(vals)[0] / 2.0) + 0.3], np.float32)
    loss, grad = pkg.distill_loss_grad(xt, torch.from_numpy(idx).cuda(), vals, teacher_lse=cuda(tl), temperature=tau)
    low = f64(xt).min()
    qr = 1 - np.exp(f64(vals)[0] / tau - float(tl[0])).sum()
    want = tau ** 2 * qr * -low / tau
    assert abs(float(loss) - want) < 1e-5 * want
    rest = np.ones(V, bool)
    rest[idx[0]] = False
    g = f64(grad)[0][rest]
    assert np.abs(g + tau * qr / (V - 8)).max() <= tau * qr / (V - 8) * (ref.ROUND[dtype] + 1e-5)


@pytest.mark.parametrize("R,V,dtype", [(R, V, d) for R, V in SIZES for d in ("bf16", "f16", "f32")] + LONG)
@pytest.mark.parametrize("tail", [False, True])
def test_distill_loss_of_rows_masked_throughout(R, V, dtype, tail):
    for labels in (True, False):
        for x, idx, vals, tl, y, tau, loss, grad in distill_masked(R, V, dtype, "whole", tail, labels):
            check_distill(x, idx, vals, tl, y, tau, dtype, loss, None, range(min(R, 4)))
            alone = pkg.distill_loss(x, torch.from_numpy(idx).cuda(), vals, teacher_lse=None if tl is None else cuda(tl),
                                     labels=torch.from_numpy(y).cuda(), temperature=tau, kd_weight=0.7, ce_weight=0.4)
            assert torch.equal(alone, loss)


@pytest.mark.parametrize("V", [300, 50257, 140000, 450001])
@pytest.mark.parametrize("offset", [-2.0 ** 20, 2.0 ** 20])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_does_not_depend_on_an_offset(V, offset, tail):
    # logits on a grid of 1/8, so that the offset of 2^20 is exact: the loss is that of the logits without it
    rng = np.random.default_rng(V)
    h = np.round(rng.standard_normal((2, V)) * 24) / 8
    x = cuda(h + offset)
    assert np.array_equal(f64(x), h + offset)
    for tau in (1.0, 2.0, 1.7):
        idx, vals, tl, y = case_of(rng, x, np.ones((2, V), bool), 40, tau, tail)
        loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, teacher_lse=None if tl is None else cuda(tl),
                                           labels=torch.from_numpy(y).cuda(), temperature=tau, kd_weight=0.7, ce_weight=0.4)
        check_distill(x, idx, vals, tl, y, tau, "f32", loss, grad, range(2))


@pytest.mark.parametrize("V,dtype", [(300, "bf16"), (50257, "f32"), (900001, "bf16")])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_masked_row_without_a_term_has_no_gradient(V, dtype, tail):
    # no word is left, the teacher no entry above -inf, and there is no label: the loss is 0, and so is its gradient
    x = torch.full((2, V), -INF, dtype=DT[dtype], device="cuda")
    idx = torch.tensor([[-1] * 4, [3, -1, 299, 7]], dtype=torch.int32, device="cuda")
    tl = torch.zeros(2, device="cuda") if tail else None
    for tau in (1.0, 2.0, 1.7):
        loss, grad = pkg.distill_loss_grad(x, idx, torch.full((2, 4), -INF, device="cuda"), teacher_lse=tl, temperature=tau, ce_weight=0.5,
                                           labels=torch.tensor([-100, -1], device="cuda"))
        assert loss.tolist() == [0.0, 0.0] and not f64(grad).any()


def bucket_gradient(V, sure):
    """(gradient of the unlisted words, their softmax among themselves, log p_rest, q_rest, x, teacher_lse) of 64 rows
    with 64 listed words, one of them with an entry above -inf (0, so that q = exp(-teacher_lse))."""
    R, k = 64, 64
    rng = np.random.default_rng(V)
    h = rng.standard_normal((R, V)) * (1.0 if sure else 0.1)
    at = np.arange(k) * (V // k) + 3
    if sure:
        h[:, at] = np.log(V / k) + rng.uniform(13.0, 15.0, (R, 1)) + rng.uniform(-3, 0, (R, k))
        tl = -np.log1p(-np.linspace(1, 40, R) * 2.0 ** -24)
    else:
        tl = -np.log(k / V * np.exp(rng.uniform(-0.1, 0.1, R)))
    tl = tl.astype(np.float32)
    x = cuda(h)
    vals = torch.full((R, k), -INF, device="cuda")
    vals[:, 5] = 0.0
    idx = torch.from_numpy(np.tile(at, (R, 1)).astype(np.int32)).cuda()
    _, grad = pkg.distill_loss_grad(x, idx, vals, teacher_lse=cuda(tl))
    rest = np.ones(V, bool)
    rest[at] = False
    h = f64(x)
    for r in range(R):
        L, Lr, Lt = ref.lse(h[r]), ref.lse(h[r, rest]), ref.lse(h[r, at])
        yield f64(grad[r])[rest], np.exp(h[r, rest] - Lr), np.exp(Lr - L), np.exp(Lt - L), float(tl[r]), ref.lse_tol(V, L)


@pytest.mark.parametrize("V", [300, 50257, 450001])
def test_distill_bucket_gradient_of_a_sure_student(V):
    # p_rest and q_rest near 1e-6: an unlisted word's gradient is (p_rest - q_rest) softmax_rest_j.  q is one expf near
    # 1, within 2 units of 2^-24, and 1 - q exact; p_rest is a sum of its own, off by a few 1e-6 of itself
    for g, soft, p_rest, _, tl, es in bucket_gradient(V, True):
        tol = 2 * 2.0 ** -24 + p_rest * 4 * es
        want = (p_rest + np.expm1(-tl)) * soft
        assert (np.abs(g - want) <= soft * tol + np.abs(want) * 4 * es + 1e-38).all(), (np.abs(g - want) / soft).max() / tol


@pytest.mark.parametrize("V", [2000, 50257, 450001])
def test_distill_bucket_gradient_of_an_unsure_student(V):
    # p_rest and q_rest near 1: the same is (q - p_listed) softmax_rest_j, each of the two off by a few 1e-6 of itself
    for g, soft, _, p_listed, tl, es in bucket_gradient(V, False):
        q = np.exp(-tl)
        tol = (q * 8 * 2.0 ** -24 + p_listed * 4 * es) + np.abs(q - p_listed) * 4 * es
        assert (np.abs(g - (q - p_listed) * soft) <= soft * tol + 1e-38).all(), tol


@pytest.mark.parametrize("R,V,k", [(700, 1003, 700), (400, 50257, 1000), (120, 131075, 400)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_many_entries_over_many_rows(R, V, k, tail):
    # more entries than threads, and several rows for each CTA or cluster, some of weight 0
    rng = np.random.default_rng(V)
    x = cuda(rng.standard_normal((R, V)).astype(np.float32) * 3, "bf16")
    z = f64(x) * 0.9 + rng.standard_normal((R, V))
    idx = np.argpartition(-z, k, axis=1)[:, :k].astype(np.int32)
    vals = cuda(np.take_along_axis(z, idx, 1))
    tl = np.array([ref.lse(r / 1.7) for r in z], np.float32) if tail else None
    y = rng.integers(V, size=R)
    w = np.where(rng.random(R) < 0.2, 0.0, 1.0).astype(np.float32)
    loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, teacher_lse=None if tl is None else cuda(tl),
                                       labels=torch.from_numpy(y).cuda(), row_weight=cuda(w), temperature=1.7, kd_weight=0.7, ce_weight=0.4)
    off = torch.from_numpy(w == 0).cuda()
    assert not grad[off].any() and not loss[off].any()
    some = [r for r in np.unique(np.concatenate([rng.integers(R, size=12), [0, R - 1]])) if w[r]]
    check_distill(x, idx, vals, tl, y, 1.7, "bf16", loss, grad, some)


# ---- routing ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("T,E,k", [(40, 8, 2), (50, 64, 6), (3000, 256, 8), (60, 300, 12), (30, 1000, 20), (200, 16, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_with_finite_masks(T, E, k, dtype, renorm):
    # some tokens masked throughout, some but for a few experts: weights, counts, the balance loss and gradients are
    # those of the shifted logits; z is the mean of lse^2, infinite where that is beyond fp32
    rng = np.random.default_rng(T + E)
    for value in MASKS:
        low = np.float32(LOWEST[dtype] if value == "lowest" else max(value, LOWEST[dtype]))
        h = (rng.standard_normal((T, E)) * 2).astype(np.float32)
        h[3::5] = low
        h[4::5, k // 2:] = low
        x = cuda(h, dtype)
        h = f64(x)
        s = shifted(h)
        cu = np.array([0, T // 3, T], np.int32)
        cut = torch.from_numpy(cu).cuda()
        idx, w, counts, live, losses = pkg.route(x, k, renormalize=renorm, cu_tokens=cut)
        rl = np.array([cu[1], T - cu[1], T, 2])
        assert np.array_equal(idx.cpu().numpy(), np.stack([ref.topk(t, k) for t in h]))
        rel = ref.U * (E / 8 + 64 + 16 * 20)
        many = ref.U * (T / 8 + 512)
        by_logit = np.exp(np.take_along_axis(s, f64(idx).astype(int), 1)
                          - np.array([ref.lse(t[i]) if renorm else ref.lse(t) for t, i in zip(s, f64(idx).astype(int))])[:, None])
        assert np.abs(f64(w) - by_logit).max() <= rel
        assert np.array_equal(live.cpu().numpy(), rl) and int(counts.sum()) == T * k
        c = f64(counts)
        p = np.exp(s - np.array([ref.lse(t) for t in s])[:, None])
        want = np.mean([(E * c[g] / (k * rl[g]) * p[cu[g]:cu[g + 1]].sum(0) / rl[g]).sum() for g in range(2)])
        assert abs(float(losses[0]) - want) <= (rel + many) * want
        L = h.max(1) + np.array([ref.lse(t) for t in s])
        z = np.mean(L ** 2)
        assert abs(float(losses[1]) - z) <= 1e-4 * z if z < 1e38 else float(losses[1]) == INF

        dw = rng.standard_normal((T, k)).astype(np.float32)
        grad = f64(pkg.route_backward(x, idx, counts, live, d_weights=cuda(dw), d_losses=torch.tensor([0.7, 0.0], device="cuda"),
                                      renormalize=renorm, cu_tokens=cut))
        wg, size = ref.route_grad(s, f64(idx).astype(int), c, rl, cu, dw.astype(np.float64), np.array([0.7, 0.0]), renorm)
        off = np.abs(grad - wg) - ((4 * rel + 16 * ref.U) * size + np.abs(wg) * ref.ROUND[dtype] + ref.TINY[dtype])
        assert off.max() <= 0, value


# ---- infinite logits --------------------------------------------------------------------------------


@pytest.mark.parametrize("R,V", [(3, 300), (3, 5000), (3, 50257), (3, 140000), (700, 3000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_topk_of_an_infinite_logit(R, V, dtype):
    rng = np.random.default_rng(V)
    h = rng.standard_normal((R, V)).astype(np.float32)
    h[0, V // 3] = INF
    h[1, [1, V - 1]] = INF
    h[2, V // 2], h[2, V // 5] = INF, np.nan
    x = cuda(h, dtype)
    idx, vals, lse = pkg.topk_logits(x, 3, temperature=2.0)
    for r in range(3):
        assert np.array_equal(idx[r].cpu().numpy(), ref.topk(f64(x)[r], 3))
    assert float(lse[0]) == INF and float(lse[1]) == INF and np.isnan(float(lse[2]))
    assert np.isfinite(f64(lse)[3:]).all()


def test_k_beyond_32_bits_is_refused():
    x = torch.zeros(1, 100, device="cuda")
    for k in (2 ** 32 + 3, -2 ** 32 + 3):
        with pytest.raises(ValueError):
            pkg.topk_logits(x, k)
        with pytest.raises(ValueError):
            pkg.route(x, k)
