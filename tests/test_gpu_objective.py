"""The training-objective operators against their definitions in 64 bits
(objective_ref.py, which also derives the bounds): every type, odd sizes and
alignments, ties, masks that leave nothing, one row and many."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import objective_ref as ref  # noqa: E402
import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from sparse_communication_distributed_gb300 import ScapeError  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")


def place(x, dtype, offset=0, pad=0):
    """x (numpy) as a CUDA view whose rows start "offset" elements into rows that are "pad" longer."""
    R, V = x.shape
    wide = torch.full((R, V + offset + pad), 7.0, dtype=DT[dtype], device="cuda")
    view = wide[:, offset:offset + V]
    view.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return view


def f64(t):
    return t.detach().double().cpu().numpy()


def logits(rng, R, V, kind="normal"):
    x = rng.standard_normal((R, V)) * 3
    if kind == "ties":
        x = np.round(x * 2) / 2
    elif kind == "equal":
        x = np.full((R, V), 1.25)
    elif kind == "rising":
        x = np.tile(np.linspace(-9, 9, V), (R, 1))
    elif kind == "masked":
        x[rng.random((R, V)) < 0.7] = -INF
        x[:, V // 2] = 0.5
    elif kind == "zeros":
        x = np.where(rng.random((R, V)) < 0.5, 0.0, -0.0)
    elif kind == "low":  # far below zero, where exp() of a logit itself is 0
        x -= 400.0
    elif kind == "high":
        x += 400.0
    elif kind == "spiked":
        x[np.arange(R), rng.integers(V, size=R)] += 60
    return x


# ---- top logits ---------------------------------------------------------------------------------

TOPK = [  # rows, vocab, k, dtype, kind, offset, pad
    (1, 1, 1, "f32", "normal", 0, 0), (3, 2, 2, "bf16", "normal", 1, 0), (5, 7, 3, "f16", "ties", 0, 3),
    (2, 31, 31, "bf16", "zeros", 3, 2), (4, 1000, 1000, "f32", "normal", 1, 0), (3, 1024, 1024, "bf16", "ties", 0, 0),
    (7, 4097, 64, "bf16", "normal", 5, 6), (2, 32000, 64, "bf16", "normal", 0, 0), (3, 32000, 8, "f16", "equal", 0, 0),
    (2, 50257, 128, "bf16", "ties", 0, 0), (5, 50257, 64, "f32", "rising", 2, 1), (2, 33000, 256, "bf16", "rising", 0, 0),
    (2, 131075, 256, "f32", "normal", 0, 0), (2, 131072, 1024, "bf16", "equal", 0, 0), (3, 70001, 17, "f16", "masked", 1, 1),
    (400, 513, 5, "bf16", "ties", 0, 0), (1, 300007, 33, "bf16", "normal", 0, 0), (2, 9000, 100, "f32", "zeros", 0, 0),
    (40, 20000, 1, "f32", "spiked", 1, 1), (1, 600000, 700, "f32", "rising", 0, 0),
]


@pytest.mark.parametrize("R,V,k,dtype,kind,offset,pad", TOPK)
def test_topk(R, V, k, dtype, kind, offset, pad):
    rng = np.random.default_rng(V + k)
    x = place(logits(rng, R, V, kind), dtype, offset, pad)
    tau = 1.7
    idx, vals, lse = pkg.topk_logits(x, k, temperature=tau)
    h = f64(x)
    for r in range(R):
        want = ref.topk(h[r], k)
        assert np.array_equal(idx[r].cpu().numpy(), want), r
    at = idx.long()
    assert torch.equal(vals.view(torch.int32 if dtype == "f32" else torch.int16),
                       torch.gather(x, 1, at).view(torch.int32 if dtype == "f32" else torch.int16))
    got = f64(lse)
    for r in range(R):
        L = ref.lse(h[r] / tau)
        assert abs(got[r] - L) <= ref.lse_tol(V, L), (r, got[r], L)


def test_topk_rows_without_a_finite_logit_and_nan():
    x = np.full((3, 5000), -INF)
    x[1, 4000] = 2.0
    x[2, 77] = np.nan
    idx, vals, lse = pkg.topk_logits(place(x, "bf16"), 3)
    assert idx.cpu().numpy().tolist() == [[0, 1, 2], [4000, 0, 1], [77, 0, 1]]
    assert f64(vals)[1].tolist() == [2.0, -INF, -INF]
    got = f64(lse)
    assert got[0] == -INF and abs(got[1] - 2.0) < 1e-6 and np.isnan(got[2])


def test_topk_repeats_bit_for_bit_and_no_rows():
    x = place(logits(np.random.default_rng(0), 300, 20011, "ties"), "bf16")
    a, b = pkg.topk_logits(x, 50), pkg.topk_logits(x, 50)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    idx, vals, lse = pkg.topk_logits(x[:0], 50)
    assert idx.shape == (0, 50) and vals.shape == (0, 50) and lse.shape == (0,)


def test_topk_past_32_bit_offsets():
    # row 5 starts 3.4e9 elements into the buffer
    R, V, stride = 6, 1000, 680_000_000
    buf = torch.zeros(5 * stride + V, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (R, V), (stride, 1))
    h = logits(np.random.default_rng(1), R, V)
    x.copy_(torch.from_numpy(h))
    idx, _, _ = pkg.topk_logits(x, 9)
    for r in range(R):
        assert np.array_equal(idx[r].cpu().numpy(), ref.topk(f64(x[r]), 9))
    w = torch.zeros(R, device="cuda")
    w[5] = 1.0
    vals = torch.ones(R, 9, device="cuda")
    _, g = pkg.distill_loss_grad(x, idx, vals, row_weight=w, grad=x)
    s = np.exp(f64(place(h, "bf16"))[5])
    want = s / s.sum()
    want[idx[5].long().cpu().numpy()] -= 1 / 9
    assert g.data_ptr() == x.data_ptr()
    assert np.abs(f64(x[5]) - want).max() < 2.0 ** -9 and not f64(x[0]).any()


@pytest.mark.parametrize("R,V,dtype,kind", [(1, 9, "f32", "low"), (3, 700, "bf16", "low"), (2, 50257, "f32", "low"),
                                            (1, 140000, "f16", "low"), (2, 33001, "bf16", "high"), (700, 300, "f32", "low")])
def test_topk_far_from_zero(R, V, dtype, kind):
    x = place(logits(np.random.default_rng(V), R, V, kind), dtype)
    k = min(V, 40)
    idx, _, lse = pkg.topk_logits(x, k, temperature=0.8)
    h, got = f64(x), f64(lse)
    for r in range(R):
        assert np.array_equal(idx[r].cpu().numpy(), ref.topk(h[r], k))
        L = ref.lse(h[r] / 0.8)
        assert abs(got[r] - L) <= ref.lse_tol(V, L)


@pytest.mark.parametrize("R,V,k,dtype", [(1, 40000, 1024, "bf16"), (2, 100000, 700, "f32"), (3, 70000, 64, "f16"), (5, 131072, 256, "f32"),
                                         (19, 33000, 100, "bf16"), (1, 16400, 3, "f32"), (1, 50257, 64, "bf16")])
@pytest.mark.parametrize("kind", ["normal", "equal", "masked"])
def test_topk_few_long_rows(R, V, k, dtype, kind):
    x = place(logits(np.random.default_rng(V + k), R, V, kind), dtype, 1, 2)
    idx, vals, lse = pkg.topk_logits(x, k)
    h, got = f64(x), f64(lse)
    for r in range(R):
        assert np.array_equal(idx[r].cpu().numpy(), ref.topk(h[r], k))
        L = ref.lse(h[r])
        assert abs(got[r] - L) <= ref.lse_tol(V, L)
    assert torch.equal(vals, torch.gather(x, 1, idx.long()))


@pytest.mark.parametrize("R,V,k,dtype,kind", [(4000, 300, 7, "f32", "ties"), (2500, 1003, 64, "bf16", "normal"), (1300, 9001, 33, "bf16", "ties"),
                                              (900, 33001, 200, "f16", "normal"), (1000, 50257, 64, "bf16", "normal"), (500, 131075, 256, "f32", "normal")])
def test_topk_many_rows(R, V, k, dtype, kind):
    # every CTA takes several rows
    x = torch.randn(R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V)).mul_(3)
    x = (x.mul(2).round().div(2) if kind == "ties" else x).to(DT[dtype])
    idx, vals, lse = pkg.topk_logits(x, k)
    # in descending order, ties by index, and nothing left out is larger than the last one (or equal, at a lower index)
    v, i = vals.float(), idx.long()
    assert torch.equal(vals, torch.gather(x, 1, i))
    assert bool(((v[:, :-1] > v[:, 1:]) | ((v[:, :-1] == v[:, 1:]) & (i[:, :-1] < i[:, 1:]))).all())
    last, at = v[:, -1:], i[:, -1:]
    better = (x.float() > last) | ((x.float() == last) & (torch.arange(V, device="cuda") <= at))
    assert bool((better.sum(1) == k).all())
    assert float((lse.double() - torch.logsumexp(x.double(), 1)).abs().max()) <= ref.lse_tol(V, 20.0)


# ---- distillation -------------------------------------------------------------------------------

DISTILL = [  # rows, vocab, k, dtype, kind, tail, ce, tau, offset, pad
    (1, 1, 1, "f32", "normal", False, True, 1.0, 0, 0), (2, 2, 1, "bf16", "normal", True, True, 2.0, 1, 0),
    (3, 9, 9, "f16", "normal", True, False, 1.0, 0, 1), (4, 33, 5, "f32", "normal", True, True, 3.0, 1, 0),
    (3, 1000, 0, "bf16", "normal", False, True, 1.0, 3, 2), (5, 4099, 64, "bf16", "normal", False, False, 2.0, 0, 0),
    (2, 32000, 64, "bf16", "normal", False, True, 2.0, 0, 0), (2, 32000, 64, "bf16", "masked", True, True, 1.0, 0, 0),
    (3, 50257, 128, "bf16", "normal", True, True, 2.0, 0, 0), (3, 50257, 32, "f16", "normal", False, True, 1.5, 1, 6),
    (2, 50257, 100, "f32", "spiked", True, True, 1.0, 0, 3), (1, 131075, 1024, "f32", "normal", False, True, 1.0, 0, 0),
    (2, 128000, 64, "bf16", "normal", True, False, 4.0, 0, 8), (1, 270001, 64, "bf16", "normal", True, True, 2.0, 0, 0),
    (300, 513, 7, "bf16", "ties", True, True, 2.0, 0, 0), (2, 16384, 16, "f32", "equal", False, True, 0.5, 0, 0),
    (1, 600011, 31, "f32", "normal", True, True, 2.0, 0, 0), (2, 65536, 1, "bf16", "spiked", True, True, 2.0, 0, 0),
]


def teacher(rng, x, k, tau, dtype):
    """A teacher near the student: its k top entries (some empty, one -inf) and its log-sum-exp."""
    R, V = x.shape
    z = np.where(np.isfinite(x), x, -20.0) * 0.9 + rng.standard_normal((R, V))
    idx = np.argsort(-z, axis=1)[:, :k].astype(np.int32)
    vals = torch.from_numpy(np.take_along_axis(z, idx, 1).copy()).to(DT[dtype]).cuda()
    for r in range(R):
        if k > 3 and r % 2:
            idx[r, rng.integers(k // 2, k):] = -1
            vals[r, 1] = -INF
    tl = np.array([ref.lse(z[r] / tau) for r in range(R)])
    return idx, vals, tl.astype(np.float32)


def check_distill(x, idx, vals, tl, y, w, tau, kd, ce, dtype, loss, grad):
    h, v, got, g = f64(x), f64(vals), f64(loss), None if grad is None else f64(grad)
    for r in range(x.shape[0]):
        want, tol, wg, gtol = ref.distill(h[r], idx[r], v[r], None if tl is None else float(tl[r]),
                                          -1 if y is None else int(y[r]), 1.0 if w is None else w[r], tau, kd, ce)
        if np.isnan(want):
            assert np.isnan(got[r])
        elif np.isinf(want):
            assert got[r] == want
        else:
            assert abs(got[r] - want) <= tol, (r, got[r], want, tol)
        if g is not None:
            off = np.abs(g[r] - wg) - (gtol + (np.abs(wg) + gtol) * ref.ROUND[dtype] + ref.TINY[dtype])
            assert off.max() <= 0, (r, int(off.argmax()), g[r][off.argmax()], wg[off.argmax()], off.max())


@pytest.mark.parametrize("R,V,k,dtype,kind,tail,ce,tau,offset,pad", DISTILL)
def test_distill(R, V, k, dtype, kind, tail, ce, tau, offset, pad):
    rng = np.random.default_rng(V * 3 + k)
    x = place(logits(rng, R, V, kind), dtype, offset, pad)
    vdt = dtype if k % 2 else "f32"
    idx, vals, tl = teacher(rng, f64(x), k, tau, vdt)
    tl = tl if tail and k else None
    y = None
    if ce:
        y = rng.integers(V, size=R)
        if k and R > 2:
            y[0], y[1], y[2] = idx[0, 0], -100, idx[2, k - 1]
        finite = np.isfinite(f64(x))
        y = np.array([c if c < 0 or finite[r, c] else V // 2 for r, c in enumerate(y)])
    w = None if R < 3 else np.where(np.arange(R) % 3 == 2, 0.0, 0.5 + np.arange(R) / R).astype(np.float32)
    args = dict(teacher_lse=None if tl is None else torch.from_numpy(tl).cuda(),
                labels=None if y is None else torch.from_numpy(y).cuda(),
                row_weight=None if w is None else torch.from_numpy(w).cuda(),
                temperature=tau, kd_weight=0.7, ce_weight=0.4)
    it = torch.from_numpy(idx).cuda()
    loss, grad = pkg.distill_loss_grad(x, it, vals, **args)
    check_distill(x, idx, vals, tl, y, w, tau, 0.7, 0.4, dtype, loss, grad)
    assert torch.equal(pkg.distill_loss(x, it, vals, **args), loss)
    again = pkg.distill_loss_grad(x, it, vals, **args)
    assert torch.equal(again[0], loss) and torch.equal(again[1], grad)
    # a gradient whose rows are aligned otherwise than the logits', then one over the logits
    other = place(np.zeros((R, V)), dtype, offset + 1, pad)
    pkg.distill_loss_grad(x, it, vals, **args, grad=other)
    assert torch.equal(other, grad)
    wide = x._base
    before, after = wide[:, :offset].clone(), wide[:, offset + V:].clone()
    pkg.distill_loss_grad(x, it, vals, **args, grad=x)
    assert torch.equal(x, grad)
    assert torch.equal(wide[:, :offset], before) and torch.equal(wide[:, offset + V:], after)


@pytest.mark.parametrize("R,V,k,dtype", [(2, 9, 3, "f32"), (3, 700, 20, "bf16"), (2, 50257, 64, "f32"), (2, 600011, 31, "f32"),
                                         (400, 300, 5, "f16"), (1, 1100003, 40, "bf16")])
@pytest.mark.parametrize("kind", ["low", "high"])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_far_from_zero(R, V, k, dtype, kind, tail):
    rng = np.random.default_rng(V)
    x = place(logits(rng, R, V, kind), dtype)
    idx, vals, tl = teacher(rng, f64(x), k, 1.5, "f32")
    tl = tl if tail else None
    y = rng.integers(V, size=R)
    args = dict(teacher_lse=None if tl is None else torch.from_numpy(tl).cuda(), labels=torch.from_numpy(y).cuda(),
                temperature=1.5, kd_weight=0.7, ce_weight=0.4)
    loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, **args)
    check_distill(x, idx, vals, tl, y, None, 1.5, 0.7, 0.4, dtype, loss, grad)


def test_distill_listed_words_masked_far_below_zero():
    # a bucket whose listed words the student masks while the others are far below zero: p_listed is 0, not NaN
    for V in (900, 600000):  # (the long row does not fit on chip)
        x = np.full((1, V), -500.0)
        x[0, :4] = -INF
        xt = place(x, "f32")
        idx = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        vals = torch.tensor([[1.0, 0.5, -INF, -INF]], device="cuda")
        tl = np.array([2.0], np.float32)
        loss, grad = pkg.distill_loss_grad(xt, idx, vals, teacher_lse=torch.from_numpy(tl).cuda())
        assert float(loss) == INF  # q > 0 where p = 0
        check_distill(xt, idx.cpu().numpy(), vals, tl, None, None, 1.0, 1.0, 0.0, "f32", loss, grad)


def test_distill_rows_of_weight_zero_are_not_read():
    x = np.full((4, 3001), np.nan)
    x[2] = logits(np.random.default_rng(2), 1, 3001)[0]
    idx = torch.arange(8, dtype=torch.int32, device="cuda").repeat(4, 1)
    vals = torch.ones(4, 8, device="cuda")
    vals[0] = np.nan
    w = torch.tensor([0.0, 0.0, 2.0, 0.0], device="cuda")
    loss, grad = pkg.distill_loss_grad(place(x, "bf16"), idx, vals, row_weight=w)
    assert f64(loss)[[0, 1, 3]].tolist() == [0, 0, 0] and np.isfinite(f64(loss)[2])
    assert not f64(grad)[[0, 1, 3]].any() and np.isfinite(f64(grad)).all()


@pytest.mark.parametrize("R,V,k,dtype,tail", [(4000, 300, 7, "f32", True), (3001, 1003, 20, "bf16", False), (1300, 9001, 33, "bf16", True),
                                              (900, 33001, 64, "f16", True), (530, 50257, 64, "bf16", False), (250, 131075, 300, "f32", True)])
def test_distill_many_rows(R, V, k, dtype, tail):
    # every CTA takes several rows, some of them of weight 0, in any order
    rng = np.random.default_rng(V)
    x = torch.randn(R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(V)).mul_(3).to(DT[dtype])
    z = x.float() * 0.9 + torch.randn(R, V, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    vals, idx = torch.topk(z, k, dim=1)
    idx = idx.int()
    tl = torch.logsumexp(z / 2.0, 1) if tail else None
    y = rng.integers(V, size=R)
    w = np.where(rng.random(R) < 0.3, 0.0, 0.5 + rng.random(R)).astype(np.float32)
    w[-3:] = 0.0
    for masked in (False, True):
        wt = torch.from_numpy(w).cuda() if masked else None
        args = dict(teacher_lse=tl, labels=torch.from_numpy(y).cuda(), row_weight=wt, temperature=2.0, kd_weight=0.7, ce_weight=0.4)
        grad = torch.full_like(x, 7.0)
        loss, _ = pkg.distill_loss_grad(x, idx, vals, **args, grad=grad)
        assert torch.equal(pkg.distill_loss(x, idx, vals, **args), loss)
        if masked:
            off = wt == 0
            assert not grad[off].any() and not loss[off].any()
        some = np.unique(np.concatenate([rng.integers(R, size=10), [0, R - 4, R - 1]]))
        st = torch.from_numpy(some).cuda()
        check_distill(x[st], idx[st].cpu().numpy(), vals[st], None if tl is None else f64(tl)[some], y[some],
                      w[some] if masked else None, 2.0, 0.7, 0.4, dtype, loss[st], grad[st])
        # all rows: a row's gradient sums to 0
        sums = grad.float().sum(1).abs() / grad.float().abs().sum(1).clamp(min=1e-20)
        assert float(sums.max()) < 0.05


def test_distill_rows_without_a_teacher():
    rng = np.random.default_rng(3)
    x = place(logits(rng, 3, 2000), "f32")
    idx = np.array([[-1] * 4, [5, 6, 7, 8], [1, 2, 3, 4]], np.int32)
    vals = torch.tensor([[1.0] * 4, [-INF] * 4, [1.0, -INF, 0.5, -INF]], device="cuda")
    y = np.array([10, -1, 3])
    for tl in (None, np.array([3.0, 3.0, 2.0], np.float32)):
        loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, labels=torch.from_numpy(y).cuda(),
                                           teacher_lse=None if tl is None else torch.from_numpy(tl).cuda(),
                                           kd_weight=0.5, ce_weight=0.5)
        check_distill(x, idx, vals, tl, y, None, 1.0, 0.5, 0.5, "f32", loss, grad)
        assert float(loss[1]) == 0.0 and not f64(grad)[1].any()


def test_distill_all_words_listed_and_none_left():
    # every coordinate listed: p_rest = 0, no bucket even though sum q < 1 by rounding or by the teacher_lse given
    rng = np.random.default_rng(4)
    x = place(logits(rng, 2, 40), "f32")
    idx = np.stack([rng.permutation(40), np.arange(40)]).astype(np.int32)
    vals = torch.from_numpy(rng.standard_normal((2, 40)).astype(np.float32)).cuda()
    tl = np.array([ref.lse(r) + 0.1 for r in f64(vals)], np.float32)
    loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, teacher_lse=torch.from_numpy(tl).cuda())
    check_distill(x, idx, vals, tl, None, None, 1.0, 1.0, 0.0, "f32", loss, grad)


def test_distill_counts_indices_out_of_range():
    rng = np.random.default_rng(5)
    x = place(logits(rng, 3, 500), "bf16")
    idx = np.array([[1, 500, 2], [3, 2 ** 31 - 1, -1], [4, 5, 6]], np.int32)
    vals = torch.from_numpy(rng.standard_normal((3, 3)).astype(np.float32)).cuda()
    y = np.array([500, 3, -100])
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, grad = pkg.distill_loss_grad(x, torch.from_numpy(idx).cuda(), vals, labels=torch.from_numpy(y).cuda(),
                                       kd_weight=1.0, ce_weight=1.0, bad_count=bad)
    assert int(bad) == 3
    check_distill(x, idx, vals, None, np.where(y >= 500, -1, y), None, 1.0, 1.0, 1.0, "bf16", loss, grad)


def test_distill_label_or_teacher_on_a_masked_word_is_infinite():
    x = np.array([[0.0, -INF, 1.0, 2.0]] * 2)
    idx = torch.tensor([[1, 2], [2, 3]], dtype=torch.int32, device="cuda")
    vals = torch.ones(2, 2, device="cuda")
    y = torch.tensor([0, 1], device="cuda")
    loss, grad = pkg.distill_loss_grad(place(x, "f32"), idx, vals, labels=y, kd_weight=1.0, ce_weight=1.0)
    assert f64(loss).tolist() == [INF, INF]
    check_distill(place(x, "f32"), idx.cpu().numpy(), vals, None, np.array([0, 1]), None, 1.0, 1.0, 1.0, "f32", loss, grad)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_against_differences(tail):
    # central differences of the operator's own loss along random directions d (|d_j| <= 1).  Along d the
    # loss' third derivative is at most tau^2 kd * 6 / tau^3 + ce * 6 < 12 (third cumulant of a variable in
    # [-1, 1], at most 2, and the bucket's), so with h = 2^-5 the quotient is off by h^2 12 / 6 = 2^-9; the
    # losses' rounding, under 1e-5 each, adds 1e-5 / h.
    rng = np.random.default_rng(6)
    R, V, k, tau, h = 4, 3000, 20, 1.5, 2.0 ** -5
    base = logits(rng, R, V)
    idx, vals, tl = teacher(rng, base, k, tau, "f32")
    y = rng.integers(V, size=R)
    args = dict(teacher_lse=torch.from_numpy(tl).cuda() if tail else None, labels=torch.from_numpy(y).cuda(),
                temperature=tau, kd_weight=0.6, ce_weight=0.5)
    it = torch.from_numpy(idx).cuda()
    x = place(base, "f32")
    _, grad = pkg.distill_loss_grad(x, it, vals, **args)
    for _ in range(4):
        d = place(rng.uniform(-1, 1, (R, V)), "f32")
        up = f64(pkg.distill_loss(x + h * d, it, vals, **args))
        dn = f64(pkg.distill_loss(x - h * d, it, vals, **args))
        want = (f64(grad) * f64(d)).sum(1)
        assert np.abs((up - dn) / (2 * h) - want).max() < 2.0 ** -9 + 1e-5 / h


def test_objective_on_another_stream():
    rng = np.random.default_rng(7)
    x = place(logits(rng, 64, 32000), "bf16")
    want = pkg.topk_logits(x, 32, temperature=2.0)
    lossw, gradw = pkg.distill_loss_grad(x, want[0], want[1], temperature=2.0)
    rw = pkg.route(x[:, :64], 4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            y = x * 1.0  # made on s just before
        got = pkg.topk_logits(y, 32, temperature=2.0, stream=stream)
        loss, grad = pkg.distill_loss_grad(y, got[0], got[1], temperature=2.0, stream=stream)
        r = pkg.route(y[:, :64], 4, stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got + (loss, grad) + r, want + (lossw, gradw) + rw))


def test_objective_in_a_graph():
    rng = np.random.default_rng(8)
    x = place(logits(rng, 33, 5003), "bf16")
    run = lambda: (lambda t: t + pkg.distill_loss_grad(x, t[0], t[1]) + pkg.route(x[:, :37], 5))(  # noqa: E731
        pkg.topk_logits(x, 20))
    run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    x.copy_(torch.from_numpy(logits(rng, 33, 5003)))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, run()))


# ---- routing ------------------------------------------------------------------------------------

ROUTE = [  # tokens, experts, k, groups, dtype, kind, renorm, offset, pad
    (1, 1, 1, 1, "f32", "normal", True, 0, 0), (1, 8, 2, 1, "bf16", "normal", True, 0, 0),
    (3, 8, 8, 2, "f16", "ties", False, 1, 0), (257, 7, 3, 4, "f32", "ties", True, 0, 2),
    (1000, 64, 6, 9, "bf16", "normal", True, 0, 0), (700, 65, 1, 1, "bf16", "ties", False, 0, 0),
    (300, 256, 8, 3, "f32", "normal", False, 0, 0), (90, 300, 32, 2, "bf16", "normal", True, 0, 0),
    (40, 512, 8, 1, "f16", "masked", True, 3, 1), (33, 1024, 32, 5, "f32", "masked", False, 0, 0),
    (2000, 16, 4, 40, "bf16", "masked", True, 8, 8), (64, 31, 31, 1, "f32", "equal", True, 0, 0),
    (0, 16, 2, 1, "bf16", "normal", True, 0, 0), (0, 16, 2, 3, "f32", "normal", True, 0, 0),
    (5000, 128, 8, 7, "bf16", "normal", True, 0, 0), (300, 48, 4, 2, "f32", "low", True, 0, 0),
    (300, 200, 7, 1, "bf16", "high", False, 0, 0), (700, 64, 6, 300, "bf16", "normal", True, 0, 0),
    (3000, 256, 8, 2, "bf16", "equal", True, 0, 0), (500, 100, 24, 3, "f32", "normal", True, 0, 0),
    (400, 64, 6, 2, "bf16", "zeros", True, 0, 0), (400, 256, 8, 2, "f32", "zeros", False, 0, 0), (300, 16, 3, 1, "f16", "zeros", True, 0, 0),
    (40000, 64, 6, 9, "bf16", "normal", True, 0, 0), (90000, 8, 2, 3, "f32", "ties", True, 0, 0),
    (20000, 256, 8, 1, "f32", "normal", False, 0, 0), (12000, 100, 3, 5, "bf16", "ties", True, 0, 0),
    (20, 1000, 20, 2, "f16", "ties", False, 0, 0), (9000, 4, 1, 2, "bf16", "normal", False, 0, 0),
]


def groups_of(rng, T, G):
    cuts = np.sort(rng.integers(T + 1, size=G - 1))
    if G > 3:
        cuts[1] = cuts[0]  # an empty group
    return np.concatenate([[0], np.sort(cuts), [T]]).astype(np.int32)


@pytest.mark.parametrize("T,E,k,G,dtype,kind,renorm,offset,pad", ROUTE)
def test_route(T, E, k, G, dtype, kind, renorm, offset, pad):
    rng = np.random.default_rng(T + 7 * E)
    h = logits(rng, T, E, kind)
    valid = rng.random(T) < 0.8 if T > 1 else np.ones(T, bool)
    if T > 20:
        h[5] = -INF  # a token whose mask leaves no expert
        h[6, 1:] = -INF
    x = place(h, dtype, offset, pad)
    cu = groups_of(rng, T, G)
    cut = torch.from_numpy(cu).cuda() if G > 1 else None
    vt = torch.from_numpy(valid).cuda()
    idx, w, counts, live, losses = pkg.route(x, k, renormalize=renorm, cu_tokens=cut, valid=vt)
    ri, rw, rc, rl, bal, z = ref.route(f64(x), k, cu, valid, renorm)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(counts.cpu().numpy(), rc) and np.array_equal(live.cpu().numpy(), rl)
    # a weight: two sums of at most E terms and exponents of up to 2 max|x|
    xm = np.abs(f64(x)[np.isfinite(f64(x))]).max(initial=0.0)
    rel = ref.U * (E / 8 + 64 + 16 * xm)
    assert np.abs(f64(w) - rw).max(initial=0.0) <= rel
    # the sums over tokens add U for each addition on a path: at most tokens / 8 + 512
    many = ref.U * (T / 8 + 512)
    got = f64(losses)
    assert abs(got[0] - bal) <= (rel + many) * abs(bal) and abs(got[1] - z) <= (2 * rel + many) * max(z, 1.0)
    again = pkg.route(x, k, renormalize=renorm, cu_tokens=cut, valid=vt)
    assert all(torch.equal(a, b) for a, b in zip(again, (idx, w, counts, live, losses)))

    dw = rng.standard_normal((T, k))
    dl = np.array([0.7, 0.05])
    dwt, dlt = torch.from_numpy(dw).float().cuda(), torch.from_numpy(dl).float().cuda()
    for a, b in ((dwt, dlt), (None, dlt), (dwt, None)):
        grad = f64(pkg.route_backward(x, idx, counts, live, d_weights=a, d_losses=b, renormalize=renorm, cu_tokens=cut))
        want, size = ref.route_grad(f64(x), ri, rc, rl, cu, f64(dwt) * (a is not None),
                                    f64(dlt) * (b is not None), renorm)
        off = np.abs(grad - want) - ((4 * rel + 16 * ref.U) * size + np.abs(want) * ref.ROUND[dtype] + ref.TINY[dtype])
        assert off.max(initial=0.0) <= 0
    assert not f64(pkg.route_backward(x, idx, counts, live, renormalize=renorm, cu_tokens=cut)).any()


@pytest.mark.parametrize("E,dtype", [(8, "f32"), (24, "bf16"), (64, "f32"), (128, "f16"), (256, "bf16"), (300, "f32"), (1000, "f32")])
def test_route_nan_and_infinities(E, dtype):
    # NaN ranks above +inf, an expert of -inf below all others; a token with one of the first two has NaN weights
    rng = np.random.default_rng(E)
    h = logits(rng, 40, E)
    h[0, 3] = np.nan
    h[1, 5] = INF
    h[2, :] = -INF
    h[2, [1, 6]] = [1.0, -2.0]
    h[3, [7, 2]] = [-np.nan, np.nan]
    x = place(h, dtype)
    idx, w, counts, live, losses = pkg.route(x, 4)
    i = idx.cpu().numpy()
    assert i[0, 0] == 3 and i[1, 0] == 5 and i[3, :2].tolist() == [2, 7]
    assert i[2].tolist() == [1, 6, 0, 2] and f64(w)[2, 2:].tolist() == [0.0, 0.0]
    for t in range(40):
        assert np.array_equal(i[t], ref.topk(f64(x[t]), 4)), t
    assert live.tolist() == [40, 40, 1] and int(counts.sum()) == 160
    assert np.isfinite(f64(w)[4:]).all() and np.isnan(f64(w)[[0, 1, 3]]).any(1).all()


def test_route_gradient_against_differences():
    # third derivatives along |d| <= 1 are below 12 for each of the three terms (weights, balance, z with
    # lse < 6); h = 2^-6 leaves 2^-12 * 2 * 3 plus the terms' rounding 2e-6 * 3 / h; a token whose choice
    # changes within h would break the formula, so logits are spaced wider than 2h
    rng = np.random.default_rng(9)
    T, E, k, h = 30, 12, 3, 2.0 ** -6
    base = rng.permuted(np.tile(np.arange(E) * 0.25, (T, 1)), axis=1)
    cu = torch.tensor([0, 11, 30], dtype=torch.int32, device="cuda")
    dw = rng.standard_normal((T, k)) / T
    dl = np.array([0.5, 0.03])
    x = place(base, "f32")
    for renorm in (True, False):
        def total(x):
            _, w, _, _, losses = pkg.route(x, k, renormalize=renorm, cu_tokens=cu)
            return (f64(w) * dw).sum() + (f64(losses) * dl).sum()
        idx, _, counts, live, _ = pkg.route(x, k, renormalize=renorm, cu_tokens=cu)
        grad = f64(pkg.route_backward(x, idx, counts, live, d_weights=torch.from_numpy(dw).float().cuda(),
                                      d_losses=torch.from_numpy(dl).float().cuda(), renormalize=renorm, cu_tokens=cu))
        for _ in range(4):
            d = place(rng.uniform(-1, 1, (T, E)), "f32")
            q = (total(x + h * d) - total(x - h * d)) / (2 * h)
            assert abs(q - (grad * f64(d)).sum()) < 6 * 2.0 ** -12 + 6e-6 / h


def test_route_tokens_outside_all_groups_are_not_live():
    x = place(logits(np.random.default_rng(10), 600, 16), "f32")
    cu = torch.tensor([100, 300, 300, 500], dtype=torch.int32, device="cuda")
    idx, w, counts, live, losses = pkg.route(x, 2, cu_tokens=cu)
    i = idx.cpu().numpy()
    assert (i[:100] == -1).all() and (i[500:] == -1).all() and (i[100:500] >= 0).all()
    assert live.tolist() == [200, 0, 200, 400, 2] and int(counts.sum()) == 800
    g = f64(pkg.route_backward(x, idx, counts, live, d_losses=torch.ones(2, device="cuda"), cu_tokens=cu))
    assert not g[:100].any() and not g[500:].any() and g[100:500].any()


# ---- refusals -----------------------------------------------------------------------------------


def test_refusals():
    x = torch.zeros(4, 100, device="cuda")
    idx = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    vals = torch.zeros(4, 3, device="cuda")
    for bad in (lambda: pkg.topk_logits(x, 0), lambda: pkg.topk_logits(x, 101), lambda: pkg.topk_logits(x, 3, temperature=0.0),
                lambda: pkg.topk_logits(x[:1].expand(4, 100), 3), lambda: pkg.distill_loss(x, idx, vals, temperature=-1.0),
                lambda: pkg.distill_loss(x, idx, vals, kd_weight=float("nan")), lambda: pkg.route(x, 33),
                lambda: pkg.route(x, 0), lambda: pkg.route(torch.zeros(4, 1025, device="cuda"), 2)):
        with pytest.raises(ScapeError):
            bad()
    for bad in (lambda: pkg.topk_logits(x.double(), 3), lambda: pkg.topk_logits(x.t(), 3), lambda: pkg.topk_logits(x.cpu(), 3),
                lambda: pkg.topk_logits(x[0], 3), lambda: pkg.distill_loss(x, idx.long(), vals),
                lambda: pkg.distill_loss(x, idx, vals[:, :2]), lambda: pkg.distill_loss(x, idx, None),
                lambda: pkg.distill_loss(x, idx, vals.t().contiguous().t()), lambda: pkg.distill_loss(x, idx.cpu(), vals),
                lambda: pkg.distill_loss(x, idx, vals, labels=torch.zeros(4, dtype=torch.int32, device="cuda")),
                lambda: pkg.distill_loss_grad(x, idx, vals, grad=x.half()), lambda: pkg.route(x, 2, cu_tokens=torch.zeros(
                    2, dtype=torch.int64, device="cuda")), lambda: pkg.route(x, 2, valid=torch.ones(3, dtype=torch.bool, device="cuda")),
                lambda: pkg.route_backward(x, idx, vals, vals)):
        with pytest.raises(ValueError):
            bad()
    assert pkg.topk_logits(x, 3)[0].tolist() == [[0, 1, 2]] * 4  # still usable
