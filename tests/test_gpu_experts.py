"""Experts' rows against their definitions in 64 bits: every type, odd lengths and
addresses, tokens without a choice, experts without a token, one token and many.

Bounds, with U = 2^-24 (fp32's unit roundoff) and half a step of the result's type:
a sum of k products by fused multiply-adds is off by at most k U of the sum of their
magnitudes; a dot product of n terms, n/32 + 5 additions on its longest path, by
(n/32 + 6) U of that sum; a product by U of itself."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as pkg  # noqa: E402
from objective_ref import ROUND, TINY, U  # noqa: E402
from sparse_communication_distributed_gb300 import ScapeError  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def choices(rng, T, k, E, kind="some"):
    """k different experts a token (as a router gives them), some tokens with none."""
    idx = np.array([rng.permutation(max(E, k))[:k] % E for _ in range(T)], np.int32).reshape(T, k)
    if kind == "some":
        idx[rng.random(T) < 0.3] = -1
        idx[rng.random((T, k)) < 0.1] = -7
    elif kind == "one":
        idx[:] = E // 2
    elif kind == "none":
        idx[:] = -1
    return idx


def plan(idx, E, align):
    T, k = idx.shape
    flat = idx.reshape(-1)
    room = T * k + min(E, T * k) * (align - 1)
    source, slots, offsets = np.full(room, -1, np.int32), np.full(T * k, -1, np.int32), np.zeros(E + 1, np.int32)
    at = 0
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        slots[mine] = at + np.arange(mine.size)
        source[at:at + mine.size] = mine
        at += -(-mine.size // align) * align
        offsets[e + 1] = at
    return offsets, slots.reshape(T, k), source


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def f64(t):
    return t.double().cpu().numpy()


PLANS = [(0, 3, 5, 1, "some"), (1, 1, 1, 1, "all"), (1, 2, 8, 128, "all"), (3, 8, 8, 16, "some"), (97, 2, 3, 1, "one"),
         (255, 8, 64, 4, "some"), (256, 8, 1024, 1, "all"), (257, 8, 64, 128, "some"), (1000, 1, 2, 7, "some"),
         (5000, 6, 33, 1, "some"), (4097, 32, 100, 65, "some"), (20000, 8, 1023, 1, "all"), (9000, 4, 16, 128, "none"),
         (70000, 3, 300, 2, "one"), (200000, 8, 256, 128, "some")]


@pytest.mark.parametrize("T,k,E,align,kind", PLANS)
def test_plan(T, k, E, align, kind):
    rng = np.random.default_rng(T + E)
    if kind == "some" and T > 10000:
        idx = rng.integers(-1, E, (T, k)).astype(np.int32)  # (the same expert twice in a token, too)
    else:
        idx = choices(rng, T, k, E, kind)
    got = pkg.expert_plan(cuda(idx), E, align=align)
    for g, w in zip(got, plan(idx, E, align)):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("T", [100, 3000])
def test_plan_counts_experts_out_of_range(T):
    rng = np.random.default_rng(T)
    idx = rng.integers(-3, 20, (T, 4)).astype(np.int32)
    idx[5, 1], idx[T - 1, 3] = 2 ** 31 - 1, -2 ** 31
    bad = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    got = pkg.expert_plan(cuda(idx), 16, bad_count=bad)
    assert int(bad) == 5 + int((idx >= 16).sum())
    for g, w in zip(got, plan(np.where(idx >= 16, -1, idx), 16, 1)):
        assert np.array_equal(g.cpu().numpy(), w)


ROWS = [(1, 1, 1, 1, 1, 0), (1, 2048, 2, 8, 1, 0), (5, 7, 2, 3, 4, 0), (33, 61, 6, 64, 1, 3), (40, 130, 3, 16, 16, 2),
        (300, 1280, 8, 128, 1, 0), (129, 2048, 6, 64, 128, 16), (50, 4104, 32, 40, 1, 0), (17, 5001, 1, 2, 8, 1),
        (1200, 64, 4, 1024, 1, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,D,k,E,align,pad", ROWS)
def test_there_and_back(T, D, k, E, align, pad, dtype):
    rng = np.random.default_rng(D + T)
    idx = choices(rng, T, k, E, "some" if T > 1 else "all")
    offsets, slots, source = pkg.expert_plan(cuda(idx), E, align=align)
    wide = cuda(rng.standard_normal((T, D + pad))).to(DT[dtype])
    x = wide[:, pad:]  # rows that start anywhere
    rows = pkg.expert_dispatch(x, slots, source)
    h_slots, h_source = slots.cpu().numpy(), source.cpu().numpy()
    want = torch.where(source[:, None] >= 0, x[(source.clamp(min=0) // k).long()], torch.zeros((), dtype=x.dtype, device="cuda"))
    assert rows.shape == (h_source.size, D) and torch.equal(rows, want)

    y = cuda(rng.standard_normal(rows.shape)).to(DT[dtype])
    w = cuda(rng.standard_normal((T, k)).astype(np.float32))
    hy, hw, on = f64(y), f64(w), h_slots >= 0
    at = np.where(on, h_slots, 0)
    for weights, ww in ((w, hw), (None, np.ones((T, k)))):
        got = f64(pkg.expert_combine(y, slots, weights))
        terms = np.where(on[:, :, None], hy[at] * ww[:, :, None], 0.0)
        ref, size = terms.sum(1), np.abs(terms).sum(1)
        assert np.all(np.abs(got - ref) <= k * U * size + ROUND[dtype] * (np.abs(ref) + k * U * size) + TINY[dtype])

    d_out = cuda(rng.standard_normal((T, D))).to(DT[dtype])
    d_y, d_w = pkg.expert_combine_backward(d_out, y, slots, source, w)
    g = f64(d_out)
    ref = np.where(h_source[:, None] >= 0, g[h_source.clip(0) // k] * hw.reshape(-1)[h_source.clip(0)][:, None], 0.0)
    got = f64(d_y)
    assert np.all(np.abs(got - ref) <= (U + ROUND[dtype]) * (1 + U) * np.abs(ref) + TINY[dtype])
    assert np.all(got[h_source < 0] == 0)
    terms = np.where(on[:, :, None], hy[at] * g[:, None, :], 0.0)
    got = f64(d_w)
    assert np.all(np.abs(got - terms.sum(2)) <= (D / 32 + 6) * U * np.abs(terms).sum(2))
    assert np.all(got[~on] == 0)
    # bit for bit again
    again = pkg.expert_combine_backward(d_out, y, slots, source, w)
    assert torch.equal(d_y, again[0]) and torch.equal(d_w, again[1])


def test_gradient_against_differences():
    # <combine(y + h v) - combine(y - h v), g> / 2h in fp32: the sum is linear in y and in w
    rng = np.random.default_rng(4)
    T, D, k, E = 20, 33, 3, 5
    offsets, slots, source = pkg.expert_plan(cuda(choices(rng, T, k, E)), E)
    y, v = (cuda(rng.standard_normal((source.numel(), D)).astype(np.float32)) for _ in range(2))
    w, u = (cuda(rng.standard_normal((T, k)).astype(np.float32)) for _ in range(2))
    g = cuda(rng.standard_normal((T, D)).astype(np.float32))
    d_y, d_w = pkg.expert_combine_backward(g, y, slots, source, w)
    h = 0.5
    n = T * D * k
    for step, along, grad in ((lambda s: pkg.expert_combine(y + s * v, slots, w), v, d_y),
                              (lambda s: pkg.expert_combine(y, slots, w + s * u), u, d_w)):
        diff = float(((f64(step(h)) - f64(step(-h))) * f64(g)).sum()) / (2 * h)
        want = float((f64(along) * f64(grad)).sum())
        # every one of the n products of magnitude up to about 5^3 is off by a few roundings, of random sign
        assert abs(diff - want) <= n * 8 * U * 125


def test_dispatch_gradient_is_combine_without_weights():
    rng = np.random.default_rng(5)
    T, D, k, E = 50, 40, 4, 9
    offsets, slots, source = pkg.expert_plan(cuda(choices(rng, T, k, E)), E, align=8)
    d_rows = cuda(rng.standard_normal((source.numel(), D)).astype(np.float32))
    got = f64(pkg.expert_combine(d_rows, slots))
    want = np.zeros((T, D))
    h = source.cpu().numpy()
    np.add.at(want, h[h >= 0] // k, f64(d_rows)[h >= 0])
    assert np.all(np.abs(got - want) <= k * U * 5 * k)


def test_tokens_without_a_choice_are_not_read():
    idx = np.array([[0, 1], [-1, -1], [1, -1]], np.int32)
    offsets, slots, source = pkg.expert_plan(cuda(idx), 2)
    x = torch.ones(3, 16, device="cuda")
    x[1] = float("nan")
    rows = pkg.expert_dispatch(x, slots, source)
    assert torch.isfinite(rows).all() and rows[3].eq(0).all()
    w = torch.ones(3, 2, device="cuda")
    w[1] = float("nan")
    w[2, 1] = float("inf")
    assert pkg.expert_combine(rows, slots, w).tolist() == [[2.0] * 16, [0.0] * 16, [1.0] * 16]
    d_out = torch.ones(3, 16, device="cuda")
    d_out[1] = float("nan")
    d_y, d_w = pkg.expert_combine_backward(d_out, rows, slots, source, w)
    assert torch.isfinite(d_y).all() and d_w.tolist() == [[16.0, 16.0], [0.0, 0.0], [16.0, 0.0]]


def test_slots_outside_the_rows_are_no_choice():
    y = torch.ones(4, 8, device="cuda")
    slots = torch.tensor([[0, 4], [3, 2 ** 31 - 1], [-5, 1]], dtype=torch.int32, device="cuda")
    assert pkg.expert_combine(y, slots).tolist() == [[1.0] * 8] * 3
    source = torch.tensor([0, 5, -1, 2], dtype=torch.int32, device="cuda")
    w = torch.full((3, 2), 2.0, device="cuda")
    d_y, d_w = pkg.expert_combine_backward(torch.ones(3, 8, device="cuda"), y, slots, source, w)
    assert d_y.tolist() == [[2.0] * 8, [2.0] * 8, [0.0] * 8, [2.0] * 8]
    assert d_w.tolist() == [[8.0, 0.0], [8.0, 0.0], [0.0, 8.0]]


def test_rows_past_32_bit_offsets():
    # the last rows start 4.9e9 bytes into the buffer
    R, D = 70000, 35008
    y = torch.zeros(R, D, dtype=torch.bfloat16, device="cuda")
    y[R - 1], y[1] = 2.0, 1.0
    slots = torch.tensor([[R - 1, 1]], dtype=torch.int32, device="cuda")
    source = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    source[R - 1], source[1] = 0, 1
    assert pkg.expert_combine(y, slots).eq(3.0).all()
    x = torch.full((1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    rows = pkg.expert_dispatch(x, slots, source)
    assert rows[R - 1].eq(5).all() and rows[1].eq(5).all() and rows[2:R - 1].eq(0).all() and rows[0].eq(0).all()


def test_after_the_router_on_another_stream_and_in_a_graph():
    T, E, k, D = 3000, 32, 4, 96
    gen = torch.Generator(device="cuda").manual_seed(0)
    logits = torch.randn(T, E, generator=gen, device="cuda")
    x = torch.randn(T, D, generator=gen, device="cuda").to(torch.bfloat16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def layer(stream=None):
        idx, w, counts, live, _ = pkg.route(logits, k, stream=stream)
        offsets, slots, source = pkg.expert_plan(idx, E, align=16, stream=stream)
        rows = pkg.expert_dispatch(x, slots, source, stream=stream)
        out = pkg.expert_combine(rows, slots, w, stream=stream)
        return [offsets, slots, source, rows, out, counts] + list(
            pkg.expert_combine_backward(x, rows, slots, source, w, stream=stream))

    want = layer()
    got = layer(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    n = want[0].diff().cpu() - want[5][0].cpu()
    assert int(n.min()) >= 0 and int(n.max()) < 16
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    logits.copy_(logits.flip(0))
    want = layer()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    i2, i1 = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    with pytest.raises(ValueError, match="idx"):
        pkg.expert_plan(i2.long(), 4)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.expert_plan(i2.cpu(), 4)
    with pytest.raises(ScapeError, match="experts=0"):
        pkg.expert_plan(i2, 0)
    with pytest.raises(ScapeError, match="align"):
        pkg.expert_plan(i2, 4, align=0)
    with pytest.raises(ValueError, match="32 bits"):
        pkg.expert_plan(i2, 1 << 40)
    with pytest.raises(ValueError, match="slots"):
        pkg.expert_dispatch(x[:3], i2, i1)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.expert_dispatch(x.T, i2, i1)
    with pytest.raises(ValueError, match="x must be"):
        pkg.expert_dispatch(x.double(), i2, i1)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.expert_combine(torch.zeros(4, 9, device="cuda")[:, :8], i2, w)
    with pytest.raises(ValueError, match="weights"):
        pkg.expert_combine(x, i2, w.double())
    with pytest.raises(ValueError, match="source"):
        pkg.expert_combine_backward(x, x, i2, i1, w)
    with pytest.raises(ValueError, match="d_out"):
        pkg.expert_combine_backward(x[:2], x, i2, i1[:4], w)
    with pytest.raises(ValueError, match="weights"):
        pkg.expert_combine_backward(x, x, i2, i1[:4], None)
