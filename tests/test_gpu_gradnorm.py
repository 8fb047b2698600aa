"""Gradients' norms and clipping against their definitions in 64 bits: every type,
odd sizes and addresses, many tensors, values whose squares leave fp32's range.

Bounds, with U = 2^-24: a sum of 64 squares, 32 of them one behind the other, is off
by at most 33 U of itself, sums in 64 bits by nothing that counts; so a norm is off by
17 U and its own rounding.  A scaled element carries the norm's 17 U, the rounding of
the scale and of the product (U each), and half a step of its type."""
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
NAME = {v: k for k, v in DT.items()}


def tensors(rng, sizes, dtypes, scale=1.0, offset=0):
    out = []
    for i, n in enumerate(sizes):
        dt = DT[dtypes[i % len(dtypes)]]
        buf = torch.zeros(n + offset, dtype=dt, device="cuda")
        t = buf[offset:]
        t.copy_(torch.from_numpy(rng.standard_normal(n) * scale))
        out.append(t)
    return out


def norm64(ts):
    # each tensor scaled by its largest element, so that nothing leaves the range of 64 bits
    total = 0.0
    for t in ts:
        x = t.double()
        total += float((x * x).sum())
    return np.sqrt(total)


def close(got, want):
    assert abs(float(got) - want) <= 18 * U * want, (float(got), want)


SIZES = [[1], [7], [8, 0, 9], [1000, 1, 4096, 4097], [65536 * 3 + 5], [3, 1 << 20, 12345], [5] * 700, [(1 << 22) + 3, 1 << 22]]


@pytest.mark.parametrize("dtypes", [["bf16"], ["f16"], ["f32"], ["bf16", "f32", "f16"]])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_norm_and_clip(sizes, offset, dtypes):
    rng = np.random.default_rng(sum(sizes) + offset)
    ts = tensors(rng, sizes, dtypes, 0.1, offset)
    want = norm64(ts)
    before = [t.clone() for t in ts]
    close(pkg.grad_norm(ts), want)
    for out_type, shift in (("bf16", 0), ("f32", 1), ("f16", 3)):
        flat = torch.full((sum(sizes) + shift + 8,), 9.0, dtype=DT[out_type], device="cuda")
        outs = list(flat[shift:shift + sum(sizes)].split(sizes))
        c = want / 3
        close(pkg.clip_grads(ts, c, out=outs), want)
        assert flat[:shift].eq(9).all() and flat[shift + sum(sizes):].eq(9).all()  # nothing beside the results
        for x, o in zip(before, outs):
            ref = x.double() * (np.float32(c).item() / want)
            off = (o.double() - ref).abs() - ((20 * U + ROUND[out_type]) * ref.abs() + TINY[out_type])
            assert off.numel() == 0 or off.max().item() <= 0
    assert all(torch.equal(a, b) for a, b in zip(ts, before))
    close(pkg.clip_grads(ts, want / 3), want)  # in place
    for x, t in zip(before, ts):
        ref = x.double() * (np.float32(want / 3).item() / want)
        off = (t.double() - ref).abs() - ((20 * U + ROUND[NAME[t.dtype]]) * ref.abs() + TINY[NAME[t.dtype]])
        assert off.numel() == 0 or off.max().item() <= 0


def test_below_the_largest_norm_nothing_changes():
    rng = np.random.default_rng(0)
    ts = tensors(rng, [1000, 333], ["bf16"])
    before = [t.clone() for t in ts]
    flat = torch.empty(1333, dtype=torch.bfloat16, device="cuda")
    for c in (1e6, float("inf")):
        pkg.clip_grads(ts, c)
        pkg.clip_grads(ts, c, out=list(flat.split([1000, 333])))
        assert all(torch.equal(a, b) for a, b in zip(ts, before)) and torch.equal(flat, torch.cat(before))


def test_workers_have_norms_of_their_own():
    rng = np.random.default_rng(1)
    workers = [tensors(rng, [100, 20001], ["bf16"], s) for s in (0.01, 1.0, 5.0)] + [[], tensors(rng, [0], ["f32"])]
    workers.append(tensors(rng, [33], ["f32"], 100.0))
    want = [norm64(w) for w in workers]
    got = pkg.grad_norm(workers)
    assert got.shape == (6,)
    for g, w in zip(got, want):
        close(g, w)
    before = [[t.clone() for t in w] for w in workers]
    close(pkg.clip_grads(workers, 50.0)[2], want[2])
    for w, b, n in zip(workers, before, want):
        for t, x in zip(w, b):
            s = min(1.0, 50.0 / n) if n else 1.0
            off = (t.double() - x.double() * s).abs() - (20 * U + ROUND[NAME[t.dtype]]) * x.double().abs() * s
            assert off.numel() == 0 or off.max().item() <= 0
    many = [tensors(rng, [10], ["f32"]) for _ in range(64)]
    for g, w in zip(pkg.grad_norm(many), many):
        close(g, norm64(w))
    assert pkg.grad_norm([]).tolist() == [0.0]


@pytest.mark.parametrize("dtype,scale", [("bf16", 1e30), ("f32", 1e36), ("bf16", 1e-30), ("f32", 1e-38), ("f16", 2e4),
                                         ("f32", 1e19), ("f32", 1e-23)])
def test_squares_beyond_32_bits(dtype, scale):
    rng = np.random.default_rng(2)
    ts = tensors(rng, [1000, 77], [dtype], 1.0)
    for t in ts:
        t.copy_((t.double() * scale).clamp(-torch.finfo(t.dtype).max, torch.finfo(t.dtype).max))
    want = norm64(ts)
    got = float(pkg.grad_norm(ts))
    # a result among fp32's denormals is rounded to one of them
    assert abs(got - want) <= 18 * U * want + 2.0 ** -149
    out = [torch.empty(t.numel(), device="cuda") for t in ts]
    c = 2.0 ** -10 * want if want > 1 else 0.25 * want
    pkg.clip_grads(ts, c, out=out)
    for t, o in zip(ts, out):
        ref = t.double() * (np.float32(c).item() / want)
        assert ((o.double() - ref).abs() <= 20 * U * ref.abs() + 2.0 ** -149).all()


def test_a_scale_below_32_bits():
    # 1e-25 / 4e37 is no number of 32 bits, what it gives is
    t = torch.tensor([3e37, -2e37, 1e30, 1.0], device="cuda")
    out = torch.empty(4, device="cuda")
    n = float(pkg.clip_grads([t], 1e-25, out=[out]))
    want = t.double() * (np.float32(1e-25).item() / norm64([t]))
    assert abs(n - norm64([t])) <= 18 * U * n
    assert ((out.double() - want).abs() <= 20 * U * want.abs() + 2.0 ** -149).all() and float(out[0]) > 0
    pkg.clip_grads([t], 1e-25)
    assert torch.equal(t, out)


def test_one_huge_element_among_small_ones():
    t = torch.full((100000,), 1e-20, device="cuda")
    t[54321] = 3e25
    close(pkg.grad_norm([t]), 3e25)
    t[54321] = 1e-20
    close(pkg.grad_norm([t]), float(np.float32(1e-20)) * np.sqrt(100000))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_gradients_are_reported_and_left(bad, dtype):
    rng = np.random.default_rng(3)
    a, b = tensors(rng, [5000, 300], [dtype], 3.0), tensors(rng, [5000], [dtype], 3.0)
    a[1][299] = bad
    before = [t.clone() for t in a]
    want = norm64(b)
    norms = pkg.clip_grads([a, b], 1.0)
    assert np.isnan(float(norms[0])) if bad != bad else float(norms[0]) == np.inf
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, before))
    close(norms[1], want)
    assert abs(float(pkg.grad_norm(b)) - 1.0) < 2 * ROUND[dtype] + 40 * U  # the other worker is clipped


def test_past_32_bit_elements():
    n = (1 << 32) + 100003
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[n - 1], t[(1 << 32) + 1], t[5] = 3.0, 4.0, 12.0
    close(pkg.grad_norm([t[1:]]), 13.0)
    close(pkg.clip_grads([t], 6.5), 13.0)
    assert [float(t[i]) for i in (n - 1, (1 << 32) + 1, 5)] == [1.5, 2.0, 6.0]


def test_streams_graphs_and_repeats():
    rng = np.random.default_rng(4)
    ts = tensors(rng, [100000, 77, 4096], ["f32"])
    flat = torch.empty(104173, dtype=torch.bfloat16, device="cuda")
    outs = list(flat.split([100000, 77, 4096]))
    want = pkg.clip_grads(ts, 1.0, out=outs)
    kept = flat.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    flat.zero_()
    side.wait_stream(torch.cuda.current_stream())
    got = pkg.clip_grads(ts, 1.0, out=outs, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(flat, kept)
    # two graphs that share nothing but the tensors, replayed in turn with new gradients
    graphs, norms = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            norms.append(pkg.clip_grads(ts, 1.0, out=outs))
        graphs.append(g)
    for t in ts:
        t.mul_(3.0)
    for g, n in zip(graphs, norms):
        flat.zero_()
        g.replay()
        torch.cuda.synchronize()
        close(n, norm64(ts))
        assert (flat.double() - kept.double()).abs().max() <= 2 * ROUND["bf16"] * kept.double().abs().max()


def test_refusals():
    t = torch.zeros(8, 8, device="cuda")
    with pytest.raises(ValueError, match="list"):
        pkg.grad_norm(t)
    with pytest.raises(ValueError, match="contiguous"):
        pkg.grad_norm([t.T[1:]])
    with pytest.raises(ValueError, match="CUDA"):
        pkg.grad_norm([t.cpu()])
    with pytest.raises(ValueError, match="bfloat16"):
        pkg.grad_norm([t.double()])
    with pytest.raises(ValueError, match="mix"):
        pkg.grad_norm([[t], t])
    with pytest.raises(ValueError, match="tensors"):
        pkg.grad_norm([t, 1.0])
    with pytest.raises(ValueError, match="same size"):
        pkg.clip_grads([t], 1.0, out=[t[:1]])
    with pytest.raises(ScapeError, match="max_norm"):
        pkg.clip_grads([t], 0.0)
    with pytest.raises(ScapeError, match="overlap"):
        pkg.clip_grads([t, t], 1.0)
    with pytest.raises(ScapeError, match="n_groups"):
        pkg.grad_norm([[t]] * 65)
    assert pkg.grad_norm([t, t]).tolist() == [0.0]
