"""The operators of a training step one behind the other, as a mixture-of-experts
language model uses them: route, plan, dispatch, experts, combine, linear cross
entropy with its gradient, the way back, clipping, and the optimizer's step."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import sparse_communication_distributed_gb300 as sc  # noqa: E402

pytestmark = pytest.mark.gpu
T, D, E, K, V, ALIGN = 300, 64, 6, 2, 1003, 16
BF = torch.bfloat16


def model(seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s, scale=1.0):
        return (torch.randn(*s, generator=gen, device="cuda") * scale)

    p = {"router": rand(D, E, scale=0.3), "w": rand(E, D, D, scale=0.125).to(BF), "head": rand(V, D, scale=0.3).to(BF)}
    x = rand(T, D).to(BF)
    y = torch.randint(V, (T,), generator=gen, device="cuda")
    valid = torch.rand(T, generator=gen, device="cuda") >= 0.1   # padding
    weight = valid.float() / valid.sum()
    return p, x, y, valid, weight


def step(p, x, y, valid, weight):
    """Loss and gradients of one worker: matrix products of the experts in torch, everything else in the library."""
    logits = x.float() @ p["router"]
    idx, w, counts, live, aux = sc.route(logits, K, valid=valid)
    offsets, slots, source = sc.expert_plan(idx, E, align=ALIGN)
    rows = sc.expert_dispatch(x, slots, source)
    # every expert on its padded segment; which rows those are is not known on the host: all experts see all rows
    owner = torch.searchsorted(offsets[1:], torch.arange(rows.shape[0], dtype=torch.int32, device="cuda"), right=True)
    mine = torch.nn.functional.one_hot(owner.clamp(max=E), E + 1)[:, :E].to(BF)
    out = torch.einsum("rd,edf,re->rf", rows.float(), p["w"].float(), mine.float()).to(BF)
    h = (x.float() + sc.expert_combine(out, slots, w).float()).to(BF)
    loss, d_h, d_head = sc.linear_ce_grad(h, p["head"], y, row_weight=weight)
    d_out, d_w = sc.expert_combine_backward(d_h, out, slots, source, w)
    d_we = torch.einsum("rd,rf,re->edf", rows.float(), d_out.float(), mine.float())
    d_rows = torch.einsum("rf,edf,re->rd", d_out.float(), p["w"].float(), mine.float()).to(BF)
    d_logits = sc.route_backward(logits, idx, counts, live, d_weights=d_w,
                                 d_losses=torch.full((2,), 0.01, device="cuda") * torch.logspace(0, -1, 2, device="cuda"))
    d_router = x.float().T @ d_logits
    d_x = d_h.float() + sc.expert_combine(d_rows, slots).float() + d_logits @ p["router"].T
    return loss, aux, {"router": d_router, "w": d_we, "head": d_head, "x": d_x}, idx


def reference(p, x, y, valid, weight, idx):
    """The same in 64 bits by autograd, the choice of experts given."""
    q = {k: v.double().requires_grad_(True) for k, v in p.items()}
    z = x.double().requires_grad_(True)
    logits = z @ q["router"]
    on = valid[:, None]
    at = idx.clamp(min=0).long()
    w = torch.softmax(logits.gather(1, at), 1) * on
    each = torch.einsum("td,edf->tef", z, q["w"])
    h = z + (each.gather(1, at[:, :, None].expand(T, K, D)) * w[:, :, None]).sum(1)
    rows = torch.nn.functional.cross_entropy(h @ q["head"].T, y, reduction="none") * weight.double()
    prob = torch.softmax(logits, 1)[valid]
    f = torch.bincount(at[valid].reshape(-1), minlength=E).double() * E / (K * len(prob))
    balance = (f * prob.mean(0)).sum()
    zl = (torch.logsumexp(logits[valid], 1) ** 2).mean()
    (rows.sum() + 0.01 * balance + 0.001 * zl).backward()
    return rows.detach(), torch.stack([balance, zl]).detach(), {**{k: v.grad for k, v in q.items()}, "x": z.grad}


def test_gradients_of_a_step():
    args = model(1)
    loss, aux, grads, idx = step(*args)
    want, waux, ref = reference(*args, idx)
    # the experts' rows, h and every gradient on the way are rounded to bf16 (half a step 2^-8 of their size, of random
    # sign): six roundings one behind the other, and the loss feels those of h through logits of norm |h| |W| <= 8 x 2.4
    assert float((loss - want).abs().max()) <= 3 * 2.0 ** -8 * 20 * float(args[4].max())
    assert float((aux - waux).abs().max()) <= 1e-5 * float(waux.abs().max())
    for k, g in grads.items():
        rel = float((g.double() - ref[k]).norm() / ref[k].norm())
        assert rel <= 6 * 2.0 ** -8, (k, rel)
    assert grads["x"][~args[3]].abs().max() == 0  # padding


def test_clipped_into_the_step():
    numel = [D * E, E * D * D, V * D]
    flats = [torch.empty(sum(numel), dtype=BF, device="cuda") for _ in range(2)]
    workers = []
    for w in range(2):
        g = step(*model(w + 2))[2]
        workers.append([g["router"], g["w"], g["head"]])  # fp32, fp32, bf16
    norms = sc.clip_grads(workers, 0.05, out=[f.split(numel) for f in flats])
    for n, ts, f in zip(norms.tolist(), workers, flats):
        flat = torch.cat([t.double().reshape(-1) for t in ts])
        assert abs(n - float(flat.norm())) <= 1e-6 * n and n > 0.05
        want = flat * (0.05 / float(flat.norm()))
        assert ((f.double() - want).abs() <= (2.0 ** -8 + 1e-6) * want.abs() + 1e-38).all()
    theta = torch.randn(sum(numel), device="cuda")
    a, b = (sc.Scape(numel, chunk=4096, W=2, density=0.1) for _ in range(2))
    for s in (a, b):
        s.load(sc.THETA, theta)
    a.step(flats)
    b.step([f.clone() for f in flats])
    got = a.read(sc.THETA)
    assert np.array_equal(got, b.read(sc.THETA)) and np.isfinite(got).all()
    assert not np.array_equal(got, theta.cpu().numpy())


def test_the_whole_step_in_a_graph():
    args = model(9)
    loss, aux, grads, _ = step(*args)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(*args)  # (cuBLAS takes its workspace)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = step(*args)
        norm = sc.grad_norm([held[2][k] for k in ("router", "w", "head")])
    p, x, y, valid, weight = args
    other = model(10)
    x.copy_(other[1])
    y.copy_(other[2])
    want = step(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held[0], want[0]) and torch.equal(held[2]["head"], want[2]["head"])
    total = sum(float(want[2][k].double().square().sum()) for k in ("router", "w", "head")) ** 0.5
    assert abs(float(norm) - total) <= 1e-5 * total
