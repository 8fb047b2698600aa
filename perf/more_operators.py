"""The operators between a model's backbone and the optimizer step, as measured cases.

ce        softmax cross entropy of hidden states through an output matrix, without the logits in memory:
          the loss of every row ("loss"), or that with the gradients of both ("grad").
experts   the tokens of a mixture of experts sorted by expert ("dispatch": the plan and the rows), the experts'
          rows summed back with their weights ("combine"), its backward pass ("backward"), and the way there and
          back in one ("around").
grads     the norm of each worker's gradients over many tensors ("norm"), and the gradients scaled down to a
          largest norm and written into the flat buffers that the optimizer step takes ("clip").

The module computes each of them either in plain torch operations (``own = False``) or through the
package's entry points (``own = True``), on the same state.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_MAX_CE = 16384 * 2048 * 32000      # rows x dim x vocab of the largest listed loss
_MAX_ROWS = 16384 * 8 * 2048 * 2    # bytes of the experts' rows
_MAX_GRADS = 1_800_000_000 * 2      # bytes of all gradients
_NO_LABEL = 0.05                    # share of the rows without a label


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # a few answers scored: latency of one reading of the output matrix (the Llama-style 1.8B layout's)
        dict(name="ce_loss_few_rows", op="ce", rows=16, dim=2048, vocab=32000, pad=0, dtype="bf16", masked=0.0, grad=False),
        # evaluation over GPT-2's odd vocabulary, part of the rows being padding; hidden rows of a wider buffer
        dict(name="ce_loss_gpt2", op="ce", rows=4096, dim=1024, vocab=50257, pad=64, dtype="bf16", masked=0.1, grad=False),
        # fine-tuning of the 500M layout in fp16: a third of the rows are prompts, which have no loss
        dict(name="ce_grad_500m_prompts", op="ce", rows=4096, dim=1280, vocab=32000, pad=0, dtype="f16", masked=0.3, grad=True),
        # the largest: pre-training of the 1.8B layout, eight sequences of 2048
        dict(name="ce_grad_1.8b", op="ce", rows=16384, dim=2048, vocab=32000, pad=0, dtype="bf16", masked=0.0, grad=True),
        # one token through its experts and back (generation)
        dict(name="experts_one_token", op="experts", what="around", tokens=1, dim=2048, experts=8, k=2, align=1, skew=0.7,
             masked=0.0, dtype="bf16"),
        # a ragged training batch, segments at multiples of a tile, some tokens padding
        dict(name="dispatch_tiles", op="experts", what="dispatch", tokens=16384, dim=2048, experts=64, k=6, align=128, skew=0.7,
             masked=0.05, dtype="bf16"),
        # many experts
        dict(name="combine_many_experts", op="experts", what="combine", tokens=16384, dim=2048, experts=256, k=8, align=1, skew=0.7,
             masked=0.0, dtype="bf16"),
        # the backward pass at training size, an odd number of tokens
        dict(name="combine_backward", op="experts", what="backward", tokens=16381, dim=1280, experts=128, k=8, align=1, skew=0.7,
             masked=0.05, dtype="bf16"),
        # the smallest gradient that the step takes: one flat tensor a worker
        dict(name="norm_flat_2^20_w4", op="grads", what="norm", layout="flat", n=1 << 20, workers=4, dtype="bf16", out="bf16"),
        # norms alone, for the log: every tensor of the 1.8B layout
        dict(name="norm_1.8b", op="grads", what="norm", layout="llama-1.8b", n=0, workers=1, dtype="bf16", out="bf16"),
        # autograd's 32-bit gradients of GPT-2-medium, clipped into the bf16 buffers of two workers
        dict(name="clip_gpt2_w2", op="grads", what="clip", layout="gpt2-medium", n=0, workers=2, dtype="f32", out="bf16"),
        # bf16 gradients of the 500M layout, clipped
        dict(name="clip_500m", op="grads", what="clip", layout="llama-500m", n=0, workers=1, dtype="bf16", out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "experts", "experts", "grads"])
    if op == "ce":
        dim = rng.choice([1024, 1280, 2048, 8 * _log_int(rng, 4, 512)])
        vocab = rng.choice([32000, 50257, _log_int(rng, 1000, 131072)])
        grad = rng.random() < 0.6
        rows = _log_int(rng, 1, min(16384, _MAX_CE // (dim * vocab)))
        return dict(op=op, rows=rows, dim=dim, vocab=vocab, pad=rng.choice([0, 0, 8 * rng.randint(1, 32)]),
                    dtype=rng.choice(["bf16", "bf16", "f16"]), masked=rng.choice([0.0, 0.1, 0.5]), grad=grad)
    if op == "experts":
        dim = rng.choice([1024, 1280, 2048, _log_int(rng, 16, 4096)])
        experts = rng.choice([8, 64, 128, 256, _log_int(rng, 2, 300)])
        k = rng.randint(1, min(8, experts))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        tokens = _log_int(rng, 1, min(131072, _MAX_ROWS // (k * dim * _SIZE[dtype])))
        return dict(op=op, what=rng.choice(["dispatch", "combine", "backward", "around"]), tokens=tokens, dim=dim,
                    experts=experts, k=k, align=rng.choice([1, 1, 16, 128]), skew=round(rng.uniform(0.0, 1.5), 2),
                    masked=rng.choice([0.0, 0.05, 0.3]), dtype=dtype)
    dtype, out = rng.choice(["bf16", "f16", "f32"]), rng.choice(["bf16", "bf16", "f32"])
    layout, workers = rng.choice(["flat", "flat", "ragged", "gpt2-medium"]), rng.randint(1, 4)
    if layout == "gpt2-medium":
        workers = 1
    n = 0 if layout == "gpt2-medium" else _log_int(rng, 1000, _MAX_GRADS // (workers * (_SIZE[dtype] + _SIZE[out])) // 4)
    return dict(op=op, what=rng.choice(["norm", "clip"]), layout=layout, n=n, workers=workers, dtype=dtype, out=out)


def _llama(d, ff, layers, vocab):
    block = [d, d * d, d * d, d * d, d * d, d, ff * d, ff * d, d * ff]
    return [vocab * d] + block * layers + [d, vocab * d]


def _gpt2_medium():
    d, ff = 1024, 4096
    block = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, ff * d, ff, d * ff, d]
    return [50257 * d, 1024 * d] + block * 24 + [d, d]


def _numel(case):
    """Elements of every tensor of one worker."""
    if case["layout"] == "flat":
        return [case["n"]]
    if case["layout"] == "ragged":  # odd sizes, one of them most of it, some next to nothing
        n = case["n"]
        parts = [n // 2 + 1, 1, n // 7, 7, n // 11, 33, n // 13]
        return parts + [n - sum(parts)] if sum(parts) < n else [n]
    return {"llama-1.8b": lambda: _llama(2048, 5632, 32, 32000), "llama-500m": lambda: _llama(1280, 3456, 24, 32000),
            "gpt2-medium": _gpt2_medium}[case["layout"]]()


# ---- inputs -----------------------------------------------------------------------------------------


def _prepare_ce(case, gen):
    T, D, V, dt = case["rows"], case["dim"], case["vocab"], _DT[case["dtype"]]

    def rand(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    # an output matrix whose words have a Zipf-like frequency along one direction, and hidden states near a likely word's row
    W = rand(V, D).mul_(0.02)
    u = torch.nn.functional.normalize(rand(D), dim=0)
    bias = -torch.log1p(torch.arange(V, device="cuda", dtype=torch.float32))[torch.randperm(V, generator=gen, device="cuda")]
    W += (bias / 8.0)[:, None] * u
    likely = torch.randint(V, (T,), generator=gen, device="cuda")
    H = rand(T, D)
    H += 8.0 * u
    near = W[likely]
    H += near * (torch.rand(T, 1, generator=gen, device="cuda") * 12 / near.square().sum(1, keepdim=True))
    wide = torch.zeros(T, D + case["pad"], dtype=dt, device="cuda")
    wide[:, :D] = H.to(dt)
    s = dict(case=case, hidden=wide[:, :D], weight=W.to(dt), row_weight=None)
    other = torch.randint(V, (T,), generator=gen, device="cuda")
    s["labels"] = torch.where(torch.rand(T, generator=gen, device="cuda") < 0.7, likely, other)
    s["labels"][torch.rand(T, generator=gen, device="cuda") < _NO_LABEL] = -100
    if case["masked"]:
        w = (torch.rand(T, generator=gen, device="cuda") >= case["masked"]).float()
        # the mean over the live rows; fp16 training scales its loss, so that small gradients stay normal numbers
        s["row_weight"] = w * ((4096.0 if case["dtype"] == "f16" else 1.0) / w.sum().clamp(min=1.0))
    return s


def _prepare_experts(case, gen):
    T, D, E, k, dt = case["tokens"], case["dim"], case["experts"], case["k"], _DT[case["dtype"]]
    # a router's choices: k different experts a token, some experts liked more; padding goes to none
    x = torch.randn(T, E, generator=gen, device="cuda") + case["skew"] * torch.randn(E, generator=gen, device="cuda")
    top = torch.topk(x, k, dim=1)
    idx = top.indices.to(torch.int32)
    weights = torch.softmax(top.values, 1)
    if case["masked"]:
        dead = torch.rand(T, 1, generator=gen, device="cuda") < case["masked"]
        idx, weights = idx.masked_fill(dead, -1), weights.masked_fill(dead, 0.0)
    s = dict(case=case, idx=idx, weights=weights)
    if case["what"] in ("dispatch", "around"):
        s["x"] = torch.randn(T, D, generator=gen, device="cuda").to(dt)
        return s
    s["offsets"], s["slots"], s["source"] = _plain_plan(idx, E, case["align"])
    s["y"] = torch.randn(s["source"].numel(), D, generator=gen, device="cuda").to(dt)
    if case["what"] == "backward":
        s["d_out"] = (torch.randn(T, D, generator=gen, device="cuda") / 8).to(dt)
    return s


def _prepare_grads(case, gen):
    numel = _numel(case)
    n = sum(numel)
    dt, grads, outs, flats = _DT[case["dtype"]], [], [], []
    for _ in range(case["workers"]):
        # tensors of different scale; the worker's norm lies between a half and four
        norm = 0.5 * 8.0 ** float(torch.rand(1, generator=gen, device="cuda"))
        grads.append([(torch.randn(m, generator=gen, device="cuda") * (norm * (0.5 + (i % 5) / 5) / math.sqrt(n))).to(dt)
                      for i, m in enumerate(numel)])
        if case["what"] == "clip":
            flats.append(torch.empty(n, dtype=_DT[case["out"]], device="cuda"))
            outs.append(list(flats[-1].split(numel)))
    return dict(case=case, grads=grads, outs=outs, flats=flats, max_norm=1.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"ce": _prepare_ce, "experts": _prepare_experts, "grads": _prepare_grads}[case["op"]](case, gen)


# ---- plain forms ------------------------------------------------------------------------------------


def _plain_ce(s, with_grad):
    H, W, y = s["hidden"].float(), s["weight"].float(), s["labels"]
    w = torch.ones(H.shape[0], device=H.device) if s["row_weight"] is None else s["row_weight"]
    on = ((y >= 0) & (w != 0))[:, None]
    x = H @ W.T
    m = x.amax(1, keepdim=True)
    x -= m
    at = y.clamp(min=0)[:, None]
    chosen = torch.gather(x, 1, at)
    x.exp_()
    total = x.sum(1, keepdim=True)
    loss = torch.where(on, w[:, None] * (torch.log(total) - chosen), 0.0).squeeze(1)
    if not with_grad:
        return [loss]
    x /= total
    x.scatter_add_(1, at, torch.full_like(chosen, -1.0))
    x *= w[:, None]
    x *= on
    return [loss, (x @ W).to(s["hidden"].dtype), (x.T @ H).to(s["weight"].dtype)]


def _plain_plan(idx, experts, align):
    T, k = idx.shape
    N = T * k
    dev = idx.device
    e = torch.where(idx >= 0, idx, experts).reshape(-1).to(torch.int64)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=dev).scatter_add_(0, e, torch.ones_like(e))
    room = (counts[:-1] + align - 1) // align * align
    offsets = torch.cat([room.new_zeros(1), room.cumsum(0)])
    order = torch.sort(e, stable=True).indices              # choices by expert, those of no expert last
    first = torch.cat([counts.new_zeros(1), counts.cumsum(0)])[:-1]
    sorted_e = e[order]
    rank = torch.arange(N, device=dev) - first[sorted_e]
    slot = torch.where(sorted_e < experts, offsets[sorted_e] + rank, -1)
    slots = torch.empty_like(e).scatter_(0, order, slot).view(T, k)
    capacity = N + min(experts, N) * (align - 1)
    source = torch.full((capacity + 1,), -1, dtype=torch.int64, device=dev)
    source[torch.where(slot >= 0, slot, capacity)] = torch.where(slot >= 0, order, -1)
    return offsets.to(torch.int32), slots.to(torch.int32), source[:capacity].to(torch.int32)


def _plain_dispatch(x, source, k):
    rows = x[source.clamp(min=0).long() // k]
    return torch.where(source[:, None] >= 0, rows, torch.zeros_like(rows[:1]))


def _plain_combine(y, slots, weights):
    rows = y[slots.clamp(min=0).long()].float()
    return torch.where(slots[:, :, None] >= 0, rows * weights[:, :, None], 0.0).sum(1).to(y.dtype)


def _plain_combine_backward(d_out, y, slots, source, weights):
    k = slots.shape[1]
    at = source.clamp(min=0).long()
    d_rows = d_out.float()[at // k] * weights.reshape(-1)[at][:, None]
    d_y = torch.where(source[:, None] >= 0, d_rows, 0.0).to(y.dtype)
    dot = (y[slots.clamp(min=0).long()].float() * d_out.float()[:, None]).sum(2)
    return d_y, torch.where(slots >= 0, dot, 0.0)


def _plain_norm(grads):
    # long sums: in 64 bits
    return torch.stack([torch.stack([g.float().square().sum(dtype=torch.float64) for g in worker]).sum().sqrt()
                        for worker in grads])


def _plain_clip(s):
    norms = _plain_norm(s["grads"])
    scale = torch.where(norms > s["max_norm"], s["max_norm"] / norms, 1.0)
    [o.copy_(g.float() * c) for worker, outs, c in zip(s["grads"], s["outs"], scale.float()) for g, o in zip(worker, outs)]
    return norms.float()


# ---- one pass ---------------------------------------------------------------------------------------


def _own_ce(s, with_grad):
    import sparse_communication_distributed_gb300 as scape
    if with_grad:
        return list(scape.linear_ce_grad(s["hidden"], s["weight"], s["labels"], row_weight=s["row_weight"]))
    return [scape.linear_ce(s["hidden"], s["weight"], s["labels"], row_weight=s["row_weight"])]


def _own_experts(s, case):
    import sparse_communication_distributed_gb300 as scape
    if case["what"] == "combine":
        return [scape.expert_combine(s["y"], s["slots"], s["weights"])]
    if case["what"] == "backward":
        return list(scape.expert_combine_backward(s["d_out"], s["y"], s["slots"], s["source"], s["weights"]))
    offsets, slots, source = scape.expert_plan(s["idx"], case["experts"], align=case["align"])
    rows = scape.expert_dispatch(s["x"], slots, source)
    if case["what"] == "dispatch":
        return [offsets, slots, source, rows]
    return [offsets, slots, source, rows, scape.expert_combine(rows, slots, s["weights"])]


def _own_grads(s, case):
    import sparse_communication_distributed_gb300 as scape
    if case["what"] == "norm":
        return [scape.grad_norm(s["grads"])]
    return [scape.clip_grads(s["grads"], s["max_norm"], out=s["outs"])] + s["flats"]


def run(state):
    s, case = state, state["case"]
    if case["op"] == "ce":
        return _own_ce(s, case["grad"]) if own else _plain_ce(s, case["grad"])
    if case["op"] == "grads":
        if own:
            return _own_grads(s, case)
        if case["what"] == "norm":
            return [_plain_norm(s["grads"]).float()]
        return [_plain_clip(s)] + s["flats"]
    if own:
        return _own_experts(s, case)
    if case["what"] == "combine":
        return [_plain_combine(s["y"], s["slots"], s["weights"])]
    if case["what"] == "backward":
        return list(_plain_combine_backward(s["d_out"], s["y"], s["slots"], s["source"], s["weights"]))
    offsets, slots, source = _plain_plan(s["idx"], case["experts"], case["align"])
    rows = _plain_dispatch(s["x"], source, case["k"])
    if case["what"] == "dispatch":
        return [offsets, slots, source, rows]
    return [offsets, slots, source, rows, _plain_combine(rows, slots, s["weights"])]


def work(case):
    if case["op"] == "ce":
        T, D, V, es = case["rows"], case["dim"], case["vocab"], _SIZE[case["dtype"]]
        live = T * (1 - case["masked"]) * (1 - _NO_LABEL)  # rows with a term
        n = live * D * es + V * D * es + T * (8 + 4 + 4 * bool(case["masked"]))
        if case["grad"]:
            return {"bytes": n + T * D * es + V * D * es, "flops": 6 * live * D * V}
        return {"bytes": n, "flops": 2 * live * D * V}
    if case["op"] == "grads":
        n = sum(_numel(case)) * case["workers"]
        if case["what"] == "norm":
            return {"bytes": n * _SIZE[case["dtype"]], "flops": 2 * n}
        return {"bytes": n * (_SIZE[case["dtype"]] + _SIZE[case["out"]]), "flops": 3 * n}
    T, D, E, k, es = case["tokens"], case["dim"], case["experts"], case["k"], _SIZE[case["dtype"]]
    live = T * (1 - case["masked"])
    capacity = T * k + min(E, T * k) * (case["align"] - 1)
    plan = T * k * 8 + capacity * 4 + (E + 1) * 4
    there = live * D * es + capacity * D * es
    back = live * k * D * es + T * k * 8 + T * D * es
    if case["what"] == "dispatch":
        return {"bytes": plan + there, "flops": 0}
    if case["what"] == "around":
        return {"bytes": plan + there + T * k * 4 + T * D * es, "flops": 2 * live * k * D}
    if case["what"] == "combine":
        return {"bytes": back, "flops": 2 * live * k * D}
    return {"bytes": live * D * es + live * k * D * es + capacity * D * es + capacity * 4 + T * k * 12, "flops": 3 * live * k * D}


# ---- 64 bits ----------------------------------------------------------------------------------------


def _exact_ce(case, s):
    T, D, V = case["rows"], case["dim"], case["vocab"]
    if T * D * V * (6 if case["grad"] else 2) > 1.2e13:
        return None
    W = s["weight"].double().requires_grad_(case["grad"])
    w = torch.ones(T, dtype=torch.float64, device="cuda") if s["row_weight"] is None else s["row_weight"].double()
    step = max(1, (1 << 26) // V)
    losses, d_hidden, d_weight = [], [], torch.zeros_like(W.detach()) if case["grad"] else None
    for r in range(0, T, step):
        h = s["hidden"][r:r + step].double().requires_grad_(case["grad"])
        row = torch.nn.functional.cross_entropy(h @ W.T, s["labels"][r:r + step], reduction="none", ignore_index=-100)
        row = row * w[r:r + step]
        losses.append(row.detach())
        if case["grad"]:
            dh, dw = torch.autograd.grad(row.sum(), (h, W))
            d_hidden.append(dh)
            d_weight += dw
    return [torch.cat(losses)] + ([torch.cat(d_hidden), d_weight] if case["grad"] else [])


def _exact_experts(case, s):
    T, k, D = case["tokens"], case["k"], case["dim"]
    what, w = case["what"], s["weights"].double()
    flat = s["idx"].reshape(-1)
    if what in ("dispatch", "around"):
        # expert by expert: its choices in ascending order, each segment filled up to a multiple
        x = s["x"].double()
        capacity = T * k + min(case["experts"], T * k) * (case["align"] - 1)
        rows = torch.zeros(capacity, D, dtype=torch.float64, device="cuda")
        out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
        at = 0
        for e in range(case["experts"]):
            mine = torch.nonzero(flat == e).squeeze(1)
            rows[at:at + mine.numel()] = x[mine // k]
            out.index_add_(0, mine // k, x[mine // k] * w.reshape(-1)[mine][:, None])
            at += -(-mine.numel() // case["align"]) * case["align"]
        return [None, None, None, rows] + ([out] if what == "around" else [])
    out = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    d_y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["slots"][:, j] >= 0).squeeze(1)
        r = s["slots"][t, j].long()
        yr = s["y"][r].double()
        if what == "combine":
            out.index_add_(0, t, yr * w[t, j, None])
        else:
            d = s["d_out"][t].double()
            d_y[r] = d * w[t, j, None]
            dw[t, j] = torch.einsum("td,td->t", d, yr)
    return [out] if what == "combine" else [d_y, dw]


def _exact_grads(case, s):
    norms, outs = [], []
    for worker in s["grads"]:
        flat = torch.cat([g.reshape(-1) for g in worker])
        step = 1 << 27
        total = sum(float(torch.dot(p, p)) for p in (flat[i:i + step].double() for i in range(0, flat.numel(), step)))
        norm = math.sqrt(total)
        norms.append(norm)
        if case["what"] == "clip":
            outs.append(flat.double().mul_(min(1.0, s["max_norm"] / norm if norm > 0 else 1.0)))
    return [torch.tensor(norms, dtype=torch.float64, device="cuda")] + outs


def exact(case, seed):
    s = prepare(case, seed)
    return {"ce": _exact_ce, "experts": _exact_experts, "grads": _exact_grads}[case["op"]](case, s)
