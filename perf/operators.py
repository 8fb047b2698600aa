"""The operators of a training objective whose gradients the optimizer step consumes, as measured cases.

Three operators, five calls:

topk      the k largest logits of every row (ties to the lower index) and the row's log-sum-exp at a
          temperature: what a teacher leaves behind for distillation.
distill   the loss of a student against those top logits, mixed with the cross entropy of a hard label,
          for each row; alone ("loss") or with the gradient of the student's logits ("grad").
route     a mixture-of-experts router: top-k experts of every token, their weights, the tokens that every
          expert of every group got, the balance loss and the z loss; and its backward pass.

The module computes each of them either in plain torch operations (``own = False``) or through the
package's entry points (``own = True``), on the same state.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_MAX_BYTES = 8192 * 50257 * 2  # logits of the largest listed case


# ---- cases ------------------------------------------------------------------------------------------


def listed():
    return [
        # a teacher that answers one token at a time (cache being written while it generates); Llama vocabulary
        dict(name="topk_one_token", op="topk", rows=1, vocab=32000, pad=0, k=64, dtype="bf16", temperature=2.0),
        # a teacher's batch of two 2048-token sequences over the GPT-2 vocabulary, whose rows have an odd length
        dict(name="topk_gpt2_bf16", op="topk", rows=4096, vocab=50257, pad=0, k=64, dtype="bf16", temperature=2.0),
        # a wide vocabulary in 32 bits, deep cache
        dict(name="topk_wide_f32", op="topk", rows=1024, vocab=131072, pad=0, k=256, dtype="f32", temperature=1.0),
        # the smallest training call: a few rows, where latency is what counts
        dict(name="grad_few_rows", op="distill", rows=4, vocab=32000, pad=0, k=32, dtype="bf16", temperature=2.0,
             tail=False, ce=True, masked=0.0, grad=True),
        # evaluation: the loss alone, over GPT-2's vocabulary padded to a multiple of 128 (a strided view)
        dict(name="loss_gpt2_padded", op="distill", rows=4096, vocab=50257, pad=47, k=64, dtype="bf16", temperature=2.0,
             tail=True, ce=True, masked=0.1, grad=False),
        # pure distillation over the Llama vocabulary, ordinary training size
        dict(name="grad_llama", op="distill", rows=8192, vocab=32000, pad=0, k=64, dtype="bf16", temperature=2.0,
             tail=False, ce=False, masked=0.0, grad=True),
        # the largest: GPT-2's odd vocabulary, tail bucket, hard labels, masked rows
        dict(name="grad_gpt2_tail_ce", op="distill", rows=8192, vocab=50257, pad=0, k=128, dtype="bf16", temperature=2.0,
             tail=True, ce=True, masked=0.1, grad=True),
        # 32-bit logits over a wide vocabulary
        dict(name="grad_wide_f32", op="distill", rows=768, vocab=131072, pad=0, k=256, dtype="f32", temperature=1.0,
             tail=False, ce=True, masked=0.0, grad=True),
        # a router answering one token
        dict(name="route_one_token", op="route", tokens=1, experts=8, k=2, groups=0, masked=0.0, renorm=True,
             dtype="bf16", backward=False),
        # a training batch of ragged sequences with padding, one balance loss for each sequence
        dict(name="route_ragged", op="route", tokens=16384, experts=64, k=6, groups=16, masked=0.05, renorm=True,
             dtype="bf16", backward=False),
        # a large global batch through many experts, 32-bit logits
        dict(name="route_large_f32", op="route", tokens=131072, experts=256, k=8, groups=0, masked=0.0, renorm=False,
             dtype="f32", backward=False),
        # the router's backward pass at training size
        dict(name="route_backward", op="route", tokens=65536, experts=128, k=8, groups=32, masked=0.05, renorm=True,
             dtype="bf16", backward=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "distill", "distill", "route"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "route":
        experts = rng.choice([8, 16, 64, 128, 256, _log_int(rng, 4, 300)])
        tokens = _log_int(rng, 1, 131072)
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(8, experts)),
                    groups=rng.choice([0, 0, _log_int(rng, 1, 64)]), masked=rng.choice([0.0, 0.05, 0.3]),
                    renorm=rng.random() < 0.5, dtype=dtype, backward=rng.random() < 0.5)
    vocab = rng.choice([32000, 50257, _log_int(rng, 1000, 200000)])
    pad = rng.choice([0, 0, rng.randint(1, 127)])
    top = min(16384, int(_MAX_BYTES * (0.4 if op == "topk" else 1.0)) // ((vocab + pad) * _SIZE[dtype]))
    case = dict(op=op, rows=_log_int(rng, 1, top), vocab=vocab, pad=pad, k=_log_int(rng, 1, 256), dtype=dtype,
                temperature=rng.choice([1.0, 2.0, round(rng.uniform(0.7, 5.0), 3)]))
    if op == "distill":
        case.update(tail=rng.random() < 0.5, ce=rng.random() < 0.5, masked=rng.choice([0.0, 0.1, 0.5]),
                    grad=rng.random() < 0.75)
    return case


# ---- inputs -----------------------------------------------------------------------------------------


def _logits(rows, vocab, pad, gen):
    """Logits as a language model gives them: a Zipf-like bias for each word, noise, one likely word a row."""
    x = torch.randn(rows, vocab + pad, generator=gen, device="cuda").mul_(2.0)
    bias = -torch.log1p(torch.arange(vocab + pad, device="cuda", dtype=torch.float32))
    x += bias[torch.randperm(vocab + pad, generator=gen, device="cuda")]
    likely = torch.randint(vocab, (rows, 1), generator=gen, device="cuda")
    x.scatter_add_(1, likely, torch.rand(rows, 1, generator=gen, device="cuda") * 12)
    return x, likely.squeeze(1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    if case["op"] == "topk":
        x, _ = _logits(case["rows"], case["vocab"], case["pad"], gen)
        return dict(case=case, logits=x.to(dt)[:, :case["vocab"]])
    if case["op"] == "distill":
        R, V = case["rows"], case["vocab"]
        x, likely = _logits(R, V, case["pad"], gen)
        z = x[:, :V] * 0.9
        z += torch.randn(R, V, generator=gen, device="cuda").mul_(0.7)
        s = dict(case=case, logits=x.to(dt)[:, :V])
        del x
        vals, idx = torch.topk(z, case["k"], dim=1)
        s["idx"], s["vals"] = idx.to(torch.int32), vals.to(dt)
        # teachers differ in how many words they keep: the last entries of some rows are empty (-1)
        keep = torch.randint(case["k"] // 2, case["k"] + 1, (R, 1), generator=gen, device="cuda")
        keep = torch.where(torch.rand(R, 1, generator=gen, device="cuda") < 0.75, case["k"], keep)
        s["idx"].masked_fill_(torch.arange(case["k"], device="cuda") >= keep, -1)
        s["teacher_lse"] = torch.logsumexp(z / case["temperature"], 1) if case["tail"] else None
        s["labels"] = None
        if case["ce"]:
            other = torch.randint(V, (R,), generator=gen, device="cuda")
            right = torch.rand(R, generator=gen, device="cuda") < 0.7
            s["labels"] = torch.where(right, likely, other)
            s["labels"][torch.rand(R, generator=gen, device="cuda") < 0.05] = -100
        s["row_weight"] = None
        if case["masked"]:
            w = (torch.rand(R, generator=gen, device="cuda") >= case["masked"]).float()
            s["row_weight"] = w / w.sum().clamp(min=1.0)
        return s
    T, E, G, k = case["tokens"], case["experts"], case["groups"], case["k"]
    x = torch.randn(T, E, generator=gen, device="cuda") + 0.7 * torch.randn(E, generator=gen, device="cuda")
    s = dict(case=case, logits=x.to(dt), cu_tokens=None, valid=None)
    if G:
        cuts = torch.randint(T + 1, (G - 1,), generator=gen, device="cuda").sort().values
        s["cu_tokens"] = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), T)]).to(torch.int32)
    if case["masked"]:
        s["valid"] = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
    if case["backward"]:
        s["idx"], _, s["counts"], s["tokens"], _ = _plain_route(s, k, case["renorm"])
        s["d_weights"] = torch.randn(T, k, generator=gen, device="cuda") / T
        s["d_losses"] = torch.tensor([0.01, 0.001], device="cuda") * (0.5 + torch.rand(2, generator=gen, device="cuda"))
    return s


# ---- plain forms ------------------------------------------------------------------------------------


def _lse(x):
    m = x.amax(1, keepdim=True)
    return torch.log(torch.exp(x - m).sum(1)) + m.squeeze(1)


def _ordered(x):
    """Whole numbers in the order of the 32-bit floats x (+0 and -0 alike), each row's lower index first among equals."""
    b = (x + 0.0).view(torch.int32).to(torch.int64)
    b = torch.where(b < 0, -1 - (b & 0x7FFFFFFF), b)
    return (b << 32) - torch.arange(x.shape[1], device=x.device)


def _plain_topk(s, k, temperature):
    x = s["logits"].float()
    idx = torch.topk(_ordered(x), k, dim=1).indices
    return idx.to(torch.int32), torch.gather(s["logits"], 1, idx), _lse(x / temperature)


def _plain_distill(s, tau, kd_weight, ce_weight, with_grad):
    x = s["logits"].float()
    idx, valid = s["idx"].clamp(min=0).long(), s["idx"] >= 0
    t = torch.where(valid, s["vals"].float() / tau, -math.inf)
    has = (t > -math.inf).any(1, keepdim=True)
    sx = x / tau
    L = _lse(sx)[:, None]
    log_p = torch.gather(sx, 1, idx) - L
    if s["teacher_lse"] is not None:
        log_q = t - s["teacher_lse"][:, None]
        log_q = torch.where(has, log_q, -math.inf)
    else:
        m = torch.where(has, t.amax(1, keepdim=True), 0.0)
        log_q = t - torch.log(torch.exp(t - m).sum(1, keepdim=True)) - m
        log_q = torch.where(has, log_q, -math.inf)
    q = torch.exp(log_q)
    kl = torch.where(q > 0, q * (log_q - log_p), 0.0).sum(1)
    total = q.sum(1, keepdim=True)
    q_tail = torch.zeros_like(total)
    if s["teacher_lse"] is not None:
        # everything outside the listed words as one bucket
        out = torch.where(valid, idx, torch.full_like(idx, x.shape[1]))
        inside = torch.zeros(x.shape[0], x.shape[1] + 1, dtype=torch.bool, device=x.device).scatter_(1, out, True)[:, :-1]
        rest = torch.where(inside, -math.inf, sx)
        m = rest.amax(1, keepdim=True)
        m = torch.where(m > -math.inf, m, 0.0)
        L_rest = torch.log(torch.exp(rest - m).sum(1, keepdim=True)) + m
        q_tail = torch.where(has & (L_rest > -math.inf), (1.0 - total).clamp(min=0.0), 0.0)
        kl = kl + torch.where(q_tail > 0, q_tail * (torch.log(q_tail) - (L_rest - L)), 0.0).squeeze(1)
    loss = kd_weight * tau * tau * kl
    if s["labels"] is not None:
        hard = s["labels"] >= 0
        y = s["labels"].clamp(min=0)[:, None]
        L1 = _lse(x)[:, None]
        ce = (L1 - torch.gather(x, 1, y)).squeeze(1)
        loss = loss + torch.where(hard, ce_weight * ce, 0.0)
    w = s["row_weight"]
    if w is not None:
        loss = torch.where(w != 0, w * loss, 0.0)
    if not with_grad:
        return [loss]
    g = torch.exp(sx - L) * (total + q_tail)
    if s["teacher_lse"] is not None:
        g = g - torch.where(inside | (q_tail == 0), 0.0, q_tail * torch.exp(sx - L_rest))
    g.scatter_add_(1, idx, -q)
    g = g * (kd_weight * tau)
    if s["labels"] is not None:
        h = torch.exp(x - L1)
        h.scatter_add_(1, y, -torch.ones_like(L1))
        g = g + torch.where(hard[:, None], ce_weight * h, 0.0)
    if w is not None:
        g = torch.where(w[:, None] != 0, w[:, None] * g, 0.0)
    return [loss, g.to(s["logits"].dtype)]


def _group_of(s, T, device):
    if s["cu_tokens"] is None:
        return torch.zeros(T, dtype=torch.int64, device=device), 1
    ends = s["cu_tokens"][1:]
    return torch.searchsorted(ends, torch.arange(T, dtype=torch.int32, device=device), right=True), ends.numel()


def _plain_route(s, k, renorm):
    x = s["logits"].float()
    T, E = x.shape
    group, G = _group_of(s, T, x.device)
    live = x.amax(1) > -math.inf
    if s["valid"] is not None:
        live = live & s["valid"]
    idx = torch.topk(_ordered(x), k, dim=1).indices
    lse = _lse(x)
    p = torch.where(live[:, None], torch.exp(x - lse[:, None]), 0.0)
    chosen = torch.gather(x, 1, idx)
    base = _lse(chosen) if renorm else lse
    weights = torch.where(live[:, None], torch.exp(chosen - base[:, None]), 0.0)
    one = live[:, None].expand(T, k).to(torch.int32).reshape(-1)
    counts = torch.zeros(G * E, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, (group[:, None] * E + idx).reshape(-1), one)
    counts = counts.view(G, E)
    per_group = torch.zeros(G, dtype=torch.int32, device=x.device).scatter_add_(0, group, live.to(torch.int32))
    n_valid, n_groups = per_group.sum(), (per_group > 0).sum()
    tokens = torch.cat([per_group, n_valid[None], n_groups[None]]).to(torch.int32)
    sums = torch.zeros(G, E, device=x.device).index_add_(0, group, p)
    tg = per_group.float().clamp(min=1.0)
    balance = ((counts.float() * sums).sum(1) * E / (k * tg * tg)).sum() / n_groups.clamp(min=1)
    z = torch.where(live, lse * lse, 0.0).sum() / n_valid.clamp(min=1)
    idx = torch.where(live[:, None], idx, -1).to(torch.int32)
    return idx, weights, counts, tokens, torch.stack([balance, z])


def _plain_route_backward(s, renorm):
    x = s["logits"].float()
    T, E = x.shape
    k = s["idx"].shape[1]
    group, G = _group_of(s, T, x.device)
    live = s["idx"][:, :1] >= 0
    idx = s["idx"].clamp(min=0).long()
    lse = _lse(x)[:, None]
    p = torch.exp(x - lse)
    tg = s["tokens"][:G].float().clamp(min=1.0)
    n_valid, n_groups = s["tokens"][G].clamp(min=1), s["tokens"][G + 1].clamp(min=1)
    a = (s["d_losses"][0] / n_groups) * E / (k * tg * tg)
    d = (a[:, None] * s["counts"].float())[group]
    g = p * (d - (p * d).sum(1, keepdim=True)) + (2 * s["d_losses"][1] / n_valid) * lse * p
    chosen = torch.gather(x, 1, idx)
    if renorm:
        w = torch.exp(chosen - _lse(chosen)[:, None])
    else:
        w = torch.exp(chosen - lse)
    dot = (w * s["d_weights"]).sum(1, keepdim=True)
    if renorm:
        g.scatter_add_(1, idx, w * (s["d_weights"] - dot))
    else:
        g = g - p * dot
        g.scatter_add_(1, idx, w * s["d_weights"])
    return torch.where(live, g, 0.0).to(s["logits"].dtype)


# ---- one pass ---------------------------------------------------------------------------------------


def _weights_of(case):
    """(kd_weight, ce_weight) of a distillation case."""
    return (0.7, 0.3) if case["ce"] else (1.0, 0.0)


def run(state):
    s, case = state, state["case"]
    if case["op"] == "topk":
        if own:
            import sparse_communication_distributed_gb300 as scape
            return list(scape.topk_logits(s["logits"], case["k"], temperature=case["temperature"]))
        return list(_plain_topk(s, case["k"], case["temperature"]))
    if case["op"] == "distill":
        kd, ce = _weights_of(case)
        if own:
            import sparse_communication_distributed_gb300 as scape
            args = dict(teacher_lse=s["teacher_lse"], labels=s["labels"], row_weight=s["row_weight"],
                        temperature=case["temperature"], kd_weight=kd, ce_weight=ce)
            if case["grad"]:
                return list(scape.distill_loss_grad(s["logits"], s["idx"], s["vals"], **args))
            return [scape.distill_loss(s["logits"], s["idx"], s["vals"], **args)]
        return _plain_distill(s, case["temperature"], kd, ce, case["grad"])
    if own:
        import sparse_communication_distributed_gb300 as scape
        if case["backward"]:
            return [scape.route_backward(s["logits"], s["idx"], s["counts"], s["tokens"], d_weights=s["d_weights"],
                                         d_losses=s["d_losses"], renormalize=case["renorm"], cu_tokens=s["cu_tokens"])]
        return list(scape.route(s["logits"], case["k"], renormalize=case["renorm"], cu_tokens=s["cu_tokens"],
                                valid=s["valid"]))
    if case["backward"]:
        return [_plain_route_backward(s, case["renorm"])]
    return list(_plain_route(s, case["k"], case["renorm"]))


def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        G = max(1, case["groups"])
        small = G * E * 4 + (G + 2) * 4 + 8 + (G + 1) * 4 * bool(case["groups"])
        if case["backward"]:
            return {"bytes": 2 * T * E * es + T * k * 8 + small, "flops": 10 * T * E}
        return {"bytes": T * E * es + T * k * 8 + T * bool(case["masked"]) + small, "flops": 6 * T * E}
    R, V, k = case["rows"], case["vocab"], case["k"]
    if case["op"] == "topk":
        return {"bytes": R * V * es + R * k * (4 + es) + R * 4, "flops": 4 * R * V}
    side = R * k * (4 + es) + R * 4 + R * 4 * case["tail"] + R * 8 * case["ce"] + R * 4 * bool(case["masked"])
    exps = 1 + case["ce"]
    return {"bytes": R * V * es * (2 if case["grad"] else 1) + side,
            "flops": R * V * (3 * exps + (3 * exps if case["grad"] else 0))}


# ---- 64 bits ----------------------------------------------------------------------------------------


def _exact_distill_rows(x, idx, vals, tlse, labels, w, tau, kd, ce, with_grad):
    """Loss of some rows and its gradient by differentiation, in 64 bits."""
    x = x.double().requires_grad_(with_grad)
    R, V = x.shape
    logp = torch.log_softmax(x / tau, 1)
    listed_ = torch.nn.functional.pad(torch.zeros(R, V, dtype=torch.bool, device=x.device), (0, 1))
    listed_.scatter_(1, torch.where(idx < 0, V, idx).long(), True)
    t = (vals.double() / tau).masked_fill(idx < 0, -math.inf)
    empty = torch.isinf(t).all(1)
    ref = t.logsumexp(1) if tlse is None else tlse.double()
    q = (t - ref[:, None]).exp().masked_fill(empty[:, None], 0.0)
    lp = torch.gather(logp, 1, idx.clamp(min=0).long())
    loss = (torch.special.xlogy(q, q) - torch.where(q > 0, q * lp, 0.0)).sum(1)
    if tlse is not None:
        outside = logp.masked_fill(listed_[:, :V], -math.inf).logsumexp(1)
        qt = torch.where(empty, 0.0, (1 - q.sum(1)).clamp(min=0))
        loss = loss + torch.special.xlogy(qt, qt) - qt * outside
    loss = loss * kd * tau ** 2
    if labels is not None:
        hard = torch.nn.functional.cross_entropy(x, labels, reduction="none", ignore_index=-100)
        loss = loss + ce * hard
    if w is not None:
        loss = loss * w.double()
    if not with_grad:
        return loss, None
    return loss.detach(), torch.autograd.grad(loss.sum(), x)[0]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "topk":
        R, V, k = case["rows"], case["vocab"], case["k"]
        step = max(1, (1 << 26) // V)
        vals, lse = [], []
        for r in range(0, R, step):
            x = s["logits"][r:r + step].double()
            vals.append(x.sort(dim=1, descending=True).values[:, :k])
            lse.append(torch.logsumexp(x / case["temperature"], 1))
        return [None, torch.cat(vals), torch.cat(lse)]
    if case["op"] == "distill":
        R, V = case["rows"], case["vocab"]
        kd, ce = _weights_of(case)
        step = max(1, (1 << 26) // V)
        losses, grads = [], []
        part = lambda v, r: None if v is None else v[r:r + step]  # noqa: E731
        for r in range(0, R, step):
            l, g = _exact_distill_rows(*(part(s[n], r) for n in ("logits", "idx", "vals", "teacher_lse", "labels",
                                                                 "row_weight")), case["temperature"], kd, ce, case["grad"])
            losses.append(l)
            if g is not None:
                grads.append(g)
        return [torch.cat(losses)] + ([torch.cat(grads)] if grads else [])
    x = s["logits"].double()
    T, E = x.shape
    k, G = case["k"], max(1, case["groups"])
    cu = [0, T] if s["cu_tokens"] is None else s["cu_tokens"].tolist()
    live = torch.ones(T, dtype=torch.bool, device=x.device) if s["valid"] is None else s["valid"]
    x.requires_grad_(True)
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    sel = x.detach().sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.softmax(torch.gather(x, 1, sel), 1) if case["renorm"] else torch.gather(p, 1, sel)
    w = w * live[:, None]
    balance, used = 0.0, 0
    for g in range(G):
        at = slice(cu[g], cu[g + 1])
        n = int(live[at].sum())
        if n:
            f = torch.bincount(sel[at][live[at]].reshape(-1), minlength=E).double() * E / (k * n)
            balance = balance + (f * p[at][live[at]].mean(0)).sum()
            used += 1
    balance = balance / max(1, used) + 0.0 * x.sum()
    z = (lse * lse * live).sum() / max(1, int(live.sum()))
    if not case["backward"]:
        return [None, w.detach(), None, None, torch.stack([balance, z]).detach()]
    total = (w * s["d_weights"].double()).sum() + balance * s["d_losses"][0].double() + z * s["d_losses"][1].double()
    return [torch.autograd.grad(total, x)[0]]
