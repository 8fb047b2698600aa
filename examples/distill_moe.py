"""A mixture-of-experts student distilled from a teacher's top logits, its
gradients stepped by SCAPE.

    python examples/distill_moe.py [--steps 60] [--workers 2]

Each worker runs its own batch through one student: an embedding, one
mixture-of-experts layer and an output matrix, with PyTorch for the matrix
products.  libscape does the rest of a step:

- ``topk_logits`` cuts the teacher's logits down to 32 words a token and the
  log-sum-exp of the row, which is all that is kept of the teacher;
- ``route`` sends every token to 2 of 8 experts and gives the balance and z
  losses of each sequence, ``route_backward`` the router's gradient;
- ``distill_loss_grad`` gives the loss against the teacher's words (the others as
  one bucket) mixed with the hard labels, and overwrites the logits by their
  gradient;
- ``Scape.step`` takes the workers' bf16 gradients and updates the parameters.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_communication_distributed_gb300 as scape  # noqa: E402

VOCAB, DIM, FF, EXPERTS, TOP = 1003, 64, 128, 8, 2
TAU, KD, CE, BALANCE, Z = 2.0, 0.7, 0.3, 0.01, 0.001
SHAPES = {"emb": (VOCAB, DIM), "router": (DIM, EXPERTS), "w1": (EXPERTS, DIM, FF), "w2": (EXPERTS, FF, DIM),
          "head": (DIM, VOCAB)}


class Route(torch.autograd.Function):
    """Choice of experts, their weights, and the balance and z losses."""

    @staticmethod
    def forward(ctx, logits, cu_tokens):
        idx, weights, counts, live, losses = scape.route(logits, TOP, cu_tokens=cu_tokens)
        ctx.save_for_backward(logits, idx, counts, live, cu_tokens)
        ctx.mark_non_differentiable(idx, counts)
        return idx, weights, counts, losses

    @staticmethod
    def backward(ctx, _idx, d_weights, _counts, d_losses):
        logits, idx, counts, live, cu_tokens = ctx.saved_tensors
        return scape.route_backward(logits, idx, counts, live, d_weights=d_weights.contiguous(),
                                    d_losses=d_losses.contiguous(), cu_tokens=cu_tokens), None


class Distill(torch.autograd.Function):
    """Mean loss over the rows; the logits are overwritten by their gradient."""

    @staticmethod
    def forward(ctx, logits, idx, vals, lse, labels):
        mean = torch.full((logits.shape[0],), 1.0 / logits.shape[0], device=logits.device)
        rows, grad = scape.distill_loss_grad(logits.detach(), idx, vals, teacher_lse=lse, labels=labels,
                                             row_weight=mean, temperature=TAU, kd_weight=KD, ce_weight=CE,
                                             grad=logits.detach())
        ctx.save_for_backward(grad)
        return rows.sum()

    @staticmethod
    def backward(ctx, d_loss):
        return ctx.saved_tensors[0] * d_loss, None, None, None, None


def student(p, tokens, cu_tokens):
    """Logits, tokens of each expert, balance and z losses."""
    h = p["emb"][tokens]
    idx, weights, counts, losses = Route.apply(h @ p["router"], cu_tokens)
    y = torch.zeros_like(h)
    for e in range(EXPERTS):
        at, slot = torch.nonzero(idx == e, as_tuple=True)
        out = torch.nn.functional.gelu(h[at] @ p["w1"][e]) @ p["w2"][e]
        y = y.index_add(0, at, out * weights[at, slot, None])
    return (h + y) @ p["head"], counts, losses


def train(steps: int, workers: int, tokens: int = 512, seed: int = 0, log=print):
    """Runs the example; returns the losses of all steps and the last expert counts."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    numel = [int(torch.Size(s).numel()) for s in SHAPES.values()]
    opt = scape.Scape(numel, chunk=4096, W=workers, density=0.1, lr=3e-3, wd=0.01)
    theta = torch.cat([torch.randn(n, generator=gen, device=dev) * (0.3 if k != "router" else 0.05)
                       for k, n in zip(SHAPES, numel)])
    opt.load(scape.THETA, theta)
    # a teacher: the logits of the next word are a function of the word
    teacher = torch.randn(VOCAB, 24, generator=gen, device=dev) @ torch.randn(24, VOCAB, generator=gen, device=dev)
    cu = torch.tensor([0, tokens // 4, tokens // 2, tokens], dtype=torch.int32, device=dev)
    grads = [torch.empty(opt.N, dtype=torch.bfloat16, device=dev) for _ in range(workers)]
    history, counts = [], None
    for step in range(steps):
        opt.read_into(scape.THETA, theta)
        total = 0.0
        for w in range(workers):
            leaf = theta.detach().clone().requires_grad_(True)
            p = {k: v.view(s) for (k, s), v in zip(SHAPES.items(), leaf.split(numel))}
            x = torch.randint(VOCAB, (tokens,), generator=gen, device=dev)
            z = teacher[x]
            labels = torch.multinomial(torch.softmax(z, 1), 1, generator=gen).squeeze(1)
            idx, vals, lse = scape.topk_logits(z, 32, temperature=TAU)
            logits, counts, aux = student(p, x, cu)
            loss = Distill.apply(logits, idx, vals, lse, labels)
            (loss + BALANCE * aux[0] + Z * aux[1]).backward()
            grads[w].copy_(leaf.grad)
            total += float(loss.detach()) / workers
        opt.step(grads)
        history.append(total)
        if log and (step % 10 == 0 or step == steps - 1):
            log(f"step {step:3d}  loss {total:.4f}  balance {aux[0].item():.4f}  tokens of each expert "
                f"{counts.sum(0).tolist()}")
    opt.close()
    return history, counts


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--workers", type=int, default=2)
    a = ap.parse_args()
    train(a.steps, a.workers)
