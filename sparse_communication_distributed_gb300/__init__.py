"""SCAPE sparse-communication optimizer step on one GB300 (sm_103a).

The CUDA kernels and the C ABI live in ``csrc/`` and build into
``libscape.so`` (``python -m sparse_communication_distributed_gb300.build``);
``scape.Scape`` is the thin ctypes binding over ``include/scape.h``, and
``objective`` binds the calls that produce the gradients of a language model, a
distilled or a mixture-of-experts one among them (linear cross entropy, teacher
top logits, distillation loss, routing),
``experts`` those that sort the tokens' rows by expert and sum them back, and
``gradients`` the norms and the clipping in front of a step.
"""
from .experts import expert_combine, expert_combine_backward, expert_dispatch, expert_plan
from .gradients import clip_grads, grad_norm
from .objective import (distill_loss, distill_loss_grad, linear_ce, linear_ce_grad, route,
                        route_backward, topk_logits)
from .scape import (E, MASK, PHASES, STEP, THETA, U, V, Scape, ScapeError, load_library)

__all__ = ["Scape", "ScapeError", "load_library", "THETA", "V", "U", "E", "MASK", "STEP", "PHASES",
           "topk_logits", "distill_loss", "distill_loss_grad", "linear_ce", "linear_ce_grad", "route",
           "route_backward",
           "expert_plan", "expert_dispatch", "expert_combine", "expert_combine_backward",
           "grad_norm", "clip_grads"]
