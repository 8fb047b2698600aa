"""SCAPE sparse-communication optimizer step on one GB300 (sm_103a).

The CUDA kernels and the C ABI live in ``csrc/`` and build into
``libscape.so`` (``python -m sparse_communication_distributed_gb300.build``);
``scape.Scape`` is the thin ctypes binding over ``include/scape.h``, and
``objective`` binds the calls that produce the gradients of a distilled or
mixture-of-experts model (teacher top logits, distillation loss, routing).
"""
from .objective import distill_loss, distill_loss_grad, route, route_backward, topk_logits
from .scape import (E, MASK, PHASES, STEP, THETA, U, V, Scape, ScapeError, load_library)

__all__ = ["Scape", "ScapeError", "load_library", "THETA", "V", "U", "E", "MASK", "STEP", "PHASES",
           "topk_logits", "distill_loss", "distill_loss_grad", "route", "route_backward"]
