"""Operators of the training step around the orthogonalised matrices, as
torch-tensor calls of the C functions with the same names: tokens sorted by
expert and back, norms of queries and keys with the position rotation, and
distillation from a teacher's top logits, each with its gradient.

Outputs and workspaces are the caller's tensors. A tensor must be on the GPU,
its type one the C function takes and its last dimension contiguous
(ValueError otherwise); the library checks the rest (NsError). Streams default
to torch's current stream.

A call on another stream (``stream=`` a torch stream or a handle) holds no
reference to its tensors: keep them until it is done, or ``record_stream`` them.

The calls record nothing for autograd: a tensor that requires gradients is
refused where they are recorded (ValueError). Under ``torch.no_grad`` and inside
an ``autograd.Function`` (examples/muon_moe_step.py has one for each operator)
it is taken.

The calls on tensors are an extension module (csrc/binding.cpp, built with the
library; missing it is an ImportError): ``help`` on each shows its arguments.
"""

from __future__ import annotations

import ctypes

import torch  # noqa: F401  (the extension links against its libraries)

from ._lib import check, lib
from ._training import (ns_distill_grad, ns_distill_loss, ns_moe_combine, ns_moe_combine_grad,  # noqa: F401
                        ns_moe_dispatch, ns_moe_dispatch_grad, ns_moe_sort, ns_qk_norm_rope, ns_qk_norm_rope_grad)


def ns_moe_rows(tokens: int, k: int, experts: int, align: int = 1, capacity: int = 0) -> int:
    """Rows that hold any routing of tokens * k slots to the experts."""
    out = ctypes.c_int64()
    check(lib.ns_moe_rows(tokens, k, experts, align, capacity, ctypes.byref(out)), "ns_moe_rows")
    return out.value


def ns_moe_sort_workspace_bytes(tokens: int, k: int, experts: int) -> int:
    out = ctypes.c_uint64()
    check(lib.ns_moe_sort_workspace_bytes(tokens, k, experts, ctypes.byref(out)), "ns_moe_sort_workspace_bytes")
    return out.value


def ns_qk_norm_rope_grad_workspace_bytes(head_dim: int) -> int:
    out = ctypes.c_uint64()
    check(lib.ns_qk_norm_rope_grad_workspace_bytes(head_dim, ctypes.byref(out)), "ns_qk_norm_rope_grad_workspace_bytes")
    return out.value


TRAINING_KERNEL_KINDS = ("moe", "qk_norm_rope", "distill")


def ns_profile_read_training(reset: bool = False):
    """({kind: launches}, {kind: summed gpu ms}) of these operators since the last reset."""
    n = (ctypes.c_int64 * len(TRAINING_KERNEL_KINDS))()
    ms = (ctypes.c_double * len(TRAINING_KERNEL_KINDS))()
    check(lib.ns_profile_read_training(1 if reset else 0, n, ms), "ns_profile_read_training")
    return dict(zip(TRAINING_KERNEL_KINDS, list(n))), dict(zip(TRAINING_KERNEL_KINDS, list(ms)))
