"""Float64 restatement of the norms around a block, the global gradient norm
with clipping, and a mixture-of-experts layer for a few tokens; gradients are
written by hand. Test infrastructure only."""

from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------- norm and clipping
def grad_norm(grads) -> float:
    """Root of the sum of squares of every value."""
    return math.sqrt(math.fsum(float(np.sum(np.square(np.asarray(g, np.float64)))) for g in grads))


def clip_scale(norm: float, max_norm: float, eps: float = 1e-6) -> float:
    return 1.0 if norm + eps <= max_norm else max_norm / (norm + eps)


# -------------------------------------------------------------- block norms
def _gate(gate):
    return 1.0 if gate is None else gate[:, None] if gate.ndim == 1 else gate


def _rms(x, eps):
    return 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)


def block_norm(branch, residual, branch_weight=1.0, weight=1.0, gate=None, post_norm=True, residual_scale=1.0,
               branch_scale=1.0, eps=1e-6):
    """(new residual, its norm); branch None: the norm alone."""
    h = residual_scale * residual
    if branch is not None:
        u = (branch * _rms(branch, eps) if post_norm else branch) * branch_weight
        h = h + branch_scale * _gate(gate) * u
    return h, h * _rms(h, eps) * weight


def block_norm_grad(grad_h, grad_n, branch, h, branch_weight=1.0, weight=1.0, gate=None, post_norm=True,
                    residual_scale=1.0, branch_scale=1.0, eps=1e-6) -> dict:
    """Gradients at the new residual h: residual, weight and, with a branch,
    branch, branch_weight and gate."""
    r2 = _rms(h, eps)
    m, v = h * r2, grad_n * weight
    t = grad_h + r2 * (v - m * (v * m).mean(-1, keepdims=True))
    out = dict(residual=residual_scale * t, weight=(grad_n * m).sum(0))
    if branch is None:
        return out
    r1 = _rms(branch, eps) if post_norm else 1.0
    y = branch * r1
    s = branch_scale * _gate(gate) * t
    z = s * branch_weight
    out["branch"] = r1 * (z - y * (z * y).mean(-1, keepdims=True)) if post_norm else z
    out["branch_weight"] = (s * y).sum(0)
    if gate is not None:
        g = branch_scale * t * y * branch_weight
        out["gate"] = g.sum(1) if gate.ndim == 1 else g
    return out


# --------------------------------------------- experts for a few tokens
def moe_few_tokens(x, ids, weights, gate_up, down):
    """y [tokens, dim]; negative ids go nowhere, weights None: 1."""
    tokens, k = ids.shape
    ffn = down.shape[2]
    y = np.zeros(x.shape)
    for t in range(tokens):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            both = gate_up[e] @ x[t]
            a, b = both[:ffn], both[ffn:]
            y[t] += (1.0 if weights is None else weights[t, j]) * (down[e] @ (a / (1 + np.exp(-a)) * b))
    return y
