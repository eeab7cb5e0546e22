"""Float64 oracle of the training-step operators: tokens sorted by expert and
back, norms of queries and keys with the position rotation, and distillation
from a teacher's top logits, each with its gradient written out by hand.

Plain numpy, in the order of the formulas of include/nsgb300.h; shares no code
with the CUDA path.
"""

from __future__ import annotations

import numpy as np


# ------------------------------------------------------- tokens and experts
def moe_sort(ids, experts: int, align: int = 1, capacity: int = 0, rows: int | None = None):
    """(row_of_slot, slot_of_row, counts, offsets) of ids [tokens, k], slot by slot."""
    ids = np.asarray(ids)
    kept = [[] for _ in range(experts)]
    for s, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts and (not capacity or len(kept[e]) < capacity):
            kept[e].append(s)
    counts = [len(x) for x in kept]
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // align) * align)
    rows = offsets[-1] if rows is None else rows
    row_of_slot, slot_of_row = np.full(ids.size, -1), np.full(rows, -1)
    for e in range(experts):
        for i, s in enumerate(kept[e]):
            row_of_slot[s] = offsets[e] + i
            slot_of_row[offsets[e] + i] = s
    return row_of_slot.reshape(ids.shape), slot_of_row, np.array(counts), np.array(offsets)


def moe_dispatch(x, row_of_slot, rows: int):
    out = np.zeros((rows, x.shape[1]))
    for t, slots in enumerate(row_of_slot):
        for r in slots:
            if r >= 0:
                out[r] = x[t]
    return out


def moe_dispatch_grad(grad_rows, row_of_slot):
    return moe_combine(grad_rows, None, row_of_slot)


def moe_combine(expert_rows, weights, row_of_slot):
    out = np.zeros((row_of_slot.shape[0], expert_rows.shape[1]))
    for t, slots in enumerate(row_of_slot):
        for j, r in enumerate(slots):
            if r >= 0:
                out[t] += (1.0 if weights is None else weights[t, j]) * expert_rows[r]
    return out


def moe_combine_grad(grad_y, expert_rows, weights, row_of_slot):
    grad_rows, grad_weights = np.zeros_like(expert_rows), np.zeros(row_of_slot.shape)
    for t, slots in enumerate(row_of_slot):
        for j, r in enumerate(slots):
            if r >= 0:
                grad_rows[r] = weights[t, j] * grad_y[t]
                grad_weights[t, j] = grad_y[t] @ expert_rows[r]
    return grad_rows, grad_weights


# ------------------------------------------------------- queries and keys
def _rotation(table, positions, rot_dim: int, dim: int, interleaved: bool):
    """One dim x dim matrix per position."""
    R = np.zeros((len(positions), dim, dim))
    R[:, range(dim), range(dim)] = 1.0
    half = rot_dim // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = table[positions, i], table[positions, half + i]
        R[:, a, a], R[:, a, b], R[:, b, a], R[:, b, b] = c, -s, s, c
    return R


def norm_rope(x, weight, table, positions, rot_dim: int, eps: float, interleaved: bool):
    """y [tokens, heads, dim] of x."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    R = _rotation(table, positions, rot_dim, x.shape[2], interleaved)
    return np.einsum("tab,thb->tha", R, x * r * weight)


def norm_rope_grad(grad_y, x, weight, table, positions, rot_dim: int, eps: float, interleaved: bool):
    """(grad_x, grad_weight)."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    R = _rotation(table, positions, rot_dim, x.shape[2], interleaved)
    u = np.einsum("tab,tha->thb", R, grad_y)
    h = u * weight
    grad_x = r * h - x * r ** 3 * (h * x).mean(-1, keepdims=True)
    return grad_x, (u * x * r).sum((0, 1))


# ------------------------------------------------------------ distillation
def teacher_probabilities(values, ids, teacher_lse, temperature: float):
    """p [tokens, top], 0 for entries left out."""
    z = np.where(ids >= 0, values, -np.inf) / temperature
    p = np.zeros(z.shape)
    for t in range(z.shape[0]):
        if (z[t] > -np.inf).any():
            if teacher_lse is not None:
                p[t] = np.exp(z[t] - teacher_lse[t])
                continue
            e = np.exp(z[t] - z[t].max())      # relative to the largest: exact for values near a type's lowest
            p[t] = e / e.sum()
    return p


def distill(logits, values, ids, weights=None, teacher_lse=None, temperature: float = 1.0):
    """(loss, lse, grad_logits)."""
    tokens, vocab = logits.shape
    p = teacher_probabilities(values, ids, teacher_lse, temperature)
    loss, lse, grad = np.zeros(tokens), np.zeros(tokens), np.zeros((tokens, vocab))
    for t in range(tokens):
        w = 1.0 if weights is None else weights[t]
        if w == 0 or not ((ids[t] >= 0) & (values[t] > -np.inf)).any():
            continue
        s = logits[t] / temperature
        lse[t] = np.logaddexp.reduce(s)
        for j in range(p.shape[1]):
            if p[t, j] > 0:
                loss[t] += w * p[t, j] * (np.log(p[t, j]) - s[ids[t, j]] + lse[t])
        grad[t] = w / temperature * p[t].sum() * np.exp(s - lse[t])
        for j in range(p.shape[1]):
            if ids[t, j] >= 0:
                grad[t, ids[t, j]] -= w / temperature * p[t, j]
    return loss, lse, grad
