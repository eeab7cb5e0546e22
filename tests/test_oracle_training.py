"""Pins of the training-step oracle, CPU only: hand-worked routing, adjoint
identities, and every gradient against central differences of the forward."""

import numpy as np
import pytest

from oracle import training as ot

STEP = 1e-5
# central differences in float64: truncation STEP^2 f''' / 6 plus rounding
# 2^-52 |f| / STEP, both below 1e-8 for values and derivatives of order 10
DIFF_TOL = 1e-7


def differences(f, x):
    """Gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += STEP
        b[i] -= STEP
        g[i] = (f(a) - f(b)) / (2 * STEP)
    return g


def test_sort_hand_case():
    ids = np.array([[1, 0], [1, -1], [0, 1], [2, 1]])
    row, slot, counts, offsets = ot.moe_sort(ids, 4, align=2, capacity=3, rows=9)
    assert counts.tolist() == [2, 3, 1, 0]
    assert offsets.tolist() == [0, 2, 6, 8, 8]
    assert row.tolist() == [[2, 0], [3, -1], [1, 4], [6, -1]]     # the fourth slot of expert 1 is dropped
    assert slot.tolist() == [1, 4, 0, 2, 5, -1, 6, -1, -1]


@pytest.mark.parametrize("seed", range(5))
def test_routing_adjoints(seed):
    g = np.random.default_rng(seed)
    T, k, E, D = 7, 3, 5, 4
    row, slot, _, off = ot.moe_sort(g.integers(-1, E, (T, k)), E, align=2, capacity=4)
    x, gr = g.standard_normal((T, D)), g.standard_normal((off[-1], D))
    gr[slot < 0] = 0
    assert np.isclose((ot.moe_dispatch(x, row, off[-1]) * gr).sum(), (x * ot.moe_dispatch_grad(gr, row)).sum())
    ys, w, dy = g.standard_normal((off[-1], D)), g.standard_normal((T, k)), g.standard_normal((T, D))
    d_rows, d_w = ot.moe_combine_grad(dy, ys, w, row)
    assert np.abs(differences(lambda v: (ot.moe_combine(v, w, row) * dy).sum(), ys) - d_rows).max() < DIFF_TOL
    assert np.abs(differences(lambda v: (ot.moe_combine(ys, v, row) * dy).sum(), w) - d_w).max() < DIFF_TOL


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 6])
def test_norm_rope_gradient(interleaved, rot):
    g = np.random.default_rng(rot)
    T, H, D, P = 3, 2, 6, 9
    angle = g.uniform(0, 6, (P, rot // 2))
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = g.integers(0, P, T)
    x, w, dy = g.standard_normal((T, H, D)), g.standard_normal(D), g.standard_normal((T, H, D))
    y = ot.norm_rope(x, w, table, pos, rot, 1e-3, interleaved)
    # a rotation keeps every pair's length
    n = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-3) * w
    assert np.allclose((y ** 2).sum(-1), (n ** 2).sum(-1))
    for t in range(T):
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = table[pos[t], i], table[pos[t], rot // 2 + i]
            assert np.allclose(y[t, :, a], n[t, :, a] * c - n[t, :, b] * s)
            assert np.allclose(y[t, :, b], n[t, :, b] * c + n[t, :, a] * s)
    dx, dw = ot.norm_rope_grad(dy, x, w, table, pos, rot, 1e-3, interleaved)
    f = lambda x, w: (ot.norm_rope(x, w, table, pos, rot, 1e-3, interleaved) * dy).sum()  # noqa: E731
    assert np.abs(differences(lambda v: f(v, w), x) - dx).max() < DIFF_TOL
    assert np.abs(differences(lambda v: f(x, v), w) - dw).max() < DIFF_TOL


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 2.0])
def test_distill_gradient(full, temperature):
    g = np.random.default_rng(3)
    T, V, K = 4, 11, 5
    s, z = g.standard_normal((T, V)), g.standard_normal((T, K))
    ids = g.integers(0, V, (T, K))
    ids[0, 1] = ids[0, 0]            # an entry named twice
    ids[1, 2:] = -1                  # padding
    z[2, 0] = -np.inf
    w = np.array([1.0, 0.5, 2.0, 0.0])
    tl = np.log(np.exp(z / temperature).sum(1) * 1.2) if full else None
    loss, lse, grad = ot.distill(s, z, ids, w, tl, temperature)
    assert np.abs(differences(lambda v: ot.distill(v, z, ids, w, tl, temperature)[0].sum(), s) - grad).max() < DIFF_TOL
    assert loss[3] == 0 and lse[3] == 0 and not grad[3].any()
    p = ot.teacher_probabilities(z, ids, tl, temperature)
    if not full:
        assert np.allclose(p.sum(1), 1) and (loss >= 0).all()
        assert np.allclose(grad.sum(1), 0)


def test_distill_without_entries_ignores_the_row():
    s = np.full((2, 4), np.nan)
    loss, lse, grad = ot.distill(s, np.array([[1.0], [-np.inf]]), np.array([[-1], [2]]))
    assert not loss.any() and not lse.any() and not grad.any()


def test_distill_of_equal_distributions_is_zero():
    g = np.random.default_rng(8)
    s = g.standard_normal((3, 6))
    ids = np.tile(np.arange(6), (3, 1))
    loss, _, grad = ot.distill(s, s + 7.0, ids)
    assert np.abs(loss).max() < 1e-14 and np.abs(grad).max() < 1e-15


def test_teacher_values_near_the_lowest_are_compared_with_each_other():
    low = float(np.finfo(np.float32).min)
    p = ot.teacher_probabilities(np.array([[low, low, -np.inf, low]]), np.array([[0, 1, 2, -1]]), None, 0.5)
    assert p.tolist() == [[0.5, 0.5, 0.0, 0.0]]
