"""The float64 oracle of the block norms, the gradient norm and the experts for
a few tokens: hand-worked values, central differences, closed forms."""

import math

import numpy as np
import pytest

from oracle import blocks as ob


def test_gradient_norm_and_clip_by_hand():
    assert ob.grad_norm([np.array([3.0]), np.array([[4.0, 0.0]]), np.zeros(0)]) == 5.0
    assert ob.grad_norm([]) == 0.0
    assert ob.clip_scale(5.0, 1.0, 0.0) == 0.2
    assert ob.clip_scale(0.5, 1.0) == 1.0
    assert ob.clip_scale(1.0, 1.0) == 1.0 / (1.0 + 1e-6)
    assert ob.clip_scale(0.0, 0.0, 0.0) == 1.0


def test_block_norm_by_hand():
    # branch (3, 4): mean square 12.5; with eps = 0 the norm is (3, 4) / sqrt(12.5)
    b, x = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    h, n = ob.block_norm(b, x, branch_weight=np.array([2.0, 1.0]), gate=np.array([0.5]), residual_scale=3.0, branch_scale=2.0, eps=0.0)
    want = np.array([3 + 6 / math.sqrt(12.5), -3 + 4 / math.sqrt(12.5)])
    assert np.allclose(h, want, rtol=1e-15)
    assert np.allclose(n, want / math.sqrt((want ** 2).mean()), rtol=1e-15)
    h, n = ob.block_norm(None, x, weight=np.array([1.0, 5.0]), residual_scale=2.0, eps=0.0)
    assert np.allclose(h, 2 * x) and np.allclose(n, [[1.0, -5.0]])
    h, _ = ob.block_norm(b, x, branch_weight=np.array([2.0, 1.0]), gate=np.array([[0.5, -1.0]]), post_norm=False)
    assert np.allclose(h, [[4.0, -5.0]])


CASES = [(post, gate, branch) for post in (True, False) for gate in (None, "token", "value") for branch in (True, False)
         if branch or (gate is None and not post)]


@pytest.mark.parametrize("post,gate,branch", CASES)
def test_block_norm_gradient_is_the_difference_quotient(post, gate, branch):
    g = np.random.default_rng(3)
    T, D = 3, 5
    x, p, w = g.normal(size=(T, D)), g.normal(size=D), g.normal(size=D)
    leaves = dict(residual=x, weight=w)
    if branch:
        leaves.update(branch=g.normal(size=(T, D)), branch_weight=p)
        if gate:
            leaves["gate"] = g.normal(size=(T, D) if gate == "value" else T)
    ch, cn = g.normal(size=(T, D)), g.normal(size=(T, D))
    more = dict(post_norm=post, residual_scale=0.7, branch_scale=1.3, eps=1e-3)

    def f(leaves):
        h, n = ob.block_norm(leaves.get("branch"), leaves["residual"], leaves.get("branch_weight", 1.0), leaves["weight"],
                             leaves.get("gate"), **more)
        return (h * ch).sum() + (n * cn).sum(), h

    h = f(leaves)[1]
    got = ob.block_norm_grad(ch, cn, leaves.get("branch"), h, leaves.get("branch_weight", 1.0), w, leaves.get("gate"), **more)
    assert set(got) == set(leaves)
    step = 1e-6
    for name, value in leaves.items():
        want = np.zeros(value.shape)
        for i in np.ndindex(value.shape):
            up, down = value.copy(), value.copy()
            up[i] += step
            down[i] -= step
            want[i] = (f({**leaves, name: up})[0] - f({**leaves, name: down})[0]) / (2 * step)
        assert np.allclose(got[name], want, rtol=1e-6, atol=1e-7), name


def test_experts_for_a_few_tokens_by_hand():
    # one expert with ffn 1: h = silu(2) * 3, D = (1, -1)
    x = np.array([[1.0, 1.0], [0.0, 0.0]])
    up = np.array([[[2.0, 0.0], [1.0, 2.0]], [[9.0, 9.0], [9.0, 9.0]]])
    down = np.array([[[1.0], [-1.0]], [[9.0], [9.0]]])
    h = 2 / (1 + math.exp(-2)) * 3
    y = ob.moe_few_tokens(x, np.array([[0, -1], [0, 0]]), np.array([[0.5, np.nan], [1.0, 1.0]]), up, down)
    assert np.allclose(y, [[0.5 * h, -0.5 * h], [0, 0]])
    # named twice: both weights count; without weights 1 each
    assert np.allclose(ob.moe_few_tokens(x, np.array([[0, 0], [-1, -1]]), None, up, down), [[2 * h, -2 * h], [0, 0]])


def test_experts_agree_with_the_sorted_path():
    # the same layer by sorting the tokens, dispatching, products and combining
    from oracle import training as ot
    g = np.random.default_rng(5)
    T, k, E, D, F = 9, 3, 4, 6, 5
    x, w, ids = g.normal(size=(T, D)), g.normal(size=(T, k)), g.integers(-1, E, (T, k))
    up, down = g.normal(size=(E, 2 * F, D)), g.normal(size=(E, D, F))
    row, slot, counts, offsets = ot.moe_sort(ids, E, 1, 0, T * k)
    rows = ot.moe_dispatch(x, row, T * k)
    out = np.zeros((T * k, D))
    for e in range(E):
        part = slice(offsets[e], offsets[e] + counts[e])
        both = rows[part] @ up[e].T
        a, b = both[:, :F], both[:, F:]
        out[part] = (a / (1 + np.exp(-a)) * b) @ down[e].T
    assert np.allclose(ob.moe_few_tokens(x, ids, w, up, down), ot.moe_combine(out, w, row), rtol=1e-12, atol=1e-12)
