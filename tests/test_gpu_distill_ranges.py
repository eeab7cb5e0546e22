"""Distillation of logits at the ends of their type's range and far from zero:
a loss and a gradient depend on the logits' distances alone, so a row whose
logits are all the type's lowest value (masked throughout) is a uniform one, and
a row moved by a constant keeps its accuracy.

Against the float64 oracle of the rows less their largest logit. Bounds, stated
before the first run, u = 2^-24: a term of the sum is a 2-ulp exp2 of a distance
rounded twice, so with d the largest distance / temperature that still counts
(120: beyond it the term is below 2^-126) a log-sum-exp is off by
e = (V / 128 + 32) u + 4 u min(d, 120), its value rounded at its own size."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from test_gpu_training_ops import DEV, ROUND, f64, gen, near, randn, status, u

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")


def rows_of(g, V, dtype):
    """Rows at the ends of the range, one ordinary."""
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x = torch.empty(7, V, dtype=dtype, device=DEV)
    x[0] = low
    x[1] = high
    x[2] = low
    x[2, V // 2:] = float("-inf")
    x[3] = high
    x[3, V // 2:] = low                                       # their distance overflows
    x[4] = (randn(g, V).to(dtype).float() * 0.25 + 1.0).mul(high / 8).to(dtype)   # only the largest carries anything
    x[5] = randn(g, V, dtype=dtype)
    x[6] = low
    x[6, :3] = randn(g, 3, dtype=dtype)
    return x


def check(logits, values, ids, tau, loss, lse, grad, weights=None):
    s, z, iv = f64(logits), f64(values), ids.cpu().numpy()
    T, V = s.shape
    K = z.shape[1]
    w = np.ones(T) if weights is None else f64(weights)
    top = s.max(1, keepdims=True)
    d = np.where(s > -np.inf, top - s, 0) / tau
    want_loss, want_lse, want_grad = ot.distill(s - top, z, iv, w, None, tau)
    p = ot.teacher_probabilities(z, iv, None, tau)
    e = (V / 128 + 32) * u + 4 * u * np.minimum(d.max(1), 120)
    ep = 32 * u + 4 * u * (np.abs(z - z.max(1, keepdims=True)) / tau).max(1)
    full = top[:, 0] / tau + want_lse
    held = np.abs(full) <= np.finfo(np.float32).max           # what fp32 can hold
    got = f64(lse)
    assert (np.abs(got - full)[held] <= (e + 8 * u * np.abs(full))[held]).all(), (got, full)
    assert (got[~held] == np.sign(full[~held]) * np.inf).all()
    at = np.take_along_axis(d, iv, 1)
    terms = (p * (np.abs(np.log(np.where(p > 0, p, 1))) + at + np.abs(want_lse)[:, None])).sum(1)
    near(loss, want_loss, w * (e + ep + (ep + 8 * u + K * u) * terms), torch.float32)
    if grad is None:
        return
    q = np.exp(-d - want_lse[:, None]) * (s > -np.inf)
    pv = np.zeros((T, V))
    np.add.at(pv, (np.arange(T)[:, None], iv), p)
    near(grad, want_grad, (w / tau)[:, None] * (2 * (e + ep + 16 * u)[:, None] * q + 2 * (ep + (K + 4) * u)[:, None] * pv), grad.dtype)


SIZES = [  # vocab, entries: a block a row, more than 128 entries, a cluster a row, a row too long for one
    (1003, 5), (2000, 200), (131072, 16), (460001, 7), (900001, 7),
]


@pytest.mark.parametrize("V,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tau", [1.0, 0.5, 3.0])
@pytest.mark.parametrize("offset", [0, 1])
def test_ends_of_the_range(V, K, dtype, tau, offset):
    g = gen(V + K)
    logits = rows_of(g, V, dtype)
    T = len(logits)
    ids = torch.randint(0, V // 2, (T, K), generator=g, device=DEV)
    ids[4] = logits[4].argmax()                               # elsewhere the loss has no value that fp32 holds
    ids[6] %= 3
    values = randn(g, T, K)
    loss, lse, loss2, lse2 = (torch.full((T,), 5.0, device=DEV) for _ in range(4))
    grad = torch.full((T * V + offset,), 5.0, dtype=dtype, device=DEV)[offset:].view(T, V)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad, temperature=tau)
    nsg.ns_distill_loss(logits, values, ids, loss2, lse2, temperature=tau)
    assert status() == nsg.NS_OK
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    check(logits, values, ids, tau, loss, lse, grad)


@pytest.mark.parametrize("V,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient_from_a_given_sum_at_the_ends_of_the_range(V, K, dtype):
    # exp(s - lse) for the lse as it is: of a row of the lowest value, 1 (fp32 cannot hold the logarithm beside it)
    g = gen(V)
    logits = torch.full((2, V), torch.finfo(dtype).min, dtype=dtype, device=DEV)
    logits[1] = torch.finfo(dtype).max
    ids, values = torch.randint(0, V, (2, K), generator=g, device=DEV), randn(g, 2, K)
    lse, grad = logits[:, 0].float().contiguous(), torch.empty_like(logits)
    nsg.ns_distill_grad(logits, values, ids, lse, grad)
    assert status() == nsg.NS_OK
    want = np.ones((2, V))
    np.add.at(want, (np.arange(2)[:, None], ids.cpu().numpy()), -ot.teacher_probabilities(f64(values), ids.cpu().numpy(), None, 1.0))
    near(grad, want, (64 + K) * u * np.ones_like(want), dtype)


@pytest.mark.parametrize("V,K", SIZES[:4])
@pytest.mark.parametrize("shift", [1e4, -3e5])
@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_rows_far_from_zero_keep_their_accuracy(V, K, shift, tau):
    g = gen(V)
    T = 4
    logits = 3 * randn(g, T, V) + shift                       # what fp32 makes of them is the input
    ids, values = torch.randint(0, V, (T, K), generator=g, device=DEV), randn(g, T, K)
    weights = torch.rand(T, generator=g, device=DEV) + 0.5
    loss, lse, grad = torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.empty(T, V, device=DEV)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad, weights=weights, temperature=tau)
    assert status() == nsg.NS_OK
    check(logits, values, ids, tau, loss, lse, grad, weights)
