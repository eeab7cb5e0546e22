"""The gradient alone, later and with other weights, for tokens that the loss
call left out: their log-sum-exp was never computed, and the gradient says so."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from test_gpu_training_ops import DEV, f64, gen, near, randn, status, u

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")


@pytest.mark.parametrize("V,K", [(301, 4), (50001, 20), (131072, 200), (900001, 5)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens_left_out_by_the_loss(V, K, dtype):
    g = gen(V)
    T = 6
    logits, values = randn(g, T, V, dtype=dtype), randn(g, T, K)
    ids = torch.randint(0, V, (T, K), generator=g, device=DEV)
    first = torch.tensor([1.0, 0.0, 0.0, 2.0, 1.0, 0.0], device=DEV)
    then = torch.tensor([0.5, 3.0, 0.0, 0.0, 1.5, -1.0], device=DEV)
    none = ids.clone()
    none[4] = -1                                           # no entry left: nothing to learn from whatever the weight
    loss, lse, grad = torch.full((T,), 5.0, device=DEV), torch.full((T,), 5.0, device=DEV), torch.full_like(logits, 5.0)
    nsg.ns_distill_loss(logits, values, none, loss, lse, weights=first)
    assert (lse[[1, 2, 4, 5]] == 0).all() and (loss[[1, 2, 4, 5]] == 0).all()
    nsg.ns_distill_grad(logits, values, none, lse, grad, weights=then)
    assert status() == nsg.NS_OK
    assert grad[[1, 5]].isnan().all()                      # a weight, but no sum to divide by
    assert not grad[[2, 3, 4]].any()
    want = ot.distill(f64(logits[:1]), f64(values[:1]), ids[:1].cpu().numpy(), f64(then[:1]))[2]
    near(grad[:1], want, (V / 128 + 64 + K) * u * np.ones_like(want), dtype)


def test_a_sum_that_is_exactly_zero_is_a_sum():
    # logits that are log-probabilities: their log-sum-exp comes out as 0
    for V in (1, 4, 1024):
        logits = torch.full((2, V), -np.log(V), device=DEV) if V > 1 else torch.zeros(2, 1, device=DEV)
        ids, values = torch.zeros(2, 1, dtype=torch.int64, device=DEV), torch.zeros(2, 1, device=DEV)
        grad = torch.full_like(logits, 5.0)
        nsg.ns_distill_grad(logits, values, ids, torch.zeros(2, device=DEV), grad)
        want = np.full((2, V), 1.0 / V)
        want[:, 0] -= 1
        near(grad, want, 64 * u * np.ones_like(want), torch.float32)
    assert status() == nsg.NS_OK


def test_the_loss_never_writes_the_mark_for_a_token_that_counts():
    logits = torch.tensor([[0.0], [-0.0], [-1e-45], [1e-45]], device=DEV)
    ids, values = torch.zeros(4, 1, dtype=torch.int64, device=DEV), torch.zeros(4, 1, device=DEV)
    loss, lse, grad = torch.empty(4, device=DEV), torch.empty(4, device=DEV), torch.full_like(logits, 5.0)
    for tau in (1.0, 1e6):
        nsg.ns_distill_loss(logits, values, ids, loss, lse, temperature=tau)
        nsg.ns_distill_grad(logits, values, ids, lse, grad, temperature=tau)
        assert not grad.any()
    assert status() == nsg.NS_OK
