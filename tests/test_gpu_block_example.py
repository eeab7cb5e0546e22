"""The example of norms around blocks, clipping and decoding: its operators under
autograd against the same formulas in 64 bits, a run of all of them together,
and decoding against the training path."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def rms(x):
    return x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()


def test_block_norms_under_autograd_match_plain_torch():
    import muon_block_step as ex
    g = torch.Generator(device="cuda").manual_seed(1)
    T, D = 96, 64

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    base = (randn(T, D), randn(D), randn(D), randn(D, D) / 8, randn(D), randn(D), randn(T), randn(D, D) / 8)
    c = randn(T, D)

    def run(leaves, own):
        x, w0, p1, m1, w1, p2, gate, m2 = leaves
        if own:
            n = ex.BlockNorm.apply(None, x, None, w0, None)
            x, n = ex.BlockNorm.apply(n @ m1, x, p1, w1, None)
            x, n = ex.BlockNorm.apply(torch.tanh(n @ m2), x, p2, w0, gate)
        else:
            n = rms(x) * w0
            x = x + rms(n @ m1) * p1
            n = rms(x) * w1
            x = x + gate[:, None] * rms(torch.tanh(n @ m2)) * p2
            n = rms(x) * w0
        loss = (n * c.to(n.dtype)).sum() + x.pow(2).sum()
        return [loss] + list(torch.autograd.grad(loss, leaves))

    got = run([t.clone().requires_grad_() for t in base], True)
    want = run([t.double().requires_grad_() for t in base], False)
    assert nsg.ns_check_status() == nsg.NS_OK
    for a, b in zip(got, want):
        # fp32 against 64 bits through two blocks of sums of 64 terms and sums over 96 tokens: (64 + 96 + 2 * 24) 2^-24 < 2e-5
        assert (a.double() - b).norm() <= 2e-5 * b.norm() + 1e-9


def test_clipping_scales_every_gradient():
    import muon_block_step as ex
    g = torch.Generator(device="cuda").manual_seed(2)
    leaves = [torch.zeros(*s, device="cuda", requires_grad=True) for s in ((30, 7), (5,), (1001,), (3, 3))]
    grads = [torch.randn(t.shape, generator=g, device="cuda") for t in leaves]
    for t, x in zip(leaves[:3], grads):
        t.grad = x.clone()
    norm = ex.clip_gradients(leaves, 0.5)              # the last has no gradient
    want = torch.cat([x.flatten() for x in grads[:3]]).double().norm()
    assert abs(norm.item() - want.item()) <= 1e-6 * want.item()
    for t, x in zip(leaves[:3], grads):
        # the scale and its product: 2 roundings of 2^-24, and the norm's own 32 2^-24
        assert (t.grad.double() - x.double() * (0.5 / (want + 1e-6))).abs().max() <= 40 * 2.0 ** -24 * x.abs().max()
    assert leaves[3].grad is None
    assert nsg.ns_check_status() == nsg.NS_OK


def test_a_run_of_all_of_them():
    import muon_block_step as ex
    model, losses, norms = ex.train(steps=4, batch=4, vocab=300, dim=128, heads=(4, 2, 32), experts=4, ffn=96, length=32)
    assert all(x == x and abs(x) != float("inf") for x in losses + norms) and min(norms) > 0
    # decoding gives what the training path gives for the last position. Both round the experts' sum and two norms to
    # bf16, the training path the experts' rows and hidden values besides: a few roundings of 2^-9 of values around 1,
    # summed over 128 columns of the head with weights of 1 / sqrt(128).
    tokens = torch.arange(4 * 9, device="cuda").view(4, 9) % model.vocab
    with torch.no_grad():
        want = model.logits(tokens).view(4, 9, -1)[:, -1].float()
    got = model.next_logits(tokens, model.expert_weights()).float()
    assert (got - want).norm() <= 0.02 * want.norm()
    assert model.generate(tokens, 3).shape == (4, 12)
    assert nsg.ns_check_status() == nsg.NS_OK
