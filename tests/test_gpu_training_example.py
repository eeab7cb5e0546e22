"""The training-step example: its operators under autograd against the same
model in plain torch operations, and a run whose loss falls."""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_operators_under_autograd_match_plain_torch():
    import muon_moe_step as ex
    g = torch.Generator(device="cuda").manual_seed(1)
    T, D, E, k, V, heads, R = 96, 64, 6, 2, 301, (4, 2, 16), 16

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    qkv, qw, kw = randn(T, 8 * 16), randn(16), randn(16)
    angle = torch.arange(T, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, R, 2, device="cuda") / R)
    table, positions = torch.cat([angle.cos(), angle.sin()], 1), torch.arange(T, device="cuda")
    x, w, expert, head = randn(T, D), randn(T, k).softmax(-1), randn(E, D, D) / 8, randn(V, D + 96)
    ids = randn(T, E).topk(k, dim=1).indices
    values, tids = randn(T, 5), torch.randint(0, V, (T, 5), generator=g, device="cuda")
    weights = torch.rand(T, generator=g, device="cuda") / T

    def rope(y):
        a, b = y.double()[..., :8], y.double()[..., 8:]
        c, s = table.double()[positions][:, None, :8], table.double()[positions][:, None, 8:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def run(leaves, own):
        qkv, qw, kw, x, w, expert = leaves
        if own:
            q, key = ex.QkNormRope.apply(qkv, qw, kw, heads, table, positions)
            row, slot, off = ex.sort_tokens(ids, E)
            rows = ex.Dispatch.apply(x, row, slot)
            out = torch.cat([rows[off[e]:off[e + 1]] @ expert[e] for e in range(E)] + [rows[off[-1]:]])
            y = ex.Combine.apply(out, w, row, slot)
        else:
            q, key = ex.split_heads(qkv, heads)[:2]
            q = rope(q / (q.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * qw)
            key = rope(key / (key.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * kw)
            y = sum(w[:, j, None] * torch.einsum("td,tde->te", x, expert[ids[:, j]]) for j in range(k))
        logits = torch.cat([y, q.flatten(1).to(y.dtype), key.flatten(1).to(y.dtype)], 1) @ head.to(y.dtype).t()
        if own:
            loss = ex.Distill.apply(logits, values, tids, weights)[0]
        else:
            p = values.double().softmax(1)
            loss = (weights.double() * (p * (p.log() - logits.log_softmax(1).gather(1, tids))).sum(1)).sum()
        return [loss] + list(torch.autograd.grad(loss, leaves))

    base = (qkv, qw, kw, x, w, expert)
    got = run([t.clone().requires_grad_() for t in base], True)
    want = run([t.double().requires_grad_() for t in base], False)
    assert nsg.ns_check_status() == nsg.NS_OK
    for a, b in zip(got, want):
        # fp32 against 64 bits through a chain of products of up to 160 terms
        assert (a.double() - b).norm() <= 2e-5 * b.norm() + 1e-9


def test_the_loss_falls():
    import muon_moe_step as ex
    losses = ex.train(steps=40)
    assert all(x == x for x in losses)
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5]), losses
