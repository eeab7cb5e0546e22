"""Head norms of inputs at the ends of fp32's range, where a product of the
formulas leaves it although the result does not: against the float64 oracle,
with the bounds of test_gpu_training_ops.py (c = (D + 16) u for a norm's value,
twice that for its gradient's two terms). Nothing in them depends on the scale."""

import numpy as np
import pytest
import torch

from oracle import training as ot
from test_gpu_training_ops import DEV, ROUND, f64, gen, near, randn, rotation_table, status, u

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

# Scale of x, eps. The squares' sum stays inside fp32: 128 * 16 * 1e36, and (1e-18)^2.
SCALES = [(1e-18, 0.0), (1e-13, 0.0), (1e-10, 1e-30), (1e15, 1e-6), (1e16, 1e-6), (2e17, 1e-6)]
FORMS = [  # dim, rot, interleaved, offset: every way a lane takes its words, then single values
    (128, 128, False, 0), (64, 32, True, 0), (72, 66, True, 0), (72, 72, False, 0), (128, 64, False, 1), (33, 6, False, 0),
]


def heads(g, T, H, D, scale, dtype, offset):
    x = (randn(g, T * H * D + offset) * scale).to(dtype)
    return x[offset:].view(T, H, D)


@pytest.mark.parametrize("scale,eps", SCALES)
@pytest.mark.parametrize("D,rot,interleaved,offset", FORMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradient(scale, eps, D, rot, interleaved, offset, dtype):
    g = gen(D + rot)
    T, H, K = 21, 4, 2
    q, k = heads(g, T, H, D, scale, dtype, offset), heads(g, T, K, D, scale, dtype, offset)
    gq, gk = heads(g, T, H, D, 1.0, dtype, offset), heads(g, T, K, D, 1.0, dtype, offset)
    qw, kw = randn(g, D, dtype=dtype), randn(g, D, dtype=dtype)
    table = rotation_table(T, rot)
    dq, dk, dqw, dkw = torch.full_like(q, 7), torch.full_like(k, 7), torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    nsg.ns_qk_norm_rope_grad(gq, gk, q, k, dq, dk, qw, kw, dqw, dkw, table, None, ws, eps=eps, interleaved=interleaved)
    assert status() == nsg.NS_OK
    at = (f64(table), np.arange(T), rot, eps, interleaved)
    R = np.abs(ot._rotation(at[0], at[1], rot, D, interleaved))
    c = (D + 16) * u
    for x, dy, dx, w, dw in ((q, gq, dq, qw, dqw), (k, gk, dk, kw, dkw)):
        xv, dyv, wv = f64(x), f64(dy), f64(w)
        r = 1 / np.sqrt((xv * xv).mean(-1, keepdims=True) + eps)
        ua = np.einsum("tab,tha->thb", R, np.abs(dyv))
        h = ua * np.abs(wv)
        want, want_w = ot.norm_rope_grad(dyv, xv, wv, *at)
        near(dx, want, 2 * c * (r * h + np.abs(xv) * r ** 3 * (h * np.abs(xv)).mean(-1, keepdims=True)), dtype)
        near(dw, want_w, ((T * x.shape[1] + 2) * u + c) * (ua * np.abs(xv) * r).sum((0, 1)), torch.float32)


# Scale of x, eps, scale of the weights: their product with r alone has no value in fp32.
WEIGHTS = [(1e15, 1e-6, 1e-28), (2e17, 1e-6, 1e-25), (1e-18, 0.0, 1e22)]


@pytest.mark.parametrize("scale,eps,weight", WEIGHTS)
@pytest.mark.parametrize("D,rot,interleaved,offset", FORMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward(scale, eps, weight, D, rot, interleaved, offset, dtype):
    g = gen(D + rot)
    T, H, K = 21, 4, 2
    q, k = heads(g, T, H, D, scale, dtype, offset), heads(g, T, K, D, scale, dtype, offset)
    qw, kw = (randn(g, D) * weight).to(dtype), (randn(g, D) * weight).to(dtype)
    table = rotation_table(T, rot)
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    nsg.ns_qk_norm_rope(q, k, qo, ko, qw, kw, table, eps=eps, interleaved=interleaved)
    assert status() == nsg.NS_OK
    at = (f64(table), np.arange(T), rot, eps, interleaved)
    R = np.abs(ot._rotation(at[0], at[1], rot, D, interleaved))
    for x, y, w in ((q, qo, qw), (k, ko, kw)):
        xv, wv = f64(x), f64(w)
        r = 1 / np.sqrt((xv * xv).mean(-1, keepdims=True) + eps)
        near(y, ot.norm_rope(xv, wv, *at), (D + 16) * u * np.einsum("tab,thb->tha", R, np.abs(xv * r * wv)), dtype)
