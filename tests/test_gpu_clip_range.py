"""Clipping by norms so large that the scale leaves fp32's normal range. The scale
is computed in 64 bits, so a value is off by the product's rounding and the
store's, 2 u and U of it (bounds as in test_gpu_block_ops.py)."""

import numpy as np
import pytest
import torch

from oracle import blocks as ob
from test_gpu_block_ops import DEV, bf16, f64, fp16, fp32, gen, near, nsg, ok, randn, run_norm, u

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [bf16, fp32])
@pytest.mark.parametrize("size,max_norm", [(1e36, 1e-4), (1e36, 0.02), (1e34, 1e-12), (1e30, 1e-9), (1e36, 1e-30)])
def test_clipping_by_a_large_norm(dtype, size, max_norm):
    g = gen(3)
    buf = (randn(g, 20011).double() * size).to(dtype)
    grads = [buf[:1], buf[3:9005], buf[9005:]]
    norm = run_norm(grads)
    want = ob.grad_norm([f64(t) for t in grads])
    assert np.isfinite(norm.item()) and abs(norm.item() - want) <= 32 * u * want
    scale = ob.clip_scale(norm.item(), np.float32(max_norm).item())
    exact = [scale * f64(t) for t in grads]
    for offset in (0, 1):               # at the inputs' places of a word, and at others
        outs = list(torch.full((20009 + offset,), 7.0, dtype=dtype, device=DEV)[offset:].split([len(t) for t in grads]))
        nsg.ns_grad_clip(grads, outs, norm, max_norm)
        for y, e in zip(outs, exact):
            near(y, e, 2 * u * np.abs(e), dtype)
    nsg.ns_grad_clip(grads, grads, norm, max_norm)
    for y, e in zip(grads, exact):
        near(y, e, 2 * u * np.abs(e), dtype)
    ok()


def test_clipping_by_a_norm_that_is_not_the_tensors():
    # of other ranks, or infinite: small values vanish, larger ones keep their bits
    norm = torch.full((1,), 3e38, device=DEV)
    x = torch.tensor([65504.0, 1.0, 0.0, -6e4], dtype=fp16, device=DEV)
    y, z = torch.full_like(x, 7), torch.full((3,), 7.0, device=DEV)
    w = torch.tensor([3e38, -1.0, 1e30], device=DEV)
    nsg.ns_grad_clip([x, w], [y, z], norm, 1e-3)
    assert not y.any()
    near(z, f64(w) * np.float32(1e-3).item() / (norm.double().item() + np.float32(1e-6).item()), 2 * u * 1e-3 * np.array([1, 0, 1e-8]), fp32)
    inf = torch.full((1,), float("inf"), device=DEV)
    nsg.ns_grad_clip([w], [z], inf, 1.0)
    assert not z.any()
    nsg.ns_grad_clip([w], [z], inf, float("inf"))
    assert torch.equal(z, w)
    ok()
