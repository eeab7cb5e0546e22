"""Inputs of the block norms' gradient that are not there, beside values of the
others that are not finite."""

import pytest
import torch

from test_gpu_block_ops import DEV, NAN, bf16, fp16, fp32, gen, nsg, ok, randn, scratch

pytestmark = pytest.mark.gpu


# Rows in words, value by value in registers, and longer than those.
@pytest.mark.parametrize("D", [64, 33, 8192, 8200])
@pytest.mark.parametrize("x,r", [(bf16, fp32), (fp16, fp16), (fp32, fp32)])
@pytest.mark.parametrize("value", [float("inf"), NAN])
def test_no_gradient_of_the_norm_no_gradient_of_its_weight(D, x, r, value):
    g = gen(D)
    T = 5
    b, dh, gate = randn(g, T, D, dtype=x), randn(g, T, D, dtype=r), randn(g, T, D, dtype=x)
    h = torch.full((T, D), value, dtype=r, device=DEV)
    ws = scratch(nsg.ns_block_norm_grad_workspace_bytes(D))
    for post in (True, False):
        for gt in (None, gate):
            out = {}
            for name, residual in (("finite", torch.zeros_like(h)), ("not", h)):
                db, dx = torch.full_like(b, NAN), torch.full_like(dh, NAN)
                dp, dw = (torch.full((D,), NAN, device=DEV) for _ in range(2))
                dg = None if gt is None else torch.full_like(gt, NAN)
                nsg.ns_block_norm_grad(dh, None, b, residual, db, dx, None, None, gt, dp, dw, dg, ws, post_norm=post)
                assert not dw.any() and torch.equal(dx, dh)
                out[name] = [db, dp] + ([] if gt is None else [dg])
            assert all(torch.equal(p, q) and p.isfinite().all() for p, q in zip(out["finite"], out["not"]))
    ok()
