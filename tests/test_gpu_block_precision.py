"""The experts' layer for a few tokens to fp32's precision at the sizes at which
a block's warps share long rows.

Elementwise bounds that hold for any data grow with the row and say little there;
these are of a token's 2-norm, for independent terms, stated before the first
run. u = 2^-24 is fp32's rounding, U the output type's.

* A sum of n such terms, added in pieces of 16 (n / 16 roundings, each at most u
  of a partial sum whose square grows evenly, and of uniform size): its error is
  u sqrt(n / 96) of its own size, in the mean.
* The two sums of the hidden value, its silu (16 u^2 for exponential, quotient
  and products), the sum down and that over the slots make
  SUMS(D, F) = 2 u sqrt(2 D / 96 + F / 96 + 16), twice the mean.
* The store adds U at most. So 16-bit results show no error below it; in the
  second test they do, because matrices of the same layer subtract what the exact
  layer gives, in parts that the type holds.
"""

import numpy as np
import pytest
import torch

from test_gpu_block_ops import DEV, TYPES, f64, few_inputs, few_reference, gen, nsg, ok, randn, run_few, u
from test_gpu_training_ops import ROUND

# tokens, k, experts, dim, ffn: one step a warp and many, teams of one to 16 warps, rows that are not whole words
SIZES = [(1, 8, 64, 2048, 1408), (64, 6, 64, 2048, 1408), (7, 2, 16, 1096, 712), (33, 8, 8, 1000, 300), (20, 1, 3, 2048, 512),
         (40, 4, 4, 1001, 777), (100, 8, 8, 512, 2816)]


def sums(D, F):
    return 2 * u * np.sqrt(2 * D / 96 + F / 96 + 16)


def rows_off(y, want):
    """Error of each row over the row's size."""
    return np.linalg.norm(y - want, axis=1) / np.maximum(np.linalg.norm(want, axis=1), 1e-300)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,D,F", SIZES)
@pytest.mark.parametrize("dtype", TYPES)
def test_few_tokens_by_their_rows(T, k, E, D, F, dtype):
    g = gen(T + D + 2 * F)
    x, ids, w, up, down = few_inputs(g, T, k, E, D, F, dtype, invalid=0.0)
    y = f64(run_few(x, ids, w, up, down))
    ok()
    want = few_reference(x, ids, w, up, down)[0]
    assert (rows_off(y, want) <= sums(D, F) + ROUND[dtype]).all(), rows_off(y, want).max()


def parts(v, dtype, n=3):
    """n values of dtype whose sum is v."""
    out = []
    for _ in range(n):
        out.append(v.to(dtype))
        v = v - out[-1].double()
    return torch.stack(out, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E,D,F", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_few_tokens_of_16_bits_by_what_is_left(T, k, E, D, F, dtype):
    g = gen(T + D + 3 * F)
    row = randn(g, 1, D, dtype=dtype)
    row[0, 0] = 1
    x = row.repeat(T, 1)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV)
    up, down = (randn(g, E, 2 * F, D) / D ** 0.5).to(dtype), (randn(g, E, D, F) / F ** 0.5).to(dtype)
    # the last three hidden values are silu(64) / 64 = 1
    up[:, F - 3:F], up[:, 2 * F - 3:] = 0, 0
    up[:, F - 3:F, 0], up[:, 2 * F - 3:, 0] = 64.0, 1 / 64
    size = torch.empty(E, dtype=torch.float64, device=DEV)
    for e in range(E):
        a, b = (up[e].double() @ row[0].double())[:, None].chunk(2)
        rest = (down[e, :, :F - 3].double() @ (a * torch.sigmoid(a) * b)[:F - 3])[:, 0]
        size[e] = rest.norm()
        down[e, :, F - 3:] = -parts(rest, dtype)
    lift = 2.0 ** 12                                            # into the type's range
    y = f64(run_few(x, ids, torch.full((T, k), lift, device=DEV), up, down)) / lift
    ok()
    # what the parts leave: 2^-24 of a sum in bf16, half of the smallest value in fp16
    left = k * np.sqrt(D) * 2.0 ** -25 if dtype == torch.float16 else 0.0
    limit = (sums(D, F) + 2.0 ** -23) * (size ** 2)[ids].sum(1).sqrt().cpu().numpy() + left
    assert (np.linalg.norm(y, axis=1) <= limit).all(), (np.linalg.norm(y, axis=1) / limit).max()


@pytest.mark.parametrize("T,k,E,D,F", [(1, 8, 64, 512, 352), (33, 8, 8, 1000, 300)])
@pytest.mark.parametrize("unit", [2.0 ** -8, 2.0 ** -11, 2.0 ** -24])
def test_the_bound_of_rows_sees_what_is_wrong(T, k, E, D, F, unit):
    # without a GPU: nothing at all, hidden values 1 % off, a step of 32 values left out
    rng = np.random.default_rng(T + D)
    x, down = rng.standard_normal((T, D)), rng.standard_normal((D, F)) / F ** 0.5
    up = rng.standard_normal((2 * F, D)) / D ** 0.5
    a, b = np.split(x @ up.T, 2, axis=1)
    h = a / (1 + np.exp(-a)) * b
    want, limit = h @ down.T, sums(D, F) + unit
    short = h.copy()
    short[:, 64:96] = 0
    for wrong in (np.zeros_like(h), h * (1 + 0.01 * rng.standard_normal(h.shape)), short):
        assert (rows_off(wrong @ down.T, want) > limit).all()
