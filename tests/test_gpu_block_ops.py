"""The gradient norm and clipping, the norms around a block and the experts for
a few tokens against the float64 oracle.

Tolerances, element by element and stated before the first run. u = 2^-24 is
fp32's rounding, U the output type's (half its eps), tiny its smallest positive
value; every store adds U |value| + tiny.

* the norm: a lane's sum of at most 80 squares in fp32, in four chains of at most
  20 that are then added, the rest in 64 bits: (20 + 4) u of the sum, half of it
  after the root, + 1 u for the store: within 32 u;
* clipping: the scale is computed in 64 bits from the fp32 norm that the test
  passes and rounded to fp32 (1 u), the product 1 u;
* a mean of D squares and its reciprocal square root: (D + 16) u relative, and
  with the products around it c = (D + 24) u;
* h = alpha x + beta g u: c A with A the sum of the two terms' magnitudes; its
  norm r2 is off by c (1 + |A| / |h|) relative (2-norms of the rows);
* backward, every quantity by the sum of the magnitudes that enter it: t by 4 c,
  what follows from it by 8 c, and a sum over T tokens by T u more;
* a product of D terms: 2 (D + 16) u of the sum of the terms' magnitudes (tensor
  cores may cut what they add at fp32's last place; an fp32 factor split in two
  leaves 2^-21 of each term); silu's slope is at most 1.1, its rounding 8 u; the
  hidden value that meets the weights is exact to 2^-17.
"""

import numpy as np
import pytest
import torch

import test_gpu_training_ops as ops
from oracle import blocks as ob
from test_gpu_training_ops import DEV, TYPES, f64, gen, near, randn, strided_rows, u

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

NAN = float("nan")
bf16, fp16, fp32 = TYPES


def ok():
    assert nsg.ns_check_status() == nsg.NS_OK


def scratch(bytes_):
    return torch.full((bytes_,), 0xFF, dtype=torch.uint8, device=DEV)


# ------------------------------------------------------- norm and clipping
def run_norm(grads, stream=None):
    norm = torch.full((1,), NAN, device=DEV)
    nsg.ns_grad_norm(grads, norm, scratch(nsg.ns_grad_norm_workspace_bytes(len(grads))), stream=stream)
    return norm


def packed(g, sizes, dtype, offset=0, scale=1.0):
    """Tensors one behind the other in one buffer that starts `offset` values past a boundary."""
    flat = randn(g, sum(sizes) + offset, dtype=fp32).mul_(scale).to(dtype)[offset:]
    return list(flat.split(sizes)) if sizes else []


SIZES = [
    [1], [3], [8], [7, 1, 9], [0, 5, 0], [4095, 1, 4097], [16383, 16384, 16385], [100000], [3 * 8192 + 5, 8192, 2],
    [1001 * 333, 1001, 77 * 1001], [2 ** 20 + 3], list(range(1, 40)),
]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [0, 1, 6])
def test_norm_and_clip(sizes, dtype, offset):
    g = gen(sum(sizes) + offset)
    grads = packed(g, sizes, dtype, offset, 3.0)
    norm = run_norm(grads)
    want = ob.grad_norm([f64(t) for t in grads])
    assert abs(norm.item() - want) <= 32 * u * want
    n = norm.item()
    for max_norm in (0.37 * n, 2 * n, 0.0, float("inf")):
        scale = ob.clip_scale(n, max_norm, 1e-3)
        for out_offset in (offset, 3):      # another place of a word than the input's
            buf = torch.full((sum(sizes) + out_offset + 1,), 7.0, dtype=dtype, device=DEV)
            outs = list(buf[out_offset:-1].split(sizes))
            nsg.ns_grad_clip(grads, outs, norm, max_norm, eps=1e-3)
            for x, y in zip(grads, outs):
                near(y, scale * f64(x), 2 * u * np.abs(scale * f64(x)), dtype)
            assert (buf[:out_offset] == 7).all() and buf[-1] == 7
    # in place gives the same bits
    want = [torch.empty_like(t) for t in grads]
    nsg.ns_grad_clip(grads, want, norm, 0.5 * n)
    nsg.ns_grad_clip(grads, grads, norm, 0.5 * n)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    ok()


def test_norm_of_many_tensors_of_all_types():
    g = gen(1)
    grads = []
    for i in range(1300):                   # several launches
        grads.append(randn(g, *((i % 7 + 1, 40 + i) if i % 3 else (i,)), dtype=TYPES[i % 3]))
    grads[5] = randn(g, 300, 70, dtype=bf16).t()                # another order of the dimensions
    grads[600] = randn(g, 4, 6, 5, 7).to(memory_format=torch.channels_last)
    norm = run_norm(grads)
    want = ob.grad_norm([f64(t) for t in grads])
    assert abs(norm.item() - want) <= 32 * u * want
    assert torch.equal(norm, run_norm(grads))                   # the same bits
    outs = [torch.empty_like(t) for t in grads]
    nsg.ns_grad_clip(grads, outs, norm, 1.0)
    scale = ob.clip_scale(norm.item(), 1.0)
    for x, y in zip(grads, outs):
        assert x.stride() == y.stride()
        near(y, scale * f64(x), 2 * u * np.abs(f64(x)) * scale, x.dtype)
    ok()


def test_norm_of_nothing():
    assert run_norm([]).item() == 0.0
    assert run_norm([torch.empty(0, device=DEV), torch.empty(0, 5, device=DEV, dtype=bf16)]).item() == 0.0
    assert run_norm([torch.zeros(70001, device=DEV, dtype=fp16)]).item() == 0.0
    nsg.ns_grad_clip([], [], torch.ones(1, device=DEV), 1.0)
    nsg.ns_grad_clip([torch.empty(0, device=DEV)], [torch.empty(0, device=DEV)], torch.ones(1, device=DEV), 1.0)
    ok()


@pytest.mark.parametrize("dtype,size", [(fp32, 1e30), (fp32, 1e-30), (fp32, 1e-42), (bf16, 1e30), (bf16, 1e-35), (fp16, 6e-8), (fp32, 1e19), (bf16, 1e-20)])
@pytest.mark.parametrize("n", [5, 9000, 300001])
def test_norm_whose_squares_leave_the_range(dtype, size, n):
    g = gen(n)
    x = (randn(g, n).double() * size).to(dtype)
    if n > 5:
        x[n // 2:] = 0                      # chunks of zeros beside them
    for t in (x, torch.cat([torch.zeros(1, dtype=dtype, device=DEV), x])[1:]):
        want = ob.grad_norm([f64(t)])
        got = run_norm([t, torch.zeros(20000, device=DEV)]).item()
        assert abs(got - want) <= 32 * u * want + 2.0 ** -149
    ok()


def test_norm_of_large_beside_small_values():
    x = torch.full((100000,), 1e-30, device=DEV)
    x[777] = 2e25
    assert run_norm([x]).item() == pytest.approx(2e25, rel=1e-6)
    big = torch.full((4,), 3e38, device=DEV)
    assert run_norm([big]).item() == float("inf")               # past fp32's largest value
    ok()


def test_infinite_and_nan_gradients():
    x, y = torch.ones(5000, device=DEV), torch.full((33,), 2.0, device=DEV, dtype=bf16)
    x[4999] = float("inf")
    norm = run_norm([y, x])
    assert norm.item() == float("inf")
    outs = [torch.empty_like(y), torch.empty_like(x)]
    nsg.ns_grad_clip([y, x], outs, norm, 1.0)
    assert not outs[0].any() and not outs[1][:4999].any() and outs[1][4999].isnan()
    nsg.ns_grad_clip([y, x], outs, norm, float("inf"))
    assert torch.equal(outs[0], y) and torch.equal(outs[1], x)
    x[3] = NAN
    norm = run_norm([y, x])
    assert norm.isnan().all()
    nsg.ns_grad_clip([y, x], outs, norm, 1.0)
    assert outs[0].isnan().all() and outs[1].isnan().all()
    ok()


def test_norm_over_several_calls():
    # the root of the sum of squares of partial norms is a norm to clip by
    g = gen(8)
    a, b = packed(g, [5000, 77], fp32), packed(g, [1234], bf16)
    both = torch.stack([run_norm(a), run_norm(b)]).square().sum().sqrt()
    want = ob.grad_norm([f64(t) for t in a + b])
    assert abs(both.item() - want) <= 64 * u * want
    nsg.ns_grad_clip(a, a, both, 1.0)
    nsg.ns_grad_clip(b, b, both, 1.0)
    assert abs(run_norm(a + b).item() - 1.0) < 4e-3
    ok()


def test_values_past_32_bits():
    n = 2 ** 32 + 4099
    x = torch.zeros(n, dtype=bf16, device=DEV)
    x[-3:], x[2 ** 31], x[0] = 2.0, 1.0, 1.0
    assert run_norm([x]).item() == pytest.approx(14 ** 0.5, rel=1e-6)
    norm = torch.full((1,), 10.0, device=DEV)
    nsg.ns_grad_clip([x], [x], norm, 5.0, eps=0.0)
    assert x[-4:].tolist() == [0, 1, 1, 1] and x[2 ** 31] == 0.5 and x[0] == 0.5 and x[1] == 0
    ok()


# ------------------------------------------------------------- block norms
BLOCKS = [  # tokens, dim, post, gate, branch, extra stride, offset
    (1, 1, True, "none", True, 0, 0), (1, 8, True, "token", True, 0, 0), (3, 64, True, "none", True, 0, 0),
    (5, 2048, True, "value", True, 0, 0), (33, 1001, True, "token", True, 0, 0), (40, 1001, False, "value", True, 3, 0),
    (7, 4096, False, "none", True, 0, 0), (300, 256, True, "token", True, 8, 0), (17, 264, True, "value", True, 0, 1),
    (2, 8192, True, "token", True, 0, 0), (3, 16384, True, "value", True, 0, 0), (2, 20008, True, "none", True, 0, 0),
    (700, 72, True, "value", True, 0, 0), (64, 2050, True, "none", True, 0, 0), (9, 520, False, "token", True, 0, 0),
    (4, 2048, False, "none", False, 0, 0), (19, 1003, False, "none", False, 5, 2), (2500, 128, True, "token", True, 0, 0),
    (1031, 1032, True, "none", True, 8, 0), (6, 12296, True, "token", True, 0, 0), (151, 4104, True, "value", True, 0, 0),
]
PAIRS = [(bf16, bf16), (bf16, fp32), (fp16, fp16), (fp16, fp32), (fp32, fp32)]


def block_inputs(g, T, D, x, r, gate, branch, extra, offset, weight_fp32, weighted=True):
    wt = fp32 if weight_fp32 else x
    b = strided_rows(g, T, D, x, extra, offset) if branch else None
    h = strided_rows(g, T, D, r, extra, offset)
    if branch and T > 2:
        b[1] = 0                            # a row of zeros has only eps to divide by
        h[2] = 0
    weights = [randn(g, D, dtype=wt) if weighted and (branch or i) else None for i in range(2)]
    gate = {"none": None, "token": randn(g, T), "value": strided_rows(g, T, D, x, extra, offset)}[gate]
    return b, h, weights, gate


def f(t):
    return None if t is None else f64(t)


def one(t):
    return 1.0 if t is None else f64(t)


def like(t, extra=0):
    """NaN, with rows `extra` wider than t's."""
    return torch.full((t.shape[0], t.shape[1] + extra), NAN, dtype=t.dtype, device=DEV)[:, :t.shape[1]]


@pytest.mark.parametrize("T,D,post,gate,branch,extra,offset", BLOCKS)
@pytest.mark.parametrize("x,r", PAIRS)
@pytest.mark.parametrize("weight_fp32", [False, True])
def test_block_norm(T, D, post, gate, branch, extra, offset, x, r, weight_fp32):
    g = gen(T + D)
    b, h_in, (p, w), gt = block_inputs(g, T, D, x, r, gate, branch, extra, offset, weight_fp32, weighted=(T + D) % 5 > 0)
    more = dict(post_norm=post, residual_scale=0.75, branch_scale=-1.25, eps=1e-5)
    h_out, out = like(h_in, extra), torch.full((T, D), NAN, dtype=x, device=DEV)
    nsg.ns_block_norm(b, h_in, h_out, out, p, w, gt, **more)
    ok()
    want_h, want_n = ob.block_norm(f(b), f64(h_in), one(p), one(w), f(gt), **more)
    c = (D + 24) * u
    A = 0.75 * np.abs(f64(h_in))
    if branch:
        with_gate = ob.block_norm(np.abs(f64(b)), np.zeros((T, D)), np.abs(one(p)), 1.0, None if gt is None else np.abs(f64(gt)),
                                  post_norm=post, branch_scale=1.25, eps=1e-5)[0]
        A = A + with_gate
    near(h_out, want_h, c * A, r)
    r2 = ob._rms(want_h, 1e-5)
    off = 1 + np.linalg.norm(A, axis=1, keepdims=True) / np.maximum(np.linalg.norm(want_h, axis=1, keepdims=True), 1e-300)
    off = np.minimum(off, 1 + np.linalg.norm(A, axis=1, keepdims=True) / np.sqrt(D * 1e-5))
    near(out, want_n, 2 * c * r2 * np.abs(one(w)) * (A + np.abs(want_h) * off), x)
    # each output alone, and both in place of inputs
    alone = [like(h_in), like(out)]
    nsg.ns_block_norm(b, h_in, alone[0], None, p, w, gt, **more)
    nsg.ns_block_norm(b, h_in, None, alone[1], p, w, gt, **more)
    assert torch.equal(alone[0], h_out) and torch.equal(alone[1], out)
    h2 = ops.same_place(h_in)
    if branch:
        b2 = ops.same_place(b)
        nsg.ns_block_norm(b2, h2, h2, b2, p, w, gt, **more)
        assert torch.equal(h2, h_out) and torch.equal(b2, out)
    else:
        nsg.ns_block_norm(None, h2, h2, out, p, w, None, **more)
        assert torch.equal(h2, h_out)
    ok()


@pytest.mark.parametrize("T,D,post,gate,branch,extra,offset", BLOCKS)
@pytest.mark.parametrize("x,r", PAIRS)
@pytest.mark.parametrize("weight_fp32", [False, True])
def test_block_norm_gradient(T, D, post, gate, branch, extra, offset, x, r, weight_fp32):
    g = gen(T + D + 1)
    b, h, (p, w), gt = block_inputs(g, T, D, x, r, gate, branch, extra, offset, weight_fp32, weighted=(T + D) % 5 > 0)
    dh, dn = strided_rows(g, T, D, r, extra, offset), strided_rows(g, T, D, x, extra, offset)
    more = dict(post_norm=post, residual_scale=0.75, branch_scale=-1.25, eps=1e-5)
    c, ws = (D + 24) * u, scratch(nsg.ns_block_norm_grad_workspace_bytes(D))
    for have_dh, have_dn in ((True, True), (True, False), (False, True)):
        gh, gn = dh if have_dh else None, dn if have_dn else None
        dx, dw = like(h, extra), torch.full((D,), NAN, device=DEV)
        db, dp = (like(b, extra), torch.full((D,), NAN, device=DEV)) if branch else (None, None)
        dg = None if gt is None else torch.full_like(gt, NAN)
        nsg.ns_block_norm_grad(gh, gn, b, h, db, dx, p, w, gt, dp, dw, dg, ws, **more)
        ok()
        gh64, gn64 = (f64(dh) if have_dh else np.zeros((T, D))), (f64(dn) if have_dn else np.zeros((T, D)))
        want = ob.block_norm_grad(gh64, gn64, f(b), f64(h), one(p), one(w), f(gt), **more)
        r2 = ob._rms(f64(h), 1e-5)
        m, v = np.abs(f64(h)) * r2, np.abs(gn64 * one(w))
        t = np.abs(gh64) + r2 * (v + m * (v * m).mean(-1, keepdims=True))
        near(dx, want["residual"], 4 * c * 0.75 * t, r)
        near(dw, want["weight"], (T * u + 2 * c) * (np.abs(gn64) * m).sum(0), fp32)
        if not branch:
            continue
        r1 = ob._rms(f64(b), 1e-5) if post else 1.0
        y = np.abs(f64(b)) * r1
        s = 1.25 * t * (1.0 if gt is None else np.abs(ob._gate(f64(gt))))
        z = s * np.abs(one(p))
        near(db, want["branch"], 8 * c * (r1 * (z + y * (z * y).mean(-1, keepdims=True)) if post else z), x)
        near(dp, want["branch_weight"], (T * u + 8 * c) * (s * y).sum(0), fp32)
        if gt is not None:
            dg_abs = 1.25 * t * y * np.abs(one(p))
            near(dg, want["gate"], 8 * c * (dg_abs.sum(1) if gt.dim() == 1 else dg_abs), gt.dtype)
    # the outputs in place of inputs of their type, without the weights' gradients
    h2, dh2, dn2 = ops.same_place(h), ops.same_place(dh), ops.same_place(dn)
    full = [like(h), like(b) if branch else None, None if gt is None else torch.full_like(gt, NAN)]
    nsg.ns_block_norm_grad(dh, dn, b, h, full[1], full[0], p, w, gt, grad_gate=full[2], **more)
    gt2 = None if gt is None else ops.same_place(gt)
    nsg.ns_block_norm_grad(dh2, dn2, b, h2, dn2 if branch else None, dh2, p, w, gt2, grad_gate=gt2, **more)
    assert torch.equal(dh2, full[0]) and torch.equal(h2, h)
    if branch:
        assert torch.equal(dn2, full[1])
        b2 = ops.same_place(b)
        nsg.ns_block_norm_grad(dh, dn, b2, h, b2, None, p, w, gt, **more)
        assert torch.equal(b2, full[1])
    if gt is not None:
        assert torch.equal(gt2, full[2])
    nsg.ns_block_norm_grad(dh, dn, b, h2, None, h2, p, w, gt, **more)
    assert torch.equal(h2, full[0])
    ok()


def test_block_norm_gradient_against_differences():
    # fp32 sums of squares of 3 x 10 values: central differences of step 2^-6 are exact to 1e-3
    g = gen(12)
    T, D = 3, 10
    x, b, p, w, gt = randn(g, T, D), randn(g, T, D), randn(g, D), randn(g, D), randn(g, T)
    ch, cn = randn(g, T, D), randn(g, T, D)

    def value(leaves):
        h, n = torch.empty(T, D, device=DEV), torch.empty(T, D, device=DEV)
        nsg.ns_block_norm(leaves["branch"], leaves["residual"], h, n, leaves["branch_weight"], leaves["weight"], leaves["gate"], eps=0.1)
        return float((h.double() * ch).sum() + (n.double() * cn).sum()), h

    leaves = dict(branch=b, residual=x, branch_weight=p, weight=w, gate=gt)
    h = value(leaves)[1]
    grads = {k: torch.empty_like(v) for k, v in leaves.items()}
    nsg.ns_block_norm_grad(ch, cn, b, h, grads["branch"], grads["residual"], p, w, gt, grads["branch_weight"], grads["weight"],
                           grads["gate"], scratch(nsg.ns_block_norm_grad_workspace_bytes(D)), eps=0.1)
    step = 2.0 ** -6
    for name, v in leaves.items():
        for i in range(v.numel()):
            up, down = v.clone(), v.clone()
            up.view(-1)[i] += step
            down.view(-1)[i] -= step
            want = (value({**leaves, name: up})[0] - value({**leaves, name: down})[0]) / (2 * step)
            assert abs(grads[name].view(-1)[i].item() - want) < 2e-2 * max(1.0, abs(want)), (name, i)
    ok()


def test_block_norm_of_nothing():
    e, D = torch.empty(0, 16, device=DEV), 16
    w = torch.full((D,), 5.0, device=DEV)
    nsg.ns_block_norm(e, e, e, e)
    ws = scratch(nsg.ns_block_norm_grad_workspace_bytes(D))
    dw = w.clone()
    nsg.ns_block_norm_grad(e, e, e, e, e, e, grad_branch_weight=w, grad_weight=dw, workspace=ws)
    assert not w.any() and not dw.any()                         # sums over no token
    z = torch.empty(3, 0, device=DEV)
    nsg.ns_block_norm(z, z, z, z)
    ok()


def test_rows_of_nan_and_infinities_stay_where_they_are():
    g = gen(5)
    T, D = 12, 256
    b, x = randn(g, T, D, dtype=bf16), randn(g, T, D, dtype=bf16)
    w = randn(g, D, dtype=bf16)
    clean = [torch.empty_like(b), torch.empty_like(b)]
    nsg.ns_block_norm(b, x, *clean, w, w)
    b[3, 7], x[8, 0] = NAN, float("inf")
    got = [torch.empty_like(b), torch.empty_like(b)]
    nsg.ns_block_norm(b, x, *got, w, w)
    keep = [t for t in range(T) if t not in (3, 8)]
    for a, c in zip(got, clean):
        assert torch.equal(a[keep], c[keep]) and a[3].isnan().all()
    dx, db = torch.empty_like(b), torch.empty_like(b)
    nsg.ns_block_norm_grad(clean[0], clean[1], b, got[0], db, dx, w, w)
    assert dx[3].isnan().all() and db[3].isnan().all() and dx[keep].isfinite().all() and db[keep].isfinite().all()
    ok()


@pytest.mark.parametrize("size", [1e-18, 1e-12, 1e12, 1e16])
def test_norms_at_the_ends_of_the_range(size):
    g = gen(9)
    T, D = 4, 2048
    b, x, dn = randn(g, T, D) * size, randn(g, T, D) * size, randn(g, T, D)
    h, n = torch.empty_like(b), torch.empty_like(b)
    nsg.ns_block_norm(b, x, h, n, branch_scale=size, eps=0.0)
    want_h, want_n = ob.block_norm(f64(b), f64(x), branch_scale=size, eps=0.0)
    assert np.abs(f64(h) - want_h).max() <= 4 * D * u * size * 6 and np.abs(f64(n) - want_n).max() <= 8 * D * u * 6
    db, dx = torch.empty_like(b), torch.empty_like(b)
    nsg.ns_block_norm_grad(None, dn, b, h, db, dx, branch_scale=size, eps=0.0)
    want = ob.block_norm_grad(np.zeros((T, D)), f64(dn), f64(b), f64(h), branch_scale=size, eps=0.0)
    for got, name in ((dx, "residual"), (db, "branch")):
        assert np.abs(f64(got) - want[name]).max() <= 16 * D * u * np.abs(want[name]).max()
    ok()


# --------------------------------------------- experts for a few tokens
FEW = [  # tokens, k, experts, dim, ffn
    (1, 1, 1, 1, 1), (1, 8, 64, 2048, 1408), (1, 2, 8, 264, 72), (3, 2, 4, 33, 17), (7, 2, 16, 1096, 712), (16, 8, 60, 512, 96),
    (9, 4, 4, 128, 64), (64, 6, 64, 256, 128), (65, 1, 1, 512, 40), (130, 3, 5, 136, 200), (256, 32, 33, 40, 24), (33, 8, 8, 1000, 300),
    (5, 3, 1024, 72, 56), (20, 1, 3, 2048, 8), (8, 2, 3, 8, 2000), (12, 2, 6, 130, 66), (40, 4, 2, 96, 32), (256, 8, 16, 64, 64),
]


def few_inputs(g, T, k, E, D, F, dtype, index=torch.int64, invalid=0.15):
    x = strided_rows(g, T, D, dtype, 0 if D % 3 else 8)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=index)
    ids[torch.rand(T, k, generator=g, device=DEV) < invalid] = -1
    w = randn(g, T, k)
    w.masked_fill_(ids < 0, NAN)                               # the weight of a slot that goes nowhere is not used
    up, down = (randn(g, E, 2 * F, D) / D ** 0.5).to(dtype), (randn(g, E, D, F) / F ** 0.5).to(dtype)
    named = torch.zeros(E, dtype=torch.bool, device=DEV)
    named[ids[ids >= 0].long()] = True
    up[~named], down[~named] = NAN, NAN                        # nor are experts that no token names
    return x, ids, w, up, down


def few_reference(x, ids, w, up, down):
    """(y, bound) in float64, slot by slot."""
    xv, iv, F = f64(x), ids.cpu().numpy(), down.shape[2]
    wv = np.ones(iv.shape) if w is None else f64(w)
    y, bound = np.zeros(xv.shape), np.zeros(xv.shape)
    D = xv.shape[1]
    for e in sorted(set(iv[(iv >= 0) & (iv < up.shape[0])].tolist())):
        U, Dn = f64(up[e]), f64(down[e])
        t, j = np.nonzero(iv == e)
        both, size = xv[t] @ U.T, 2 * (D + 16) * u * (np.abs(xv[t]) @ np.abs(U).T)
        a, b, da, db = both[:, :F], both[:, F:], size[:, :F], size[:, F:]
        silu = a / (1 + np.exp(-a))
        h = silu * b
        dh = 1.1 * da * (np.abs(b) + db) + np.abs(silu) * db + (8 * u + 2.0 ** -17) * np.abs(h)
        np.add.at(y, t, wv[t, j][:, None] * (h @ Dn.T))
        np.add.at(bound, t, np.abs(wv[t, j])[:, None] * (dh @ np.abs(Dn).T + (2 * (F + 16) + iv.shape[1] + 2) * u * (np.abs(h) @ np.abs(Dn).T)))
    return y, bound


def run_few(x, ids, w, up, down, stream=None, y=None):
    T, D = x.shape
    y = torch.full((T, D), NAN, dtype=x.dtype, device=DEV) if y is None else y
    ws = scratch(nsg.ns_moe_few_tokens_workspace_bytes(T, ids.shape[1], D, down.shape[2]))
    nsg.ns_moe_few_tokens(x, ids, w, up, down, y, ws, stream=stream)
    return y


@pytest.mark.parametrize("T,k,E,D,F", FEW)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_few_tokens(T, k, E, D, F, dtype, index):
    g = gen(T + D + F)
    x, ids, w, up, down = few_inputs(g, T, k, E, D, F, dtype, index)
    y = run_few(x, ids, w, up, down)
    ok()
    near(y, *few_reference(x, ids, w, up, down), dtype)
    assert torch.equal(y, run_few(x, ids, w, up, down))         # the same bits
    # without weights; y in place of x, whose rows may lie apart
    near(run_few(x, ids, None, up, down), *few_reference(x, ids, None, up, down), dtype)
    x2 = ops.same_place(x)
    assert torch.equal(run_few(x2, ids, w, up, down, y=x2), y)
    ok()


def test_few_tokens_that_go_nowhere():
    g = gen(3)
    x, ids, w, up, down = few_inputs(g, 6, 2, 4, 64, 32, bf16, invalid=0.0)
    ids[2], w[2] = -1, NAN
    x[2] = NAN                                                  # nor is their row
    y = run_few(x, ids, w, up, down)
    assert not y[2].any() and y[[0, 1, 3, 4, 5]].isfinite().all()
    ids[:] = -5
    assert not run_few(x, ids, w, up, down).any()
    assert run_few(x[:0], ids[:0], w[:0], up, down).shape == (0, 64)
    ok()


def test_few_tokens_refuse_ids_past_the_last_expert():
    g = gen(4)
    for index, far in ((torch.int64, 2 ** 40), (torch.int32, 2 ** 30)):
        x, ids, w, up, down = few_inputs(g, 3, 2, 4, 64, 32, fp32, index, invalid=0.0)
        good = ids.clone()
        ids[0, 1], ids[2, 0] = 4, far
        y = run_few(x, ids, w, up, down)
        assert nsg.ns_check_status() == nsg.NS_ERR_DEVICE_CHECK
        good[0, 1] = good[2, 0] = -1
        assert torch.equal(y, run_few(x, good, w, up, down))
        ok()


@pytest.mark.parametrize("dtype", TYPES)
def test_few_tokens_all_to_one_expert_twice(dtype):
    g = gen(6)
    x, ids, w, up, down = few_inputs(g, 70, 2, 3, 72, 40, dtype, invalid=0.0)
    ids[:] = 1
    up[[0, 2]], down[[0, 2]] = NAN, NAN
    up[1], down[1] = randn(g, 80, 72).to(dtype), randn(g, 72, 40).to(dtype)
    near(run_few(x, ids, w, up, down), *few_reference(x, ids, w, up, down), dtype)
    ok()


def test_few_tokens_hidden_values_past_the_types_range():
    # hidden values of 2.6e5 do not fit fp16; the result does
    x, ids = torch.full((2, 16), 8.0, dtype=fp16, device=DEV), torch.zeros(2, 1, dtype=torch.int64, device=DEV)
    up = torch.full((1, 16, 16), 4.0, dtype=fp16, device=DEV)
    down = torch.full((1, 16, 8), 2.0 ** -14, dtype=fp16, device=DEV)
    y = run_few(x, ids, None, up, down)
    want = 512.0 * 512.0 * 8 * 2.0 ** -14
    assert (y.double() - want).abs().max() <= want * 2.0 ** -11
    # and values far below: 2^-20 each
    x, up = torch.full((2, 16), 2.0 ** -10, dtype=fp16, device=DEV), torch.full((1, 16, 16), 1.0, dtype=fp16, device=DEV)
    a = 2.0 ** -6
    want = a / (1 + np.exp(-a)) * a * 8
    y = run_few(x, ids, None, up, torch.ones_like(down))
    assert (y.double() - want).abs().max() <= want * 2.0 ** -11 * 1.01
    ok()


def test_one_token_does_not_change_with_the_batch():
    # a NaN in a token's row reaches only that token
    g = gen(7)
    x, ids, w, up, down = few_inputs(g, 30, 3, 5, 200, 88, bf16, invalid=0.0)
    clean = run_few(x, ids, w, up, down)
    x[11] = NAN
    got = run_few(x, ids, w, up, down)
    keep = [t for t in range(30) if t != 11]
    assert torch.equal(got[keep], clean[keep]) and got[11].isnan().all()
    ok()


# ------------------------------------------------ streams, graphs, launches
def test_other_streams_and_graphs():
    g = gen(10)
    T, D, F, E, k = 24, 256, 96, 8, 2
    x, ids, w, up, down = few_inputs(g, T, k, E, D, F, bf16, invalid=0.0)
    b, p = randn(g, T, D, dtype=bf16), randn(g, D, dtype=bf16)
    bufs = {n: torch.empty(T, D, dtype=bf16, device=DEV) for n in ("h", "n", "y", "dx", "db")}
    dw, dp = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    norm = torch.empty(1, device=DEV)
    ws = [scratch(nsg.ns_moe_few_tokens_workspace_bytes(T, k, D, F)), scratch(nsg.ns_block_norm_grad_workspace_bytes(D)),
          scratch(nsg.ns_grad_norm_workspace_bytes(4))]
    outs = [torch.empty_like(t) for t in (bufs["dx"], bufs["db"], dw, dp)]

    def step(stream=None):
        grads = [bufs["dx"], bufs["db"], dw, dp]
        nsg.ns_block_norm(b, x, bufs["h"], bufs["n"], p, p, stream=stream)
        nsg.ns_moe_few_tokens(bufs["n"], ids, w, up, down, bufs["y"], ws[0], stream=stream)
        nsg.ns_block_norm_grad(bufs["y"], bufs["n"], b, bufs["h"], bufs["db"], bufs["dx"], p, p, None, dp, dw, None, ws[1], stream=stream)
        nsg.ns_grad_norm(grads, norm, ws[2], stream=stream)
        nsg.ns_grad_clip(grads, outs, norm, 0.5, stream=stream)

    def take():
        got = [t.clone() for t in (*bufs.values(), dw, dp, norm, *outs)]
        for t in (*bufs.values(), dw, dp, norm, *outs):
            t.fill_(9)
        torch.cuda.synchronize()
        return got

    step()
    want = take()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        step(s)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(take(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(take(), want))
    # new inputs in the same buffers
    x.copy_(randn(g, T, D, dtype=bf16))
    b.copy_(randn(g, T, D, dtype=bf16))
    graph.replay()
    got = take()
    step()
    assert all(torch.equal(a, c) for a, c in zip(got, take()))
    ok()


def test_launch_counts():
    nsg.ns_profile_read_blocks(reset=True)
    nsg.ns_profile_read_training(reset=True)
    x = torch.ones(4, 64, device=DEV)
    nsg.ns_block_norm(x, x, torch.empty_like(x), torch.empty_like(x))
    nsg.ns_grad_clip([x], [x], torch.ones(1, device=DEV), 1.0)
    assert nsg.ns_profile_read_blocks(reset=True)[0] == {"grad_norm": 1, "block_norm": 1}
    run_few(x, torch.zeros(4, 1, dtype=torch.int64, device=DEV), None, torch.ones(1, 32, 64, device=DEV), torch.ones(1, 64, 16, device=DEV))
    assert nsg.ns_profile_read_training(reset=True)[0]["moe"] == 3
    ok()
