"""The training-step operators against the float64 oracle.

Tolerances, element by element and stated before the first run. u = 2^-24 is
fp32's rounding, U the output type's (half its eps), tiny its smallest positive
value:

* copies (sort, dispatch) are exact;
* a sum of n products: (n + 2) u times the sum of the terms' magnitudes, plus
  U |value| + tiny for the store;
* norms: the mean of squares is a sum of D terms, the reciprocal square root and
  each factor add a few u: (D + 16) u relative;
* a log-sum-exp: terms come from a 2-ulp exp2 of an argument rounded at its
  size: (V / 128 + 32) u + 4 u max|s / tau| absolute; the loss adds the same for
  each unit of mass and 8 u for each of its terms' magnitudes; a gradient is its
  two terms, each with the log-sum-exp's relative error.
"""

import numpy as np
import pytest
import torch

from oracle import training as ot

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

DEV = "cuda"
u = 2.0 ** -24
ROUND = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -126}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.double().cpu().numpy()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def near(got, want, bound, dtype):
    got = f64(got)
    assert got.shape == want.shape
    lim = bound + ROUND[dtype] * (np.abs(want) + bound) + TINY[dtype]
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want) / np.maximum(lim, 1e-300))))


def same_place(t):
    """A copy with t's strides and alignment (what decides the kernel)."""
    return torch.empty(0, dtype=t.dtype, device=DEV).set_(t.untyped_storage().clone(), t.storage_offset(), t.size(), t.stride())


def status():
    return nsg.ns_check_status()


def strided_rows(g, n, d, dtype, extra, offset=0):
    """[n, d] with a row stride of d + extra, starting `offset` elements into its buffer."""
    buf = randn(g, n * (d + extra) + offset + 16).to(dtype)
    return buf[offset:offset + n * (d + extra)].view(n, d + extra)[:, :d]


# ------------------------------------------------------- tokens and experts
def run_sort(ids, E, align=1, capacity=0, extra_rows=0, stream=None):
    T, k = ids.shape
    rows = nsg.ns_moe_rows(T, k, E, align, capacity) + extra_rows
    out = [torch.full(s, -7, dtype=torch.int32, device=DEV) for s in ((T, k), (rows,), (E,), (E + 1,))]
    ws = torch.full((max(1, nsg.ns_moe_sort_workspace_bytes(T, k, E)),), 0x5A, dtype=torch.uint8, device=DEV)
    nsg.ns_moe_sort(ids, E, *out, ws, align=align, capacity=capacity, stream=stream)
    return out


SORTS = [  # tokens, k, experts, align, capacity, extra rows
    (0, 2, 4, 1, 0, 0), (0, 2, 4, 1, 0, 5), (1, 1, 1, 1, 0, 0), (1, 8, 8, 16, 0, 3), (7, 3, 5, 1, 0, 0),
    (33, 2, 1, 4, 10, 0), (64, 8, 1024, 8, 0, 0), (129, 5, 60, 1, 3, 7), (1000, 6, 64, 128, 0, 0),
    (2048, 1, 256, 1, 0, 0), (2049, 1, 3, 7, 500, 1), (5000, 8, 160, 16, 0, 0), (70001, 3, 64, 1, 2000, 0),
    (90000, 8, 1000, 2, 0, 9), (4096, 32, 33, 1, 0, 0),
]


@pytest.mark.parametrize("T,k,E,align,capacity,extra", SORTS)
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_sort(T, k, E, align, capacity, extra, index):
    g = gen(T + k)
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV, dtype=index)
    got = run_sort(ids, E, align, capacity, extra)
    want = ot.moe_sort(ids.cpu().numpy(), E, align, capacity, got[1].numel())
    assert status() == nsg.NS_OK
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_sort_one_expert_gets_all_and_none():
    for E, value in ((64, 5), (64, -1), (1024, 1023)):
        ids = torch.full((9000, 4), value, dtype=torch.int64, device=DEV)
        got = run_sort(ids, E, align=128)
        want = ot.moe_sort(ids.cpu().numpy(), E, 128, 0, got[1].numel())
        for a, b in zip(got, want):
            assert np.array_equal(a.cpu().numpy(), b)
    assert status() == nsg.NS_OK


def test_sort_refuses_ids_past_the_last_expert():
    ids = torch.tensor([[0, 4], [2 ** 40, 3]], device=DEV)
    row, slot, counts, _ = run_sort(ids, 4)
    assert status() == nsg.NS_ERR_DEVICE_CHECK and status() == nsg.NS_OK
    assert row.tolist() == [[0, -1], [-1, 1]] and slot.tolist() == [0, 3, -1, -1] and counts.tolist() == [1, 0, 0, 1]


ROWS = [  # tokens, k, experts, dim, align, capacity, extra stride, offset
    (1, 1, 1, 1, 1, 0, 0, 0), (1, 8, 16, 4096, 1, 0, 0, 0), (5, 2, 3, 8, 4, 0, 0, 0), (33, 6, 8, 1408, 16, 9, 0, 0),
    (40, 3, 4, 1001, 1, 0, 0, 0), (17, 32, 64, 96, 2, 0, 8, 0), (64, 4, 8, 264, 1, 12, 3, 1), (301, 6, 64, 2048, 8, 0, 0, 0),
    (9, 2, 4, 8200, 1, 0, 0, 0), (12, 5, 7, 130, 1, 0, 0, 2), (2500, 2, 16, 40, 1, 0, 0, 0),
]


def routed(g, T, k, E, align, capacity):
    ids = torch.randint(-1, E, (T, k), generator=g, device=DEV)
    row, slot, _, _ = run_sort(ids, E, align, capacity)
    return row, slot


@pytest.mark.parametrize("T,k,E,D,align,capacity,extra,offset", ROWS)
@pytest.mark.parametrize("dtype", TYPES)
def test_dispatch_and_gradient(T, k, E, D, align, capacity, extra, offset, dtype):
    g = gen(D)
    row, slot = routed(g, T, k, E, align, capacity)
    R = slot.numel()
    x = strided_rows(g, T, D, dtype, extra, offset)
    out = torch.full((R, D + extra), float("nan"), dtype=dtype, device=DEV)
    nsg.ns_moe_dispatch(x, row, slot, out[:, :D])
    r = row.cpu().numpy()
    assert np.array_equal(f64(out[:, :D]), ot.moe_dispatch(f64(x), r, R))
    assert extra == 0 or out[:, D:].isnan().all()
    gr = strided_rows(g, R, D, dtype, extra, offset)
    gr.masked_fill_((slot < 0)[:, None], float("nan"))          # rows without a slot are never read
    dx = torch.full((T, D), float("nan"), dtype=dtype, device=DEV)
    nsg.ns_moe_dispatch_grad(gr, row, dx)
    v = np.nan_to_num(f64(gr))
    near(dx, ot.moe_dispatch_grad(v, r), (k + 2) * u * ot.moe_dispatch_grad(np.abs(v), r), dtype)
    assert status() == nsg.NS_OK


@pytest.mark.parametrize("T,k,E,D,align,capacity,extra,offset", ROWS)
@pytest.mark.parametrize("dtype", TYPES)
def test_combine_and_gradient(T, k, E, D, align, capacity, extra, offset, dtype):
    g = gen(D + 1)
    row, slot = routed(g, T, k, E, align, capacity)
    R = slot.numel()
    ys = strided_rows(g, R, D, dtype, extra, offset)
    ys.masked_fill_((slot < 0)[:, None], float("nan"))
    w = randn(g, T, k)
    w.masked_fill_(row < 0, float("nan"))                       # nor is the weight of a dropped slot
    y = torch.full((T, D), float("nan"), dtype=dtype, device=DEV)
    nsg.ns_moe_combine(ys, w, row, y)
    r, yv, wv = row.cpu().numpy(), np.nan_to_num(f64(ys)), np.nan_to_num(f64(w))
    near(y, ot.moe_combine(yv, wv, r), (k + 2) * u * ot.moe_combine(np.abs(yv), np.abs(wv), r), dtype)

    dy = strided_rows(g, T, D, dtype, extra, offset)
    gr = torch.full((R, D + extra), float("nan"), dtype=dtype, device=DEV)
    dw = torch.full((T, k), float("nan"), device=DEV)
    nsg.ns_moe_combine_grad(dy, ys, w, row, slot, gr[:, :D], dw)
    want_r, want_w = ot.moe_combine_grad(f64(dy), yv, wv, r)
    near(gr[:, :D], want_r, 2 * u * np.abs(want_r), dtype)
    assert extra == 0 or gr[:, D:].isnan().all()
    near(dw, want_w, (D + 2) * u * ot.moe_combine_grad(np.abs(f64(dy)), np.abs(yv), wv, r)[1], torch.float32)
    # in place over the experts' rows
    if extra == 0 and offset == 0:
        again = ys.clone()
        dw2 = torch.empty_like(dw)
        nsg.ns_moe_combine_grad(dy, again, w, row, slot, again, dw2)
        assert torch.equal(again, gr) and torch.equal(dw2, dw)
    assert status() == nsg.NS_OK


def test_rows_outside_the_buffer_are_refused():
    g = gen(4)
    row = torch.tensor([[0, 9], [2, -1]], dtype=torch.int32, device=DEV)      # 9 is past the 3 rows
    slot = torch.tensor([0, -1, 2], dtype=torch.int32, device=DEV)
    x, ys = randn(g, 2, 8), randn(g, 3, 8)
    out = torch.full((3, 8), float("nan"), device=DEV)
    nsg.ns_moe_dispatch(x, row, slot, out)
    assert status() == nsg.NS_ERR_DEVICE_CHECK
    assert torch.equal(out, torch.stack([x[0], torch.zeros(8, device=DEV), x[1]]))
    y = torch.empty(2, 8, device=DEV)
    nsg.ns_moe_combine(ys, None, row, y)
    assert status() == nsg.NS_ERR_DEVICE_CHECK
    assert torch.equal(y, ys[[0, 2]])
    dw = torch.empty(2, 2, device=DEV)
    nsg.ns_moe_combine_grad(x, ys, torch.ones(2, 2, device=DEV), row, slot, torch.empty_like(ys), dw)
    assert status() == nsg.NS_ERR_DEVICE_CHECK and dw[0, 1] == 0 and dw[1, 1] == 0


def test_dispatch_and_its_gradient_are_adjoint():
    # <dispatch(x), g> = <x, dispatch_grad(g)> with whole numbers, exact in fp32
    g = gen(6)
    row, slot = routed(g, 200, 4, 16, 8, 30)
    x = torch.randint(-8, 9, (200, 72), generator=g, device=DEV).float()
    gr = torch.randint(-8, 9, (slot.numel(), 72), generator=g, device=DEV).float()
    out, dx = torch.empty_like(gr), torch.empty_like(x)
    nsg.ns_moe_dispatch(x, row, slot, out)
    nsg.ns_moe_dispatch_grad(gr, row, dx)
    assert (out.double() * gr.double()).sum() == (x.double() * dx.double()).sum()


# ------------------------------------------------------- queries and keys
def rotation_table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


QKS = [  # tokens, q heads, k heads, dim, rot, interleaved, weights, layout
    (1, 1, 1, 2, 2, False, True, "plain"), (1, 32, 8, 128, 128, False, True, "fused"),
    (3, 5, 1, 64, 32, True, True, "fused"), (17, 13, 13, 80, 32, True, True, "plain"),
    (9, 4, 2, 96, 96, False, False, "swapped"), (33, 3, 0, 256, 128, False, True, "plain"),
    (5, 0, 3, 112, 0, False, True, "plain"), (70, 6, 2, 72, 48, False, True, "fused"),
    (11, 2, 1, 33, 6, False, True, "plain"), (11, 2, 1, 33, 6, True, True, "plain"),
    (6, 3, 3, 1024, 512, False, True, "plain"), (130, 8, 2, 64, 64, False, True, "offset"),
    (50, 2, 2, 40, 20, True, False, "fused"), (257, 7, 7, 32, 32, True, True, "fused"),
    (19, 4, 4, 128, 64, False, True, "fused"),
]


def head_tensors(g, T, H, K, D, dtype, layout):
    if layout == "fused":
        qkv = randn(g, T, (H + 2 * K) * D, dtype=dtype)
        return qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + K) * D].view(T, K, D)
    if layout == "swapped":      # heads outermost
        return randn(g, H, T, D, dtype=dtype).transpose(0, 1), randn(g, K, T, D, dtype=dtype).transpose(0, 1)
    if layout == "offset":       # one element past an aligned address
        return (randn(g, T * H * D + 1, dtype=dtype)[1:].view(T, H, D), randn(g, T * K * D + 1, dtype=dtype)[1:].view(T, K, D))
    return randn(g, T, H, D, dtype=dtype), randn(g, T, K, D, dtype=dtype)


@pytest.mark.parametrize("T,H,K,D,rot,interleaved,weighted,layout", QKS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("weight_fp32", [False, True])
def test_qk_norm_rope_and_gradient(T, H, K, D, rot, interleaved, weighted, layout, dtype, weight_fp32):
    g = gen(D + T)
    eps = 1e-5
    q, k = head_tensors(g, T, H, K, D, dtype, layout)
    q[T // 2:T // 2 + 1] = 0                                    # a head of zeros has only eps to divide by
    table = rotation_table(100 + T, rot) if rot else None
    pos = torch.randint(0, 100 + T, (T,), generator=g, device=DEV, dtype=torch.int64 if D % 3 else torch.int32)
    wt = torch.float32 if weight_fp32 else dtype
    qw, kw = (randn(g, D).to(wt), randn(g, D).to(wt)) if weighted else (None, None)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    nsg.ns_qk_norm_rope(q, k, qo, ko, qw, kw, table, pos, eps=eps, interleaved=interleaved)
    gq, gk = head_tensors(g, T, H, K, D, dtype, layout)
    dq, dk = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    dqw, dkw = (torch.full((D,), float("nan"), device=DEV) for _ in range(2))
    ws = torch.full((nsg.ns_qk_norm_rope_grad_workspace_bytes(D),), 0xFF, dtype=torch.uint8, device=DEV)
    nsg.ns_qk_norm_rope_grad(gq, gk, q, k, dq, dk, qw, kw, dqw, dkw, table, pos, ws, eps=eps, interleaved=interleaved)
    assert status() == nsg.NS_OK
    tb, ps = (f64(table), pos.cpu().numpy()) if rot else (np.zeros((1, 0)), np.zeros(T, int))
    c = (D + 16) * u
    for x, y, dy, dx, w, dw in ((q, qo, gq, dq, qw, dqw), (k, ko, gk, dk, kw, dkw)):
        xv, dyv, wv = f64(x), f64(dy), f64(w) if weighted else np.ones(D)
        at = (tb, ps, rot, eps, interleaved)
        R_abs = np.abs(ot._rotation(tb, ps, rot, D, interleaved))
        r = 1 / np.sqrt((xv * xv).mean(-1, keepdims=True) + eps)
        n = np.abs(xv * r * wv)
        near(y, ot.norm_rope(xv, wv, *at), c * np.einsum("tab,thb->tha", R_abs, n), dtype)
        want_dx, want_dw = ot.norm_rope_grad(dyv, xv, wv, *at)
        ua = np.einsum("tab,tha->thb", R_abs, np.abs(dyv))
        h = ua * np.abs(wv)
        near(dx, want_dx, 2 * c * (r * h + np.abs(xv) * r ** 3 * (h * np.abs(xv)).mean(-1, keepdims=True)), dtype)
        near(dw, want_dw, ((T * x.shape[1] + 2) * u + c) * (ua * np.abs(xv) * r).sum((0, 1)), torch.float32)
    # in place, and without the weights' gradients
    q2, k2 = same_place(q), same_place(k)
    nsg.ns_qk_norm_rope(q2, k2, q2, k2, qw, kw, table, pos, eps=eps, interleaved=interleaved)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    g2, h2 = same_place(gq), same_place(gk)
    nsg.ns_qk_norm_rope_grad(g2, h2, q, k, g2, h2, qw, kw, table=table, positions=pos, eps=eps, interleaved=interleaved)
    assert torch.equal(g2, dq) and torch.equal(h2, dk)
    assert status() == nsg.NS_OK


def test_qk_neighbours_of_strided_outputs_are_untouched():
    g = gen(2)
    T, H, K, D = 21, 6, 2, 64
    q, k = head_tensors(g, T, H, K, D, torch.bfloat16, "fused")
    buf = torch.full((T, (H + 2 * K) * D), 3.0, dtype=torch.bfloat16, device=DEV)
    nsg.ns_qk_norm_rope(q, k, buf[:, :H * D].view(T, H, D), buf[:, H * D:(H + K) * D].view(T, K, D),
                        table=rotation_table(T, D))
    assert status() == nsg.NS_OK
    assert (buf[:, (H + K) * D:] == 3.0).all()


@pytest.mark.parametrize("D", [64, 33])
def test_qk_positions_outside_the_table_are_refused(D):
    g = gen(3)
    rot = 32 if D == 64 else 6
    q, k = randn(g, 4, 2, D), randn(g, 4, 1, D)
    table = rotation_table(10, rot)
    pos = torch.tensor([1, 10, -1, 9], device=DEV)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    nsg.ns_qk_norm_rope(q, k, qo, ko, table=table, positions=pos)
    assert status() == nsg.NS_ERR_DEVICE_CHECK
    assert (qo[1:3] == 7).all() and (ko[1:3] == 7).all() and (qo[[0, 3]] != 7).any()
    dw = torch.empty(D, device=DEV)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    dq, dk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    nsg.ns_qk_norm_rope_grad(q, k, q, k, dq, dk, grad_q_weight=dw, table=table, positions=pos, workspace=ws)
    assert status() == nsg.NS_ERR_DEVICE_CHECK
    assert (dq[1:3] == 7).all() and (dk[1:3] == 7).all()
    keep = [0, 3]
    want = ot.norm_rope_grad(f64(q[keep]), f64(q[keep]), np.ones(D), f64(table), np.array([1, 9]), rot, 1e-6, False)[1]
    assert np.abs(f64(dw) - want).max() <= (D + 32) * u * np.abs(f64(q)).sum((0, 1)).max() * 4


# ------------------------------------------------------------ distillation
DISTILLS = [  # tokens, vocab, top, temperature, full, extra stride, offset
    (1, 1, 1, 1.0, False, 0, 0), (3, 7, 7, 2.0, False, 0, 0), (1, 131072, 64, 1.0, False, 0, 0),
    (5, 50001, 20, 0.7, True, 0, 0), (17, 1000, 128, 1.0, False, 24, 0), (9, 4099, 33, 1.5, False, 5, 3),
    (4, 8192, 1024, 1.0, True, 0, 0), (300, 513, 8, 1.0, False, 0, 1), (2, 250007, 100, 3.0, False, 1, 0),
    (40, 32000, 16, 0.25, False, 0, 0),
]


def distill_inputs(g, T, V, K, tau, full, dtype, extra=0, offset=0):
    logits = strided_rows(g, T, V, dtype, extra, offset)
    ids = torch.randint(0, V, (T, K), generator=g, device=DEV)        # some entries are named twice
    values = (3 * randn(g, T, K)).to(dtype)
    drop = torch.rand(T, K, generator=g, device=DEV)
    ids[drop < 0.1] = -1
    values[drop < 0.1] = float("nan")                                 # what a left-out entry holds does not matter
    values[(drop > 0.1) & (drop < 0.15)] = float("-inf")
    ids[T // 3] = -1 if T > 2 else ids[T // 3]                        # a row with no entry left
    weights = torch.rand(T, generator=g, device=DEV) + 0.5
    if T > 2:
        weights[T - 1] = 0
        logits[T - 1] = float("nan")                                  # ignored with its weight
    tl = None
    if full:
        z = torch.where(ids >= 0, values.float() / tau, torch.full((), float("-inf"), device=DEV))
        tl = torch.logsumexp(z, 1).clamp(min=-100) + 0.1
    return logits, values, ids, weights, tl


@pytest.mark.parametrize("T,V,K,tau,full,extra,offset", DISTILLS)
@pytest.mark.parametrize("dtype", TYPES)
def test_distill(T, V, K, tau, full, extra, offset, dtype):
    g = gen(V)
    logits, values, ids, weights, tl = distill_inputs(g, T, V, K, tau, full, dtype, extra, offset)
    loss, lse, loss2, lse2 = (torch.full((T,), float("nan"), device=DEV) for _ in range(4))
    grad = torch.full((T, V + extra), float("nan"), dtype=dtype, device=DEV)
    args = dict(weights=weights, teacher_lse=tl, temperature=tau)
    nsg.ns_distill_loss(logits, values, ids, loss2, lse2, **args)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad[:, :V], **args)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    assert extra == 0 or grad[:, V:].isnan().all()
    later = torch.full((T, V), float("nan"), dtype=dtype, device=DEV)
    nsg.ns_distill_grad(logits, values, ids, lse, later, **args)
    assert status() == nsg.NS_OK

    s, z, iv, wv = f64(logits), f64(values), ids.cpu().numpy(), f64(weights)
    tlv = None if tl is None else f64(tl)
    want_loss, want_lse, want_grad = ot.distill(s, np.where(iv >= 0, z, 0), iv, wv, tlv, tau)
    p = ot.teacher_probabilities(np.where(iv >= 0, z, 0), iv, tlv, tau)
    live = (wv != 0) & (p > 0).any(1)
    s = np.where(live[:, None], s, 0)
    e = (V / 128 + 32) * u + 4 * u * np.abs(s / tau).max(1)           # of the log-sum-exp
    ep = 32 * u + 4 * u * np.abs(np.where(p > 0, z, 0) / tau).max(1) + (0 if tl is None else 4 * u * np.abs(tlv))  # of log p
    near(lse, want_lse, np.where(live, e, 0), torch.float32)
    terms = np.zeros(T)
    for j in range(K):
        logp = np.log(np.where(p[:, j] > 0, p[:, j], 1))
        at = s[np.arange(T), np.maximum(iv[:, j], 0)] / tau
        terms += p[:, j] * (np.abs(logp) + np.abs(at) + np.abs(want_lse))
    near(loss, want_loss, wv * live * (p.sum(1) * (e + ep) + (ep + 8 * u + K * u) * terms), torch.float32)
    q = np.exp(s / tau - want_lse[:, None])
    q[~live] = 0
    scale = (wv / tau)[:, None]
    pv = np.zeros((T, V))
    for j in range(K):
        np.add.at(pv, (np.arange(T), np.maximum(iv[:, j], 0)), p[:, j])
    bound = scale * (2 * (e + ep + 16 * u)[:, None] * p.sum(1)[:, None] * q + 2 * (ep + (K + 4) * u)[:, None] * pv)
    near(grad[:, :V], want_grad, bound, dtype)
    near(later, want_grad, bound, dtype)
    # over the logits themselves
    if offset == 0 and extra == 0:
        over = logits.clone()
        nsg.ns_distill_loss(over, values, ids, loss2, lse2, grad_logits=over, **args)
        assert torch.equal(over, grad) and torch.equal(loss, loss2)
        over = logits.clone()
        nsg.ns_distill_grad(over, values, ids, lse, over, **args)
        assert torch.equal(over, later)
    assert status() == nsg.NS_OK


@pytest.mark.parametrize("dtype", TYPES)
def test_distill_masked_vocabulary(dtype):
    # entries masked with -inf or the type's lowest value have probability and gradient 0
    g = gen(1)
    T, V, K = 6, 1003, 4
    logits = randn(g, T, V, dtype=dtype)
    logits[:, 500:] = float("-inf")
    logits[1, :499] = torch.finfo(dtype).min
    logits[2, 1:] = float("-inf")                              # one entry carries everything
    ids = torch.randint(0, 499, (T, K), generator=g, device=DEV, dtype=torch.int32)
    ids[1], ids[2] = 499, 0
    values = randn(g, T, K).to(dtype)
    values[3, 1:] = torch.finfo(dtype).min
    values[4] = torch.finfo(dtype).min                         # equal, if absurd: uniform
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    for tau in (1.0, 0.5):
        grad = torch.full((T, V), float("nan"), dtype=dtype, device=DEV)
        nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad, temperature=tau)
        assert status() == nsg.NS_OK
        want_loss, want_lse, want_grad = ot.distill(f64(logits), f64(values), ids.cpu().numpy(), None, None, tau)
        assert (grad[:, 500:] == 0).all() and (grad[1, :499] == 0).all()
        assert np.isfinite(f64(loss)).all()
        assert np.abs(f64(lse) - want_lse).max() <= 64 * u * (1 + np.abs(want_lse).max())
        assert np.abs(f64(loss) - want_loss).max() <= 256 * u * (1 + np.abs(want_loss).max())
        near(grad, want_grad, 256 * u * np.ones_like(want_grad), dtype)


def test_distill_nan_stays_in_its_row():
    g = gen(5)
    logits, values, ids, _, _ = distill_inputs(g, 2, 3000, 4, 1.0, False, torch.float32)
    ids.clamp_(min=0)
    values = randn(g, 2, 4)
    logits[0, 2999] = float("nan")
    loss, lse, grad = torch.empty(2, device=DEV), torch.empty(2, device=DEV), torch.empty(2, 3000, device=DEV)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad)
    assert loss[0].isnan() and lse[0].isnan() and loss[1].isfinite() and grad[1].isfinite().all()


def test_distill_refuses_ids_past_the_vocabulary():
    g = gen(7)
    logits, values = randn(g, 2, 50), randn(g, 2, 3)
    ids = torch.tensor([[1, 50, 2], [3, 2 ** 33, 4]], device=DEV)
    loss, lse, grad = torch.empty(2, device=DEV), torch.empty(2, device=DEV), torch.empty(2, 50, device=DEV)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad)
    assert status() == nsg.NS_ERR_DEVICE_CHECK
    ids[:, 1] = -1
    loss2, grad2 = torch.empty_like(loss), torch.empty_like(grad)
    nsg.ns_distill_loss(logits, values, ids, loss2, lse, grad_logits=grad2)
    assert status() == nsg.NS_OK and torch.equal(loss, loss2) and torch.equal(grad, grad2)


def test_distill_gradient_against_differences():
    # loss(s + h d) - loss(s - h d) over 2 h against <grad, d>, fp32, per token: truncation h^2 |f'''| / 6 with
    # |f'''| <= 2 max|d|^3, rounding of the two losses 2 e / (2 h)
    g = gen(9)
    T, V, K, h = 8, 700, 6, 2.0 ** -5
    logits, values = randn(g, T, V), randn(g, T, K)
    ids = torch.randint(0, V, (T, K), generator=g, device=DEV)
    d = torch.rand(T, V, generator=g, device=DEV) * 2 - 1

    def loss_at(x, grad=None):
        loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        nsg.ns_distill_loss(x, values, ids, loss, lse, grad_logits=grad)
        return loss.double()

    grad = torch.empty(T, V, device=DEV)
    loss_at(logits, grad)
    slope = (loss_at(logits + h * d) - loss_at(logits - h * d)) / (2 * h)
    assert (slope - (grad.double() * d.double()).sum(1)).abs().max().item() <= h * h / 3 + 100 * u * 10 / h


# ------------------------------------------------- streams, graphs, sizes
def test_another_stream_and_a_graph():
    g = gen(11)
    T, k, E, D = 700, 4, 16, 256
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV)
    x, w = randn(g, T, D, dtype=torch.bfloat16), torch.rand(T, k, generator=g, device=DEV)
    row, slot, counts, off = run_sort(ids, E)
    R = slot.numel()
    xs, y = torch.empty(R, D, dtype=torch.bfloat16, device=DEV), torch.empty_like(x)
    ws = torch.empty(max(1, nsg.ns_moe_sort_workspace_bytes(T, k, E)), dtype=torch.uint8, device=DEV)
    logits, values, tid = randn(g, 9, 5000), randn(g, 9, 4), torch.randint(0, 5000, (9, 4), generator=g, device=DEV)
    loss, lse, grad = torch.empty(9, device=DEV), torch.empty(9, device=DEV), torch.empty(9, 5000, device=DEV)
    q, kk = randn(g, 33, 4, 64), randn(g, 33, 2, 64)
    qo, ko, dqw = torch.empty_like(q), torch.empty_like(kk), torch.empty(64, device=DEV)
    table = rotation_table(40, 64)
    qws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    dq, dk = torch.empty_like(q), torch.empty_like(kk)

    def step(stream=None):
        nsg.ns_moe_sort(ids, E, row, slot, counts, off, ws, stream=stream)
        nsg.ns_moe_dispatch(x, row, slot, xs, stream=stream)
        nsg.ns_moe_combine(xs, w, row, y, stream=stream)
        nsg.ns_distill_loss(logits, values, tid, loss, lse, grad_logits=grad, stream=stream)
        nsg.ns_qk_norm_rope(q, kk, qo, ko, table=table, stream=stream)
        nsg.ns_qk_norm_rope_grad(qo, ko, q, kk, dq, dk, grad_q_weight=dqw, table=table, workspace=qws, stream=stream)

    outs = [row, slot, xs, y, loss, grad, qo, ko, dq, dk, dqw]
    step()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in outs:
        t.zero_()
    x.mul_(2)                       # a replay reads what the buffers hold now
    graph.replay()
    torch.cuda.synchronize()
    assert status() == nsg.NS_OK
    assert torch.equal(y, (want[3].float() * 2).to(y.dtype))
    assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(outs, want)) if i not in (2, 3))


def test_offsets_past_32_bits():
    # rows beyond the 2^32nd byte and the 2^31st element of their buffers
    T, V = 17, 1 << 27
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device=DEV)
    ids = torch.full((T, 1), V - 1, device=DEV)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    logits[T - 1, V - 1] = 10.0
    nsg.ns_distill_loss(logits, torch.zeros(T, 1, device=DEV), ids, loss, lse, grad_logits=logits)
    assert status() == nsg.NS_OK
    want = np.log(V)
    assert abs(loss[0].item() - want) < 1e-4 and abs(loss[T - 1].item() - (np.log(V - 1 + np.exp(10.0)) - 10)) < 1e-4
    assert logits[T - 1, V - 1].item() == pytest.approx(np.exp(10.0) / (V - 1 + np.exp(10.0)) - 1, abs=0.01)
    del logits
    R, D = 70000, 32768
    src = torch.zeros(R, D, dtype=torch.bfloat16, device=DEV)
    src[R - 1] = 2.0
    row = torch.tensor([[R - 1, 0]], dtype=torch.int32, device=DEV)
    y = torch.empty(1, D, dtype=torch.bfloat16, device=DEV)
    nsg.ns_moe_combine(src, None, row, y)
    assert status() == nsg.NS_OK and (y == 2.0).all()
    x = src[R - 1:].clone()
    slot = torch.full((R,), -1, dtype=torch.int32, device=DEV)
    slot[R - 1], slot[0] = 0, 1
    src.fill_(5.0)
    nsg.ns_moe_dispatch(x, row, slot, src)
    assert status() == nsg.NS_OK
    assert (src[R - 1] == 2.0).all() and (src[0] == 2.0).all() and not src[1:R - 1].any()


def test_same_call_twice_gives_the_same_bits():
    g = gen(13)
    T, k, E, D = 3000, 6, 64, 512
    row, slot = routed(g, T, k, E, 1, 0)
    ys, dy, w = randn(g, slot.numel(), D), randn(g, T, D), randn(g, T, k)
    q, kk, gq, gk = randn(g, T, 8, 64), randn(g, T, 2, 64), randn(g, T, 8, 64), randn(g, T, 2, 64)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    seen = []
    for _ in range(2):
        y, gr, dw = torch.empty_like(dy), torch.empty_like(ys), torch.empty_like(w)
        nsg.ns_moe_combine(ys, w, row, y)
        nsg.ns_moe_combine_grad(dy, ys, w, row, slot, gr, dw)
        dq, dk, dqw, dkw = torch.empty_like(q), torch.empty_like(kk), torch.empty(64, device=DEV), torch.empty(64, device=DEV)
        nsg.ns_qk_norm_rope_grad(gq, gk, q, kk, dq, dk, grad_q_weight=dqw, grad_k_weight=dkw, table=rotation_table(T, 64), workspace=ws)
        seen.append([y, gr, dw, dq, dk, dqw, dkw])
    assert all(torch.equal(a, b) for a, b in zip(*seen))
