"""The training-step operators at the edges of their domains: nothing to do,
odd rotations, rows too long for shared memory, many teacher entries, calls on
the same buffers in a row. Against the float64 oracle; tolerances as in
test_gpu_training_ops.py (u = 2^-24, U half the output type's eps)."""

import subprocess
import sys
from pathlib import Path

import numpy as np
import pytest
import torch

import test_gpu_training_ops as ops
from oracle import training as ot

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

DEV = "cuda"
u = 2.0 ** -24


def f64(t):
    return t.double().cpu().numpy()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


def empty(*shape, dtype=torch.float32):
    return torch.full(shape, 5, dtype=dtype, device=DEV)


def ok():
    assert nsg.ns_check_status() == nsg.NS_OK


def test_nothing_to_do():
    i32 = torch.int32
    row, slot, counts, off = empty(0, 2, dtype=i32), empty(0, dtype=i32), empty(3, dtype=i32), empty(4, dtype=i32)
    nsg.ns_moe_sort(torch.empty(0, 2, dtype=torch.int64, device=DEV), 3, row, slot, counts, off, None)
    assert counts.tolist() == [0, 0, 0] and off.tolist() == [0, 0, 0, 0]
    nsg.ns_moe_dispatch(empty(0, 8), row, slot, empty(0, 8))
    nsg.ns_moe_dispatch_grad(empty(0, 8), row, empty(0, 8))
    nsg.ns_moe_combine(empty(0, 8), empty(0, 2), row, empty(0, 8))
    nsg.ns_moe_combine_grad(empty(0, 8), empty(0, 8), empty(0, 2), row, slot, empty(0, 8), empty(0, 2))
    # tokens, but no rows: everything was dropped
    none = torch.full((3, 2), -1, dtype=i32, device=DEV)
    y, dw = empty(3, 8), empty(3, 2)
    nsg.ns_moe_combine(empty(0, 8), empty(3, 2), none, y)
    nsg.ns_moe_combine_grad(empty(3, 8), empty(0, 8), empty(3, 2), none, slot, empty(0, 8), dw)
    assert not y.any() and not dw.any()
    # rows, but no tokens: all of them are padding
    rows = empty(5, 8)
    nsg.ns_moe_dispatch(empty(0, 8), row, torch.full((5,), -1, dtype=i32, device=DEV), rows)
    assert not rows.any()
    e, dqw = empty(0, 2, 8), empty(8)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(8), dtype=torch.uint8, device=DEV)
    nsg.ns_qk_norm_rope(e, e, e, e)
    nsg.ns_qk_norm_rope_grad(e, e, e, e, e, e, grad_q_weight=dqw, workspace=ws)
    assert not dqw.any()
    nsg.ns_distill_loss(empty(0, 9), empty(0, 2), torch.empty(0, 2, dtype=torch.int64, device=DEV), empty(0), empty(0))
    ok()


ROTATIONS = [  # dim, rot, interleaved
    (128, 34, False), (128, 34, True), (72, 72, False), (72, 36, False), (72, 38, True), (40, 40, False), (8, 2, False),
    (8, 6, True), (16, 14, False), (112, 112, False), (112, 50, True), (24, 24, False), (192, 130, False), (256, 250, True),
    (512, 510, False), (160, 160, False), (64, 2, True),
]


@pytest.mark.parametrize("D,rot,interleaved", ROTATIONS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,K", [(37, 5, 2), (300, 3, 3)])
def test_rotations_of_any_even_width(D, rot, interleaved, dtype, T, H, K):
    g = gen(D + rot)
    q, k, gq, gk = randn(g, T, H, D, dtype=dtype), randn(g, T, K, D, dtype=dtype), randn(g, T, H, D, dtype=dtype), randn(g, T, K, D, dtype=dtype)
    qw, kw = randn(g, D, dtype=dtype), randn(g, D, dtype=dtype)
    angle = torch.rand(T + 9, rot // 2, generator=g, device=DEV, dtype=torch.float64) * 6
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    pos = torch.randint(0, T + 9, (T,), generator=g, device=DEV)
    qo, ko, dq, dk = (torch.full_like(t, float("nan")) for t in (q, k, q, k))
    dqw, dkw = empty(D), empty(D)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(D), dtype=torch.uint8, device=DEV)
    nsg.ns_qk_norm_rope(q, k, qo, ko, qw, kw, table, pos, interleaved=interleaved)
    nsg.ns_qk_norm_rope_grad(gq, gk, q, k, dq, dk, qw, kw, dqw, dkw, table, pos, ws, interleaved=interleaved)
    ok()
    U, tiny, c = torch.finfo(dtype).eps / 2, float(torch.finfo(dtype).tiny) * float(torch.finfo(dtype).eps), (D + 16) * u
    at = (f64(table), pos.cpu().numpy(), rot, 1e-6, interleaved)
    R = np.abs(ot._rotation(at[0], at[1], rot, D, interleaved))
    for x, y, dy, dx, w, dw in ((q, qo, gq, dq, qw, dqw), (k, ko, gk, dk, kw, dkw)):
        xv, dyv, wv = f64(x), f64(dy), f64(w)
        r = 1 / np.sqrt((xv * xv).mean(-1, keepdims=True) + 1e-6)
        want, bound = ot.norm_rope(xv, wv, *at), c * np.einsum("tab,thb->tha", R, np.abs(xv * r * wv))
        assert (np.abs(f64(y) - want) <= bound + U * (np.abs(want) + bound) + tiny).all()
        want, want_w = ot.norm_rope_grad(dyv, xv, wv, *at)
        ua = np.einsum("tab,tha->thb", R, np.abs(dyv))
        h = ua * np.abs(wv)
        bound = 2 * c * (r * h + np.abs(xv) * r ** 3 * (h * np.abs(xv)).mean(-1, keepdims=True))
        assert (np.abs(f64(dx) - want) <= bound + U * (np.abs(want) + bound) + tiny).all()
        assert (np.abs(f64(dw) - want_w) <= ((T * x.shape[1] + 2) * u + c) * (ua * np.abs(xv) * r).sum((0, 1)) + u).all()


# Many heads, so that the same warps take queries and then keys: heads of an odd
# number of 16-byte words (3, 9, 5) beside one of an even number.
MANY_HEADS = [  # T, H, K, dim, rot, interleaved, dtype
    (100, 2000, 1500, 24, 16, False, torch.bfloat16), (100, 2000, 1500, 24, 24, True, torch.float16),
    (100, 2000, 1500, 24, 24, False, torch.bfloat16), (100, 2000, 1500, 12, 8, False, torch.float32),
    (100, 2000, 1500, 12, 12, False, torch.float32), (100, 800, 900, 72, 64, False, torch.bfloat16),
    (100, 1200, 1300, 40, 16, False, torch.float16), (100, 1000, 800, 64, 64, False, torch.bfloat16),
]


@pytest.mark.parametrize("T,H,K,D,rot,interleaved,dtype", MANY_HEADS)
def test_rotations_of_many_heads(T, H, K, D, rot, interleaved, dtype):
    test_rotations_of_any_even_width(D, rot, interleaved, dtype, T, H, K)


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 900001), (torch.float32, 450000)])
def test_rows_too_long_for_a_cluster(dtype, V):
    g = gen(V)
    T, K = 3, 9
    logits = randn(g, T, V, dtype=dtype)
    ids, values = torch.randint(0, V, (T, K), generator=g, device=DEV), randn(g, T, K)
    ids[0, 1], ids[1] = ids[0, 0], -1
    loss, lse, grad, later = empty(T), empty(T), empty(T, V, dtype=dtype), empty(T, V, dtype=dtype)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad, temperature=0.8)
    nsg.ns_distill_grad(logits, values, ids, lse, later, temperature=0.8)
    ok()
    want_loss, want_lse, want = ot.distill(f64(logits), f64(values), ids.cpu().numpy(), None, None, 0.8)
    e = (V / 128 + 64) * u
    assert np.abs(f64(lse) - want_lse).max() <= e * 20 and np.abs(f64(loss) - want_loss).max() <= e * 40
    U = torch.finfo(dtype).eps / 2
    for got in (grad, later):
        assert (np.abs(f64(got) - want) <= U * np.abs(want) + 4 * e * (np.abs(want) + 1e-3)).all()


# Every entry's gradient where a warp that enters the ids also computes, and
# where it has to be done before a short row is.
@pytest.mark.parametrize("dtype,V,K", [(torch.float32, 512296, 1024), (torch.bfloat16, 1011385, 1024), (torch.float16, 830001, 200),
                                       (torch.bfloat16, 1200, 1024), (torch.float32, 50021, 1000), (torch.bfloat16, 151, 129)])
def test_gradients_of_many_entries(dtype, V, K):
    g = gen(V)
    T = 5
    logits = randn(g, T, V, dtype=dtype)
    ids, values = torch.randint(0, V, (T, K), generator=g, device=DEV), randn(g, T, K)
    loss, lse, grad, later = empty(T), empty(T), empty(T, V, dtype=dtype), empty(T, V, dtype=dtype)
    nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad, temperature=0.8)
    nsg.ns_distill_grad(logits, values, ids, lse, later, temperature=0.8)
    ok()
    want_loss, want_lse, want = ot.distill(f64(logits), f64(values), ids.cpu().numpy(), None, None, 0.8)
    e = (V / 128 + 64) * u
    assert np.abs(f64(lse) - want_lse).max() <= e * 20 and np.abs(f64(loss) - want_loss).max() <= e * 40
    U = torch.finfo(dtype).eps / 2
    sums = np.zeros((T, V))                                     # what is subtracted: its sum in fp32 has its own error
    p = np.exp(f64(values) / 0.8)
    np.add.at(sums, (np.arange(T)[:, None], ids.cpu().numpy()), p / p.sum(1, keepdims=True) / 0.8)
    for got in (grad, later):
        assert (np.abs(f64(got) - want) <= U * np.abs(want) + 4 * e * (np.abs(want) + sums + 1e-6) + 2.0 ** -25).all()
    again = logits.clone()
    nsg.ns_distill_loss(again, values, ids, loss, lse, grad_logits=again, temperature=0.8)
    ok()
    assert torch.equal(again, grad)


def test_the_most_teacher_entries_with_every_one_repeated():
    g = gen(3)
    T, V, K = 5, 2000, 1024
    logits, values = randn(g, T, V), randn(g, T, K)
    ids = torch.randint(0, 300, (T, K), generator=g, device=DEV, dtype=torch.int32)
    ids[4] = 7                                             # one entry, 1024 times
    loss, lse, grad = empty(T), empty(T), empty(T, V)
    for _ in range(2):                                     # the second call finds the first one's outputs
        nsg.ns_distill_loss(logits, values, ids, loss, lse, grad_logits=grad)
    ok()
    want_loss, want_lse, want = ot.distill(f64(logits), f64(values), ids.cpu().numpy())
    assert np.abs(f64(loss) - want_loss).max() <= 1100 * u * 16
    assert np.abs(f64(grad) - want).max() <= 1100 * u


def test_other_weights_later():
    g = gen(4)
    T, V, K = 6, 3001, 8
    logits, values, ids = randn(g, T, V), randn(g, T, K), torch.randint(0, V, (T, K), generator=g, device=DEV)
    w = torch.tensor([1.0, -2.0, 0.0, 3.0, 0.5, 0.0], device=DEV)
    loss, lse, grad = empty(T), empty(T), empty(T, V)
    nsg.ns_distill_loss(logits, values, ids, loss, lse)     # weights 1
    nsg.ns_distill_grad(logits, values, ids, lse, grad, weights=w)
    ok()
    want = ot.distill(f64(logits), f64(values), ids.cpu().numpy(), f64(w))[2]
    assert np.abs(f64(grad) - want).max() <= 64 * u * 3
    assert not grad[2].any() and not grad[5].any()


def test_infinite_weights_and_rows_stay_where_they_are():
    # an infinity in one expert row or weight reaches only the tokens that use it
    row = torch.tensor([[0, 1], [2, 3], [-1, 4]], dtype=torch.int32, device=DEV)
    slot = torch.tensor([0, 1, 2, 3, 5], dtype=torch.int32, device=DEV)
    ys, w = torch.ones(5, 16, device=DEV), torch.ones(3, 2, device=DEV)
    ys[0, 3], w[1, 0] = float("inf"), float("inf")
    y = empty(3, 16)
    nsg.ns_moe_combine(ys, w, row, y)
    assert y[0, 3].isinf() and (y[0, 4:] == 2).all() and y[1].isinf().all() and (y[2] == 1).all()
    grad_rows, dw = empty(5, 16), empty(3, 2)
    nsg.ns_moe_combine_grad(torch.ones(3, 16, device=DEV), ys, w, row, slot, grad_rows, dw)
    ok()
    assert dw[0, 0].isinf() and dw[0, 1] == 16 and dw[2].tolist() == [0, 16]
    assert grad_rows[2].isinf().all() and (grad_rows[[0, 1, 3, 4]] == 1).all()


FEW_ROWS = [  # tokens, k, dim: on both sides of the limits at which a lane takes more of a row
    (2500, 1, 2048), (2500, 4, 776), (2500, 2, 768), (2500, 5, 1032), (2400, 4, 1024), (2431, 3, 392), (2440, 4, 384),
    (61, 1, 481), (61, 2, 480), (61, 2, 962), (61, 1, 960), (61, 3, 1023), (61, 2, 1541), (61, 1, 3001), (700, 2, 2046),
]


@pytest.mark.parametrize("T,k,D", FEW_ROWS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sums_of_few_rows(T, k, D, dtype):
    g = gen(T + k + D)
    R = T * k + 5
    row = torch.randint(-1, R, (T, k), generator=g, device=DEV, dtype=torch.int32)
    ys, w = randn(g, R, D, dtype=dtype), randn(g, T, k)
    y, dx = (torch.full((T, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    nsg.ns_moe_combine(ys, w, row, y)
    nsg.ns_moe_dispatch_grad(ys, row, dx)
    ok()
    r, v, wv = row.cpu().numpy(), f64(ys), f64(w)
    U, tiny = torch.finfo(dtype).eps / 2, float(torch.finfo(dtype).tiny) * float(torch.finfo(dtype).eps)
    for got, want, size in ((y, ot.moe_combine(v, wv, r), ot.moe_combine(np.abs(v), np.abs(wv), r)),
                            (dx, ot.moe_dispatch_grad(v, r), ot.moe_dispatch_grad(np.abs(v), r))):
        assert (np.abs(f64(got) - want) <= (k + 2) * u * size + U * np.abs(want) * (1 + 1e-6) + tiny + U * (k + 2) * u * size).all()


# Widths on both sides of those at which a lane takes more words of a row.
@pytest.mark.parametrize("D", [256, 264, 512, 520, 64, 66, 128, 130, 258, 32, 33, 65, 129, 124, 132])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("k", [2, 5])
def test_rows_of_few_words(D, dtype, k):
    ops.test_combine_and_gradient(41, k, 6, D, 4, 0, 0, 0, dtype)
    ops.test_dispatch_and_gradient(41, k, 6, D, 4, 0, 0, 0, dtype)


# Few tokens whose rows many warps share, and one or two slots of long rows.
@pytest.mark.parametrize("T,k,D", [(13, 8, 3761), (7, 3, 6402), (1, 8, 4104), (3, 32, 5001), (9, 2, 8192), (650, 1, 1001), (650, 2, 1002), (650, 2, 483)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("align", [1, 16])
def test_gradients_of_long_rows(T, k, D, dtype, align):
    ops.test_combine_and_gradient(T, k, 6, D, align, 0, 0, 0, dtype)


FIRST_CALLS = {  # dynamic shared memory just below 48 KB, which the static part takes past it
    "distill": "V, K = 192289, 32\n"
               "x, z, ids = torch.randn(2, V, device='cuda').half(), torch.randn(2, K, device='cuda'), torch.zeros(2, K, dtype=torch.int64, device='cuda')\n"
               "out = torch.empty(2, 2, device='cuda')\n"
               "nsg.ns_distill_loss(x, z, ids, out[0], out[1], grad_logits=torch.empty_like(x))\n",
    "sort": "E = 646\n"
            "ids = torch.arange(64, device='cuda').view(32, 2)\n"
            "i = [torch.empty(n, dtype=torch.int32, device='cuda') for n in (64, 64, E, E + 1)]\n"
            "nsg.ns_moe_sort(ids, E, i[0].view(32, 2), *i[1:], None)\n"
            "assert torch.equal(i[0], torch.arange(64, device='cuda', dtype=torch.int32))\n",
}


@pytest.mark.parametrize("name", FIRST_CALLS)
def test_first_call_of_a_process_near_the_shared_memory_limit(name):
    code = "import torch, newton_schulz_shape_gb300 as nsg\n" + FIRST_CALLS[name] + "assert nsg.ns_check_status() == nsg.NS_OK\n"
    run = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parent.parent, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]


def test_strides_of_one_token_and_one_head_reach_nothing():
    g = gen(12)
    for shape, odd in (((1, 5, 64), (331, 64, 1)), ((7, 1, 64), (64, 99, 1))):
        q, k = randn(g, *shape, dtype=torch.bfloat16), randn(g, *shape, dtype=torch.bfloat16)
        qs, ks, qo, ko = (torch.empty_strided(shape, odd, dtype=torch.bfloat16, device=DEV) for _ in range(4))
        qs.copy_(q)
        ks.copy_(k)
        want_q, want_k = torch.empty_like(q), torch.empty_like(k)
        nsg.ns_qk_norm_rope(q, k, want_q, want_k)
        nsg.ns_qk_norm_rope(qs, ks, qo, ko)
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k)
    ok()


def test_launch_counts():
    nsg.ns_profile_read_training(reset=True)
    x = torch.ones(4, 2, 64, device=DEV)
    nsg.ns_qk_norm_rope(x, x, torch.empty_like(x), torch.empty_like(x))
    launches, _ = nsg.ns_profile_read_training(reset=True)
    assert launches == {"moe": 0, "qk_norm_rope": 1, "distill": 0}


def test_binding_arguments():
    x = torch.ones(4, 2, 64, device=DEV)
    with pytest.raises(TypeError, match="k_out"):
        nsg.ns_qk_norm_rope(x, x, x)
    with pytest.raises(TypeError, match="unexpected"):
        nsg.ns_qk_norm_rope(x, x, x, x, epsilon=1.0)
    with pytest.raises(TypeError, match="multiple"):
        nsg.ns_qk_norm_rope(x, x, x, x, q=x)
    with pytest.raises(ValueError, match="k_out"):
        nsg.ns_qk_norm_rope(x, x, x, x[:, :1])
    with pytest.raises(ValueError, match="q:.*contiguous heads"):
        nsg.ns_qk_norm_rope(x[..., ::2], x, x, x)
    with pytest.raises(ValueError, match="q_weight"):
        nsg.ns_qk_norm_rope(x, x, x, x, torch.ones(64, dtype=torch.float64, device=DEV))
    with pytest.raises(ValueError, match="positions"):
        nsg.ns_qk_norm_rope(x, x, x, x, table=torch.ones(4, 2, device=DEV), positions=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="logits"):
        nsg.ns_distill_loss(x[0].t(), x[0], x[0], x, x)
    with pytest.raises(ValueError, match="weights"):
        nsg.ns_moe_combine(torch.ones(4, 8, device=DEV), torch.ones(2, 2, device=DEV).half(),
                           torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, 8, device=DEV))
    with pytest.raises(nsg.NsError) as e:
        nsg.ns_qk_norm_rope(x, x, x, x, eps=-1.0)
    assert e.value.code == nsg.NS_ERR_ARG
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, None):
        nsg.ns_qk_norm_rope(x, x, torch.empty_like(x), torch.empty_like(x), stream=stream)
    torch.cuda.synchronize()
    ok()
