"""Refusals of the training-step operators, CPU only: every argument check
answers on the host, before any CUDA call."""

import ctypes

import numpy as np
import pytest
import torch

nsg = pytest.importorskip("newton_schulz_shape_gb300")

P = 1 << 20          # an address that no call below may touch
BF, FP = nsg.NS_DT_BF16, nsg.NS_DT_FP32
ARG, SHAPE, UNSUP, WS = nsg.NS_ERR_ARG, nsg.NS_ERR_SHAPE, nsg.NS_ERR_UNSUPPORTED, nsg.NS_ERR_WORKSPACE


def call(name, base, **changed):
    args = dict(base)
    for k, v in changed.items():
        assert k in args, k
        args[k] = v
    return getattr(nsg.lib, name)(*args.values())


SORT = dict(ids=P, id_bytes=8, tokens=8192, k=4, experts=8, align=1, capacity=0, rows=32768, row_of_slot=P,
            slot_of_row=P, counts=P, offsets=P, ws=P, ws_bytes=1 << 20, stream=None)
ROWS_FWD = dict(x=P, x_ld=64, dtype=BF, tokens=8, k=4, dim=64, row_of_slot=P, slot_of_row=P, rows=32, out=P, out_ld=64,
                stream=None)
GATHER = dict(rows_in=P, rows_ld=64, dtype=BF, tokens=8, k=4, dim=64, row_of_slot=P, weights=P, rows=32, y=P, y_ld=64,
              stream=None)
COMBINE_GRAD = dict(dy=P, dy_ld=64, ys=P, ys_ld=64, dtype=BF, tokens=8, k=4, dim=64, row_of_slot=P, slot_of_row=P,
                    weights=P, rows=32, grad_rows=P, gr_ld=64, grad_weights=P, stream=None)
STRIDES = (ctypes.c_int64 * 12)(*[64] * 12)
QK = dict(q=P, k=P, q_out=P, k_out=P, strides=STRIDES, dtype=BF, tokens=4, q_heads=2, k_heads=1, dim=64, rot=64,
          interleaved=0, qw=P, kw=P, w_dtype=BF, eps=1e-6, table=P, table_rows=4, positions=P, position_bytes=8,
          stream=None)
QK_GRAD = dict(gq=P, gk=P, q=P, k=P, dq=P, dk=P, strides=STRIDES, dtype=BF, tokens=4, q_heads=2, k_heads=1, dim=64,
               rot=64, interleaved=0, qw=P, kw=P, w_dtype=FP, dqw=P, dkw=P, eps=1e-6, table=P, table_rows=4,
               positions=P, position_bytes=8, ws=P, ws_bytes=1 << 22, stream=None)
LOSS = dict(logits=P, ld=100, dtype=BF, tokens=4, vocab=100, tv=P, t_dtype=FP, ids=P, id_bytes=8, top=4, weights=None,
            t_lse=None, temperature=1.0, loss=P, lse=P, grad=P, grad_ld=100, stream=None)
GRAD = dict(logits=P, ld=100, dtype=BF, tokens=4, vocab=100, tv=P, t_dtype=FP, ids=P, id_bytes=8, top=4, weights=None,
            t_lse=None, temperature=1.0, lse=P, grad=P, grad_ld=100, stream=None)

CASES = [
    ("ns_moe_sort", SORT, dict(ids=None), ARG), ("ns_moe_sort", SORT, dict(id_bytes=2), ARG),
    ("ns_moe_sort", SORT, dict(tokens=-1), ARG), ("ns_moe_sort", SORT, dict(k=0), ARG),
    ("ns_moe_sort", SORT, dict(k=33), UNSUP), ("ns_moe_sort", SORT, dict(experts=0), ARG),
    ("ns_moe_sort", SORT, dict(experts=1025), UNSUP), ("ns_moe_sort", SORT, dict(align=0), ARG),
    ("ns_moe_sort", SORT, dict(capacity=-1), ARG), ("ns_moe_sort", SORT, dict(rows=32767), SHAPE),
    ("ns_moe_sort", SORT, dict(rows=1 << 31), SHAPE), ("ns_moe_sort", SORT, dict(tokens=1 << 30), SHAPE),
    ("ns_moe_sort", SORT, dict(counts=None), ARG), ("ns_moe_sort", SORT, dict(offsets=None), ARG),
    ("ns_moe_sort", SORT, dict(row_of_slot=None), ARG), ("ns_moe_sort", SORT, dict(slot_of_row=None), ARG),
    ("ns_moe_sort", SORT, dict(ws=None), WS), ("ns_moe_sort", SORT, dict(ws=P + 16), WS),
    ("ns_moe_sort", SORT, dict(ws_bytes=8), WS),
    ("ns_moe_dispatch", ROWS_FWD, dict(x=None), ARG), ("ns_moe_dispatch", ROWS_FWD, dict(out=None), ARG),
    ("ns_moe_dispatch", ROWS_FWD, dict(dtype=3), ARG), ("ns_moe_dispatch", ROWS_FWD, dict(x_ld=63), SHAPE),
    ("ns_moe_dispatch", ROWS_FWD, dict(out_ld=63), SHAPE), ("ns_moe_dispatch", ROWS_FWD, dict(k=33), UNSUP),
    ("ns_moe_dispatch", ROWS_FWD, dict(rows=1 << 31), SHAPE), ("ns_moe_dispatch", ROWS_FWD, dict(dim=-1), ARG),
    ("ns_moe_dispatch", ROWS_FWD, dict(slot_of_row=None), ARG),
    ("ns_moe_combine", GATHER, dict(rows_in=None), ARG), ("ns_moe_combine", GATHER, dict(y=None), ARG),
    ("ns_moe_combine", GATHER, dict(row_of_slot=None), ARG), ("ns_moe_combine", GATHER, dict(rows_ld=1), SHAPE),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(weights=None), ARG),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(grad_weights=None), ARG),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(dy=None), ARG), ("ns_moe_combine_grad", COMBINE_GRAD, dict(ys_ld=9), SHAPE),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(tokens=1 << 31), SHAPE),
    ("ns_qk_norm_rope", QK, dict(q=None), ARG), ("ns_qk_norm_rope", QK, dict(k_out=None), ARG),
    ("ns_qk_norm_rope", QK, dict(dtype=-1), ARG), ("ns_qk_norm_rope", QK, dict(w_dtype=nsg.NS_DT_FP16), ARG),
    ("ns_qk_norm_rope", QK, dict(rot=63), SHAPE), ("ns_qk_norm_rope", QK, dict(rot=66), SHAPE),
    ("ns_qk_norm_rope", QK, dict(dim=1025), UNSUP), ("ns_qk_norm_rope", QK, dict(table=None), ARG),
    ("ns_qk_norm_rope", QK, dict(interleaved=2), ARG), ("ns_qk_norm_rope", QK, dict(position_bytes=2), ARG),
    ("ns_qk_norm_rope", QK, dict(eps=-1.0), ARG), ("ns_qk_norm_rope", QK, dict(eps=float("nan")), ARG),
    ("ns_qk_norm_rope", QK, dict(strides=None), ARG), ("ns_qk_norm_rope", QK, dict(tokens=1 << 62), SHAPE),
    ("ns_qk_norm_rope_grad", QK_GRAD, dict(gq=None), ARG), ("ns_qk_norm_rope_grad", QK_GRAD, dict(dk=None), ARG),
    ("ns_qk_norm_rope_grad", QK_GRAD, dict(ws=None), WS), ("ns_qk_norm_rope_grad", QK_GRAD, dict(ws=P + 8), WS),
    ("ns_qk_norm_rope_grad", QK_GRAD, dict(ws_bytes=64), WS),
    ("ns_distill_loss", LOSS, dict(logits=None), ARG), ("ns_distill_loss", LOSS, dict(loss=None), ARG),
    ("ns_distill_loss", LOSS, dict(lse=None), ARG), ("ns_distill_loss", LOSS, dict(ld=99), SHAPE),
    ("ns_distill_loss", LOSS, dict(grad_ld=99), SHAPE), ("ns_distill_loss", LOSS, dict(temperature=0.0), ARG),
    ("ns_distill_loss", LOSS, dict(temperature=float("nan")), ARG), ("ns_distill_loss", LOSS, dict(top=0), ARG),
    ("ns_distill_loss", LOSS, dict(temperature=float("inf")), ARG),
    ("ns_distill_loss", LOSS, dict(top=1025), UNSUP), ("ns_distill_loss", LOSS, dict(vocab=0), ARG),
    ("ns_distill_loss", LOSS, dict(vocab=1 << 31, ld=1 << 31, grad_ld=1 << 31), SHAPE),
    ("ns_distill_loss", LOSS, dict(id_bytes=1), ARG), ("ns_distill_loss", LOSS, dict(t_dtype=7), ARG),
    ("ns_distill_loss", LOSS, dict(grad_ld=104), ARG),          # in place needs the same stride
    ("ns_distill_grad", GRAD, dict(grad=None), ARG), ("ns_distill_grad", GRAD, dict(lse=None), ARG),
]


@pytest.mark.parametrize("name,base,changed,want", CASES)
def test_refusals(name, base, changed, want):
    assert call(name, base, **changed) == want


def test_nothing_to_do_makes_no_call():
    # without a GPU a launch would answer NS_ERR_CUDA
    assert call("ns_moe_dispatch", ROWS_FWD, rows=0) == nsg.NS_OK
    assert call("ns_moe_dispatch", ROWS_FWD, dim=0, x=None, out=None) == nsg.NS_OK
    assert call("ns_moe_combine", GATHER, tokens=0, y=None) == nsg.NS_OK
    assert call("ns_moe_combine_grad", COMBINE_GRAD, tokens=0, rows=0, dy=None) == nsg.NS_OK
    assert call("ns_qk_norm_rope", QK, tokens=0, q=None) == nsg.NS_OK
    assert call("ns_qk_norm_rope", QK, q_heads=0, k_heads=0, q=None) == nsg.NS_OK
    assert call("ns_qk_norm_rope_grad", QK_GRAD, tokens=0, dqw=None, dkw=None, ws=None) == nsg.NS_OK
    assert call("ns_distill_loss", LOSS, tokens=0, loss=None, logits=None) == nsg.NS_OK
    assert call("ns_distill_grad", GRAD, tokens=0, grad=None) == nsg.NS_OK


@pytest.mark.parametrize("seed", range(30))
def test_rows_hold_the_worst_routing(seed):
    from oracle import training as ot
    g = np.random.default_rng(seed)
    T, k, E = int(g.integers(0, 30)), int(g.integers(1, 5)), int(g.integers(1, 9))
    align, cap = int(g.choice([1, 4, 16])), int(g.choice([0, 1, 5, 1000]))
    rows = nsg.ns_moe_rows(T, k, E, align, cap)
    for _ in range(20):
        ids = g.integers(-1, E, (T, k)) if g.random() < 0.5 else np.full((T, k), g.integers(0, E))
        assert ot.moe_sort(ids, E, align, cap)[3][-1] <= rows
    # the bound is reached: one slot in as many experts as possible, the rest in one of them
    if not cap and T * k:
        worst = np.zeros(T * k, int)
        worst[:min(E, T * k)] = np.arange(min(E, T * k))
        if align == 1:
            assert ot.moe_sort(worst.reshape(T, k), E, align, cap)[3][-1] == rows


def test_workspace_sizes():
    assert nsg.ns_moe_sort_workspace_bytes(1, 1, 4) == 0
    assert nsg.ns_qk_norm_rope_grad_workspace_bytes(128) % (2 * 128 * 4) == 0
    with pytest.raises(nsg.NsError) as e:
        nsg.ns_moe_rows(4, 40, 4)
    assert e.value.code == UNSUP
    with pytest.raises(nsg.NsError) as e:
        nsg.ns_qk_norm_rope_grad_workspace_bytes(2000)
    assert e.value.code == UNSUP


def test_binding_refuses_tensors_it_cannot_pass():
    ids, x = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 8)
    i32 = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="expert_ids"):
        nsg.ns_moe_sort(ids, 2, i32, i32, i32[:2], i32[:3], None)          # not on the GPU
    with pytest.raises(ValueError, match="row_of_slot"):
        nsg.ns_moe_dispatch(x, i32, i32, x)                               # not [tokens, k]
    with pytest.raises(ValueError, match="GPU"):
        nsg.ns_qk_norm_rope(x.view(4, 1, 8), x.view(4, 1, 8), x.view(4, 1, 8), x.view(4, 1, 8))
    with pytest.raises(ValueError, match="logits"):
        nsg.ns_distill_loss(x, x, ids, x, x)


def test_module_attributes():
    assert callable(nsg.ns_moe_sort)
    with pytest.raises(AttributeError):
        nsg.ns_no_such_operator
