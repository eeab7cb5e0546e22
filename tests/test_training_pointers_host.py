"""Addresses that their elements cannot have are refused on the host, before
any CUDA call: a kernel would fault on them."""

import pytest

from test_training_host import COMBINE_GRAD, GATHER, GRAD, LOSS, P, QK, QK_GRAD, ROWS_FWD, SORT, call, nsg

OFF = [
    ("ns_moe_sort", SORT, dict(ids=P + 4)), ("ns_moe_sort", SORT, dict(id_bytes=4, ids=P + 2)),
    ("ns_moe_sort", SORT, dict(row_of_slot=P + 2)), ("ns_moe_sort", SORT, dict(slot_of_row=P + 1)),
    ("ns_moe_sort", SORT, dict(counts=P + 2)), ("ns_moe_sort", SORT, dict(offsets=P + 3)),
    ("ns_moe_dispatch", ROWS_FWD, dict(x=P + 1)), ("ns_moe_dispatch", ROWS_FWD, dict(dtype=nsg.NS_DT_FP32, out=P + 2)),
    ("ns_moe_dispatch", ROWS_FWD, dict(row_of_slot=P + 2)), ("ns_moe_dispatch", ROWS_FWD, dict(slot_of_row=P + 2)),
    ("ns_moe_combine", GATHER, dict(rows_in=P + 1)), ("ns_moe_combine", GATHER, dict(weights=P + 2)),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(dy=P + 1)), ("ns_moe_combine_grad", COMBINE_GRAD, dict(grad_rows=P + 1)),
    ("ns_moe_combine_grad", COMBINE_GRAD, dict(grad_weights=P + 2)),
    ("ns_qk_norm_rope", QK, dict(q=P + 1)), ("ns_qk_norm_rope", QK, dict(k_out=P + 1)),
    ("ns_qk_norm_rope", QK, dict(kw=P + 1)), ("ns_qk_norm_rope", QK, dict(w_dtype=nsg.NS_DT_FP32, qw=P + 2)),
    ("ns_qk_norm_rope", QK, dict(table=P + 2)), ("ns_qk_norm_rope", QK, dict(positions=P + 4)),
    ("ns_qk_norm_rope_grad", QK_GRAD, dict(gq=P + 1)), ("ns_qk_norm_rope_grad", QK_GRAD, dict(dqw=P + 2)),
    ("ns_distill_loss", LOSS, dict(logits=P + 1)), ("ns_distill_loss", LOSS, dict(grad=P + 1)),
    ("ns_distill_loss", LOSS, dict(tv=P + 2)), ("ns_distill_loss", LOSS, dict(ids=P + 4)),
    ("ns_distill_loss", LOSS, dict(weights=P + 1)), ("ns_distill_loss", LOSS, dict(t_lse=P + 2)),
    ("ns_distill_loss", LOSS, dict(loss=P + 2)), ("ns_distill_grad", GRAD, dict(lse=P + 1)),
]


@pytest.mark.parametrize("name,base,changed", OFF)
def test_misaligned_addresses(name, base, changed):
    assert call(name, base, **changed) == nsg.NS_ERR_ARG


@pytest.mark.parametrize("none", [dict(tokens=0), dict(q_heads=0, k_heads=0), dict(k_heads=0)])
def test_weight_gradients_are_checked_without_tokens_too(none):
    for off in (dict(dqw=P + 2), dict(dkw=P + 1)):
        assert call("ns_qk_norm_rope_grad", QK_GRAD, **none, **off) == nsg.NS_ERR_ARG


def test_temperatures_whose_inverse_is_not_finite():
    for t in (1e-40, 1e-31, 2e30, float("inf"), -1.0):
        assert call("ns_distill_loss", LOSS, temperature=t) == nsg.NS_ERR_ARG
