"""The operators beside autograd: they record nothing, so a call that would cut
a graph is refused."""

import pytest
import torch

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

DEV = "cuda"


def calls():
    """(name, tensors, call) of every operator on small inputs: the floating ones by name; call takes a dict of them."""
    def f(*shape):
        return torch.ones(*shape, device=DEV)

    row = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device=DEV)
    slot = torch.arange(4, dtype=torch.int32, device=DEV)
    ids = torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(16), dtype=torch.uint8, device=DEV)
    heads = dict(q=f(2, 2, 16), k=f(2, 1, 16), q_weight=f(16), k_weight=f(16), table=f(2, 16))
    teacher = dict(logits=f(2, 9), teacher_values=f(2, 3), weights=f(2), teacher_lse=f(2))
    return [
        ("ns_moe_dispatch", dict(x=f(2, 8), out=f(4, 8)), dict(row_of_slot=row, slot_of_row=slot), ["out"]),
        ("ns_moe_dispatch_grad", dict(grad_rows=f(4, 8), grad_x=f(2, 8)), dict(row_of_slot=row), ["grad_x"]),
        ("ns_moe_combine", dict(expert_rows=f(4, 8), weights=f(2, 2), y=f(2, 8)), dict(row_of_slot=row), ["y"]),
        ("ns_moe_combine_grad", dict(grad_y=f(2, 8), expert_rows=f(4, 8), weights=f(2, 2), grad_rows=f(4, 8), grad_weights=f(2, 2)),
         dict(row_of_slot=row, slot_of_row=slot), ["grad_rows", "grad_weights"]),
        ("ns_qk_norm_rope", dict(heads, q_out=f(2, 2, 16), k_out=f(2, 1, 16)), {}, ["q_out", "k_out"]),
        ("ns_qk_norm_rope_grad", dict(heads, grad_q_out=f(2, 2, 16), grad_k_out=f(2, 1, 16), grad_q=f(2, 2, 16), grad_k=f(2, 1, 16),
                                      grad_q_weight=f(16), grad_k_weight=f(16)), dict(workspace=ws),
         ["grad_q", "grad_k", "grad_q_weight", "grad_k_weight"]),
        ("ns_distill_loss", dict(teacher, loss=f(2), lse=f(2), grad_logits=f(2, 9)), dict(teacher_ids=ids), ["loss", "lse", "grad_logits"]),
        ("ns_distill_grad", dict(teacher, lse=f(2), grad_logits=f(2, 9)), dict(teacher_ids=ids), ["grad_logits"]),
    ]


NAMES = ["ns_moe_dispatch", "ns_moe_dispatch_grad", "ns_moe_combine", "ns_moe_combine_grad", "ns_qk_norm_rope", "ns_qk_norm_rope_grad",
         "ns_distill_loss", "ns_distill_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_require_gradients_are_refused_where_a_graph_is_recorded(name):
    _, floats, rest, _ = next(c for c in calls() if c[0] == name)
    op = getattr(nsg, name)
    op(**floats, **rest)
    for one in floats:
        given = {k: v.clone().requires_grad_() if k == one else v for k, v in floats.items()}
        with pytest.raises(ValueError, match=rf"^{one}: .*gradient"):
            op(**given, **rest)
        with torch.no_grad():
            op(**given, **rest)
        with torch.inference_mode():
            op(**given, **rest)
    torch.cuda.synchronize()
    assert nsg.ns_check_status() == nsg.NS_OK


@pytest.mark.parametrize("name", NAMES + ["ns_moe_sort"])
def test_outputs_count_as_written(name):
    # so that autograd can tell that what it saved is no longer there
    if name == "ns_moe_sort":
        i32 = [torch.empty(n, dtype=torch.int32, device=DEV) for n in ((2, 2), 4, 3, 4)]
        floats = dict(zip(("row_of_slot", "slot_of_row", "counts", "offsets"), i32))
        rest = dict(expert_ids=torch.zeros(2, 2, dtype=torch.int64, device=DEV), experts=3, workspace=None)
        written = list(floats)
    else:
        _, floats, rest, written = next(c for c in calls() if c[0] == name)
    op = getattr(nsg, name)
    before = {k: v._version for k, v in floats.items()}
    op(**floats, **rest)
    assert {k for k, v in floats.items() if v._version != before[k]} == set(written)
    # a view counts for what it is a view of, a refused call for nothing
    big = {k: torch.empty(2, *v.shape, dtype=v.dtype, device=DEV) for k, v in floats.items() if k in written}
    op(**{**floats, **{k: v[0] for k, v in big.items()}}, **rest)
    assert all(v._version == 1 for v in big.values())
    before = {k: v._version for k, v in floats.items()}
    with pytest.raises(ValueError):
        op(**{**floats, written[-1]: floats[written[-1]].cpu()}, **rest)
    assert all(v._version == before[k] for k, v in floats.items())
    # tensors of inference mode have no count
    with torch.inference_mode():
        made = {k: v.clone() for k, v in floats.items()}
    op(**made, **rest)
    torch.cuda.synchronize()
    assert nsg.ns_check_status() == nsg.NS_OK


def test_a_saved_tensor_that_was_written_over_stops_the_backward_pass():
    x = torch.ones(2, 2, 16, device=DEV, requires_grad=True)
    y = x * 2
    z = (y * y).sum()                    # saves y
    with torch.no_grad():
        nsg.ns_qk_norm_rope(y.detach(), y.detach(), y.detach(), torch.empty_like(y))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
