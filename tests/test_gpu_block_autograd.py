"""Gradient norm, clipping, block norms and the experts for a few tokens beside
autograd: they record nothing, so a call that would cut a graph is refused; what
they wrote counts as written."""

import pytest
import torch

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")

DEV = "cuda"


def f(*shape):
    return torch.ones(*shape, device=DEV)


def calls():
    """name: (floating tensors by name, other arguments, those written)."""
    rows = dict(branch=f(2, 16), branch_weight=f(16), weight=f(16), gate=f(2))
    return {
        "ns_block_norm": (dict(rows, residual=f(2, 16), residual_out=f(2, 16), out=f(2, 16)), {}, ["residual_out", "out"]),
        "ns_block_norm_grad": (dict(rows, grad_residual_out=f(2, 16), grad_out=f(2, 16), residual_out=f(2, 16), grad_branch=f(2, 16),
                                    grad_residual=f(2, 16), grad_branch_weight=f(16), grad_weight=f(16), grad_gate=f(2)),
                               dict(workspace=torch.empty(nsg.ns_block_norm_grad_workspace_bytes(16), dtype=torch.uint8, device=DEV)),
                               ["grad_branch", "grad_residual", "grad_branch_weight", "grad_weight", "grad_gate"]),
        "ns_moe_few_tokens": (dict(x=f(2, 16), weights=f(2, 3), gate_up=f(4, 10, 16), down=f(4, 16, 5), y=f(2, 16)),
                              dict(expert_ids=torch.zeros(2, 3, dtype=torch.int64, device=DEV),
                                   workspace=torch.empty(nsg.ns_moe_few_tokens_workspace_bytes(2, 3, 16, 5), dtype=torch.uint8, device=DEV)),
                              ["y"]),
        "ns_grad_norm": (dict(norm=f(1)), dict(grads=[f(3)], workspace=torch.empty(nsg.ns_grad_norm_workspace_bytes(1), dtype=torch.uint8,
                                                                                    device=DEV)), ["norm"]),
        "ns_grad_clip": (dict(norm=f(1)), dict(grads=[f(3)], outs=[f(3)], max_norm=1.0), []),
    }


@pytest.mark.parametrize("name", ["ns_block_norm", "ns_block_norm_grad", "ns_moe_few_tokens", "ns_grad_norm", "ns_grad_clip"])
def test_tensors_that_require_gradients_are_refused_where_a_graph_is_recorded(name):
    floats, rest, written = calls()[name]
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
    # what a call wrote, and only that, counts as written
    before = {k: v._version for k, v in floats.items()}
    op(**floats, **rest)
    assert {k for k, v in floats.items() if v._version != before[k]} == set(written)
    before = {k: v._version for k, v in floats.items()}
    if written:
        with pytest.raises(ValueError):
            op(**{**floats, written[-1]: floats[written[-1]].cpu()}, **rest)
    assert all(v._version == before[k] for k, v in floats.items())
    torch.cuda.synchronize()
    assert nsg.ns_check_status() == nsg.NS_OK


def test_lists_of_tensors():
    norm, x, y = f(1), f(3), f(3)
    ws = torch.empty(nsg.ns_grad_norm_workspace_bytes(2), dtype=torch.uint8, device=DEV)
    for where in ("grads", "outs"):
        leaf = f(3).requires_grad_()
        lists = dict(grads=[x, x], outs=[y, torch.empty_like(y)])
        lists[where] = [lists[where][0], leaf]
        with pytest.raises(ValueError, match=rf"^{where}\[1\]: .*gradient"):
            nsg.ns_grad_clip(**lists, norm=norm, max_norm=1.0)
    with pytest.raises(ValueError, match=r"^grads\[1\]: .*gradient"):
        nsg.ns_grad_norm([x, f(3).requires_grad_()], norm, ws)
    before = x._version, y._version
    nsg.ns_grad_clip((x,), (y,), norm, 1.0)
    assert (x._version, y._version) == (before[0], before[1] + 1)
    nsg.ns_grad_clip([x, y], [x, y], norm, 1.0)
    assert (x._version, y._version) == (before[0] + 1, before[1] + 2)
    big = f(4, 6)
    for grads, outs, match in (([x], [x, y], "as many"), ([x], [f(4)], r"outs\[0\]"), ([x], [x.half()], r"outs\[0\]"),
                               ([big], [f(6, 4).t()], r"outs\[0\].*strides"), ([big[:, ::2]], [f(4, 3)], r"grads\[0\].*gaps"),
                               ([x.double()], [x.double()], r"grads\[0\]"), ([x.expand(2, 3)], [f(2, 3)], r"grads\[0\].*gaps")):
        with pytest.raises(ValueError, match=match):
            nsg.ns_grad_clip(grads, outs, norm, 1.0)
    with pytest.raises(ValueError, match="norm"):
        nsg.ns_grad_norm([x], f(2), ws)
    with pytest.raises(nsg.NsError) as e:
        nsg.ns_grad_norm([x] * 2000, norm, ws[:64])
    assert e.value.code == nsg.NS_ERR_WORKSPACE
    assert nsg.ns_check_status() == nsg.NS_OK


def test_arguments():
    x, w = f(4, 16), f(16)
    for kwargs, match in ((dict(branch=f(4, 8)), "branch"), (dict(out=f(3, 16)), "out"), (dict(residual_out=x.half()), "residual_out"),
                          (dict(weight=f(15)), "weight"), (dict(weight=w.half()), "weight"), (dict(branch_weight=w, weight=w.half()), "weight"),
                          (dict(gate=f(3)), "gate"), (dict(gate=f(4, 8)), "gate"), (dict(gate=f(4).half()), "gate"),
                          (dict(out=f(4, 32)[:, ::2]), "out: contiguous rows")):
        with pytest.raises(ValueError, match=match):
            nsg.ns_block_norm(**{**dict(branch=x, residual=x, residual_out=torch.empty_like(x), out=torch.empty_like(x)), **kwargs})
    with pytest.raises(nsg.NsError) as e:
        nsg.ns_block_norm(x.half(), x.bfloat16(), None, torch.empty_like(x).half())     # a residual of another 16-bit type
    assert e.value.code == nsg.NS_ERR_ARG
    with pytest.raises(ValueError, match="grad_gate"):
        nsg.ns_block_norm_grad(x, x, x, x, None, None, grad_gate=f(4))
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    up, down, ws = f(3, 10, 16), f(3, 16, 5), torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    for args, match in (((x, ids[:3], None, up, down), "expert_ids"), ((x, ids.float(), None, up, down), "expert_ids"),
                        ((x, ids, f(4), up, down), "weights"), ((x, ids, None, f(3, 9, 16), down), "gate_up"),
                        ((x, ids, None, up, f(2, 16, 5)), "down"), ((x, ids, None, up.half(), down), "gate_up"),
                        ((x, ids, None, up, f(3, 32, 5)[:, ::2]), "down")):
        with pytest.raises(ValueError, match=match):
            nsg.ns_moe_few_tokens(*args, torch.empty_like(x), ws)
    assert nsg.ns_check_status() == nsg.NS_OK
