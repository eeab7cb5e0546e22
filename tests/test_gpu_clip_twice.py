"""Clipping refuses a tensor that it would write from two places of its list."""

import pytest
import torch

from test_gpu_block_ops import DEV, bf16, nsg, ok

pytestmark = pytest.mark.gpu


def shuffled(n):
    """n tensors that do not lie in the order of their places."""
    t = [torch.ones(5 + i % 3, device=DEV) for i in range(n)]
    return t[::2] + t[1::2][::-1]


@pytest.mark.parametrize("n", [2, 3, 100, 1200])
@pytest.mark.parametrize("order", [sorted, list])
def test_a_tensor_named_twice_is_refused(n, order):
    norm = torch.full((1,), 4.0, device=DEV)
    grads = order(shuffled(n), key=torch.Tensor.data_ptr) if order is sorted else shuffled(n)
    fresh = [torch.zeros_like(t) for t in grads]
    for i, j in {(0, n - 1), (n // 2 - 1, n // 2)}:
        tied = list(grads)
        tied[j] = tied[i].view(-1)
        with pytest.raises(ValueError, match=r"outs\[\d+\]: a tensor that the call names in no other place"):
            nsg.ns_grad_clip(tied, tied, norm, 1.0)
        same = [t if t.shape == u.shape else u for t, u in zip([fresh[i] if k == j else t for k, t in enumerate(fresh)], grads)]
        if same[j] is fresh[i]:
            with pytest.raises(ValueError, match="outs"):
                nsg.ns_grad_clip(grads, same, norm, 1.0)
        # an output where another place has its input
        if grads[i].shape == grads[j].shape:
            outs = list(fresh)
            outs[j] = grads[i]
            with pytest.raises(ValueError, match=rf"outs\[{j}\]"):
                nsg.ns_grad_clip(grads, outs, norm, 1.0)
    assert all((t == 1).all() and t._version == 0 for t in grads)       # nothing was written
    # the same input twice, other outputs: only read
    tied = [grads[0]] * n
    outs = [torch.zeros_like(grads[0]) for _ in range(n)]
    nsg.ns_grad_clip(tied, outs, norm, 1.0, eps=0.0)
    assert all((t == 0.25).all() for t in outs)
    nsg.ns_grad_clip(grads, grads, norm, 1.0, eps=0.0)
    nsg.ns_grad_clip(grads, list(grads), norm, 1.0, eps=0.0)            # another list of the same tensors
    assert all((t == 0.0625).all() for t in grads)
    ok()


def test_empty_tensors_and_flat_buffers_are_no_other_place():
    norm = torch.full((1,), 4.0, device=DEV)
    flat = torch.ones(1000, dtype=bf16, device=DEV)
    parts = list(flat.split([7, 0, 0, 500, 493]))
    nsg.ns_grad_clip(parts, parts, norm, 1.0, eps=0.0)
    empty = torch.empty(0, device=DEV)
    nsg.ns_grad_clip([empty, empty, parts[4], parts[0]], [empty, empty, parts[4], parts[0]], norm, 1.0, eps=0.0)
    assert (flat[7:507] == 0.25).all() and (flat[:7] == 0.0625).all() and (flat[507:] == 0.0625).all()
    # halves of one buffer clipped into each other's place, outputs in order: the inputs are some of them
    a, b = torch.ones(64, device=DEV).split(32)
    with pytest.raises(ValueError, match="outs"):
        nsg.ns_grad_clip([b, a], [a, b], norm, 1.0)
    ok()
