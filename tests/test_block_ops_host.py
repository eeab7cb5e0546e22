"""Refusals of the gradient norm and clipping, the block norms and the experts
for a few tokens, CPU only: every argument check answers on the host, before any
CUDA call."""

import ctypes

import pytest
import torch

from test_training_host import ARG, BF, FP, P, SHAPE, UNSUP, WS, call, nsg

HALF = nsg.NS_DT_FP16


def pointers(*at):
    return (ctypes.c_void_p * len(at))(*at)


def sizes(*n):
    return (ctypes.c_int64 * len(n))(*n)


def types(*t):
    return (ctypes.c_int32 * len(t))(*t)


NORM = dict(grads=pointers(P, P), numels=sizes(8, 3), dtypes=types(BF, FP), count=2, norm=P, ws=P, ws_bytes=1 << 16, stream=None)
CLIP = dict(grads=pointers(P, P), outs=pointers(P, P), numels=sizes(8, 3), dtypes=types(BF, FP), count=2, norm=P, max_norm=1.0,
            eps=1e-6, stream=None)
BLOCK = dict(branch=P, residual=P, residual_out=P, out=P, strides=sizes(*[64] * 8), dtype=BF, r_dtype=FP, tokens=4, dim=64, bw=P, w=P,
             w_dtype=FP, gate=P, gate_kind=2, post=1, alpha=1.0, beta=1.0, eps=1e-6, stream=None)
BLOCK_GRAD = dict(gh=P, gn=P, branch=P, h=P, gb=P, gx=P, strides=sizes(*[64] * 8), dtype=BF, r_dtype=BF, tokens=4, dim=64, bw=P, w=P,
                  w_dtype=BF, gate=P, gate_kind=1, gbw=P, gw=P, gg=P, post=1, alpha=1.0, beta=1.0, eps=1e-6, ws=P, ws_bytes=1 << 20,
                  stream=None)
FEW = dict(x=P, x_ld=64, dtype=BF, tokens=4, k=2, dim=64, ffn=32, experts=8, ids=P, id_bytes=8, weights=P, up=P, down=P, y=P, y_ld=64,
           ws=P, ws_bytes=1 << 20, stream=None)


def strides(i, v):
    s = [64] * 8
    s[i] = v
    return sizes(*s)


CASES = [
    ("ns_grad_norm", NORM, dict(grads=None), ARG), ("ns_grad_norm", NORM, dict(numels=None), ARG),
    ("ns_grad_norm", NORM, dict(dtypes=None), ARG), ("ns_grad_norm", NORM, dict(count=-1), ARG),
    ("ns_grad_norm", NORM, dict(norm=None), ARG), ("ns_grad_norm", NORM, dict(norm=P + 2), ARG),
    ("ns_grad_norm", NORM, dict(grads=pointers(P, None)), ARG), ("ns_grad_norm", NORM, dict(grads=pointers(P + 1, P)), ARG),
    ("ns_grad_norm", NORM, dict(grads=pointers(P, P + 2)), ARG), ("ns_grad_norm", NORM, dict(dtypes=types(BF, 3)), ARG),
    ("ns_grad_norm", NORM, dict(numels=sizes(8, -1)), ARG), ("ns_grad_norm", NORM, dict(numels=sizes(8, 1 << 50)), SHAPE),
    ("ns_grad_norm", NORM, dict(numels=sizes(1 << 41, 1 << 41)), SHAPE), ("ns_grad_norm", NORM, dict(count=(1 << 20) + 1), UNSUP),
    ("ns_grad_norm", NORM, dict(ws=None), WS), ("ns_grad_norm", NORM, dict(ws=P + 16), WS), ("ns_grad_norm", NORM, dict(ws_bytes=64), WS),
    ("ns_grad_clip", CLIP, dict(outs=None), ARG), ("ns_grad_clip", CLIP, dict(outs=pointers(None, P)), ARG),
    ("ns_grad_clip", CLIP, dict(outs=pointers(P, P + 2)), ARG), ("ns_grad_clip", CLIP, dict(max_norm=-1.0), ARG),
    ("ns_grad_clip", CLIP, dict(max_norm=float("nan")), ARG), ("ns_grad_clip", CLIP, dict(eps=-1e-9), ARG),
    ("ns_grad_clip", CLIP, dict(eps=float("inf")), ARG), ("ns_grad_clip", CLIP, dict(norm=None), ARG),
    ("ns_grad_clip", CLIP, dict(grads=pointers(None, P)), ARG),
    ("ns_block_norm", BLOCK, dict(residual=None), ARG), ("ns_block_norm", BLOCK, dict(strides=None), ARG),
    ("ns_block_norm", BLOCK, dict(dtype=3), ARG), ("ns_block_norm", BLOCK, dict(r_dtype=HALF), ARG),
    ("ns_block_norm", BLOCK, dict(w_dtype=HALF), ARG), ("ns_block_norm", BLOCK, dict(tokens=-1), ARG),
    ("ns_block_norm", BLOCK, dict(dim=-1), ARG), ("ns_block_norm", BLOCK, dict(dim=(1 << 20) + 1), UNSUP),
    ("ns_block_norm", BLOCK, dict(tokens=1 << 40), SHAPE), ("ns_block_norm", BLOCK, dict(gate=None), ARG),
    ("ns_block_norm", BLOCK, dict(gate_kind=3), ARG), ("ns_block_norm", BLOCK, dict(post=2), ARG),
    ("ns_block_norm", BLOCK, dict(eps=-1.0), ARG), ("ns_block_norm", BLOCK, dict(alpha=float("inf")), ARG),
    ("ns_block_norm", BLOCK, dict(beta=float("nan")), ARG),
    *[("ns_block_norm", BLOCK, dict(strides=strides(i, 63)), SHAPE) for i in range(5)],
    *[("ns_block_norm", BLOCK, {n: P + 1}, ARG) for n in ("branch", "residual", "residual_out", "out", "bw", "w", "gate")],
    ("ns_block_norm", BLOCK, dict(gate_kind=1, gate=P + 2), ARG),
    ("ns_block_norm_grad", BLOCK_GRAD, dict(h=None), ARG), ("ns_block_norm_grad", BLOCK_GRAD, dict(gh=None, gn=None), ARG),
    ("ns_block_norm_grad", BLOCK_GRAD, dict(branch=None), ARG), ("ns_block_norm_grad", BLOCK_GRAD, dict(gate_kind=0), ARG),
    ("ns_block_norm_grad", BLOCK_GRAD, dict(ws=None), WS), ("ns_block_norm_grad", BLOCK_GRAD, dict(ws=P + 8), WS),
    ("ns_block_norm_grad", BLOCK_GRAD, dict(ws_bytes=1 << 10), WS),
    *[("ns_block_norm_grad", BLOCK_GRAD, dict(gate_kind=2, strides=strides(i, 63)), SHAPE) for i in range(8)],
    *[("ns_block_norm_grad", BLOCK_GRAD, {n: P + 1}, ARG) for n in ("gh", "gn", "branch", "h", "gb", "gx", "bw", "w", "gbw", "gw", "gg", "gate")],
    ("ns_moe_few_tokens", FEW, dict(x=None), ARG), ("ns_moe_few_tokens", FEW, dict(ids=None), ARG),
    ("ns_moe_few_tokens", FEW, dict(up=None), ARG), ("ns_moe_few_tokens", FEW, dict(down=None), ARG),
    ("ns_moe_few_tokens", FEW, dict(y=None), ARG), ("ns_moe_few_tokens", FEW, dict(dtype=-1), ARG),
    ("ns_moe_few_tokens", FEW, dict(id_bytes=2), ARG), ("ns_moe_few_tokens", FEW, dict(tokens=-1), ARG),
    ("ns_moe_few_tokens", FEW, dict(tokens=257), UNSUP), ("ns_moe_few_tokens", FEW, dict(k=0), ARG),
    ("ns_moe_few_tokens", FEW, dict(k=33), UNSUP), ("ns_moe_few_tokens", FEW, dict(experts=0), ARG),
    ("ns_moe_few_tokens", FEW, dict(experts=1025), UNSUP), ("ns_moe_few_tokens", FEW, dict(ffn=0), ARG),
    ("ns_moe_few_tokens", FEW, dict(dim=1 << 20, x_ld=1 << 20, y_ld=1 << 20), UNSUP), ("ns_moe_few_tokens", FEW, dict(ffn=1 << 20), UNSUP),
    ("ns_moe_few_tokens", FEW, dict(x_ld=63), SHAPE), ("ns_moe_few_tokens", FEW, dict(y_ld=63), SHAPE),
    ("ns_moe_few_tokens", FEW, dict(ws=None), WS), ("ns_moe_few_tokens", FEW, dict(ws=P + 16), WS),
    ("ns_moe_few_tokens", FEW, dict(ws_bytes=16), WS),
    *[("ns_moe_few_tokens", FEW, {n: P + 1}, ARG) for n in ("x", "ids", "weights", "up", "down", "y")],
]


@pytest.mark.parametrize("name,base,changed,want", CASES)
def test_refusals(name, base, changed, want):
    assert call(name, base, **changed) == want


def test_nothing_to_do_makes_no_call():
    # without a GPU a launch would answer NS_ERR_CUDA
    assert call("ns_grad_clip", CLIP, count=0, grads=None, outs=None, numels=None, dtypes=None) == nsg.NS_OK
    assert call("ns_grad_clip", CLIP, numels=sizes(0, 0), grads=pointers(None, None), outs=pointers(None, None)) == nsg.NS_OK
    assert call("ns_block_norm", BLOCK, tokens=0, residual=None, gate=None) == nsg.NS_OK
    assert call("ns_block_norm", BLOCK, dim=0, branch=None, residual=None) == nsg.NS_OK
    assert call("ns_block_norm", BLOCK, residual_out=None, out=None) == nsg.NS_OK
    assert call("ns_block_norm_grad", BLOCK_GRAD, tokens=0, gbw=None, gw=None, ws=None, h=None) == nsg.NS_OK
    assert call("ns_block_norm_grad", BLOCK_GRAD, dim=0, h=None) == nsg.NS_OK
    assert call("ns_moe_few_tokens", FEW, tokens=0, x=None) == nsg.NS_OK
    assert call("ns_moe_few_tokens", FEW, dim=0, x=None, y=None) == nsg.NS_OK


def test_workspace_sizes():
    assert nsg.ns_grad_norm_workspace_bytes(0) > 0
    assert nsg.ns_grad_norm_workspace_bytes(5000) > nsg.ns_grad_norm_workspace_bytes(1)
    assert nsg.ns_block_norm_grad_workspace_bytes(128) % (2 * 128 * 4) == 0
    assert nsg.ns_moe_few_tokens_workspace_bytes(0, 1, 1, 1) >= 0
    for fn, args in ((nsg.ns_grad_norm_workspace_bytes, ((1 << 20) + 1,)), (nsg.ns_block_norm_grad_workspace_bytes, (1 << 21,)),
                     (nsg.ns_moe_few_tokens_workspace_bytes, (257, 1, 8, 8)), (nsg.ns_moe_few_tokens_workspace_bytes, (1, 33, 8, 8))):
        with pytest.raises(nsg.NsError) as e:
            fn(*args)
        assert e.value.code == UNSUP
    for fn, args in ((nsg.ns_grad_norm_workspace_bytes, (-1,)), (nsg.ns_block_norm_grad_workspace_bytes, (-1,)),
                     (nsg.ns_moe_few_tokens_workspace_bytes, (1, 1, 8, 0))):
        with pytest.raises(nsg.NsError) as e:
            fn(*args)
        assert e.value.code == ARG


def test_binding_refuses_tensors_it_cannot_pass():
    x, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
    one = torch.zeros(1)
    with pytest.raises(ValueError, match=r"grads\[0\].*GPU"):
        nsg.ns_grad_norm([x], one, None)
    with pytest.raises(ValueError, match=r"grads\[1\]: a tensor, got NoneType"):
        nsg.ns_grad_clip([x, None], [x, x], one, 1.0)
    with pytest.raises(ValueError, match="grads: a list of tensors"):
        nsg.ns_grad_norm(3, one, None)
    with pytest.raises(ValueError, match="residual"):
        nsg.ns_block_norm(x, x, x, x)
    with pytest.raises(ValueError, match="residual_out"):
        nsg.ns_block_norm_grad(x, x, x, x, x, x)
    with pytest.raises(ValueError, match="x: "):
        nsg.ns_moe_few_tokens(x, ids, None, x, x, x, None)
    with pytest.raises(TypeError, match="max_norm"):
        nsg.ns_grad_clip([], [], one)
