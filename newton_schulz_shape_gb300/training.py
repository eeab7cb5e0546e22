"""Operators of the training step around the orthogonalised matrices, as
torch-tensor calls of the C functions with the same names: tokens sorted by
expert and back, norms of queries and keys with the position rotation, and
distillation from a teacher's top logits, each with its gradient.

Outputs and workspaces are the caller's tensors. A tensor must be on the GPU,
its type one the C function takes and its last dimension contiguous
(ValueError otherwise); the library checks the rest (NsError). Streams default
to torch's current stream.
"""

from __future__ import annotations

import ctypes
import struct

import torch

from ._lib import NS_DT_BF16, NS_DT_FP16, NS_DT_FP32, check, lib

_DTYPES = {torch.bfloat16: NS_DT_BF16, torch.float16: NS_DT_FP16, torch.float32: NS_DT_FP32}
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}


# The calls below are written for few attribute reads and calls: at the sizes
# of a decoding step the host's part is most of a call.
_raw_stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream) -> int:
    if stream is None:
        # the handle alone: building a torch.cuda.Stream object costs 3.5 us
        return _raw_stream(_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _bad(name, t, want):
    got = f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}" if isinstance(t, torch.Tensor) else type(t).__name__
    raise ValueError(f"{name}: {want}, got {got}")


def _rows2d(name, t, dtype, rows=None, cols=None):
    """Address and row stride of a [rows, cols] tensor with contiguous rows."""
    shape = t.shape
    if not t.is_cuda or t.dtype is not dtype or len(shape) != 2:
        _bad(name, t, f"a GPU matrix of {dtype}")
    n, d = shape
    if (rows is not None and n != rows) or (cols is not None and d != cols):
        _bad(name, t, f"shape ({rows}, {cols})")
    ld, inner = t.stride()
    if inner != 1 and d > 1:
        _bad(name, t, "contiguous rows")
    return t.data_ptr(), ld if n > 1 else max(ld, d)


def _whole(name, t, dtype, numel):
    """Address of a contiguous tensor of `numel` values; None passes as NULL."""
    if t is None:
        return 0
    if not t.is_cuda or t.dtype is not dtype or t.numel() != numel or not t.is_contiguous():
        _bad(name, t, f"{numel} contiguous GPU values of {dtype}")
    return t.data_ptr()


def _indices(name, t, numel):
    size = _INDEX_BYTES.get(t.dtype)
    if size is None or not t.is_cuda or t.numel() != numel or not t.is_contiguous():
        _bad(name, t, f"{numel} contiguous GPU indices (int32 or int64)")
    return t.data_ptr(), size


def _scratch(t):
    if t is None:
        return 0, 0
    if not t.is_cuda or not t.is_contiguous():
        _bad("workspace", t, "a contiguous GPU tensor")
    return t.data_ptr(), t.nbytes


def _dtype(name, t):
    code = _DTYPES.get(t.dtype)
    if code is None:
        _bad(name, t, "bfloat16, float16 or float32")
    return code


# ------------------------------------------------------- tokens and experts
def ns_moe_rows(tokens: int, k: int, experts: int, align: int = 1, capacity: int = 0) -> int:
    """Rows that hold any routing of tokens * k slots to the experts."""
    out = ctypes.c_int64()
    check(lib.ns_moe_rows(tokens, k, experts, align, capacity, ctypes.byref(out)), "ns_moe_rows")
    return out.value


def ns_moe_sort_workspace_bytes(tokens: int, k: int, experts: int) -> int:
    out = ctypes.c_uint64()
    check(lib.ns_moe_sort_workspace_bytes(tokens, k, experts, ctypes.byref(out)), "ns_moe_sort_workspace_bytes")
    return out.value


def ns_moe_sort(expert_ids, experts: int, row_of_slot, slot_of_row, counts, offsets, workspace, align: int = 1,
                capacity: int = 0, stream=None) -> None:
    """Stable sort of the slots of expert_ids [tokens, k] by expert: writes
    row_of_slot [tokens, k], slot_of_row [rows], counts [experts] and offsets
    [experts + 1], all int32 (-1: no row, no slot). Negative ids go nowhere."""
    if expert_ids.dim() != 2:
        _bad("expert_ids", expert_ids, "a [tokens, k] matrix")
    tokens, k = expert_ids.shape
    ids, id_bytes = _indices("expert_ids", expert_ids, tokens * k)
    rows = slot_of_row.numel()
    ws, ws_bytes = _scratch(workspace)
    check(lib.ns_moe_sort(ids, id_bytes, tokens, k, experts, align, capacity, rows,
                          _whole("row_of_slot", row_of_slot, torch.int32, tokens * k),
                          _whole("slot_of_row", slot_of_row, torch.int32, rows),
                          _whole("counts", counts, torch.int32, experts),
                          _whole("offsets", offsets, torch.int32, experts + 1), ws, ws_bytes, _stream(stream)),
          "ns_moe_sort")


def _slots(row_of_slot):
    if row_of_slot.dim() != 2:
        _bad("row_of_slot", row_of_slot, "a [tokens, k] matrix")
    tokens, k = row_of_slot.shape
    return tokens, k, _whole("row_of_slot", row_of_slot, torch.int32, tokens * k)


def ns_moe_dispatch(x, row_of_slot, slot_of_row, out, stream=None) -> None:
    """out [rows, dim]: the token of each row's slot, zero in rows without one."""
    tokens, k, slots = _slots(row_of_slot)
    xp, x_ld = _rows2d("x", x, x.dtype, tokens)
    op, o_ld = _rows2d("out", out, x.dtype, slot_of_row.numel(), x.shape[1])
    check(lib.ns_moe_dispatch(xp, x_ld, _dtype("x", x), tokens, k, x.shape[1], slots,
                              _whole("slot_of_row", slot_of_row, torch.int32, out.shape[0]), out.shape[0], op, o_ld,
                              _stream(stream)), "ns_moe_dispatch")


def ns_moe_dispatch_grad(grad_rows, row_of_slot, grad_x, stream=None) -> None:
    """grad_x [tokens, dim]: the sum of each token's kept rows of grad_rows."""
    tokens, k, slots = _slots(row_of_slot)
    gp, g_ld = _rows2d("grad_rows", grad_rows, grad_rows.dtype)
    rows, dim = grad_rows.shape
    xp, x_ld = _rows2d("grad_x", grad_x, grad_rows.dtype, tokens, dim)
    check(lib.ns_moe_dispatch_grad(gp, g_ld, _dtype("grad_rows", grad_rows), tokens, k, dim, slots, rows, xp, x_ld,
                                   _stream(stream)), "ns_moe_dispatch_grad")


def ns_moe_combine(expert_rows, weights, row_of_slot, y, stream=None) -> None:
    """y [tokens, dim]: the sum of each token's kept rows times their fp32
    weights [tokens, k] (None: 1)."""
    tokens, k, slots = _slots(row_of_slot)
    ep, e_ld = _rows2d("expert_rows", expert_rows, expert_rows.dtype)
    rows, dim = expert_rows.shape
    yp, y_ld = _rows2d("y", y, expert_rows.dtype, tokens, dim)
    check(lib.ns_moe_combine(ep, e_ld, _dtype("expert_rows", expert_rows), tokens, k, dim, slots,
                             _whole("weights", weights, torch.float32, tokens * k), rows, yp, y_ld, _stream(stream)),
          "ns_moe_combine")


def ns_moe_combine_grad(grad_y, expert_rows, weights, row_of_slot, slot_of_row, grad_rows, grad_weights,
                        stream=None) -> None:
    """grad_rows [rows, dim] = weight * grad_y of each row's token (zero in rows
    without a slot) and grad_weights [tokens, k] fp32."""
    tokens, k, slots = _slots(row_of_slot)
    ep, e_ld = _rows2d("expert_rows", expert_rows, expert_rows.dtype, slot_of_row.numel())
    rows, dim = expert_rows.shape
    yp, y_ld = _rows2d("grad_y", grad_y, expert_rows.dtype, tokens, dim)
    gp, g_ld = _rows2d("grad_rows", grad_rows, expert_rows.dtype, rows, dim)
    check(lib.ns_moe_combine_grad(yp, y_ld, ep, e_ld, _dtype("expert_rows", expert_rows), tokens, k, dim, slots,
                                  _whole("slot_of_row", slot_of_row, torch.int32, rows),
                                  _whole("weights", weights, torch.float32, tokens * k), rows, gp, g_ld,
                                  _whole("grad_weights", grad_weights, torch.float32, tokens * k), _stream(stream)),
          "ns_moe_combine_grad")


# ------------------------------------------------------- queries and keys
_pack8, _pack12 = struct.Struct("8q").pack, struct.Struct("12q").pack


def _check_heads(names, tensors, q, k):
    """Say what is wrong with queries, keys or what has their shapes."""
    for name, t, like in zip(names, tensors, (q, k) * 3):
        if not t.is_cuda or t.dim() != 3:
            _bad(name, t, "a GPU tensor [tokens, heads, dim]")
        if t.dtype is not q.dtype:
            _bad(name, t, f"{q.dtype}, as q")
        if t.shape != like.shape:
            _bad(name, t, f"shape {tuple(like.shape)}")
    if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        _bad("k", k, f"({q.shape[0]}, heads, {q.shape[2]})")


def _heads(name, t, dim):
    """(token stride, head stride) of a [tokens, heads, dim] tensor."""
    token, head, inner = t.stride()
    if inner != 1 and dim > 1:
        _bad(name, t, "contiguous heads")
    return token, head


def _qk_common(q, dim, tokens, q_weight, k_weight, table, positions):
    wt = q_weight.dtype if q_weight is not None else k_weight.dtype if k_weight is not None else q.dtype
    if wt is not q.dtype and wt is not torch.float32:
        _bad("q_weight" if q_weight is not None else "k_weight", q_weight if q_weight is not None else k_weight,
             f"{q.dtype} or float32")
    qw, kw = _whole("q_weight", q_weight, wt, dim), _whole("k_weight", k_weight, wt, dim)
    tp, table_rows, rot = 0, 0, 0
    if table is not None:
        if table.dim() != 2:
            _bad("table", table, "a [positions, rot_dim] matrix")
        table_rows, rot = table.shape
        tp = _whole("table", table, torch.float32, table_rows * rot)
    pp, pb = (0, 4) if positions is None else _indices("positions", positions, tokens)
    return qw, kw, _DTYPES[wt] if wt in _DTYPES else _dtype("q", q), tp, table_rows, rot, pp, pb


def ns_qk_norm_rope(q, k, q_out, k_out, q_weight=None, k_weight=None, table=None, positions=None, eps: float = 1e-6,
                    interleaved: bool = False, stream=None) -> None:
    """Root-mean-square norm of every head of q and k [tokens, heads, dim], then
    the rotation by table [positions, rot_dim] (cosines, then sines) at
    positions [tokens] (None: 0, 1, ...). Tokens and heads may be strided."""
    dtype, shape, k_shape = q.dtype, q.shape, k.shape
    if not (q.is_cuda and k.is_cuda and q_out.is_cuda and k_out.is_cuda and len(shape) == 3 and len(k_shape) == 3
            and k.dtype is dtype and q_out.dtype is dtype and k_out.dtype is dtype and q_out.shape == shape
            and k_out.shape == k_shape and k_shape[0] == shape[0] and k_shape[2] == shape[2]):
        _check_heads(("q", "k", "q_out", "k_out"), (q, k, q_out, k_out), q, k)
    tokens, heads, dim = shape
    qw, kw, wt, tp, table_rows, rot, pp, pb = _qk_common(q, dim, tokens, q_weight, k_weight, table, positions)
    strides = _pack8(*_heads("q", q, dim), *_heads("k", k, dim), *_heads("q_out", q_out, dim), *_heads("k_out", k_out, dim))
    rc = lib.ns_qk_norm_rope(q.data_ptr(), k.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), strides, _dtype("q", q), tokens,
                             heads, k_shape[1], dim, rot, 1 if interleaved else 0, qw, kw, wt, eps, tp, table_rows, pp,
                             pb, _stream(stream))
    if rc:
        check(rc, "ns_qk_norm_rope")


def ns_qk_norm_rope_grad_workspace_bytes(head_dim: int) -> int:
    out = ctypes.c_uint64()
    check(lib.ns_qk_norm_rope_grad_workspace_bytes(head_dim, ctypes.byref(out)), "ns_qk_norm_rope_grad_workspace_bytes")
    return out.value


def ns_qk_norm_rope_grad(grad_q_out, grad_k_out, q, k, grad_q, grad_k, q_weight=None, k_weight=None,
                         grad_q_weight=None, grad_k_weight=None, table=None, positions=None, workspace=None,
                         eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Gradient of ns_qk_norm_rope: grad_q, grad_k and, where given, the fp32
    weight gradients [dim] (these need the workspace)."""
    _check_heads(("q", "k", "grad_q", "grad_k", "grad_q_out", "grad_k_out"),
                 (q, k, grad_q, grad_k, grad_q_out, grad_k_out), q, k)
    tokens, heads, dim = q.shape
    qw, kw, wt, tp, table_rows, rot, pp, pb = _qk_common(q, dim, tokens, q_weight, k_weight, table, positions)
    strides = _pack12(*_heads("q", q, dim), *_heads("k", k, dim), *_heads("grad_q", grad_q, dim),
                      *_heads("grad_k", grad_k, dim), *_heads("grad_q_out", grad_q_out, dim),
                      *_heads("grad_k_out", grad_k_out, dim))
    ws, ws_bytes = _scratch(workspace)
    check(lib.ns_qk_norm_rope_grad(grad_q_out.data_ptr(), grad_k_out.data_ptr(), q.data_ptr(), k.data_ptr(),
                                   grad_q.data_ptr(), grad_k.data_ptr(), strides, _dtype("q", q), tokens, heads,
                                   k.shape[1], dim, rot, 1 if interleaved else 0, qw, kw, wt,
                                   _whole("grad_q_weight", grad_q_weight, torch.float32, dim),
                                   _whole("grad_k_weight", grad_k_weight, torch.float32, dim), eps, tp, table_rows, pp,
                                   pb, ws, ws_bytes, _stream(stream)), "ns_qk_norm_rope_grad")


# ------------------------------------------------------------ distillation
def _distill_args(logits, teacher_values, teacher_ids, weights, teacher_lse, temperature, grad_logits):
    """The common arguments, up to the temperature, and the gradient's address and stride."""
    dtype = logits.dtype
    lp, ld = _rows2d("logits", logits, dtype)
    tokens, vocab = logits.shape
    shape = teacher_values.shape
    if len(shape) != 2 or teacher_ids.shape != shape:
        _bad("teacher_ids", teacher_ids, f"the shape of teacher_values, ({tokens}, top)")
    top = shape[1]
    n = tokens * top
    ids, id_bytes = _indices("teacher_ids", teacher_ids, n)
    t_dtype = teacher_values.dtype
    values = _whole("teacher_values", teacher_values, t_dtype, n)
    grad = (0, 0) if grad_logits is None else _rows2d("grad_logits", grad_logits, dtype, tokens, vocab)
    return (lp, ld, _dtype("logits", logits), tokens, vocab, values, _dtype("teacher_values", teacher_values), ids,
            id_bytes, top, 0 if weights is None else _whole("weights", weights, torch.float32, tokens),
            0 if teacher_lse is None else _whole("teacher_lse", teacher_lse, torch.float32, tokens), temperature), grad


def ns_distill_loss(logits, teacher_values, teacher_ids, loss, lse, grad_logits=None, weights=None, teacher_lse=None,
                    temperature: float = 1.0, stream=None) -> None:
    """Divergence of the student's softmax from the teacher's top entries:
    loss and lse fp32 [tokens] and, if grad_logits is given, the gradient in the
    logits [tokens, vocab] in the same pass. grad_logits may be logits itself."""
    args, (gp, g_ld) = _distill_args(logits, teacher_values, teacher_ids, weights, teacher_lse, temperature, grad_logits)
    tokens = args[3]
    rc = lib.ns_distill_loss(*args, _whole("loss", loss, torch.float32, tokens),
                             _whole("lse", lse, torch.float32, tokens), gp, g_ld, _stream(stream))
    if rc:
        check(rc, "ns_distill_loss")


def ns_distill_grad(logits, teacher_values, teacher_ids, lse, grad_logits, weights=None, teacher_lse=None,
                    temperature: float = 1.0, stream=None) -> None:
    """The gradient alone, from the lse that ns_distill_loss wrote."""
    args, (gp, g_ld) = _distill_args(logits, teacher_values, teacher_ids, weights, teacher_lse, temperature, grad_logits)
    rc = lib.ns_distill_grad(*args, _whole("lse", lse, torch.float32, args[3]), gp, g_ld, _stream(stream))
    if rc:
        check(rc, "ns_distill_grad")


TRAINING_KERNEL_KINDS = ("moe", "qk_norm_rope", "distill")


def ns_profile_read_training(reset: bool = False):
    """({kind: launches}, {kind: summed gpu ms}) of these operators since the last reset."""
    n = (ctypes.c_int64 * len(TRAINING_KERNEL_KINDS))()
    ms = (ctypes.c_double * len(TRAINING_KERNEL_KINDS))()
    check(lib.ns_profile_read_training(1 if reset else 0, n, ms), "ns_profile_read_training")
    return dict(zip(TRAINING_KERNEL_KINDS, list(n))), dict(zip(TRAINING_KERNEL_KINDS, list(ms)))
