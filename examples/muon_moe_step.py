"""Distillation steps of a one-layer mixture-of-experts model trained with
Muon, on the library's operators:

  tokens -> fused QKV projection -> norms of queries and keys with the rotation
  (ns_qk_norm_rope) -> attention -> router -> tokens sorted by expert
  (ns_moe_sort, ns_moe_dispatch) -> experts -> weighted sum (ns_moe_combine)
  -> logits -> distillation from a teacher's top entries (ns_distill_loss)

and back through their gradients to the momentum of every matrix, which
ns_orthogonalize_batched turns into the update. Matrix products and the softmax
of attention are torch's.

  python examples/muon_moe_step.py            # 60 steps on cuda:0
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_shape_gb300 as nsg  # noqa: E402


# --------------------------------------------- the operators under autograd
class QkNormRope(torch.autograd.Function):
    """Queries and keys of a fused projection, normalised and rotated."""

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, heads, table, positions):
        q_heads, k_heads, dim = heads
        q, k = split_heads(qkv, heads)[:2]
        q_out, k_out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty_like(k, memory_format=torch.contiguous_format)
        nsg.ns_qk_norm_rope(q, k, q_out, k_out, q_weight, k_weight, table, positions)
        ctx.save_for_backward(qkv, q_weight, k_weight, table, positions)
        ctx.heads = heads
        return q_out, k_out

    @staticmethod
    def backward(ctx, grad_q_out, grad_k_out):
        qkv, q_weight, k_weight, table, positions = ctx.saved_tensors
        dim = ctx.heads[2]
        grad = torch.zeros_like(qkv)                     # the values' columns get theirs elsewhere
        (q, k, _), (gq, gk, _) = split_heads(qkv, ctx.heads), split_heads(grad, ctx.heads)
        gqw, gkw = torch.empty(dim, device=qkv.device), torch.empty(dim, device=qkv.device)
        ws = torch.empty(nsg.ns_qk_norm_rope_grad_workspace_bytes(dim), dtype=torch.uint8, device=qkv.device)
        nsg.ns_qk_norm_rope_grad(grad_q_out.contiguous(), grad_k_out.contiguous(), q, k, gq, gk, q_weight, k_weight, gqw,
                                 gkw, table, positions, ws)
        return grad, gqw.to(q_weight.dtype), gkw.to(k_weight.dtype), None, None, None


def split_heads(qkv, heads):
    """q, k, v views [tokens, heads, dim] of a fused projection."""
    q_heads, k_heads, dim = heads
    q, k, v = qkv.split([q_heads * dim, k_heads * dim, k_heads * dim], dim=1)
    return q.view(-1, q_heads, dim), k.view(-1, k_heads, dim), v.view(-1, k_heads, dim)


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_of_slot, slot_of_row):
        out = torch.empty(slot_of_row.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        nsg.ns_moe_dispatch(x, row_of_slot, slot_of_row, out)
        ctx.save_for_backward(row_of_slot)
        return out

    @staticmethod
    def backward(ctx, grad_rows):
        (row_of_slot,) = ctx.saved_tensors
        grad_x = torch.empty(row_of_slot.shape[0], grad_rows.shape[1], dtype=grad_rows.dtype, device=grad_rows.device)
        nsg.ns_moe_dispatch_grad(grad_rows.contiguous(), row_of_slot, grad_x)
        return grad_x, None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, expert_rows, weights, row_of_slot, slot_of_row):
        y = torch.empty(row_of_slot.shape[0], expert_rows.shape[1], dtype=expert_rows.dtype, device=expert_rows.device)
        nsg.ns_moe_combine(expert_rows, weights, row_of_slot, y)
        ctx.save_for_backward(expert_rows, weights, row_of_slot, slot_of_row)
        return y

    @staticmethod
    def backward(ctx, grad_y):
        expert_rows, weights, row_of_slot, slot_of_row = ctx.saved_tensors
        grad_rows, grad_weights = torch.empty_like(expert_rows), torch.empty_like(weights)
        nsg.ns_moe_combine_grad(grad_y.contiguous(), expert_rows, weights, row_of_slot, slot_of_row, grad_rows, grad_weights)
        return grad_rows, grad_weights, None, None


class Distill(torch.autograd.Function):
    """Mean loss over the tokens of a batch; the logits' gradient is computed in
    the same pass, in place of the logits."""

    @staticmethod
    def forward(ctx, logits, teacher_values, teacher_ids, weights):
        loss, lse = torch.empty(len(logits), device=logits.device), torch.empty(len(logits), device=logits.device)
        nsg.ns_distill_loss(logits, teacher_values, teacher_ids, loss, lse, grad_logits=logits, weights=weights)
        ctx.mark_dirty(logits)
        ctx.save_for_backward(logits)
        return loss.sum(), logits

    @staticmethod
    def backward(ctx, grad_loss, _):
        (grad,) = ctx.saved_tensors
        return grad * grad_loss, None, None, None


def sort_tokens(expert_ids, experts, align=16):
    """row_of_slot, slot_of_row, and the experts' segments as host integers."""
    tokens, k = expert_ids.shape
    dev = expert_ids.device
    rows = nsg.ns_moe_rows(tokens, k, experts, align)
    row_of_slot, slot_of_row, counts, offsets = (torch.empty(n, dtype=torch.int32, device=dev)
                                                 for n in ((tokens, k), rows, experts, experts + 1))
    ws = torch.empty(nsg.ns_moe_sort_workspace_bytes(tokens, k, experts), dtype=torch.uint8, device=dev)
    nsg.ns_moe_sort(expert_ids, experts, row_of_slot, slot_of_row, counts, offsets, ws, align=align)
    return row_of_slot, slot_of_row, offsets.tolist()


# ------------------------------------------------------------------ a model
class Model:
    """One layer: attention with normalised heads and a mixture of experts."""

    def __init__(self, vocab=1000, dim=256, heads=(8, 2, 32), experts=8, k=2, ffn=192, length=128, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.vocab, self.dim, self.heads, self.experts, self.k, self.length = vocab, dim, heads, experts, k, length
        q, kv, hd = heads

        def matrix(rows, cols):
            return torch.randn(rows, cols, generator=g, device=device) / math.sqrt(cols)

        # the matrices that Muon updates
        self.matrices = [matrix((q + 2 * kv) * hd, dim), matrix(dim, q * hd)]
        self.matrices += [m for _ in range(experts) for m in (matrix(2 * ffn, dim), matrix(dim, ffn))]
        # the rest: embedding, head, router, norms
        self.others = [torch.randn(vocab, dim, generator=g, device=device), matrix(vocab, dim), matrix(experts, dim),
                       torch.ones(hd, device=device), torch.ones(hd, device=device)]
        for p in self.matrices + self.others:
            p.requires_grad_()
        freq = 10000.0 ** (-torch.arange(0, hd, 2, device=device) / hd)
        angle = torch.arange(length, device=device)[:, None] * freq
        self.table = torch.cat([angle.cos(), angle.sin()], 1)

    def logits(self, tokens):
        """[batch * length, vocab] in bf16."""
        bf = torch.bfloat16
        q_heads, k_heads, hd = self.heads
        wqkv, wo = (m.to(bf) for m in self.matrices[:2])
        embed, head, router, q_weight, k_weight = self.others
        batch, n = tokens.shape
        x = embed[tokens.reshape(-1)].to(bf)
        positions = torch.arange(n, device=x.device).repeat(batch)
        qkv = x @ wqkv.t()
        q, key = QkNormRope.apply(qkv, q_weight, k_weight, self.heads, self.table, positions)
        v = split_heads(qkv, self.heads)[2]
        q, key, v = (t.view(batch, n, -1, hd).transpose(1, 2) for t in (q, key, v))
        key, v = (t.repeat_interleave(q_heads // k_heads, dim=1) for t in (key, v))
        scores = (q.float() @ key.float().transpose(-1, -2)) / math.sqrt(hd)
        scores = scores.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -math.inf)
        att = (scores.softmax(-1).to(bf) @ v).transpose(1, 2).reshape(batch * n, -1)
        x = x + att @ wo.t()
        # the experts
        top = (x.float() @ router.t()).softmax(-1).topk(self.k, dim=-1)
        weights = top.values / top.values.sum(-1, keepdim=True)
        row_of_slot, slot_of_row, offsets = sort_tokens(top.indices, self.experts)
        rows = Dispatch.apply(x, row_of_slot, slot_of_row)
        out = []
        for e in range(self.experts):
            up, down = (m.to(bf) for m in self.matrices[2 + 2 * e:4 + 2 * e])
            gate, value = (rows[offsets[e]:offsets[e + 1]] @ up.t()).chunk(2, dim=-1)
            out.append((torch.nn.functional.silu(gate) * value) @ down.t())
        out.append(rows[offsets[-1]:])                       # rows without a token: zero
        x = x + Combine.apply(torch.cat(out), weights, row_of_slot, slot_of_row)
        return x @ head.to(bf).t()


class Muon:
    """Momentum of the model's matrices, orthogonalised in one batched call."""

    def __init__(self, matrices, lr=0.02, momentum=0.9):
        self.matrices, self.lr, self.momentum = matrices, lr, momentum
        self.buffers = [torch.zeros_like(m) for m in matrices]
        self.plan = nsg.ns_plan_create([tuple(m.shape) for m in matrices])
        self.inputs = [torch.empty_like(m, dtype=torch.bfloat16) for m in matrices]
        self.outputs = [torch.empty_like(t) for t in self.inputs]
        self.workspace = torch.empty(max(1, self.plan.workspace_bytes()), dtype=torch.uint8, device=matrices[0].device)

    @torch.no_grad()
    def step(self):
        for m, b, t in zip(self.matrices, self.buffers, self.inputs):
            b.mul_(self.momentum).add_(m.grad)
            t.copy_(b)
        nsg.ns_orthogonalize_batched(self.plan, self.inputs, self.outputs, self.workspace)
        for m, o in zip(self.matrices, self.outputs):
            m.sub_(o.float() * (self.lr * math.sqrt(max(1.0, m.shape[0] / m.shape[1]))))
            m.grad = None


def teacher_top(vocab, top, seed, device="cuda"):
    """A teacher that knows a token's successors: values and ids [vocab, top]."""
    g = torch.Generator(device=device).manual_seed(seed)
    logits = 3 * torch.randn(vocab, vocab, generator=g, device=device)
    return logits.topk(top, dim=1)


def train(steps=60, batch=8, top=16, seed=0, log=None, **sizes):
    """Losses of `steps` steps."""
    model = Model(seed=seed, **sizes)
    muon, rest = Muon(model.matrices), torch.optim.Adam(model.others, lr=3e-3)
    teacher = teacher_top(model.vocab, top, seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    losses = []
    for step in range(steps):
        tokens = torch.randint(0, model.vocab, (batch, model.length), generator=g, device="cuda")
        flat = tokens.reshape(-1)
        weights = torch.full((flat.numel(),), 1.0 / flat.numel(), device="cuda")
        loss, _ = Distill.apply(model.logits(tokens), teacher.values[flat], teacher.indices[flat], weights)
        loss.backward()
        muon.step()
        rest.step()
        rest.zero_grad(set_to_none=True)
        losses.append(loss.item())
        if log:
            log(f"step {step:3d}  loss {losses[-1]:.4f}")
    status = nsg.ns_check_status()
    if status != nsg.NS_OK:
        raise RuntimeError(nsg.ns_status_string(status))
    return losses


if __name__ == "__main__":
    train(log=print)
