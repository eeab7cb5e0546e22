"""The mixture-of-experts model of muon_moe_step.py with a norm before and after
each block, its gradients clipped by their global norm, and its next tokens
decoded through the experts' form for a few tokens:

  tokens -> norm (ns_block_norm) -> attention -> norm, residual sum and norm in
  one pass (ns_block_norm) -> experts -> the same, with a gate for each token
  -> logits -> distillation; back through ns_block_norm_grad; then ns_grad_norm
  and ns_grad_clip over every gradient, Muon for the matrices

and, for decoding, ns_moe_few_tokens on the last position of each sequence.

  python examples/muon_block_step.py          # 60 steps on cuda:0
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import muon_moe_step as moe  # noqa: E402

nsg = moe.nsg


class BlockNorm(torch.autograd.Function):
    """(new residual, its norm) of a block's output and the residual; without a
    block (branch None) the norm of the residual."""

    @staticmethod
    def forward(ctx, branch, residual, branch_weight, weight, gate):
        new = torch.empty_like(residual) if branch is not None else None
        out = torch.empty_like(residual, dtype=residual.dtype if branch is None else branch.dtype)
        nsg.ns_block_norm(branch, residual, new, out, branch_weight, weight, gate)
        ctx.save_for_backward(branch, residual if new is None else new, branch_weight, weight, gate)
        if new is None:
            return out
        return new, out

    @staticmethod
    def backward(ctx, *grads):
        branch, h, branch_weight, weight, gate = ctx.saved_tensors
        grad_new, grad_out = (None, grads[0]) if branch is None else grads
        grad_branch, grad_gate = (None if t is None else torch.empty_like(t) for t in (branch, gate))
        grad_residual, grad_weight = torch.empty_like(h), torch.empty(h.shape[1], device=h.device)
        grad_branch_weight = None if branch is None else torch.empty_like(grad_weight)
        ws = torch.empty(nsg.ns_block_norm_grad_workspace_bytes(h.shape[1]), dtype=torch.uint8, device=h.device)
        nsg.ns_block_norm_grad(None if grad_new is None else grad_new.contiguous(), grad_out.contiguous(), branch, h, grad_branch,
                               grad_residual, branch_weight, weight, gate, grad_branch_weight, grad_weight, grad_gate, ws)
        if grad_branch_weight is not None:
            grad_branch_weight = grad_branch_weight.to(branch_weight.dtype)
        return grad_branch, grad_residual, grad_branch_weight, grad_weight.to(weight.dtype), grad_gate


def clip_gradients(tensors, max_norm):
    """Scales the gradients of the tensors in place to a global norm of at most
    max_norm; the norm before, on the GPU."""
    grads = [t.grad for t in tensors if t.grad is not None]
    norm = torch.empty(1, device=grads[0].device)
    ws = torch.empty(nsg.ns_grad_norm_workspace_bytes(len(grads)), dtype=torch.uint8, device=grads[0].device)
    nsg.ns_grad_norm(grads, norm, ws)
    nsg.ns_grad_clip(grads, grads, norm, max_norm)
    return norm


class Model(moe.Model):
    """The layer of muon_moe_step.py between norms."""

    def __init__(self, **sizes):
        super().__init__(**sizes)
        device = self.others[0].device
        # before attention; after it, before the experts; after them, before the head
        self.norms = [torch.ones(self.dim, device=device).requires_grad_() for _ in range(5)]
        self.others = self.others + self.norms

    def attention(self, tokens):
        """(residual, its norm) after attention, [batch * length, dim]."""
        bf = torch.bfloat16
        q_heads, k_heads, hd = self.heads
        wqkv, wo = (m.to(bf) for m in self.matrices[:2])
        embed, q_weight, k_weight = self.others[0], *self.others[3:5]
        batch, n = tokens.shape
        x = embed[tokens.reshape(-1)].to(bf)
        positions = torch.arange(n, device=x.device).repeat(batch)
        qkv = BlockNorm.apply(None, x, None, self.norms[0], None) @ wqkv.t()
        q, key = moe.QkNormRope.apply(qkv, q_weight, k_weight, self.heads, self.table, positions)
        v = moe.split_heads(qkv, self.heads)[2]
        q, key, v = (t.view(batch, n, -1, hd).transpose(1, 2) for t in (q, key, v))
        key, v = (t.repeat_interleave(q_heads // k_heads, dim=1) for t in (key, v))
        scores = (q.float() @ key.float().transpose(-1, -2)) / math.sqrt(hd)
        scores = scores.masked_fill(torch.ones(n, n, dtype=torch.bool, device=x.device).triu(1), -math.inf)
        att = (scores.softmax(-1).to(bf) @ v).transpose(1, 2).reshape(batch * n, -1)
        return BlockNorm.apply(att @ wo.t(), x, self.norms[1], self.norms[2], None)

    def choose(self, n):
        """Experts of each token, their weights, and the token's gate: the probability that they have together."""
        top = (n.float() @ self.others[2].t()).softmax(-1).topk(self.k, dim=-1)
        gate = top.values.sum(-1)
        return top.indices, top.values / gate[:, None], gate

    def logits(self, tokens):
        """[batch * length, vocab] in bf16."""
        bf = torch.bfloat16
        x, n = self.attention(tokens)
        ids, weights, gate = self.choose(n)
        row_of_slot, slot_of_row, offsets = moe.sort_tokens(ids, self.experts)
        rows = moe.Dispatch.apply(n, row_of_slot, slot_of_row)
        out = []
        for e in range(self.experts):
            up, down = (m.to(bf) for m in self.matrices[2 + 2 * e:4 + 2 * e])
            a, b = (rows[offsets[e]:offsets[e + 1]] @ up.t()).chunk(2, dim=-1)
            out.append((torch.nn.functional.silu(a) * b) @ down.t())
        out.append(rows[offsets[-1]:])                       # rows without a token: zero
        y = moe.Combine.apply(torch.cat(out), weights, row_of_slot, slot_of_row)
        return BlockNorm.apply(y, x, self.norms[3], self.norms[4], gate)[1] @ self.others[1].to(bf).t()

    def expert_weights(self):
        """The experts' matrices as ns_moe_few_tokens takes them; made once for many decoded tokens."""
        bf = torch.bfloat16
        return torch.stack(self.matrices[2::2]).detach().to(bf), torch.stack(self.matrices[3::2]).detach().to(bf)

    @torch.no_grad()
    def next_logits(self, tokens, experts):
        """[batch, vocab] of the position after each sequence."""
        batch, n = tokens.shape
        x, normed = (t.view(batch, n, -1)[:, -1] for t in self.attention(tokens))
        ids, weights, gate = self.choose(normed)
        y = torch.empty(batch, self.dim, dtype=x.dtype, device=x.device)
        size = nsg.ns_moe_few_tokens_workspace_bytes(batch, self.k, self.dim, experts[1].shape[2])
        nsg.ns_moe_few_tokens(normed, ids, weights, *experts, y, torch.empty(size, dtype=torch.uint8, device=x.device))
        out = torch.empty_like(y)
        nsg.ns_block_norm(y, x, None, out, self.norms[3], self.norms[4], gate)
        return out @ self.others[1].to(out.dtype).t()

    def generate(self, tokens, count):
        """`count` more tokens of each sequence, the likeliest each time."""
        experts = self.expert_weights()
        for _ in range(count):
            tokens = torch.cat([tokens, self.next_logits(tokens, experts).argmax(-1, keepdim=True)], 1)
        return tokens


def train(steps=60, batch=8, top=16, seed=0, max_norm=1.0, log=None, **sizes):
    """(model, losses, gradient norms before clipping) of `steps` steps."""
    model = Model(seed=seed, **sizes)
    muon, rest = moe.Muon(model.matrices), torch.optim.Adam(model.others, lr=3e-3)
    teacher = moe.teacher_top(model.vocab, top, seed + 1)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    losses, norms = [], []
    for step in range(steps):
        tokens = torch.randint(0, model.vocab, (batch, model.length), generator=g, device="cuda")
        flat = tokens.reshape(-1)
        weights = torch.full((flat.numel(),), 1.0 / flat.numel(), device="cuda")
        loss, _ = moe.Distill.apply(model.logits(tokens), teacher.values[flat], teacher.indices[flat], weights)
        loss.backward()
        norms.append(clip_gradients(model.matrices + model.others, max_norm))
        muon.step()
        rest.step()
        rest.zero_grad(set_to_none=True)
        losses.append(loss.item())
        if log:
            log(f"step {step:3d}  loss {losses[-1]:.4f}  gradient norm {norms[-1].item():.4f}")
    status = nsg.ns_check_status()
    if status != nsg.NS_OK:
        raise RuntimeError(nsg.ns_status_string(status))
    return model, losses, [n.item() for n in norms]


if __name__ == "__main__":
    trained = train(log=print)[0]
    start = torch.arange(4, device="cuda")[:, None]
    print(trained.generate(start, 12).tolist())
