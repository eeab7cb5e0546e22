"""The training-step operators as measured cases: tokens sorted by expert and
back (sort, dispatch, combine), norms of queries and keys with the position
rotation, and distillation from a teacher's top logits; each direction.

With ``own`` false, ``run`` computes an operator in its plain form: elementary
torch operations in fp32, rounded once at the end. With ``own`` true it calls
the library.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MOST_BYTES = 2_100_000_000          # a drawn case moves no more than the largest listed one


def _lib():
    import newton_schulz_shape_gb300 as nsg
    return nsg


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 32 sequences through a 128-expert layer
        dict(name="sort decode", op="sort", tokens=32, k=8, experts=128, align=1, capacity=0, invalid=0.0),
        # a training micro-batch over 64 experts, segments padded to 128-row product tiles
        dict(name="sort train", op="sort", tokens=32768, k=6, experts=64, align=128, capacity=0, invalid=0.0),
        # the same layer's rows, hidden size 2048
        dict(name="dispatch train", op="dispatch", dir="fwd", tokens=8192, k=6, experts=64, dim=2048, dtype="bf16",
             align=128, capacity=0, invalid=0.0),
        # an odd width in fp32 (rows not 16-byte aligned) with a tenth of the slots dropped
        dict(name="dispatch grad odd", op="dispatch", dir="bwd", tokens=3001, k=3, experts=20, dim=1001, dtype="fp32",
             align=1, capacity=0, invalid=0.1),
        # decoding: few tokens, wide rows
        dict(name="combine decode", op="combine", dir="fwd", tokens=16, k=8, experts=128, dim=4096, dtype="fp16",
             align=1, capacity=0, invalid=0.0),
        # training backward, the largest routing case
        dict(name="combine grad train", op="combine", dir="bwd", tokens=16384, k=6, experts=64, dim=2048, dtype="bf16",
             align=1, capacity=2048, invalid=0.0),
        # decoding: 32 query and 8 key heads of 128 out of a fused projection
        dict(name="qk decode", op="qk", dir="fwd", tokens=16, q_heads=32, k_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, dtype="bf16", fused=True),
        # ragged: 80-wide heads, a partial interleaved rotation, separate buffers
        dict(name="qk ragged", op="qk", dir="fwd", tokens=5003, q_heads=13, k_heads=13, head_dim=80, rot_dim=32,
             interleaved=True, dtype="fp16", fused=False),
        # training backward of the 32/8-head layer
        dict(name="qk grad train", op="qk", dir="bwd", tokens=16384, q_heads=32, k_heads=8, head_dim=128, rot_dim=128,
             interleaved=False, dtype="bf16", fused=True),
        # few rows of a large vocabulary: a row has to be split
        dict(name="distill few rows", op="distill", dir="both", tokens=8, vocab=131072, top=64, dtype="bf16",
             temperature=1.0, masked=0.0, full=False),
        # odd vocabulary in fp32, prompt tokens masked, gradient from a kept log-sum-exp
        dict(name="distill grad odd", op="distill", dir="grad", tokens=1531, vocab=50001, top=20, dtype="fp32",
             temperature=2.0, masked=0.3, full=True),
        # a training micro-batch: the largest case
        dict(name="distill train", op="distill", dir="both", tokens=4096, vocab=131072, top=64, dtype="bf16",
             temperature=1.0, masked=0.0, full=False),
    ]


def _size(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.3:
        n |= 1
    n = min(max(n, low), high)
    return n + 1 if n == 3072 else n


def _shrunk(case):
    while work(case)["bytes"] > MOST_BYTES:
        case["tokens"] = max(1, case["tokens"] // 2)
    return case


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "qk", "distill"])
    if op == "qk":
        head_dim = rng.choice([32, 64, 72, 80, 96, 112, 128, 160, 192, 256])
        q_heads, group = rng.choice([(8, 1), (12, 3), (13, 1), (16, 4), (20, 5), (32, 4), (40, 5), (64, 8)])
        return _shrunk(dict(op=op, dir=rng.choice(["fwd", "bwd"]), tokens=_size(rng, 1, 16384), q_heads=q_heads,
                            k_heads=q_heads // group, head_dim=head_dim,
                            rot_dim=rng.choice([head_dim, head_dim, head_dim // 2, 2 * rng.randint(1, head_dim // 2)]),
                            interleaved=rng.random() < 0.4, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                            fused=rng.random() < 0.6))
    if op == "distill":
        vocab = _size(rng, 1000, 200000)
        return _shrunk(dict(op=op, dir=rng.choice(["both", "both", "loss", "grad"]), tokens=_size(rng, 1, 4096),
                            vocab=vocab, top=rng.choice([1, 8, 20, 32, 64, 100, 128]),
                            dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                            temperature=rng.choice([0.7, 1.0, 2.0]), masked=rng.choice([0.0, 0.0, 0.2, 0.5]),
                            full=rng.random() < 0.4))
    experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    tokens = _size(rng, 1, 32768)
    case = dict(op=op, tokens=tokens, k=k, experts=experts, align=rng.choice([1, 1, 16, 128]), capacity=0,
                invalid=rng.choice([0.0, 0.0, 0.1]))
    if rng.random() < 0.3:
        case["capacity"] = max(1, int(tokens * k / experts * rng.choice([1.0, 1.25, 2.0])))
    if op != "sort":
        case.update(dir=rng.choice(["fwd", "bwd"]), dim=_size(rng, 64, 8192), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    return _shrunk(case)


def _rows(case):
    """Rows that hold any routing of the case."""
    slots, experts, align, cap = case["tokens"] * case["k"], case["experts"], case["align"], case["capacity"]
    rows = slots + min(experts, slots) * (align - 1)
    if cap:
        rows = min(rows, experts * ((cap + align - 1) // align * align))
    return rows


def work(case):
    T, op = case["tokens"], case["op"]
    if op == "qk":
        size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
        values = T * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
        n = 2 if case["dir"] == "fwd" else 3
        return {"bytes": values * size * n + T * (4 * case["rot_dim"] + 8) + 2 * case["head_dim"] * (size + 4 * (n - 2)),
                "flops": values * (6 if case["dir"] == "fwd" else 12)}
    if op == "distill":
        size = torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
        live = int(round(T * (1 - case["masked"])))
        teacher = live * case["top"] * (size + 8) + T * 16
        read = live * case["vocab"] * size
        write = 0 if case["dir"] == "loss" else T * case["vocab"] * size
        return {"bytes": read + write + teacher, "flops": live * case["vocab"] * (4 if case["dir"] == "both" else 3)}
    slots, rows = T * case["k"], _rows(case)
    if op == "sort":
        return {"bytes": 8 * slots + 4 * slots + 4 * rows + 8 * case["experts"], "flops": 2 * slots}
    row = case["dim"] * torch.empty(0, dtype=DTYPES[case["dtype"]]).element_size()
    kept = int(min(slots * (1 - case["invalid"]), rows))
    forward = case["dir"] == "fwd"
    if op == "dispatch":
        bytes_ = T * row + rows * row + 4 * rows if forward else kept * row + T * row + 4 * slots
        return {"bytes": bytes_, "flops": 0 if forward else kept * case["dim"]}
    if forward:
        return {"bytes": kept * row + T * row + 8 * slots, "flops": 2 * kept * case["dim"]}
    return {"bytes": T * row + kept * row + rows * row + 12 * slots + 4 * rows, "flops": 3 * kept * case["dim"]}


# ------------------------------------------------------------------ inputs
def _routing(case, gen):
    """Expert choices as a router makes them: distinct for a token, some experts
    liked more; a share of the tokens is padding and goes nowhere (-1)."""
    T, k, E = case["tokens"], case["k"], case["experts"]
    liking = torch.randn(E, generator=gen, device="cuda") * 0.5
    ids = (torch.randn(T, E, generator=gen, device="cuda") + liking).topk(k, dim=1).indices
    if case["invalid"]:
        ids[torch.rand(T, generator=gen, device="cuda") < case["invalid"]] = -1
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)
    T, op = case["tokens"], case["op"]

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype) * scale

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if op == "qk":
        dt, H, K, D, R = DTYPES[case["dtype"]], case["q_heads"], case["k_heads"], case["head_dim"], case["rot_dim"]

        def heads(make):
            if case["fused"]:        # q and k are columns of one projection [q heads | k heads | v heads]
                qkv = make(T, (H + 2 * K) * D, dtype=dt)
                return qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + K) * D].view(T, K, D)
            return make(T, H, D, dtype=dt), make(T, K, D, dtype=dt)

        s["q"], s["k"] = heads(randn)
        s["q_weight"], s["k_weight"] = (1 + 0.1 * randn(D)).to(dt), (1 + 0.1 * randn(D)).to(dt)
        freq = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float32) / R)
        limit = 32768
        angle = torch.arange(limit, device="cuda", dtype=torch.float32)[:, None] * freq
        s["table"] = torch.cat([angle.cos(), angle.sin()], dim=1).contiguous()
        start = int(torch.randint(0, limit - T + 1, (1,), generator=gen, device="cuda"))
        s["positions"] = torch.arange(start, start + T, device="cuda", dtype=torch.int64)
        s["eps"] = 1e-6
        if case["dir"] == "fwd":
            s["q_out"], s["k_out"] = empty(T, H, D, dtype=dt), empty(T, K, D, dtype=dt)
        else:
            s["dq_out"], s["dk_out"] = randn(T, H, D, dtype=dt), randn(T, K, D, dtype=dt)
            s["dq"], s["dk"] = heads(empty)
            s["dq_weight"], s["dk_weight"] = empty(D), empty(D)
            if own:
                s["workspace"] = empty(_lib().ns_qk_norm_rope_grad_workspace_bytes(D), dtype=torch.uint8)
        return s

    if op == "distill":
        dt, V, K = DTYPES[case["dtype"]], case["vocab"], case["top"]
        s["logits"] = randn(T, V, dtype=dt, scale=2.0)
        first = torch.randint(0, V, (T, 1), generator=gen, device="cuda")
        s["teacher_ids"] = (first + torch.arange(K, device="cuda") * (V // K)) % V
        s["teacher_values"] = (4 + 2 * randn(T, K)).sort(dim=1, descending=True).values.to(dt)
        # the student is near the teacher on its top entries
        s["logits"].scatter_add_(1, s["teacher_ids"], (4 + randn(T, K)).to(dt))
        s["weights"] = (torch.rand(T, generator=gen, device="cuda") >= case["masked"]).float() / T
        s["teacher_lse"] = (s["teacher_values"].float() / case["temperature"]).exp().sum(1).mul(1.05).log() if case["full"] else None
        s["loss"], s["lse"] = empty(T), empty(T)
        if case["dir"] != "loss":
            s["grad"] = empty(T, V, dtype=dt)
        if case["dir"] == "grad":
            s["lse"] = _plain_lse(s["logits"], case["temperature"])
        return s

    slots, rows = T * case["k"], _rows(case)
    s["rows"] = rows
    ids = _routing(case, gen)
    if op == "sort":
        s["ids"] = ids
        s["row_of_slot"], s["slot_of_row"] = empty(T, case["k"], dtype=torch.int32), empty(rows, dtype=torch.int32)
        s["counts"], s["offsets"] = empty(case["experts"], dtype=torch.int32), empty(case["experts"] + 1, dtype=torch.int32)
        if own:
            s["workspace"] = empty(_lib().ns_moe_sort_workspace_bytes(T, case["k"], case["experts"]), dtype=torch.uint8)
        return s
    dt, D = DTYPES[case["dtype"]], case["dim"]
    s["row_of_slot"], s["slot_of_row"], _, _ = _plain_sort(ids, case["experts"], case["align"], case["capacity"], rows)
    if op == "combine":
        s["weights"] = torch.softmax(randn(T, case["k"]), dim=1)
        s["expert_rows"] = randn(rows, D, dtype=dt)
    if op == "dispatch" and case["dir"] == "fwd":
        s["x"], s["out"] = randn(T, D, dtype=dt), empty(rows, D, dtype=dt)
    elif op == "dispatch":
        s["grad_rows"], s["out"] = randn(rows, D, dtype=dt), empty(T, D, dtype=dt)
    elif case["dir"] == "fwd":
        s["out"] = empty(T, D, dtype=dt)
    else:
        s["dy"], s["out"], s["dw"] = randn(T, D, dtype=dt), empty(rows, D, dtype=dt), empty(T, case["k"])
    return s


# ------------------------------------------------------------- plain forms
def _plain_sort(ids, experts, align, capacity, rows):
    flat = ids.reshape(-1)
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts).long()
    order = torch.sort(key, stable=True).indices
    key = key[order]
    total = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).index_add_(0, key, torch.ones_like(key))
    kept = total.clone()
    if capacity:
        kept.clamp_(max=capacity)
    kept[experts] = 0
    segment = (kept + (align - 1)) // align * align
    offsets = segment.cumsum(0) - segment          # one past the last expert: the rows in use
    rank = torch.arange(n, device=ids.device) - (total.cumsum(0) - total)[key]
    keep = rank < kept[key]
    row = offsets[key] + rank
    row_of_slot = torch.empty(n, dtype=torch.int32, device=ids.device)
    row_of_slot[order] = torch.where(keep, row, -1).int()
    slot_of_row = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    slot_of_row[torch.where(keep, row, rows)] = order.int()
    return row_of_slot.view(ids.shape), slot_of_row[:rows], kept[:experts].int(), offsets.int()


def _take_rows(rows, row_of_slot):
    """fp32 [T, k, D]: the row of each slot, zero where the slot was dropped."""
    got = rows[row_of_slot.clamp(min=0).long()].float()
    return got * (row_of_slot >= 0)[..., None]


def _put_rows(x, slot_of_row, k, weights=None):
    """fp32 [R, D]: the token of each row, zero in padding."""
    slot = slot_of_row.clamp(min=0).long()
    got = x[slot // k].float()
    if weights is not None:
        got = got * weights.reshape(-1)[slot][:, None]
    return got * (slot_of_row >= 0)[:, None]


def _plain_rotate(x, table, positions, rot, interleaved, back):
    cos, sin = table[positions][:, None, :rot // 2], table[positions][:, None, rot // 2:]
    sin = -sin if back else sin
    part, rest = x[..., :rot], x[..., rot:]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    part = torch.stack([u, v], dim=-1).flatten(-2) if interleaved else torch.cat([u, v], dim=-1)
    return torch.cat([part, rest], dim=-1)


def _plain_norm_rope(s, x, weight):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    return _plain_rotate(x * r * weight.float(), s["table"], s["positions"], s["rot_dim"], s["interleaved"], False)


def _plain_norm_rope_grad(s, x, weight, dy):
    u = _plain_rotate(dy.float(), s["table"], s["positions"], s["rot_dim"], s["interleaved"], True)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    n = x * r
    g = u * weight.float()
    return r * (g - n * (g * n).mean(-1, keepdim=True)), (u * n).sum((0, 1))


def _plain_lse(logits, temperature):
    x = logits.float() / temperature
    top = x.max(dim=1, keepdim=True).values
    return ((x - top).exp().sum(dim=1).log() + top[:, 0])


def _plain_distill(s):
    tau, V = s["temperature"], s["vocab"]
    z = s["teacher_values"].float() / tau
    ids = s["teacher_ids"]
    valid = (ids >= 0) & (z > -math.inf)
    live = (s["weights"] != 0) & valid.any(dim=1)
    z = torch.where(valid, z, -math.inf)
    if s["teacher_lse"] is None:
        top = torch.where(live, z.max(dim=1).values, torch.zeros(()).cuda())[:, None]
        logz = (z - top).exp().sum(dim=1, keepdim=True).log() + top
    else:
        logz = s["teacher_lse"][:, None]
    logp = z - logz
    p = logp.exp()
    at = ids.clamp(min=0)
    out = []
    lse = s["lse"]
    if s["dir"] != "grad":
        lse = _plain_lse(s["logits"], tau)
        student = s["logits"].gather(1, at).float() / tau
        terms = torch.where(p > 0, p * (logp - student + lse[:, None]), torch.zeros(()).cuda())
        loss = torch.where(live, s["weights"] * terms.sum(dim=1), torch.zeros(()).cuda())
        lse = torch.where(live, lse, torch.zeros(()).cuda())
        out = [loss, lse]
    if s["dir"] != "loss":
        scale = s["weights"] / tau
        grad = (s["logits"].float() / tau - lse[:, None]).exp_()
        grad *= (scale * p.sum(dim=1))[:, None]
        grad.scatter_add_(1, at, -scale[:, None] * p)
        grad[~live] = 0
        out.append(grad.to(s["logits"].dtype))
    return out


def _run_plain(s):
    op, forward = s["op"], s.get("dir") == "fwd"
    if op == "sort":
        return _plain_sort(s["ids"], s["experts"], s["align"], s["capacity"], s["rows"])
    if op == "dispatch" and forward:
        return _put_rows(s["x"], s["slot_of_row"], s["k"]).to(s["x"].dtype)
    if op == "dispatch":
        return _take_rows(s["grad_rows"], s["row_of_slot"]).sum(1).to(s["grad_rows"].dtype)
    if op == "combine" and forward:
        return (_take_rows(s["expert_rows"], s["row_of_slot"]) * s["weights"][..., None]).sum(1).to(s["expert_rows"].dtype)
    if op == "combine":
        d_rows = _put_rows(s["dy"], s["slot_of_row"], s["k"], s["weights"]).to(s["dy"].dtype)
        return d_rows, (_take_rows(s["expert_rows"], s["row_of_slot"]) * s["dy"].float()[:, None]).sum(-1)
    if op == "qk" and forward:
        return (_plain_norm_rope(s, s["q"], s["q_weight"]).to(s["q"].dtype), _plain_norm_rope(s, s["k"], s["k_weight"]).to(s["q"].dtype))
    if op == "qk":
        dq, dq_weight = _plain_norm_rope_grad(s, s["q"], s["q_weight"], s["dq_out"])
        dk, dk_weight = _plain_norm_rope_grad(s, s["k"], s["k_weight"], s["dk_out"])
        return dq.to(s["q"].dtype), dk.to(s["q"].dtype), dq_weight, dk_weight
    return _plain_distill(s)


# --------------------------------------------------------- the library's
def _run_own(s):
    nsg = _lib()
    op, forward = s["op"], s.get("dir") == "fwd"
    if op == "sort":
        nsg.ns_moe_sort(s["ids"], s["experts"], s["row_of_slot"], s["slot_of_row"], s["counts"], s["offsets"], s["workspace"],
                        align=s["align"], capacity=s["capacity"])
        return s["row_of_slot"], s["slot_of_row"], s["counts"], s["offsets"]
    if op == "dispatch" and forward:
        nsg.ns_moe_dispatch(s["x"], s["row_of_slot"], s["slot_of_row"], s["out"])
        return s["out"]
    if op == "dispatch":
        nsg.ns_moe_dispatch_grad(s["grad_rows"], s["row_of_slot"], s["out"])
        return s["out"]
    if op == "combine" and forward:
        nsg.ns_moe_combine(s["expert_rows"], s["weights"], s["row_of_slot"], s["out"])
        return s["out"]
    if op == "combine":
        nsg.ns_moe_combine_grad(s["dy"], s["expert_rows"], s["weights"], s["row_of_slot"], s["slot_of_row"], s["out"], s["dw"])
        return s["out"], s["dw"]
    if op == "qk" and forward:
        nsg.ns_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["q_weight"], s["k_weight"], s["table"], s["positions"],
                            eps=s["eps"], interleaved=s["interleaved"])
        return s["q_out"], s["k_out"]
    if op == "qk":
        nsg.ns_qk_norm_rope_grad(s["dq_out"], s["dk_out"], s["q"], s["k"], s["dq"], s["dk"], s["q_weight"], s["k_weight"],
                                 s["dq_weight"], s["dk_weight"], s["table"], s["positions"], s["workspace"],
                                 eps=s["eps"], interleaved=s["interleaved"])
        return s["dq"], s["dk"], s["dq_weight"], s["dk_weight"]
    if s["dir"] == "grad":
        nsg.ns_distill_grad(s["logits"], s["teacher_values"], s["teacher_ids"], s["lse"], s["grad"], weights=s["weights"],
                            teacher_lse=s["teacher_lse"], temperature=s["temperature"])
        return [s["grad"]]
    nsg.ns_distill_loss(s["logits"], s["teacher_values"], s["teacher_ids"], s["loss"], s["lse"], grad_logits=s.get("grad"),
                        weights=s["weights"], teacher_lse=s["teacher_lse"], temperature=s["temperature"])
    return [s["loss"], s["lse"], s["grad"]] if s["dir"] == "both" else [s["loss"], s["lse"]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- in 64 bits
def _exact_qk(s, x, weight):
    """Norm and rotation as a complex product, position by position."""
    R, D = s["rot_dim"], s["head_dim"]
    y = x / ((x ** 2).sum(-1, keepdim=True) / D + s["eps"]).sqrt() * weight
    row = s["table"].double()[s["positions"]][:, None]
    turn = torch.complex(row[..., :R // 2], row[..., R // 2:])
    pairs = y[..., :R].unflatten(-1, (R // 2, 2)) if s["interleaved"] else y[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    turned = turned.flatten(-2) if s["interleaved"] else turned.transpose(-1, -2).flatten(-2)
    return torch.cat([turned, y[..., R:]], -1)


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None                     # whole numbers: compared bit for bit
    s = prepare(case, seed)
    if op == "qk":
        leaves = [s[n].double().requires_grad_() for n in ("q", "k", "q_weight", "k_weight")]
        q, k = _exact_qk(s, leaves[0], leaves[2]), _exact_qk(s, leaves[1], leaves[3])
        if case["dir"] == "fwd":
            return q.detach(), k.detach()
        return torch.autograd.grad([q, k], leaves, [s["dq_out"].double(), s["dk_out"].double()])
    if op == "distill":
        tau = case["temperature"]
        x = s["logits"].double().requires_grad_()
        logq = torch.log_softmax(x / tau, dim=1)
        z = s["teacher_values"].double() / tau
        logp = torch.log_softmax(z, dim=1) if s["teacher_lse"] is None else z - s["teacher_lse"].double()[:, None]
        if case["dir"] == "grad":       # the given log-sum-exp is an input of the gradient
            logq = x / tau - s["lse"].double()[:, None]
            with torch.no_grad():
                grad = logq.exp().mul_(logp.exp().sum(1, keepdim=True)).scatter_add_(1, s["teacher_ids"], -logp.exp())
                return [grad.mul_((s["weights"].double() / tau)[:, None])]
        loss = s["weights"].double() * (logp.exp() * (logp - logq.gather(1, s["teacher_ids"]))).sum(1)
        lse = torch.where(s["weights"] != 0, torch.logsumexp(x.detach() / tau, dim=1), 0.0)
        out = [loss.detach(), lse]
        if case["dir"] == "both":
            out += torch.autograd.grad(loss.sum(), x)
        return out
    T, k = case["tokens"], case["k"]
    rows = s["row_of_slot"].reshape(-1).long()
    slots = torch.nonzero(rows >= 0)[:, 0]
    rows, tokens = rows[slots], slots // k
    R, D = s["rows"], case["dim"]

    def zeros(n):
        return torch.zeros(n, D, dtype=torch.float64, device="cuda")

    if op == "dispatch" and case["dir"] == "fwd":
        return zeros(R).index_copy_(0, rows, s["x"].double()[tokens])
    if op == "dispatch":
        return zeros(T).index_add_(0, tokens, s["grad_rows"].double()[rows])
    y, w = s["expert_rows"].double(), s["weights"].double().reshape(-1)
    if case["dir"] == "fwd":
        return zeros(T).index_add_(0, tokens, y[rows] * w[slots][:, None])
    dy = s["dy"].double()[tokens]
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda").index_copy_(0, slots, torch.linalg.vecdot(dy, y[rows]))
    return zeros(R).index_copy_(0, rows, dy * w[slots][:, None]), dw.view(T, k)
