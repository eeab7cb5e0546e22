"""More operators as measured cases: the global gradient norm over many tensors
and clipping, the norms after and before a block with its gate and residual
scale (each direction), and a whole mixture-of-experts layer for a few tokens.

With ``own`` false, ``run`` computes an operator in its plain form: elementary
torch operations in fp32, rounded once at the end. With ``own`` true it calls
the library.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
MOST_BYTES = 2_250_000_000          # a drawn case moves no more than the largest listed one


def _lib():
    import newton_schulz_shape_gb300 as nsg
    return nsg


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the gradients of a small one-layer model with 8 experts (18 matrices, 5 other tensors): latency
        dict(name="grad norm small", op="norm", layers=1, dim=256, qkv=384, ffn=192, experts=8, vectors=5, dtype="fp32"),
        # the matrices of 24 layers (d = 2048, gate and up as one matrix of 8192 rows), the norms' weights in fp32
        dict(name="grad norm train", op="norm", layers=24, dim=2048, qkv=6144, ffn=4096, experts=1, vectors=4, dtype="mixed"),
        # odd shapes packed one behind the other in a flat buffer: most tensors start off a 16-byte boundary
        dict(name="grad clip odd", op="clip", layers=7, dim=1001, qkv=1203, ffn=333, experts=2, vectors=3, dtype="fp16"),
        # a layer of 64 experts of 1408 x 2048, gradients kept and clipped into other buffers: the largest case
        dict(name="grad clip experts", op="clip", layers=1, dim=2048, qkv=6144, ffn=1408, experts=64, vectors=4, dtype="bf16"),
        # one decoding step of 16 sequences: norm of the block's output, residual sum, norm before the next block
        dict(name="block norm decode", op="block", dir="fwd", tokens=16, dim=2048, dtype="bf16", residual="bf16",
             post=True, gate="none", branch=True),
        # a training micro-batch with the residual stream in fp32
        dict(name="block norm train", op="block", dir="fwd", tokens=16384, dim=4096, dtype="bf16", residual="fp32",
             post=True, gate="none", branch=True),
        # the plain norm before the first block, an odd width
        dict(name="norm odd", op="block", dir="fwd", tokens=5003, dim=1001, dtype="fp16", residual="fp16",
             post=False, gate="none", branch=False),
        # a few thousand tokens with a gate for every value
        dict(name="block norm grad gated", op="block", dir="bwd", tokens=2999, dim=2048, dtype="fp32", residual="fp32",
             post=False, gate="value", branch=True),
        # training backward, a gate for each token
        dict(name="block norm grad train", op="block", dir="bwd", tokens=16384, dim=2048, dtype="bf16", residual="bf16",
             post=True, gate="token", branch=True),
        # decoding one sequence through 64 experts of 1408 x 2048
        dict(name="moe one token", op="moe", tokens=1, k=8, experts=64, dim=2048, ffn=1408, dtype="bf16", invalid=0.0),
        # a few tokens in fp16, ragged sizes, padding among the tokens
        dict(name="moe ragged", op="moe", tokens=7, k=2, experts=16, dim=1096, ffn=712, dtype="fp16", invalid=0.3),
        # 64 sequences: every expert is named, some by many tokens
        dict(name="moe 64 tokens", op="moe", tokens=64, k=6, experts=64, dim=2048, ffn=1408, dtype="bf16", invalid=0.0),
    ]


def _size(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return min(n | 1 if rng.random() < 0.3 else n, high)


def draw(rng):
    case, shrinks = _any_case(rng)
    while work(case)["bytes"] > MOST_BYTES:
        name = next(n for n in shrinks if case[n] > 1)
        case[name] //= 2
    return case


def _any_case(rng):
    """A case of any size, and what may be halved until it is small enough."""
    op = rng.choice(["norm", "clip", "block", "block", "moe"])
    if op in ("norm", "clip"):
        dim = _size(rng, 64, 4096)
        case = dict(op=op, layers=_size(rng, 1, 24), dim=dim, qkv=dim + 2 * _size(rng, 32, dim), ffn=_size(rng, 64, 4 * dim),
                    experts=rng.choice([1, 1, 2, 8, 32]), vectors=rng.randint(0, 6), dtype=rng.choice(["bf16", "fp16", "fp32", "mixed"]))
        return case, ["layers", "experts"]
    if op == "block":
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        branch = rng.random() < 0.85
        dim = _size(rng, 64, 8192)
        if rng.random() < 0.7:
            dim = (dim + 7) // 8 * 8
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), tokens=_size(rng, 1, 32768), dim=dim, dtype=dtype,
                    residual=rng.choice([dtype, dtype, "fp32"]), post=branch and rng.random() < 0.7,
                    gate=rng.choice(["none", "token", "value"]) if branch else "none", branch=branch), ["tokens"]
    experts = rng.choice([4, 8, 16, 60, 64, 128])
    dim, ffn = _size(rng, 128, 4096), _size(rng, 64, 4096)
    if rng.random() < 0.8:
        dim, ffn = (dim + 7) // 8 * 8, (ffn + 7) // 8 * 8
    return dict(op=op, tokens=_size(rng, 1, 64), k=rng.choice([1, 2, 4]) if experts == 4 else rng.choice([1, 2, 4, 6, 8]),
                experts=experts, dim=dim, ffn=ffn, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                invalid=rng.choice([0.0, 0.0, 0.3])), ["ffn"]


def _shapes(case):
    """(shapes of the matrices, lengths of the vectors): projections, experts, norms."""
    d = case["dim"]
    experts = [(2 * case["ffn"], d), (d, case["ffn"])] * case["experts"]
    return ([(case["qkv"], d), (d, d)] + experts) * case["layers"], [d] * (case["vectors"] * case["layers"])


def _bytes(name):
    return 4 if name == "fp32" else 2


def work(case):
    if case["op"] in ("norm", "clip"):
        matrices, vectors = _shapes(case)
        big, small = sum(a * b for a, b in matrices), sum(vectors)
        size = big * _bytes(case["dtype"]) + small * (4 if case["dtype"] == "mixed" else _bytes(case["dtype"]))
        both = case["op"] == "clip"
        return {"bytes": size * (2 if both else 1) + 4, "flops": (big + small) * (3 if both else 2)}
    T, D = case["tokens"], case["dim"]
    if case["op"] == "block":
        x, r, n = _bytes(case["dtype"]), _bytes(case["residual"]), T * D
        weights = D * x * (2 if case["branch"] else 1)
        gate = {"none": 0, "token": 4 * T, "value": n * x}[case["gate"]]
        if case["dir"] == "fwd":
            # branch, residual and gate in, the new residual and its norm out
            moved = n * (x + r) + (n * (x + r) if case["branch"] else 0) + gate
            return {"bytes": moved + weights, "flops": n * (12 if case["branch"] else 4)}
        # gradients of the new residual and of its norm, the new residual, branch and gate in; the inputs' gradients out
        moved = n * (x + 3 * r) + (n * 2 * x if case["branch"] else 0) + 2 * gate
        return {"bytes": moved + weights + 4 * D * (2 if case["branch"] else 1), "flops": n * (26 if case["branch"] else 11)}
    F, E, slots = case["ffn"], case["experts"], int(math.ceil(T * (1 - case["invalid"]))) * case["k"]
    named = min(E, max(case["k"], E * (1 - (1 - case["k"] / E) ** (slots / case["k"]))))     # experts that random choices name
    x = _bytes(case["dtype"])
    return {"bytes": int(named * 3 * D * F * x + 2 * T * D * x + T * case["k"] * 12), "flops": slots * 6 * D * F}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype).mul_(scale)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, device="cuda", dtype=dtype)

    if case["op"] in ("norm", "clip"):
        matrices, vectors = _shapes(case)
        mixed = case["dtype"] == "mixed"
        kinds = [(torch.bfloat16, matrices, 0.02), (torch.float32, [(n,) for n in vectors], 0.1)] if mixed else \
                [(DTYPES[case["dtype"]], matrices + [(n,) for n in vectors], 0.02)]
        s["flat"], s["grads"], s["flat_out"], s["outs"] = [], [], [], []
        for dtype, shapes, scale in kinds:
            if not shapes:
                continue
            sizes = [math.prod(shape) for shape in shapes]
            flat = randn(sum(sizes), dtype=dtype, scale=scale)
            s["flat"].append(flat)
            s["grads"] += [part.view(shape) for part, shape in zip(flat.split(sizes), shapes)]
            if case["op"] == "clip":
                out = torch.empty_like(flat)
                s["flat_out"].append(out)
                s["outs"] += [part.view(shape) for part, shape in zip(out.split(sizes), shapes)]
        s["norm"], s["max_norm"], s["eps"] = empty(1), 1.0, 1e-6
        if own:
            s["workspace"] = empty(_lib().ns_grad_norm_workspace_bytes(len(s["grads"])), dtype=torch.uint8)
        return s

    T, D, x = case["tokens"], case["dim"], DTYPES[case["dtype"]]
    if case["op"] == "block":
        r, back = DTYPES[case["residual"]], case["dir"] == "bwd"
        s["eps"], s["residual_scale"], s["branch_scale"] = 1e-6, 1.0, 0.5 if case["branch"] else 1.0
        s["weight"] = (1 + randn(D, scale=0.1)).to(x)
        s["branch"], s["branch_weight"], s["gate"] = None, None, None
        if case["branch"]:
            s["branch"], s["branch_weight"] = randn(T, D, dtype=x), (1 + randn(D, scale=0.1)).to(x)
        if case["gate"] == "token":
            s["gate"] = torch.sigmoid(randn(T))
        elif case["gate"] == "value":
            s["gate"] = torch.sigmoid(randn(T, D)).to(x)
        if not back:
            s["residual"] = randn(T, D, dtype=r, scale=3.0)
            s["residual_out"], s["out"] = empty(T, D, dtype=r) if case["branch"] else None, empty(T, D, dtype=x)
            return s
        s["residual_out"] = randn(T, D, dtype=r, scale=3.0)
        s["grad_residual_out"], s["grad_out"] = randn(T, D, dtype=r), randn(T, D, dtype=x)
        s["grad_residual"], s["grad_weight"] = empty(T, D, dtype=r), empty(D)
        s["grad_branch"], s["grad_branch_weight"] = (empty(T, D, dtype=x), empty(D)) if case["branch"] else (None, None)
        s["grad_gate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
        if own:
            s["workspace"] = empty(_lib().ns_block_norm_grad_workspace_bytes(D), dtype=torch.uint8)
        return s

    k, E, F = case["k"], case["experts"], case["ffn"]
    s["x"] = randn(T, D, dtype=x)
    s["gate_up"], s["down"] = randn(E, 2 * F, D, dtype=x, scale=D ** -0.5), randn(E, D, F, dtype=x, scale=F ** -0.5)
    liking = randn(E, scale=0.5)                    # some experts are liked more
    top = (randn(T, E) + liking).topk(k, dim=1)
    s["ids"], s["weights"] = top.indices, torch.softmax(top.values, dim=1)
    if case["invalid"]:                             # padding tokens go nowhere
        s["ids"][torch.rand(T, generator=gen, device="cuda") < case["invalid"]] = -1
    s["y"] = empty(T, D, dtype=x)
    if own:
        s["workspace"] = empty(_lib().ns_moe_few_tokens_workspace_bytes(T, k, D, F), dtype=torch.uint8)
    return s


# ------------------------------------------------------------- plain forms
def _plain_norm(s):
    sums = [flat.float().square().sum().double() for flat in s["flat"]]
    return torch.stack(sums).sum().sqrt()


def _plain_clip(s):
    norm = _plain_norm(s)
    scale = (s["max_norm"] / (norm + s["eps"])).clamp(max=1.0).float()
    return [norm.float().view(1)] + [(flat.float() * scale).to(flat.dtype) for flat in s["flat"]]


def _rms(x, eps):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)


def _plain_block(s):
    h = s["residual"].float() * s["residual_scale"]
    if s["branch"] is not None:
        u = s["branch"].float()
        if s["post"]:
            u = u * _rms(u, s["eps"])
        u = u * s["branch_weight"].float()
        if s["gate"] is not None:
            u = u * (s["gate"].float() if s["gate"].dim() == 2 else s["gate"][:, None])
        h = h + s["branch_scale"] * u
    out = (h * _rms(h, s["eps"]) * s["weight"].float()).to(s["out"].dtype)
    return (out,) if s["branch"] is None else (h.to(s["residual"].dtype), out)


def _plain_norm_grad(x, r, dy):
    """Gradient of n = x r in x, given dy = that of n; and n."""
    n = x * r
    return r * (dy - n * (dy * n).mean(-1, keepdim=True)), n


def _plain_block_grad(s):
    h, dn = s["residual_out"].float(), s["grad_out"].float()
    t, n = _plain_norm_grad(h, _rms(h, s["eps"]), dn * s["weight"].float())
    t = t + s["grad_residual_out"].float()
    grads = [(t * s["residual_scale"]).to(s["residual_out"].dtype), (dn * n).sum(0)]
    if s["branch"] is None:
        return grads
    b, w, t = s["branch"].float(), s["branch_weight"].float(), t * s["branch_scale"]
    gate = None if s["gate"] is None else s["gate"].float() if s["gate"].dim() == 2 else s["gate"][:, None]
    du = t if gate is None else t * gate
    y = b
    db = du * w
    if s["post"]:
        db, y = _plain_norm_grad(b, _rms(b, s["eps"]), db)
    grads += [db.to(s["branch"].dtype), (du * y).sum(0)]
    if gate is not None:
        dg = t * y * w
        grads.append(dg.to(s["gate"].dtype) if s["gate"].dim() == 2 else dg.sum(1))
    return grads


def _plain_moe(s):
    ids = s["ids"]
    T, k = ids.shape
    valid, slot_ids = ids >= 0, ids.clamp(min=0).reshape(-1)
    x = s["x"].float().repeat_interleave(k, dim=0)[:, :, None]
    gate, up = torch.bmm(s["gate_up"][slot_ids].float(), x)[:, :, 0].chunk(2, dim=1)
    hidden = gate / (1 + (-gate).exp()) * up
    rows = torch.bmm(s["down"][slot_ids].float(), hidden[:, :, None]).view(T, k, -1)
    return (torch.where(valid, s["weights"], 0.0)[:, :, None] * rows).sum(1).to(s["x"].dtype)


def _run_plain(s):
    if s["op"] == "norm":
        return _plain_norm(s).float().view(1)
    if s["op"] == "clip":
        return _plain_clip(s)
    if s["op"] == "block":
        return _plain_block(s) if s["dir"] == "fwd" else _plain_block_grad(s)
    return _plain_moe(s)


# --------------------------------------------------------- the library's
def _run_own(s):
    nsg = _lib()
    if s["op"] == "norm":
        nsg.ns_grad_norm(s["grads"], s["norm"], s["workspace"])
        return s["norm"]
    if s["op"] == "clip":
        nsg.ns_grad_norm(s["grads"], s["norm"], s["workspace"])
        nsg.ns_grad_clip(s["grads"], s["outs"], s["norm"], s["max_norm"], eps=s["eps"])
        return [s["norm"]] + s["flat_out"]
    if s["op"] == "moe":
        nsg.ns_moe_few_tokens(s["x"], s["ids"], s["weights"], s["gate_up"], s["down"], s["y"], s["workspace"])
        return s["y"]
    scales = dict(post_norm=s["post"], residual_scale=s["residual_scale"], branch_scale=s["branch_scale"], eps=s["eps"])
    if s["dir"] == "fwd":
        nsg.ns_block_norm(s["branch"], s["residual"], s["residual_out"], s["out"], s["branch_weight"], s["weight"], s["gate"],
                          **scales)
        return (s["out"],) if s["branch"] is None else (s["residual_out"], s["out"])
    nsg.ns_block_norm_grad(s["grad_residual_out"], s["grad_out"], s["branch"], s["residual_out"], s["grad_branch"],
                           s["grad_residual"], s["branch_weight"], s["weight"], s["gate"], s["grad_branch_weight"],
                           s["grad_weight"], s["grad_gate"], s["workspace"], **scales)
    grads = [s["grad_residual"], s["grad_weight"]]
    if s["branch"] is not None:
        grads += [s["grad_branch"], s["grad_branch_weight"]]
    return grads if s["gate"] is None else grads + [s["grad_gate"]]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# -------------------------------------------------------------- in 64 bits
def _exact_norm(x, eps):
    return x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + eps).sqrt()


def _exact_block(s, residual, branch, branch_weight, gate):
    u = (_exact_norm(branch, s["eps"]) if s["post"] else branch) * branch_weight
    if gate is not None:
        u = u * (gate if gate.dim() == 2 else gate.unsqueeze(1))
    return s["residual_scale"] * residual + s["branch_scale"] * u


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        norm = math.sqrt(math.fsum(float(torch.linalg.vecdot(g, g)) for g in (t.reshape(-1).double() for t in s["grads"])))
        out = torch.tensor([norm], dtype=torch.float64, device="cuda")
        if case["op"] == "norm":
            return out
        return [out] + [flat.double() * min(1.0, s["max_norm"] / (norm + s["eps"])) for flat in s["flat"]]
    if case["op"] == "block":
        wide = {n: None if s[n] is None else s[n].double() for n in ("branch", "branch_weight", "gate", "weight")}
        if case["dir"] == "fwd":
            h = s["residual"].double() * s["residual_scale"]
            if s["branch"] is not None:
                h = _exact_block(s, s["residual"].double(), wide["branch"], wide["branch_weight"], wide["gate"])
            out = _exact_norm(h, s["eps"]) * wide["weight"]
            return (out,) if s["branch"] is None else (h, out)
        # the norm is differentiated at the new residual as it was stored
        h, w = s["residual_out"].double().requires_grad_(), wide["weight"].requires_grad_()
        t, grad_weight = torch.autograd.grad(_exact_norm(h, s["eps"]) * w, [h, w], s["grad_out"].double())
        t = t + s["grad_residual_out"].double()
        if s["branch"] is None:
            return [t * s["residual_scale"], grad_weight]
        leaves = [torch.zeros_like(h)] + [wide[n] for n in ("branch", "branch_weight", "gate") if wide[n] is not None]
        leaves = [leaf.detach().requires_grad_() for leaf in leaves]
        got = torch.autograd.grad(_exact_block(s, *leaves[:3], leaves[3] if len(leaves) > 3 else None), leaves, t)
        return [got[0], grad_weight] + list(got[1:])
    y = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
    for e in torch.unique(s["ids"][s["ids"] >= 0]).tolist():
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        both = s["x"][t].double() @ s["gate_up"][e].double().t()
        gate, up = both[:, :case["ffn"]], both[:, case["ffn"]:]
        y.index_add_(0, t, s["weights"][t, j].double()[:, None] * ((torch.sigmoid(gate) * gate * up) @ s["down"][e].double().t()))
    return y
