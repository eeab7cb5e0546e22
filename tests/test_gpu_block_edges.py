"""Gradient norm, clipping, block norms and the experts for a few tokens at the
edges of their domains: the largest routings, matrices past 32 bits and off a
word's boundary, neighbours that must not be read or written, calls from several
host threads, a workspace shared by two graphs. Tolerances as in
test_gpu_block_ops.py."""

import threading

import numpy as np
import pytest
import torch

import test_gpu_block_ops as bo
from oracle import blocks as ob
from test_gpu_block_ops import DEV, NAN, bf16, f64, few_inputs, few_reference, fp16, fp32, gen, near, nsg, ok, randn, run_few, scratch, u

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E,D,F,dtype", [(256, 32, 1024, 64, 40, bf16), (256, 32, 1024, 33, 24, fp32), (256, 32, 1, 40, 16, fp16),
                                             (1, 32, 2, 72, 24, bf16), (4, 8, 1, 64, 64, bf16), (33, 1, 1, 64, 64, fp32)])
@pytest.mark.parametrize("invalid", [0.0, 0.97])
def test_few_tokens_of_the_largest_and_oddest_routings(T, k, E, D, F, dtype, invalid):
    g = gen(T + k + D)
    x, ids, w, up, down = few_inputs(g, T, k, E, D, F, dtype, invalid=invalid)
    y = run_few(x, ids, w, up, down)
    ok()
    near(y, *few_reference(x, ids, w, up, down), dtype)


@pytest.mark.parametrize("dtype,D,F", [(bf16, 131, 67), (bf16, 130, 66), (fp16, 64, 33), (fp32, 35, 21), (bf16, 64, 40), (fp32, 64, 40)])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_few_tokens_of_matrices_anywhere_in_memory(dtype, D, F, offset):
    # the matrices lie in larger buffers of NaN, at any value's place: nothing beside them counts
    g = gen(D + F + offset)
    T, k, E = 11, 2, 3
    x, ids, w, up, down = few_inputs(g, T, k, E, D, F, dtype, invalid=0.0)
    ids[0, 0], ids[1, 0] = 0, E - 1
    up, down = (torch.where(t.isnan(), torch.ones_like(t), t) for t in (up, down))

    def moved(t):
        buf = torch.full((t.numel() + 2 * offset + 2,), NAN, dtype=dtype, device=DEV)
        view = buf[1 + offset:1 + offset + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    want = few_reference(x, ids, w, up, down)
    near(run_few(moved(x.contiguous()), ids, w, moved(up), moved(down)), *want, dtype)
    near(run_few(x, ids, w, up, moved(down)), *want, dtype)
    ok()


def test_few_tokens_leave_their_neighbours():
    g = gen(5)
    x, ids, w, up, down = few_inputs(g, 9, 2, 4, 100, 24, bf16, invalid=0.2)
    buf = torch.full((11, 130), 3.0, dtype=bf16, device=DEV)
    y = run_few(x, ids, w, up, down, y=buf[1:10, 8:108])
    assert torch.equal(y, run_few(x, ids, w, up, down))
    buf[1:10, 8:108] = 3
    assert (buf == 3).all()
    size = nsg.ns_moe_few_tokens_workspace_bytes(9, 2, 100, 24)
    ws = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device=DEV)
    nsg.ns_moe_few_tokens(x, ids, w, up, down, y, ws[:size])
    assert (ws[size:] == 0x5A).all()
    ok()


def test_few_tokens_of_matrices_past_32_bits():
    E, D, F = 40, 8192, 8192                # 5.4e9 values of gate_up, 2.7e9 of down
    up, down = torch.zeros(E, 2 * F, D, dtype=bf16, device=DEV), torch.zeros(E, D, F, dtype=bf16, device=DEV)
    g = gen(1)
    # rows of zeros but for some; their places are the oracle's as well
    rows = [0, 1, 77, F - 1]
    x = randn(g, 2, D, dtype=bf16)
    for r in rows:
        up[E - 1, r], up[E - 1, F + r] = randn(g, D, dtype=bf16) / 64, randn(g, D, dtype=bf16) / 64
    down[E - 1, D - 5:] = randn(g, 5, F, dtype=bf16) / 2
    ids = torch.tensor([[E - 1], [3]], device=DEV)
    y = run_few(x, ids, None, up, down)
    ok()
    assert not y[1].any() and not y[0, :D - 5].any()
    small_up = torch.cat([up[E - 1, rows], up[E - 1, [F + r for r in rows]]])[None]
    small_down = down[E - 1, D - 5:, rows].contiguous()[None]
    xv = f64(x[:1])
    want = ob.moe_few_tokens(xv, np.zeros((1, 1), int), None, f64(small_up), np.pad(f64(small_down), ((0, 0), (0, D - 5), (0, 0))))[:, :5]
    both = np.abs(f64(small_up[0])) @ np.abs(xv[0])
    a, b = both[:4], both[4:]
    size = 2 * (D + 16) * u
    dh = 1.1 * size * a * (b + size * b) + a * size * b + (8 * u + 2.0 ** -17) * a * b
    bound = (np.abs(f64(small_down[0])) @ (dh + 2 * (F + 17) * u * a * b))[None]
    near(y[:1, D - 5:], want, bound, bf16)


def test_block_norms_leave_their_neighbours():
    g = gen(6)
    for D, dtype, residual in ((64, bf16, fp32), (200, bf16, bf16), (33, fp16, fp32), (72, fp32, fp32)):
        T = 21
        b, x, dn, dh = (randn(g, T, D, dtype=t) for t in (dtype, residual, dtype, residual))
        gate = randn(g, T, D, dtype=dtype)
        bufs = [torch.full((T + 2, D + 16), 3.0, dtype=t, device=DEV) for t in (residual, dtype, dtype, residual, dtype)]
        h, n, db, dx, dg = (t[1:-1, 8:8 + D] for t in bufs)
        w = randn(g, D, dtype=dtype)
        sums = torch.full((2, D + 8), 3.0, device=DEV)
        size = nsg.ns_block_norm_grad_workspace_bytes(D)
        ws = torch.full((size + 256,), 0x5A, dtype=torch.uint8, device=DEV)
        nsg.ns_block_norm(b, x, h, n, w, w, gate)
        nsg.ns_block_norm_grad(dh, dn, b, h, db, dx, w, w, gate, sums[0, :D], sums[1, 4:4 + D], dg, ws[:size])
        ok()
        for t in (h, n, db, dx, dg):
            assert t.isfinite().all() and (t != 3).any()
            t.fill_(3)
        assert all((t == 3).all() for t in bufs) and (sums[0, D:] == 3).all() and (sums[1, :4] == 3).all() and (sums[1, 4 + D:] == 3).all()
        assert (ws[size:] == 0x5A).all()


# The gradient that is taken without choices for each row, and its neighbours that are not; rows at the limits of a team.
@pytest.mark.parametrize("D", [248, 256, 264, 2048, 4096, 4104, 8192, 8200, 255, 257, 4095, 8191, 8193])
@pytest.mark.parametrize("x,r", [(bf16, bf16), (bf16, fp32), (fp32, fp32)])
@pytest.mark.parametrize("gate", ["none", "value"])
def test_rows_at_the_limits_of_a_team(D, x, r, gate):
    for T in (1, 5, 160):
        bo.test_block_norm(T, D, True, gate, True, 0, 0, x, r, False)
        bo.test_block_norm_gradient(T, D, True, gate, True, 0, 0, x, r, False)


# Rows in words, value by value in registers, and longer than those.
@pytest.mark.parametrize("D", [64, 33, 4097, 8200])
@pytest.mark.parametrize("gate", ["none", "token", "value"])
def test_every_output_of_the_gradient_in_place_of_every_input(D, gate):
    g = gen(D)
    T = 9
    dh, dn, b, h = (randn(g, T, D) for _ in range(4))
    gt = dict(none=None, token=randn(g, T), value=randn(g, T, D))[gate]
    p, w = randn(g, D), randn(g, D)
    ins = dict(dh=dh, dn=dn, b=b, h=h, **({"gt": gt} if gate == "value" else {}))
    names = ["db", "dx"] + (["dg"] if gate == "value" else [])

    def run(ins, outs):
        nsg.ns_block_norm_grad(ins["dh"], ins["dn"], ins["b"], ins["h"], outs["db"], outs["dx"], p, w, ins.get("gt", gt),
                               grad_gate=outs.get("dg"), residual_scale=0.75, branch_scale=1.5)
        return outs

    want = run(ins, {n: torch.empty(T, D, device=DEV) for n in names})
    for n in names:
        for at in ins:
            now = {k: v.clone() for k, v in ins.items()}
            got = run(now, {m: now[at] if m == n else torch.empty(T, D, device=DEV) for m in names})
            assert all(torch.equal(got[m], want[m]) for m in names), (n, at)
            assert all(torch.equal(now[k], ins[k]) for k in ins if k != at)
    ok()


def test_rows_past_32_bits():
    T, D = (2 ** 32 + 2 ** 20) // 8192 + 3, 8192
    x = torch.zeros(T, D, dtype=bf16, device=DEV)
    x[-1], x[T // 2, 0] = 2.0, 1.0
    h, n = torch.empty_like(x), torch.empty_like(x)
    nsg.ns_block_norm(x, x, h, n, eps=0.25)
    ok()
    assert (h[-1] == torch.tensor(2.0 + 2.0 / 4.25 ** 0.5, dtype=bf16)).all() and not h[-2].any() and n[T // 2, 0] != 0
    dw = torch.empty(D, device=DEV)
    nsg.ns_block_norm_grad(None, x, None, h, None, n, grad_weight=dw, workspace=scratch(nsg.ns_block_norm_grad_workspace_bytes(D)), eps=0.25)
    ok()
    m = f64(h[-1])[1] / np.sqrt(f64(h[-1])[1] ** 2 + 0.25)
    assert abs(dw[1].item() - 2 * m) <= 2.0 ** -18


def test_the_sum_of_a_row_that_is_not_given_is_not_needed():
    # h as infinite as it likes: without a gradient of its norm only the branch is normalised
    g = gen(8)
    b, dh = randn(g, 3, 64), randn(g, 3, 64)
    h = torch.full((3, 64), float("inf"), device=DEV)
    db, dx = torch.empty_like(b), torch.empty_like(b)
    nsg.ns_block_norm_grad(dh, None, b, h, db, dx)
    assert torch.equal(dx, dh) and db.isfinite().all()
    h.fill_(NAN)
    nsg.ns_block_norm_grad(dh, None, b, h, db, dx)
    assert torch.equal(dx, dh) and db.isfinite().all()
    nsg.ns_block_norm_grad(dh, None, b, h, db, dx, post_norm=False)
    assert torch.equal(db, dh)
    ok()


def test_calls_from_several_host_threads():
    g = gen(9)
    few = [few_inputs(g, T, 2, 8, D, 48, bf16, invalid=0.0) for T, D in ((1, 64), (40, 512), (200, 100), (9, 2048))]
    rows = [randn(g, T, D, dtype=bf16) for T, D in ((3, 64), (500, 2048), (70, 1001), (9, 8192))]
    grads = [[randn(g, n) for n in sizes] for sizes in ((5,), (70000, 3), (1 << 20,), (100,) * 40)]

    def calls(i):
        y = run_few(*few[i])
        h, n = torch.empty_like(rows[i]), torch.empty_like(rows[i])
        nsg.ns_block_norm(rows[i], rows[i], h, n)
        d = torch.empty_like(h)
        dw = torch.empty(h.shape[1], device=DEV)
        nsg.ns_block_norm_grad(h, n, rows[i], h, None, d, grad_weight=dw, workspace=scratch(nsg.ns_block_norm_grad_workspace_bytes(h.shape[1])))
        return y, h, n, d, dw, bo.run_norm(grads[i])

    want = [calls(i) for i in range(4)]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got[i] = calls(i)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    ok()


def test_two_graphs_share_their_workspaces():
    g = gen(10)
    x, ids, w, up, down = few_inputs(g, 20, 2, 4, 256, 64, bf16, invalid=0.0)
    other = few_inputs(g, 3, 2, 4, 256, 64, bf16, invalid=0.0)
    size = max(nsg.ns_moe_few_tokens_workspace_bytes(T, 2, 256, 64) for T in (20, 3))
    ws, wb = scratch(size), scratch(nsg.ns_block_norm_grad_workspace_bytes(256))
    out = [torch.empty(20, 256, dtype=bf16, device=DEV), torch.empty(3, 256, dtype=bf16, device=DEV)]
    sums = [torch.empty(256, device=DEV) for _ in range(2)]

    def run(i):
        a = (x, ids, w, up, down) if i == 0 else other
        nsg.ns_moe_few_tokens(*a, out[i], ws)
        nsg.ns_block_norm_grad(out[i], out[i], None, a[0], None, None, grad_weight=sums[i], workspace=wb)

    for i in range(2):
        run(i)
    want = [t.clone() for t in out + sums]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            run(i)
    for i in (0, 1, 1, 0, 1):
        for t in (out[i], sums[i]):
            t.fill_(9)
        graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out + sums, want))
    ok()


def test_gradients_that_a_captured_step_clips():
    # the norm, and with it the scale, is of the replay's gradients
    g = gen(11)
    grads = [randn(g, 3000), randn(g, 17, dtype=fp16)]
    outs = [torch.empty_like(t) for t in grads]
    norm, ws = torch.empty(1, device=DEV), scratch(nsg.ns_grad_norm_workspace_bytes(2))
    nsg.ns_grad_norm(grads, norm, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsg.ns_grad_norm(grads, norm, ws)
        nsg.ns_grad_clip(grads, outs, norm, 1.0)
    for scale in (1.0, 1e-4, 30.0):
        for t in grads:
            t.mul_(scale)
        graph.replay()
        n = ob.grad_norm([f64(t) for t in grads])
        assert abs(norm.item() - n) <= 32 * u * n
        for a, b in zip(grads, outs):
            c = ob.clip_scale(norm.item(), 1.0)
            near(b, c * f64(a), 2 * u * np.abs(c * f64(a)), a.dtype)
    ok()


def test_a_list_that_changes_during_the_call():
    # python code that runs between the look at the tensors and the launch empties the list
    grads = [torch.ones(1000, device=DEV) for _ in range(50)]
    norm = torch.full((1,), 4.0, device=DEV)

    class Number:
        def __float__(self):
            grads.clear()
            return 1.0

    kept = list(grads)
    nsg.ns_grad_clip(grads, grads, norm, Number(), eps=0.0)
    assert not grads
    assert all(t._version == 1 for t in kept)       # as the write counts
    assert all((t == 0.25).all() for t in kept)
    for given in (tuple(kept), iter(kept)):
        nsg.ns_grad_norm(given, norm, scratch(nsg.ns_grad_norm_workspace_bytes(50)))
        assert abs(norm.item() - (50 * 1000 / 16) ** 0.5) <= 32 * u * norm.item()
    ok()
