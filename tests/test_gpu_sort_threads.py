"""The token sort called from several host threads at once: what one call sets
for its launch must not reach another's."""

import threading

import numpy as np
import pytest
import torch

from oracle import training as ot

pytestmark = pytest.mark.gpu
nsg = pytest.importorskip("newton_schulz_shape_gb300")


def test_sorts_of_different_sizes_from_several_threads():
    # 540 to 1024 experts take more shared memory than a kernel has by default, each its own amount;
    # the C function is called without the interpreter's lock
    T, k, calls = 64, 2, 2000
    answers, wrong = [], []

    def work(E, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
        out = [torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (T * k, T * k, E, E + 1)]
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        start.wait()
        rcs = [nsg.lib.ns_moe_sort(ids.data_ptr(), 8, T, k, E, 1, 0, T * k, *[t.data_ptr() for t in out], None, 0,
                                   stream.cuda_stream) for _ in range(calls)]
        stream.synchronize()
        answers.extend(rcs)
        want = ot.moe_sort(ids.cpu().numpy(), E, 1, 0, T * k)
        if not all(np.array_equal(a.cpu().numpy(), b.reshape(-1)) for a, b in zip(out, want)):
            wrong.append(E)

    experts = [540, 1024, 700, 1000]
    start = threading.Barrier(len(experts))
    threads = [threading.Thread(target=work, args=(E, E)) for E in experts]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(answers) == calls * len(experts)
    assert all(rc == nsg.NS_OK for rc in answers), sum(rc != nsg.NS_OK for rc in answers)
    assert not wrong
    assert nsg.ns_check_status() == nsg.NS_OK
