"""The rule of test_kernel_sources_host.py on the block operators' kernels: no
data before the wait for earlier kernels, CPU only."""

import re

import pytest

from test_kernel_sources_host import CSRC, bodies, without_comments

HEAD = r"__global__ void __launch_bounds__\(.*\) (\w+)\(const __grid_constant__"
FILES = ("grad_norm.cu", "block_norm.cu", "moe_few.cu")
KERNELS = {name: body for f in FILES for name, body in bodies(without_comments((CSRC / f).read_text()), HEAD)}


def test_every_kernel_is_found():
    text = "".join(without_comments((CSRC / f).read_text()) for f in FILES)
    assert len(KERNELS) == len(re.findall(r"__global__", text)) > 0


@pytest.mark.parametrize("name", KERNELS)
def test_no_data_before_the_wait(name):
    body = KERNELS[name]
    waits = [m.start() for m in re.finditer(r"griddep_wait\(\);", body)]
    assert len(waits) == 1
    before = body[:waits[0]]
    assert before.rsplit("\n", 1)[1].strip() == "nsptx::"       # on no condition
    assert not re.search(r"\bp\.|\[", re.sub(r"__shared__[^;]*;|extern[^;]*;", "", before))
    assert body.index("griddep_launch_dependents") > waits[0]
