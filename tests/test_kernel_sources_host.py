"""Rules of the kernels' sources that no run can be trusted to show, CPU only.

A warp-wide (``.aligned``) barrier that lanes reach apart is undefined: the run
may hang or pass by luck. So its wrapper brings the warp together first."""

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "newton_schulz_shape_gb300" / "csrc"


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def bodies(text, head):
    """(name, body) of the functions whose heads match, braces counted."""
    for m in re.finditer(head, text):
        i = text.index("{", m.end())
        depth, j = 1, i + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[j], 0)
            j += 1
        yield m.group(1), text[i + 1:j - 1]


PTX = without_comments((CSRC / "ptx.cuh").read_text())
CLUSTER_BARRIERS = {name: body for name, body in bodies(PTX, r"__device__ __forceinline__ \w+ (\w+)\(") if "barrier.cluster" in body}


def test_the_cluster_barriers_are_found():
    assert {"cluster_arrive_relaxed", "cluster_wait", "cluster_sync_all"} <= set(CLUSTER_BARRIERS)


@pytest.mark.parametrize("name", CLUSTER_BARRIERS)
def test_warps_are_together_at_cluster_barriers(name):
    body = CLUSTER_BARRIERS[name]
    assert ".aligned" in body
    assert "__syncwarp();" in body[:body.index("asm")]


def test_warps_are_together_at_the_barriers_of_the_distillation_kernel():
    # the statements before them are some lanes' only
    text = without_comments((CSRC / "distill.cu").read_text())
    assert re.search(r"if \(lane == 0\) \*te\.any = any;\s*__syncwarp\(\);", text)
    assert re.search(r"if \(has_edge\) grad\[edge\] = from_float<T>\(mass[^\n]*\s*__syncwarp\(\);\s*__syncthreads\(\);", text)


# A kernel that starts while its predecessor runs may touch no data before its
# wait, which alone promises that what earlier kernels wrote is seen.
KERNELS = {name: body for f in ("moe.cu", "qk_rope.cu", "distill.cu")
           for name, body in bodies(without_comments((CSRC / f).read_text()), r"__global__ void __launch_bounds__\(.*\) (\w+)\(const __grid_constant__")}
DATA = r"slot_expert|load_index|load_teacher|few_entries|table_row|lane_row|lane_weights|cp_async16|load_vec|atomicOr\(p\.status" \
       r"|p\.(ids|block_counts|row_of_slot|slot_of_row|src|rows_in|weights|side|positions|partial|logits|teacher|lse)\b"


def test_the_kernels_are_found():
    assert len(KERNELS) == 10


@pytest.mark.parametrize("name", KERNELS)
def test_no_data_before_the_wait(name):
    body = KERNELS[name]
    waits = [m.start() for m in re.finditer(r"griddep_wait\(\);", body)]
    assert len(waits) == 1
    line = body[:waits[0]].rsplit("\n", 1)[1]
    assert line.strip() == "nsptx::"                       # on no condition
    assert not re.search(DATA, body[:waits[0]])
    assert body.index("griddep_launch_dependents") > waits[0]
