"""Waits that no clock ends stand where what they wait for cannot be missing. Read from the sources: a
kernel that never ends is nothing to try on a GPU.

The allocation of tensor memory for a pair of CTAs waits for a warp of each, and for columns that others
hold on either SM. So it stands behind a cluster barrier (both CTAs run) and behind the wait for the
stream's kernels before (none of them holds columns any more)."""
import glob
import os
import re

import pytest

from moe_ffn_expert_gb300 import build as mm_build


def kernels_of_pairs():
    """(file:name, text of the body) of every kernel that allocates tensor memory for a pair."""
    found = []
    for path in sorted(glob.glob(os.path.join(mm_build.CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for part in re.split(r"\b__global__\b", text)[1:]:
            name = re.search(r"\b(k_\w+)\s*\(", part).group(1)
            body = part[part.index("{"):part.index("\n}")]
            if "tmem_alloc_pair(" in body:
                found.append((f"{os.path.basename(path)}:{name}", body))
    return found


def test_the_kernels_are_found():
    assert [name for name, _ in kernels_of_pairs()] == ["mm_gemm.cu:k_gemm", "mm_grouped.cu:k_grouped"]


@pytest.mark.parametrize("name,body", kernels_of_pairs(), ids=[n for n, _ in kernels_of_pairs()])
def test_tensor_memory_of_a_pair_is_allocated_behind_what_it_waits_for(name, body):
    before = body[:body.index("tmem_alloc_pair(")]
    assert "pdl_wait();" in before and "cluster_sync();" in before
    assert before.index("pdl_wait();") < before.rindex("cluster_sync();")


ALIGNED = r"bar\.sync|bar\.red|barrier\.cluster|setmaxnreg"
TOGETHER = r"__syncwarp\(\)|__syncthreads\w*\(|_sync\(0x"


def test_aligned_barriers_of_the_grouped_products_find_their_warps_together():
    """A barrier in its aligned form counts a warp whose lanes come apart twice: in front of each stands, in
    the same few lines, what brings them together."""
    for name in ("mm_grouped.cu", "mm_device.cuh"):
        lines = re.sub(r"//[^\n]*", "", open(os.path.join(mm_build.CSRC, name)).read()).split("\n")
        found = [i for i, line in enumerate(lines) if re.search(ALIGNED, line)]
        assert found
        for i in found:
            if "setmaxnreg.inc" in lines[i]:  # the other branch of the same decision
                continue
            assert re.search(TOGETHER, "\n".join(lines[max(0, i - 6):i])), (name, lines[i])
