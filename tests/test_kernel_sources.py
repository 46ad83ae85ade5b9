"""Rules of the kernels' code that no result shows, read from the sources (no GPU)."""
from __future__ import annotations

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_gemm_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def _kernels(path):
    """(name, body) of every __global__ function, comments taken out."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\(", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield m.group(1), text[at:end]


KERNELS = [(os.path.basename(f), name, body) for f in FILES for name, body in _kernels(f)]


def test_kernels_are_found():
    names = {name for _, name, _ in KERNELS}
    assert {"pair_gemm_kernel", "thin_gemm_kernel", "residual_norm_bwd_kernel", "few_rows_kernel"} <= names


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[f"{f}:{n}" for f, n, _ in KERNELS])
def test_other_blocks_memory_is_touched_after_a_cluster_barrier(file, name, body):
    """Shared memory of another block of the cluster may be accessed only once that block runs:
    a cluster barrier's wait comes before the first such access."""
    access = re.search(r"mapa\.shared|map_to_rank\(|st_cluster_v4\(|st\.shared::cluster|dsmem_addr\(|"
                       r"mbar_arrive_rank0\(", body)
    if access is None:
        return
    wait = re.search(r"barrier\.cluster\.wait|cluster_wait\(|cluster_sync\w*\(", body)
    assert wait is not None and wait.start() < access.start(), f"{name}: {access.group()} first"


@pytest.mark.parametrize("name", ["pair_gemm_kernel", "thin_gemm_kernel"])
def test_bounded_waits_answer_for_the_whole_warp(name):
    """A wait that runs out may do so in some lanes of a warp only; warp-collective work
    (tcgen05.ld, __syncwarp) may follow only an answer that its lanes share, warp_wait's."""
    (body,) = [b for _, n, b in KERNELS if n == name]
    assert "tc::warp_wait(" in body and "mbar_wait(" not in body
