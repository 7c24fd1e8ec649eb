"""Order of the launch steps in the kernels' source (CPU only).

A kernel lets its dependents start with pdl_trigger().  If a CTA does that
before it holds its tensor memory, a dependent's CTA on the same SM can take the
columns first and then wait for this grid, which waits for the columns: neither
ends.  So every kernel triggers behind its allocation, in the order of its
text."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "sparse_mixture_experts_noisy_b200", "csrc", "*.cu")))


def kernels(path):
    """(name, body) of every __global__ function of a file, comments left out."""
    text = re.sub(r"//[^\n]*", "", open(path, encoding="utf-8").read())
    parts = re.split(r"__global__", text)[1:]
    for p in parts:
        name = re.search(r"(\w+_kernel)\s*\(", p)
        depth, start = 0, p.index("{")
        for i in range(start, len(p)):
            depth += {"{": 1, "}": -1}.get(p[i], 0)
            if depth == 0:
                break
        yield name.group(1), p[start:i + 1]


FOUND = [(os.path.basename(f), name, body) for f in SOURCES for name, body in kernels(f) if "tmem_alloc" in body]


def test_the_kernels_are_found():
    names = {n for _, n, _ in FOUND}
    assert {"linear_pair_kernel", "linear_split_kernel", "route_tc_kernel", "tc_gemm_kernel", "tc2_gemm_kernel",
            "tc_wgrad_kernel", "tc_wgrad2_kernel", "decode_fused_kernel"} <= names


@pytest.mark.parametrize("file,name,body", FOUND, ids=[n for _, n, _ in FOUND])
def test_dependents_start_behind_the_allocation(file, name, body):
    alloc = max(m.start() for m in re.finditer(r"tmem_alloc", body))
    for m in re.finditer(r"pdl_trigger\(\)", body):
        # a barrier of the block lies between: every warp's trigger is behind warp 1's allocation
        assert m.start() > alloc and "__syncthreads()" in body[alloc:m.start()], (file, name)


@pytest.mark.parametrize("file", sorted({f for f, _, _ in FOUND}))
def test_launches_keep_room_for_tensor_memory(file):
    """Every launch of such a kernel is held to tmem_room(), so that no SM gets
    CTAs that need more than its 512 columns together."""
    text = re.sub(r"//[^\n]*", "", open(next(f for f in SOURCES if f.endswith(os.sep + file)), encoding="utf-8").read())
    assert text.count("tmem_room(") >= sum(f == file for f, _, _ in FOUND)
