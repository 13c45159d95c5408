"""Kernels that let the next one start early and take tensor memory take it first: a successor's CTA that got the
columns would hold them while it waits for the very grid that waits for them."""
import os
import re

import pytest

import entropy_logits_bf16_gb300 as rlk

CSRC = os.path.join(os.path.dirname(os.path.abspath(rlk.__file__)), "csrc")


def kernels():
    """(file, name, body) of every __global__ function of the sources."""
    for name in sorted(os.listdir(CSRC)):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
        for m in re.finditer(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", text):
            at = depth = 0
            start = text.index("{", m.end())
            for at in range(start, len(text)):
                depth += (text[at] == "{") - (text[at] == "}")
                if depth == 0:
                    break
            yield name, m.group(1), text[start:at]


FOUND = [k for k in kernels() if "tc::alloc<" in k[2] and "pdl_trigger()" in k[2]]


def test_there_are_such_kernels():
    assert {(f, k) for f, k, _ in FOUND} >= {("gemm.cuh", "gemm_tiles_kernel"), ("orthogonalise.cu", "orth_resident_kernel")}


@pytest.mark.parametrize("file,name,body", FOUND, ids=[k[1] for k in FOUND])
def test_tensor_memory_comes_before_the_trigger(file, name, body):
    alloc, trigger = body.index("tc::alloc<"), body.index("pdl_trigger()")
    assert alloc < trigger
    assert "__syncthreads()" in body[alloc:trigger], "another warp may raise the trigger before the allocation returns"
