"""Orders in the kernels' sources that no run on the GPU may try out."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hybrid_gated_deltanet_q4k_gb300", "csrc")


def _kernels(path):
    """Bodies of the __global__ functions of a source."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__", text):
        at = text.index("{", m.end())
        depth, end = 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(text[end], 0)
            end += 1
            if depth == 0:
                break
        yield text[at:end]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_a_dependent_kernel_takes_tensor_memory_after_its_wait(path):
    """A programmatic dependent that allocates before its wait can hold the tensor memory that the kernel it waits for
    has yet to allocate, and one that triggers before its allocation does that to itself: neither ends."""
    for body in _kernels(path):
        alloc = [m.start() for m in re.finditer(r"t5::alloc", body)]
        waits = [m.start() for m in re.finditer(r"pdl_wait\(\)|griddepcontrol\.wait", body)]
        triggers = [m.start() for m in re.finditer(r"pdl_trigger\(\)", body)]
        if alloc and waits:
            assert min(waits) < min(alloc)
        if alloc and triggers:
            assert max(alloc) < min(triggers)
