"""CPU checks of the training operators: what their kernels' sources have to
keep to, and refusals beyond those of single arguments."""
import glob
import os
import re

from host_streamed_nf4_b200 import build


def test_tensor_memory_is_allocated_before_the_next_kernel_is_let_in():
    """A kernel let in early may allocate tensor memory and hold it until the
    grid before it has ended: that grid's CTAs must have theirs by then, or
    both wait for good (nothing bounds the wait of an allocation)."""
    seen = 0
    for path in glob.glob(os.path.join(build.CSRC, "*.cu")):
        with open(path) as fh:
            kernels = re.split(r"\b__global__\b", fh.read())[1:]
        for body in kernels:
            alloc = re.search(r"\btmem_alloc(_pair)?\(", body)
            if not alloc:
                continue
            seen += 1
            release = re.search(r"\bpdl_(wait_then_)?release\(", body)
            if release:
                between = body[alloc.end():release.start()]
                assert "__syncthreads" in between or "cluster_sync" in between, \
                    os.path.basename(path) + ": " + body[:90].strip()
    assert seen >= 8
