"""CPU checks of the training operators: what their kernels' sources have to
keep to, and refusals beyond those of single arguments."""
import glob
import os
import re

import pytest
import torch

from host_streamed_nf4_b200 import build, hsnf4, synth
from host_streamed_nf4_b200.decoder import DecoderStack


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


TINY = synth.Family("tiny", hidden=256, inter=640, heads=2, kv_heads=1, head_dim=128, layers=2)


@pytest.mark.parametrize("positions,error", [
    (torch.zeros(1, 64, dtype=torch.int64), TypeError), (torch.zeros(1, 64), TypeError),
    (torch.zeros(1, 64, dtype=torch.int32), ValueError),  # not on the GPU
    (torch.zeros(64, dtype=torch.int32), ValueError), (torch.zeros(2, 64), ValueError)])
def test_stack_refuses_positions_when_it_is_made(positions, error):
    """Not in the middle of its first step, after a layer has been computed."""
    rope = hsnf4.Rope(128, hsnf4.rope_inv_freq(128, 1e4))
    with pytest.raises(error, match="positions"):
        DecoderStack(TINY, 1, 64, streamed=False, rope=rope, positions=positions)


def test_stack_refuses_lengths_and_ropes_when_it_is_made():
    for kw in (dict(seq_lens=[10, 20]), dict(seq_lens=[-1, 65]), dict(seq_lens=[]),
               dict(rope=hsnf4.Rope(64, [1.0] * 32)),
               dict(positions=torch.zeros(1, 64, dtype=torch.int32))):
        with pytest.raises(ValueError):
            DecoderStack(TINY, 1, 64, streamed=False, **kw)
