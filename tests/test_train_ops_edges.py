"""CPU checks of the training operators: what their kernels' sources have to
keep to, and refusals beyond those of single arguments."""
import ctypes
import glob
import os
import re
import subprocess

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


FAKE = 0x10000  # never dereferenced: validation fails first


def _refused(rc, *words):
    assert rc == hsnf4.ERR_INVALID, (rc, hsnf4.last_error())
    for w in words:
        assert w in hsnf4.last_error(), hsnf4.last_error()


@pytest.mark.parametrize("name,at", [("cu_q", FAKE * 64), ("cu_k", FAKE * 80)])
def test_attention_outputs_on_the_lengths_are_refused(name, at):
    """Lengths that an earlier CTA or kernel of the call has overwritten."""
    L = hsnf4.lib()
    a = hsnf4.PackedAttentionC(FAKE, FAKE * 16, FAKE * 32, 0, 0, 0, FAKE * 64, FAKE * 80, 8, 8, 2,
                               4, 2, 128, 1, 0.1)
    r, near = ctypes.byref(a), at - 16  # (three lengths: 12 bytes)
    _refused(L.decoder_attention_packed_fwd(r, near, 0, FAKE * 256, None), "o overlaps", name)
    _refused(L.decoder_attention_packed_fwd(r, FAKE * 128, 0, near, None), "lse overlaps", name)
    need = hsnf4.attention_packed_workspace_bytes(8, 8, 2, 4, 2, 128)

    def bwd(dq=FAKE * 400, dk=FAKE * 500, dv=FAKE * 600, ws=FAKE * 1024):
        return L.decoder_attention_packed_bwd(r, FAKE * 128, 0, FAKE * 256, FAKE * 300, 0, dq, 0, dk,
                                              0, dv, 0, ws, need, None)

    _refused(bwd(dq=near), "dq overlaps", name)
    _refused(bwd(dk=near), "dk overlaps", name)
    _refused(bwd(dv=near), "dv overlaps", name)
    _refused(bwd(ws=at), "workspace overlaps", name)


def test_gradient_table_workspace_and_norm_apart():
    """The table holds addresses that kernels write to: nothing else may."""
    L = hsnf4.lib()
    size = int(L.lora_grad_table_bytes(2))
    grads = (hsnf4.GradC * 2)(hsnf4.GradC(FAKE, FAKE * 2, 100, 0, 0),
                              hsnf4.GradC(FAKE * 4, FAKE * 4, 100, 1, 0))
    plan = hsnf4.GradPlanC()
    for table, i in ((FAKE + 384, 0), (FAKE * 2 - size + 16, 0), (FAKE * 4 + 192, 1)):
        _refused(L.lora_grad_plan(grads, 2, table, size, ctypes.byref(plan), None), "the table",
                 f"tensor {i}")
    plan = hsnf4.GradPlanC(FAKE, 3, 100, 2, 0)
    p, need = ctypes.byref(plan), int(L.lora_grad_workspace(ctypes.byref(plan)))
    for call in (L.lora_grad_norm, lambda p, *a: L.lora_grad_clip(p, 1.0, *a)):
        _refused(call(p, FAKE * 2, FAKE, need, None), "workspace overlaps the plan's table")
        _refused(call(p, FAKE + size - 4, FAKE * 2, need, None), "norm overlaps the plan's table")
        _refused(call(p, FAKE * 2 + 4, FAKE * 2, need, None), "workspace overlaps norm")


def test_lengths_of_any_int32_stay_inside_the_tensor(tmp_path):
    """The kernels' clamping of cumulative lengths, run on the CPU: the ends
    of int32 among them, whose difference is none."""
    src = tmp_path / "span.cu"
    src.write_text("""
#include <stdio.h>
#include "packed.cuh"
int main() {
  int start, end, T;
  while (scanf("%d %d %d", &start, &end, &T) == 3) {
    const hsnf4::Span s = hsnf4::span_of(start, end, T);
    printf("%d %d\\n", s.at, s.len);
  }
}
""")
    exe = tmp_path / "span"
    subprocess.run([build.NVCC, *build.ARCH, *build.CFLAGS, str(src), "-o", str(exe)], check=True,
                   capture_output=True)
    ends = [-2 ** 31, -2 ** 31 + 1, -50, -1, 0, 1, 99, 100, 101, 400, 1 << 24, 1 << 30, 2 ** 31 - 1]
    cases = [(a, b, T) for a in ends for b in ends for T in (1, 100, 2000, 1 << 24)]
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % c for c in cases), check=True,
                         capture_output=True, text=True).stdout.split()
    assert len(out) == 2 * len(cases)
    for (a, b, T), at, n in zip(cases, out[::2], out[1::2]):
        lo, hi = min(max(a, 0), T), min(max(b, 0), T)
        assert (int(at), int(n)) == (lo, max(hi - lo, 0)), (a, b, T)
