"""The packed decoder stack in calls at the edges of what it allows."""
import pytest
import torch

from host_streamed_nf4_b200 import hsnf4
from host_streamed_nf4_b200.decoder import DecoderStack
from test_gpu_packed_decoder import LENS, TINY, _stack

pytestmark = pytest.mark.gpu


def test_first_clip_of_a_stack_is_captured():
    """clip_grads needs nothing made by an earlier call of it."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        st = _stack(streamed=False, block_size=2)
    st.step()
    torch.cuda.synchronize()
    before = st.grad_flat.double()
    want = before.norm()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        norm = st.clip_grads(0.5)
    assert torch.equal(st.grad_flat.double(), before)  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(norm) - float(want)) <= 2.0 ** -22 * float(want)
    exact = before * min(1.0, 0.5 / (float(norm) + 1e-6))
    assert ((st.grad_flat.double() - exact).abs() <= 2.0 ** -21 * exact.abs()).all()
    st.close()
