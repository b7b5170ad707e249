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


def _cu(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()


def test_lengths_filled_anew():
    """A stack whose lengths are replaced between steps computes what one
    that was made with them does, whatever the step before left behind."""
    a = _stack(streamed=False, block_size=1, dropout=0.0)
    a.step()
    for lens in ([5, 100, 50, 41], [0, 196, 0, 0], [64, 64, 64, 4]):
        rope, pos = a.rope, a.positions.flip(1).contiguous()
        b = DecoderStack(TINY, 2, sum(LENS), streamed=False, block_size=1, rope=rope,
                         positions=pos, seq_lens=lens)
        a.cu.copy_(_cu(lens))
        a.positions.copy_(pos)
        for st in (a, b):
            st.step()
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0
        for x, y in ((a.h_cur, b.h_cur), (a.dh_cur, b.dh_cur), (a.grad_flat, b.grad_flat)):
            assert torch.equal(x, y), lens
        b.close()
    a.close()


def test_padding_is_a_sequence_of_its_own():
    """With no gradient arriving in its rows, what the padding holds changes
    no bit of the other sequences' results or of any gradient."""
    outs = []
    for fill in (0.0, 3.0, None):
        st = _stack(streamed=False, block_size=2)
        n = sum(LENS[:3]) - 30  # the third sequence shrinks, the padding grows
        st.cu.copy_(_cu([40, 1, 100, 55]))
        st.dh_top[n:] = 0
        if fill is not None:
            st.h_in[n:] = fill
        st.step()
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0
        assert not st.dh_cur[n:].any()
        outs.append([t.clone() for t in (st.h_cur[:n], st.dh_cur[:n], st.grad_flat,
                                         st.clip_grads(0.1), st.grad_flat)])
        st.close()
    for other in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], other))
