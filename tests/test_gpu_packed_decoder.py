"""The decoder stack on packed sequences with rotary positions of several
axes, through a whole step and the clipping of its gradients, against the
oracle's layers."""
import numpy as np
import pytest
import torch

from oracle import decoder as odec
from host_streamed_nf4_b200 import hsnf4, synth
from host_streamed_nf4_b200.decoder import DecoderStack
from gpu_util import assert_lora_close, bf16_bits, bf16_to_f64

pytestmark = pytest.mark.gpu

TINY = synth.Family("tiny", hidden=256, inter=640, heads=2, kv_heads=1, head_dim=128, layers=2)
LENS = [40, 1, 130, 25]

# As for the single-sequence stack: about ten chained bf16 roundings per layer
# (and two more, of the turned q, k and their gradients), sqrt(12) x 1.1e-3,
# and about as much again from the attention backward's bf16 P and dS.
STACK_FRO = 1e-2


def _stack(**kw):
    rope = hsnf4.Rope(128, hsnf4.rope_inv_freq(128, 1e4), sections=[16, 24, 24])
    T = sum(LENS)
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 5000, (3, T), generator=g, dtype=torch.int32).cuda()
    return DecoderStack(TINY, 2, T, rope=rope, positions=pos, seq_lens=LENS, **kw)


def _angles(st):
    half = st.rope.c.rot_dim // 2
    f = np.array(st.rope.c.inv_freq[:half], np.float64)
    return st.positions.cpu().numpy().astype(np.float64)[list(st.rope.c.axis[:half])].T * f


def test_packed_stack_vs_oracle(orc):
    st = _stack(streamed=False, block_size=2)
    st.step()
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    layers = []
    for l in range(st.L):
        lin = {}
        for p, (name, n, k) in enumerate(st.projs):
            codes, absmax = orc.quantize(bf16_bits(st.base_weight_bf16(l, p)))
            lin[name] = odec.Linear(n, k, A=bf16_bits(st.A[l][p]), B=bf16_bits(st.B[l][p]),
                                    codes=codes, absmax=absmax)
        layers.append(odec.Layer(H=st.H, KV=st.KV, d=128, g1=bf16_to_f64(st.g1[l]),
                                 g2=bf16_to_f64(st.g2[l]), lin=lin, alpha=st.alpha,
                                 angles=_angles(st), lens=LENS))
    h, acts = bf16_to_f64(st.h_in), []
    for L in layers:
        acts.append(odec.layer_forward(L, h))
        h = acts[-1]["h2"]
    assert_lora_close(bf16_to_f64(st.h_cur), h, "stack output", fro_rel=STACK_FRO)
    dh, squares = bf16_to_f64(st.dh_top), 0.0
    for l in reversed(range(len(layers))):
        dh, grads = odec.layer_backward(layers[l], acts[l], dh)
        for p, name in enumerate(odec.PROJ):
            for got, ref, what in zip((st.dA[l][p], st.dB[l][p]), grads[name], ("dA", "dB")):
                assert_lora_close(got.cpu().numpy(), ref, f"layer {l} {name} {what}",
                                  fro_rel=STACK_FRO)
                squares += float(np.sum(np.asarray(ref, np.float64) ** 2))
    assert_lora_close(bf16_to_f64(st.dh_cur), dh, "stack input gradient", fro_rel=STACK_FRO)
    # clipping: the norm of everything (each gradient within STACK_FRO of the oracle's, so
    # the norm too), and the same factor on every gradient
    before = st.grad_flat.clone()
    norm = st.clip_grads(0.25 * np.sqrt(squares))
    torch.cuda.synchronize()
    assert abs(float(norm) - np.sqrt(squares)) <= STACK_FRO * np.sqrt(squares)
    exact = before.double() * min(1.0, 0.25 * np.sqrt(squares) / (float(norm) + 1e-6))
    assert ((st.grad_flat.double() - exact).abs() <= 2.0 ** -21 * exact.abs()).all()
    st.close()


def test_packed_streamed_equals_resident_bitwise_and_recompute():
    def run(**kw):
        st = _stack(**kw)
        rec = {}
        for _ in range(2):
            st.step(lambda l, p, n, t: rec.__setitem__((l, n), t.clone()))
        norm = st.clip_grads(1.0)
        torch.cuda.synchronize()
        out = [st.h_cur.clone(), st.dh_cur.clone(), st.grad_flat.clone(), norm]
        st.close()
        return out, rec

    ref, _ = run(streamed=False, block_size=2, dropout=0.05)
    for bs in (1, 2):
        got, rec = run(streamed=True, block_size=bs, dropout=0.05)
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), bs
        if bs == 1:  # block 0 is recomputed in the backward
            assert torch.equal(rec[(0, "h_out")], rec[(0, "h_out_recomputed")])


def test_one_packed_sequence_agrees_with_the_plain_stack():
    """seq_lens = [T] without positions is the plain stack's computation."""
    T = 96
    a = DecoderStack(TINY, 2, T, streamed=False, block_size=2)
    b = DecoderStack(TINY, 2, T, streamed=False, block_size=2, seq_lens=[T])
    for st in (a, b):
        st.step()
    torch.cuda.synchronize()
    assert_lora_close(bf16_to_f64(b.h_cur), bf16_to_f64(a.h_cur), "output", fro_rel=STACK_FRO)
    assert_lora_close(b.grad_flat.cpu().numpy(), a.grad_flat.cpu().numpy(), "gradients",
                      fro_rel=2 * STACK_FRO)
    a.close()
    b.close()


def test_packed_stack_refusals():
    with pytest.raises(ValueError):
        DecoderStack(TINY, 1, 64, streamed=False, seq_lens=[10, 20])
    with pytest.raises(ValueError):
        DecoderStack(TINY, 1, 64, streamed=False, rope=hsnf4.Rope(64, [1.0] * 32))
