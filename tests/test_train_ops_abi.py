"""CPU checks of the rotary, packed-attention and gradient-clipping entry
points: every bad argument is refused before anything is enqueued."""
import ctypes
import math

import pytest
import torch

from host_streamed_nf4_b200 import hsnf4

FAKE = 0x10000  # never dereferenced: validation fails first


def _refused(rc, status, *words):
    assert rc == status, (rc, hsnf4.last_error())
    for w in words:
        assert w in hsnf4.last_error(), hsnf4.last_error()


def test_transposed_positions_and_lse_are_refused():
    """As many values in another shape would be read in the wrong order."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    rope = hsnf4.Rope(64, hsnf4.rope_inv_freq(64, 1e4), [8, 12, 12])
    pos, cu = torch.zeros(5, 3, dtype=torch.int32), torch.tensor([0, 5], dtype=torch.int32)
    with pytest.raises(ValueError, match="pos must be"):
        hsnf4.rope_fwd(rope, pos, bf(5, 64))
    lse, t = torch.zeros(5, 2), bf(5, 128)
    with pytest.raises(ValueError, match="lse must be"):
        hsnf4.attention_packed_fwd(t, t, t, cu, 2, 2, o=bf(5, 128), lse=lse)
    with pytest.raises(ValueError, match="lse must be"):
        hsnf4.attention_packed_bwd(t, t, t, t, lse, t, cu, 2, 2)


def test_rows_that_overlap_are_refused():
    """An expanded tensor has row stride 0, which the library reads as
    contiguous rows: it would leave the tensor's memory."""
    one = torch.zeros(1, 64, dtype=torch.bfloat16)
    assert hsnf4._rows(one, "q", -1, (1, 64)) == 64
    wide = torch.zeros(5, 96, dtype=torch.bfloat16)
    assert hsnf4._rows(wide[:, 16:80], "q", -1, (5, 64)) == 96
    for t in (one.expand(5, 64), wide.view(-1).as_strided((5, 64), (32, 1))):
        with pytest.raises(ValueError, match="q must be"):
            hsnf4._rows(t, "q", -1, (5, 64))


# ---------------------------------------------------------------- rotary positions

def _rope(**kw):
    a = dict(head_dim=128, inv_freq=hsnf4.rope_inv_freq(128, 10000.0), sections=[16, 24, 24])
    a.update(kw)
    return hsnf4.Rope(**a)


def _rope_call(rope, T=4, H=2, KV=1, q=FAKE, qs=0, k=FAKE * 16, ks=0, qo=FAKE * 32, qos=0,
               ko=FAKE * 64, kos=0, pos=FAKE * 128, fn="decoder_rope_fwd"):
    return getattr(hsnf4.lib(), fn)(rope._ref, pos, T, H, KV, q, qs, k, ks, qo, qos, ko, kos, None)


def test_rope_axes_of_sections():
    r = _rope()
    assert list(r.c.axis[:64]) == [0] * 16 + [1] * 24 + [2] * 24 and r.n_axes == 3
    r = _rope(sections=[4, 2, 2], inv_freq=[1.0] * 8, head_dim=16, interleaved=True)
    assert list(r.c.axis[:8]) == [0, 1, 2, 0, 1, 2, 0, 0]
    f = hsnf4.rope_inv_freq(128, 10000.0)
    assert f[0] == 1.0 and math.isclose(float(f[63]), 10000.0 ** (-126 / 128), rel_tol=2 ** -24)
    with pytest.raises(ValueError):
        _rope(sections=[16, 24, 23])
    with pytest.raises(ValueError):
        _rope(pairing="other")
    with pytest.raises(ValueError):
        hsnf4.Rope(512, [1.0] * 129)


@pytest.mark.parametrize("fn", ["decoder_rope_fwd", "decoder_rope_bwd"])
def test_rope_refusals(fn):
    bad = hsnf4.ERR_INVALID
    call = lambda rope=None, **kw: _rope_call(rope or _rope(), fn=fn, **kw)
    _refused(hsnf4.lib().decoder_rope_fwd(None, FAKE, 4, 2, 1, *[FAKE, 0] * 4, None), bad, "NULL")
    _refused(call(_rope(head_dim=120)), bad, "rot_dim")  # rot_dim 128 of 120
    _refused(call(_rope(head_dim=260)), bad, "head_dim")
    _refused(call(_rope(head_dim=64, inv_freq=[1.0] * 12, sections=[12])), bad, "rot_dim")
    _refused(call(_rope(scale=float("nan"))), bad, "scale")
    _refused(call(_rope(inv_freq=[float("inf")] * 64)), bad, "inv_freq[0]")
    r = _rope()
    r.c.axis[3] = 3
    _refused(call(r), bad, "axis[3]")
    r = _rope()
    r.c.n_axes = 9
    _refused(call(r), bad, "n_axes")
    r = _rope()
    r.c.pairing = 2
    _refused(call(r), bad, "pairing")
    for kw in (dict(T=0), dict(H=0), dict(KV=-1), dict(H=1025), dict(T=2 ** 31)):
        _refused(call(**kw), bad, "need 1 <= T")
    _refused(call(q=None), bad, "NULL")
    _refused(call(q=FAKE + 8), bad, "aligned")
    _refused(call(pos=None), bad, "pos")
    _refused(call(pos=FAKE * 128 + 2), bad, "pos")
    _refused(call(KV=0), bad, "KV = 0")
    _refused(call(qs=128), bad, "q_stride")  # below the row of 256
    _refused(call(kos=132), bad, "k_out_stride")
    # overlaps: out on another input, partly on its own input, on pos
    _refused(call(qo=FAKE * 16), bad, "overlaps")
    _refused(call(qo=FAKE + 16), bad, "overlaps")
    _refused(call(qo=FAKE, qos=512), bad, "overlaps")
    _refused(call(pos=FAKE * 32 + 4), bad, "overlaps")


# ---------------------------------------------------------------- packed attention

def _attn(**kw):
    a = dict(q=FAKE, k=FAKE * 16, v=FAKE * 32, q_stride=0, k_stride=0, v_stride=0, cu_q=FAKE * 64,
             cu_k=FAKE * 64, Tq=8, Tk=8, n_seq=2, H=4, KV=2, head_dim=128, causal=1, scale=0.1)
    a.update(kw)
    return hsnf4.PackedAttentionC(*[a[f[0]] for f in hsnf4.PackedAttentionC._fields_])


BAD_ATTN = [(dict(Tq=0), "Tq"), (dict(Tk=2 ** 24 + 1), "Tk"), (dict(n_seq=0), "n_seq"),
            (dict(n_seq=65536), "n_seq"), (dict(H=5), "multiple of KV"), (dict(KV=0), "KV"),
            (dict(H=2048, KV=1024), "H"), (dict(head_dim=80), "head_dim"), (dict(q=None), "q is"),
            (dict(v=FAKE * 32 + 2), "aligned"), (dict(cu_q=None), "cu_q"),
            (dict(cu_k=FAKE + 1), "cu_k"), (dict(causal=2), "causal"),
            (dict(scale=float("inf")), "scale"), (dict(scale=0.0), "scale"),
            (dict(q_stride=504), "q_stride"), (dict(k_stride=260), "k_stride")]


@pytest.mark.parametrize("kw,word", BAD_ATTN)
def test_attention_refusals(kw, word):
    L = hsnf4.lib()
    a = ctypes.byref(_attn(**kw))
    out = [FAKE * 128, 0, FAKE * 256]
    _refused(L.decoder_attention_packed_fwd(a, *out, None), hsnf4.ERR_INVALID, word)
    _refused(L.decoder_attention_packed_bwd(a, *out, FAKE * 300, 0, FAKE * 400, 0, FAKE * 500, 0,
                                            FAKE * 600, 0, FAKE * 1024, 1 << 30, None),
             hsnf4.ERR_INVALID, word)


def test_attention_outputs_refused():
    L = hsnf4.lib()
    a = ctypes.byref(_attn())
    bad = hsnf4.ERR_INVALID
    fwd = lambda o=FAKE * 128, os=0, lse=FAKE * 256: L.decoder_attention_packed_fwd(a, o, os, lse,
                                                                                   None)
    _refused(L.decoder_attention_packed_fwd(None, FAKE, 0, FAKE, None), bad, "NULL")
    _refused(fwd(o=None), bad, "o is NULL")
    _refused(fwd(os=500), bad, "o_stride")
    _refused(fwd(o=FAKE), bad, "overlaps q")
    _refused(fwd(lse=FAKE * 32), bad, "overlaps v")
    _refused(fwd(lse=FAKE * 128 + 64), bad, "overlaps")
    need = hsnf4.attention_packed_workspace_bytes(8, 8, 2, 4, 2, 128)
    assert need >= 4 * 8 * 4

    def bwd(o=FAKE * 128, dout=FAKE * 300, dq=FAKE * 400, dqs=0, dk=FAKE * 500, dks=0,
            dv=FAKE * 600, dvs=0, ws=FAKE * 1024, n=need):
        return L.decoder_attention_packed_bwd(a, o, 0, FAKE * 256, dout, 0, dq, dqs, dk, dks, dv,
                                              dvs, ws, n, None)

    _refused(bwd(n=need - 1), hsnf4.ERR_OOM, "need", str(need - 1))
    _refused(bwd(ws=FAKE * 1024 + 16), bad, "256-byte")
    _refused(bwd(ws=None), bad, "workspace")
    _refused(bwd(dv=None), bad, "dv")
    _refused(bwd(dq=FAKE * 300), bad, "overlaps dout")
    _refused(bwd(dk=FAKE * 600), bad, "overlaps")
    _refused(bwd(dv=FAKE * 1024), bad, "overlaps workspace")
    # dk and dv as columns of one tensor that share a column
    _refused(bwd(dk=FAKE * 500, dks=1024, dv=FAKE * 500 + 2 * 248, dvs=1024), bad, "overlaps")
    with pytest.raises(hsnf4.HsNf4Error):
        hsnf4.attention_packed_workspace_bytes(8, 8, 2, 4, 2, 96)


# ---------------------------------------------------------------- gradient norm

def _plan(grads, table=FAKE * 4096, size=1 << 20, n=None):
    arr = (hsnf4.GradC * max(len(grads), 1))(*[hsnf4.GradC(*g) for g in grads])
    plan = hsnf4.GradPlanC()
    return hsnf4.lib().lora_grad_plan(arr, len(grads) if n is None else n, table, size,
                                      ctypes.byref(plan), None)


def test_grad_plan_refusals():
    bad = hsnf4.ERR_INVALID
    ok = (FAKE, FAKE, 100, 0, 0)
    _refused(_plan([ok], n=0), bad, "1..65536")
    _refused(_plan([ok], table=None), bad, "table")
    _refused(_plan([ok], size=8), hsnf4.ERR_OOM, "need")
    _refused(_plan([(FAKE, FAKE, 100, 3, 0)]), bad, "type 3")
    _refused(_plan([(FAKE, FAKE, -1, 0, 0)]), bad, "-1 elements")
    _refused(_plan([(FAKE + 2, FAKE + 2, 8, 0, 0)]), bad, "aligned")
    _refused(_plan([(0, FAKE, 8, 0, 0)]), bad, "NULL")
    _refused(_plan([ok, ok]), bad, "overlap")  # the same tensor twice
    _refused(_plan([ok, (FAKE + 396, FAKE + 396, 4, 0, 0)]), bad, "overlap")
    _refused(_plan([(FAKE, FAKE + 4, 100, 0, 0)]), bad, "overlap")  # its own out, shifted
    # a long read-only range hides behind a shorter one that starts later
    _refused(_plan([(FAKE, FAKE * 2, 1000, 0, 0), (FAKE + 40, FAKE * 3, 2, 0, 0),
                    (FAKE * 4, FAKE + 2000, 10, 0, 0)]), bad, "overlap")
    _refused(_plan([(FAKE, FAKE * 2, 10, 0, 0), (FAKE * 4, FAKE * 2 + 36, 10, 0, 0)]), bad,
             "overlap")


def test_grad_calls_refused():
    L = hsnf4.lib()
    bad = hsnf4.ERR_INVALID
    plan = hsnf4.GradPlanC(FAKE, 3, 100, 1, 0)
    need = int(L.lora_grad_workspace(ctypes.byref(plan)))
    assert need >= 24 and need % 256 == 0
    p = ctypes.byref(plan)
    _refused(L.lora_grad_norm(None, FAKE, FAKE, need, None), bad, "plan")
    _refused(L.lora_grad_norm(ctypes.byref(hsnf4.GradPlanC()), FAKE, FAKE, need, None), bad, "plan")
    _refused(L.lora_grad_norm(p, None, FAKE, need, None), bad, "norm")
    _refused(L.lora_grad_norm(p, FAKE, FAKE, need - 1, None), hsnf4.ERR_OOM, "need")
    _refused(L.lora_grad_clip(p, -1.0, FAKE, FAKE, need, None), bad, "max_norm")
    _refused(L.lora_grad_clip(p, float("nan"), FAKE, FAKE, need, None), bad, "max_norm")
    _refused(L.lora_grad_clip(p, 1.0, FAKE, FAKE + 8, need, None), bad, "256-byte")
    with pytest.raises(ValueError):
        hsnf4.GradSet([])
    with pytest.raises(TypeError):
        hsnf4.GradSet([torch.zeros(3, dtype=torch.float64)])
    with pytest.raises(ValueError):
        hsnf4.GradSet([torch.zeros(3)])  # not on a GPU
