"""Rotary positions, packed attention and gradient clipping on the GPU
against plain implementations in 64 bits, at the sizes, masks, strides and
values where they can go wrong.

Tolerances.  A result rounded to bf16 is off by at most u = 2^-8 of itself.
A product whose bf16 operand was rounded once (the probabilities, and dS) is
off by at most u times the sum of its terms' magnitudes.  Scores are sums of
at most 128 exact products in fp32: off by at most 128 * 2^-24 times the sum
of the magnitudes, here below 2^-13 absolutely, which changes a probability
by as much relatively; exp2 and the fp32 arithmetic add a few 2^-22 more, so
w = 2^-12 times the terms' magnitudes covers both."""
import numpy as np
import pytest
import torch

from host_streamed_nf4_b200 import hsnf4

pytestmark = pytest.mark.gpu

U, W = 2.0 ** -8, 2.0 ** -12
NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _within(got, ref, tol, what):
    assert torch.isfinite(got).all(), what
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max()):.2f} "
                           "of the tolerance")


# ---------------------------------------------------------------- rotary positions

def _rope_ref(rope, pos, x, n, sign):
    """The rotation of x [T, n * d] in 64 bits, and the sum of the magnitudes."""
    c, T = rope.c, x.shape[0]
    half = c.rot_dim // 2
    f = torch.tensor(list(c.inv_freq[:half]), dtype=torch.float64, device="cuda")
    ax = torch.tensor(list(c.axis[:half]), device="cuda")
    a = pos.view(-1, T).double()[ax].T * f
    cos, sin = (a.cos() * c.scale)[:, None], (a.sin() * c.scale * sign)[:, None]
    x = x.double().reshape(T, n, c.head_dim)
    y, m = x.clone(), torch.zeros_like(x)
    i = (slice(0, half), slice(half, 2 * half)) if c.pairing == 0 else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    x1, x2 = x[..., i[0]], x[..., i[1]]
    y[..., i[0]], y[..., i[1]] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    m[..., i[0]] = m[..., i[1]] = (x1.abs() + x2.abs()) * abs(c.scale)
    return y.reshape(T, -1), m.reshape(T, -1)


# cos and sin: the angle's fp32 rounding (pi 2^-24 of half a turn) and
# sincospi's two units give 2^-21; two fp32 roundings of the products add less
ROPE_W = 2.0 ** -20

ROPE_CASES = [(1, 2, 1, 128, 64, None, "half"), (3, 1, 1, 16, 8, None, "adjacent"),
              (64, 28, 4, 128, 64, [16, 24, 24], "half"), (37, 5, 3, 80, 40, [10, 30], "half"),
              (129, 64, 8, 128, 64, [16, 24, 24], "adjacent"), (50, 3, 1, 96, 24, None, "half"),
              (33, 2, 2, 256, 128, [40, 44, 44], "half"), (17, 16, 16, 64, 16, [4, 4, 8], "adjacent"),
              (1000, 8, 8, 72, 8, None, "half")]


@pytest.mark.parametrize("T,H,KV,d,half,sections,pairing", ROPE_CASES)
@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("form", ["plain", "fused", "in_place"])
def test_rope(T, H, KV, d, half, sections, pairing, way, form):
    g = _gen(T + d)
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(2 * half, 1e4), sections, pairing=pairing,
                      scale=1.25 if form == "plain" else 1.0)
    pos = torch.randint(-5, 200_000, (rope.n_axes, T), generator=g, device="cuda",
                        dtype=torch.int32)
    if form == "fused":
        buf = _normal((T, (H + 2 * KV) * d), g)
        q, k = buf[:, :H * d], buf[:, H * d:(H + KV) * d]
    else:
        q, k = _normal((T, H * d), g), _normal((T, KV * d), g)
    fn = hsnf4.rope_fwd if way == "fwd" else hsnf4.rope_bwd
    refs = [_rope_ref(rope, pos, x, n, 1 if way == "fwd" else -1) for x, n in ((q, H), (k, KV))]
    keep = [q.clone(), k.clone()]
    got = fn(rope, pos, q, k, *((q, k) if form == "in_place" else ()))
    torch.cuda.synchronize()
    for y, (ref, mag), x, x0, n in zip(got, refs, (q, k), keep, (H, KV)):
        _within(y, ref, U * ref.abs() + ROPE_W * mag, f"rope {way}")
        rest = y.reshape(T, n, d)[..., 2 * half:]  # passed unchanged, bitwise
        assert torch.equal(rest, x0.reshape(T, n, d)[..., 2 * half:])
        if form != "in_place":
            assert torch.equal(x, x0)


@pytest.mark.parametrize("T,H,KV,d,half,sections,pairing", [
    # several tokens and turns a CTA, the last one's partly behind the end
    (40001, 2, 1, 64, 32, [10, 11, 11], "half"), (9000, 1, 1, 256, 128, None, "adjacent"),
    (70003, 1, 0, 16, 8, None, "half"), (11111, 28, 4, 128, 64, None, "half")])
def test_rope_long(T, H, KV, d, half, sections, pairing):
    if KV:
        return test_rope(T, H, KV, d, half, sections, pairing, "fwd", "in_place")
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(2 * half, 1e4), sections, pairing=pairing)
    pos, q = torch.arange(T, dtype=torch.int32, device="cuda"), _normal((T, H * d), _gen(T))
    ref, mag = _rope_ref(rope, pos, q, H, 1)
    _within(hsnf4.rope_fwd(rope, pos, q), ref, U * ref.abs() + ROPE_W * mag, "rope")


def test_rope_far_positions_and_ends():
    """Positions at the ends of int32 keep their angle, position 0 turns
    nothing, and the backward undoes the forward to rounding."""
    g = _gen(5)
    rope = hsnf4.Rope(128, hsnf4.rope_inv_freq(128, 1e6))
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9], dtype=torch.int32,
                       device="cuda")
    q = _normal((7, 256), g)
    y = hsnf4.rope_fwd(rope, pos, q)
    ref, mag = _rope_ref(rope, pos, q, 2, 1)
    # a product of 31 and 24 bits is rounded to 53 bits: at most 2^-23 of a
    # radian at 2^31, and 1/pi and its product add as much again
    _within(y, ref, U * ref.abs() + (ROPE_W + 2.0 ** -21) * mag, "far positions")
    assert torch.equal(y[0], q[0])
    back = hsnf4.rope_bwd(rope, pos, y)
    _within(back, q.double(), U * q.double().abs() + (2 * U) * mag, "there and back")


def test_rope_gradient_differences():
    """<dq, e> equals the difference of <dy, rope(q + e) - rope(q)> (the
    operator is linear), in exact inputs."""
    g = _gen(6)
    rope = hsnf4.Rope(64, hsnf4.rope_inv_freq(64, 1e4), [8, 12, 12])
    pos = torch.randint(0, 5000, (3, 20), generator=g, device="cuda", dtype=torch.int32)
    q, e, dy = (_normal((20, 4 * 64), g) for _ in range(3))
    dq = hsnf4.rope_bwd(rope, pos, dy).double()
    diff = _rope_ref(rope, pos, q.double() + e.double(), 4, 1)[0] - _rope_ref(rope, pos, q, 4, 1)[0]
    a, b = (dq * e.double()).sum(), (diff * dy.double()).sum()
    tol = (U * dq.abs() * e.double().abs()).sum() + 1e-3
    assert abs(a - b) <= tol


# ---------------------------------------------------------------- packed attention

def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _attn_ref(q, k, v, lq, lk, H, KV, causal, scale, o=None, lse=None, do=None):
    """Forward (o, lse, tolerances) or gradients (and tolerances) in 64 bits,
    sequence by sequence."""
    d = q.shape[1] // H
    z = lambda t, n: torch.zeros(t, n, d, dtype=torch.float64, device="cuda")
    Tq, Tk, G = q.shape[0], k.shape[0], H // KV
    O, TO = z(Tq, H), z(Tq, H)
    L = torch.zeros(H, Tq, dtype=torch.float64, device="cuda")
    DQ, DK, DV, TQ, TK, TV = z(Tq, H), z(Tk, KV), z(Tk, KV), z(Tq, H), z(Tk, KV), z(Tk, KV)
    q3, k3, v3 = (x.double().reshape(x.shape[0], -1, d) for x in (q, k, v))
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        rows, keys = slice(q0, q0 + a), slice(k0, k0 + b)
        q0, k0 = q0 + a, k0 + b
        mask = torch.ones(a, b, dtype=torch.bool, device="cuda")
        if causal:
            mask = mask.tril(b - a)
        for h in range(H):
            c = h // G
            s = (q3[rows, h] @ k3[keys, c].T) * scale
            s = s.masked_fill(~mask, -float("inf"))
            if do is None:
                l = torch.logsumexp(s, 1) if b else torch.full((a,), -float("inf"),
                                                               dtype=torch.float64, device="cuda")
                p = torch.where(mask, (s - l[:, None]).exp(), 0.0)
                L[h, rows] = l
                O[rows, h] = p @ v3[keys, c]
                TO[rows, h] = U * O[rows, h].abs() + (U + W) * (p @ v3[keys, c].abs())
                continue
            g = do[rows].double().reshape(a, H, d)[:, h]
            oo = o[rows].double().reshape(a, H, d)[:, h]
            l = lse[h, rows].double()[:, None]
            p = torch.where(mask, (s - l).exp(), 0.0)
            dP, D = g @ v3[keys, c].T, (g * oo).sum(1, keepdim=True)
            mag = g.abs() @ v3[keys, c].abs().T + (g * oo).abs().sum(1, keepdim=True)
            ds = p * (dP - D)
            tds = U * ds.abs() + W * p * mag
            DQ[rows, h] = scale * ds @ k3[keys, c]
            TQ[rows, h] = scale * tds @ k3[keys, c].abs()
            DK[keys, c] += scale * ds.T @ q3[rows, h]
            TK[keys, c] += scale * tds.T @ q3[rows, h].abs()
            DV[keys, c] += p.T @ g
            TV[keys, c] += (U + W) * p.T @ g.abs()
    if do is None:
        return O.flatten(1), L, TO.flatten(1)
    return [(x.flatten(1), (t + U * x.abs()).flatten(1) + 1e-30)
            for x, t in ((DQ, TQ), (DK, TK), (DV, TV))]


def _lse_within(got, ref, what):
    none = torch.isneginf(ref)
    assert torch.equal(torch.isneginf(got), none), what
    assert ((got.double() - ref)[~none].abs() <= 2.0 ** -12 + 2.0 ** -20 * ref[~none].abs()).all(), \
        what


ATTN_CASES = [
    # lens of queries, of keys (None: the same), H, KV, causal
    ([1], None, 1, 1, True), ([1, 1, 1], None, 2, 1, False), ([64], None, 2, 2, True),
    ([65], None, 2, 1, True), ([128], None, 4, 1, False), ([129], None, 3, 1, True),
    ([0, 5, 0, 0, 130, 0], None, 2, 1, True), ([100, 28], None, 4, 2, True),
    ([127, 1, 256, 2], None, 2, 1, True), ([300], None, 6, 2, False), ([257, 511], None, 7, 1, True),
    ([5, 70, 3], [200, 10, 0], 4, 2, True),   # more queries than keys: rows without a key
    ([5, 70, 3], [200, 10, 0], 4, 2, False),
    ([0, 40], [33, 0], 2, 1, True),           # keys without queries, queries without keys
    ([1, 1, 1], [1, 129, 700], 4, 1, True),   # single tokens over longer keys
    ([200], [1], 2, 1, True), ([130, 131], [640, 129], 2, 2, True),
    ([1000], None, 2, 1, True), ([33] * 40, None, 2, 1, True), ([3] * 70, None, 1, 1, False),
]


def _attn_inputs(lq, lk, H, KV, d, form, seed):
    g = _gen(seed)
    Tq, Tk = sum(lq), sum(lk)
    pad = 70 if form == "padded" else 0
    Tq, Tk = max(Tq, 1) + pad, max(Tk, 1) + pad
    if form == "fused" and Tq == Tk:
        buf = _normal((Tq, (H + 2 * KV) * d), g)
        q, k, v = buf[:, :H * d], buf[:, H * d:(H + KV) * d], buf[:, (H + KV) * d:]
    else:
        q, k, v = _normal((Tq, H * d), g), _normal((Tk, KV * d), g), _normal((Tk, KV * d), g)
    do = _normal((Tq, H * d), g)
    if form == "padded":  # rows behind the last sequence hold NaN
        for t, n in ((q, sum(lq)), (k, sum(lk)), (v, sum(lk)), (do, sum(lq))):
            t[n:] = NAN
    return q, k, v, do


@pytest.mark.parametrize("lq,lk,H,KV,causal", ATTN_CASES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("form", ["plain", "fused", "padded"])
def test_packed_attention(lq, lk, H, KV, causal, d, form):
    lk = lq if lk is None else lk
    q, k, v, do = _attn_inputs(lq, lk, H, KV, d, form, sum(lq) + d)
    cu_q, cu_k = _cu(lq), _cu(lk)
    nq, nk, scale = sum(lq), sum(lk), d ** -0.5
    mark = 7.0  # what rows outside every sequence keep
    o, dq = torch.full_like(do, mark), torch.full_like(do, mark)
    lse = torch.full((H, q.shape[0]), mark, device="cuda")
    dk = torch.full((k.shape[0], KV * d), mark, dtype=torch.bfloat16, device="cuda")
    dv = dk.clone()
    hsnf4.attention_packed_fwd(q, k, v, cu_q, H, KV, causal=causal, cu_k=cu_k, o=o, lse=lse)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    ro, rl, to = _attn_ref(q[:nq], k[:nk], v[:nk], lq, lk, H, KV, causal, scale)
    _within(o[:nq], ro, to + 1e-30, "o")
    _lse_within(lse[:, :nq], rl, "lse")
    ws = torch.full((hsnf4.attention_packed_workspace_bytes(q.shape[0], k.shape[0], len(lq), H, KV,
                                                            d),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    if form == "padded":
        o[nq:], lse[:, nq:] = NAN, NAN
    hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu_q, H, KV, causal=causal, cu_k=cu_k, dq=dq,
                               dk=dk, dv=dv, workspace=ws)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    refs = _attn_ref(q[:nq], k[:nk], v[:nk], lq, lk, H, KV, causal, scale, o[:nq], lse[:, :nq],
                     do[:nq])
    for got, (ref, tol), n, name in zip((dq, dk, dv), refs, (nq, nk, nk), ("dq", "dk", "dv")):
        _within(got[:n], ref, tol, name)
        assert (got[n:] == mark).all(), name
    if form != "padded":
        assert (o[nq:] == mark).all() and (lse[:, nq:] == mark).all()


@pytest.mark.parametrize("lq,lk,H,KV,causal", [
    # key tiles in the order of their work: long sequences among short and empty ones
    ([700, 0, 5, 640, 200, 1300, 1], None, 4, 1, True),
    ([700, 0, 5, 640, 200, 1300, 1], None, 2, 1, False), ([400, 400, 400], None, 7, 1, True),
    ([5, 600, 300, 0, 1], [900, 100, 700, 400, 0], 4, 2, True),
    ([5, 600, 300, 0, 1], [900, 100, 700, 400, 0], 4, 2, False),
    ([1] * 100 + [3000] * 2 + [1] * 26, [3] * 100 + [24500] * 2 + [2] * 26, 2, 1, False),
])
def test_packed_attention_sorted_tiles(lq, lk, H, KV, causal):
    test_packed_attention(lq, lk, H, KV, causal, 64, "padded")


def _many_heads(lq):
    """Heads that fill the device with query tiles, four per SM."""
    tiles = sum(lq) // 128 + min(len(lq), max(sum(lq), 1))
    n = torch.cuda.get_device_properties(0).multi_processor_count
    return 2 * -(-2 * n // tiles)


@pytest.mark.parametrize("lq,lk,causal", [(c[0], c[1], c[4]) for c in ATTN_CASES])
@pytest.mark.parametrize("form", ["fused", "padded"])
def test_packed_attention_many_heads(lq, lk, causal, form):
    """head_dim 64 with so many tiles that the forward takes 64 keys a step."""
    d, H, KV, lk = 64, _many_heads(lq), 2, lq if lk is None else lk
    q, k, v, _ = _attn_inputs(lq, lk, H, KV, d, form, sum(lq))
    nq, nk = sum(lq), sum(lk)
    o, lse = torch.full_like(q.contiguous(), 7.0), torch.full((H, q.shape[0]), 7.0, device="cuda")
    hsnf4.attention_packed_fwd(q, k, v, _cu(lq), H, KV, causal=causal, cu_k=_cu(lk), o=o, lse=lse)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    ro, rl, to = _attn_ref(q[:nq], k[:nk], v[:nk], lq, lk, H, KV, causal, d ** -0.5)
    _within(o[:nq], ro, to + 1e-30, "o")
    _lse_within(lse[:, :nq], rl, "lse")
    assert (o[nq:] == 7.0).all() and (lse[:, nq:] == 7.0).all()


@pytest.mark.parametrize("lq,lk,causal", [(c[0], c[1], c[4]) for c in ATTN_CASES])
@pytest.mark.parametrize("group", [1, 2])
def test_packed_attention_many_kv_heads(lq, lk, causal, group):
    """head_dim 64 with so many key tiles that two dK/dV kernels share an SM;
    two query heads a KV head share the work out where tiles are few."""
    d, lk = 64, lq if lk is None else lk
    nq, nk = sum(lq), sum(lk)
    tiles = nk // 128 + min(len(lk), max(nk, 1))
    n = torch.cuda.get_device_properties(0).multi_processor_count
    KV = -(-(2 if nk <= 128 * len(lk) else 4) * n // tiles)
    group = group if group * KV <= 1024 else 1
    H = KV * group
    q, k, v, do = _attn_inputs(lq, lk, H, KV, d, "padded", nk)
    cu_q, cu_k, scale = _cu(lq), _cu(lk), d ** -0.5
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu_q, H, KV, causal=causal, cu_k=cu_k)
    out = [torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda") for t in (q, k, v)]
    hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu_q, H, KV, causal=causal, cu_k=cu_k,
                               dq=out[0], dk=out[1], dv=out[2])
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    refs = _attn_ref(q[:nq], k[:nk], v[:nk], lq, lk, H, KV, causal, scale, o[:nq], lse[:, :nq],
                     do[:nq])
    for got, (ref, tol), rows, name in zip(out, refs, (nq, nk, nk), ("dq", "dk", "dv")):
        _within(got[:rows], ref, tol, name)
        assert (got[rows:] == 7.0).all(), name


def test_packed_attention_many_heads_large_scores_and_not_finite():
    d, KV, lens = 64, 2, [70, 50, 331, 9]
    H = _many_heads(lens)
    q, k, v, _ = _attn_inputs(lens, lens, H, KV, d, "plain", 6)
    cu = _cu(lens)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
    o4, lse4 = hsnf4.attention_packed_fwd(4 * q, k, v, cu, H, KV, scale=1.0)
    ro, rl, _ = _attn_ref(4 * q, k, v, lens, lens, H, KV, True, 1.0)
    # scores of deviation 32, their partial sums below 512: each of 64 additions is
    # off by half a step of 2^-15 there, 2^-10 in all, and 2^-9 covers exp2 too
    assert (o4.double() - ro).abs().max() <= (2 * U + 2 * 2.0 ** -9) * v.double().abs().max()
    assert (lse4.double() - rl).abs().max() <= 2.0 ** -9
    bad_q, bad_k, bad_v = q.clone(), k.clone(), v.clone()
    bad_q[70:120], bad_k[70:120], bad_v[70:120] = NAN, float("inf"), NAN
    bad_q[300, d + 3], bad_k[400, 5] = float("inf"), NAN  # head 1; KV head 0
    o2, lse2 = hsnf4.attention_packed_fwd(bad_q, bad_k, bad_v, cu, H, KV)
    torch.cuda.synchronize()
    same = (o2 == o).view(460, H, d).all(2) & (lse2 == lse).T
    want = torch.ones_like(same)
    want[70:120], want[300, 1], want[400:451, :H // 2] = False, False, False
    assert torch.equal(same, want)
    assert o2[300, d:2 * d].isnan().all() and o2[400:451, :H // 2 * d].isnan().all()
    assert lse2[1, 300].isnan() and lse2[:H // 2, 400:451].isnan().all()


def test_packed_attention_large_scores():
    """Scores in the hundreds (softmax near one key) and a scale of one."""
    d, H, KV, lens = 128, 2, 1, [200, 77]
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 3)
    q = q * 4
    cu = _cu(lens)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV, scale=1.0)
    ro, rl, _ = _attn_ref(q, k, v, lens, lens, H, KV, True, 1.0)
    # scores up to 500: their fp32 sums are off by up to 128 * 2^-24 * 128 * 16 = 2^-6 at
    # the very most (all magnitudes aligned); 2^-9 leaves room for the random sums here
    p_off = 2.0 ** -9
    mag = v.double().abs().max()
    assert (o.double() - ro).abs().max() <= (2 * U + 2 * p_off) * mag
    assert (lse.double() - rl).abs().max() <= p_off
    dq, dk, dv = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV, scale=1.0)
    torch.cuda.synchronize()
    refs = _attn_ref(q, k, v, lens, lens, H, KV, True, 1.0, o, lse, do)
    for got, (ref, tol) in zip((dq, dk, dv), refs):
        # the W part of the tolerance stands for scores off by 2^-13; here 2^-9
        _within(got, ref, tol * 16, "large scores")


def test_packed_attention_sequences_do_not_meet():
    """A sequence of NaN and infinities changes no bit of its neighbours."""
    d, H, KV, lens = 128, 4, 2, [70, 50, 131, 9]
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 4)
    cu = _cu(lens)

    def all_of(q, k, v, do):
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
        return [o, lse.T.contiguous()] + list(
            hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV))

    good = all_of(q, k, v, do)
    a, b = 70, 120  # the second sequence
    q, k, v, do = (t.clone() for t in (q, k, v, do))
    q[a:b], k[a:b], v[a:b], do[a:b] = NAN, float("inf"), NAN, -float("inf")
    bad = all_of(q, k, v, do)
    torch.cuda.synchronize()
    for x, y in zip(good, bad):
        assert torch.equal(x[:a], y[:a]) and torch.equal(x[b:], y[b:])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_packed_attention_keeps_what_is_not_finite(d, value):
    """A query, and a key, with a NaN or infinite value: every result that
    the formula makes NaN is NaN, rows that do not see it stay as they were."""
    H, KV, lens = 4, 2, [40, 200]
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 5)
    cu = _cu(lens)

    def all_of(q, k):
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
        return [o, lse.T.contiguous()] + list(
            hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV))

    good = all_of(q, k)
    for i in range(131, 163):  # all 32 columns that a thread may hold it in
        bad_q = q.clone()
        bad_q[i, d + 3] = value  # head 1, of KV head 0; its scores are infinite or NaN
        o, lse, dq, dk, dv = all_of(bad_q, k)
        torch.cuda.synchronize()
        assert o[i, d:2 * d].isnan().all() and dq[i, d:2 * d].isnan().all()
        assert dk[40:i + 1, :d].isnan().all() and dv[40:i + 1, :d].isnan().all()
        for x, y, n in ((o, good[0], H), (lse, good[1], H), (dq, good[2], H)):
            same = (x == y).reshape(240, n, -1)
            same[i, 1] = True
            assert same.all()
        assert torch.equal(dk[:, d:], good[3][:, d:]) and torch.equal(dv[:, d:], good[4][:, d:])
        assert torch.equal(dk[:40], good[3][:40]) and torch.equal(dv[:40], good[4][:40])
        assert torch.equal(dv[i + 1:, :d], good[4][i + 1:, :d])
    bad_k = k.clone()
    bad_k[140, :d] = NAN
    o, lse, dq, dk, dv = all_of(q, bad_k)
    torch.cuda.synchronize()
    assert o[140:, :2 * d].isnan().all() and lse[140:, :2].isnan().all()
    assert dq[140:, :2 * d].isnan().all() and dk[140, :d].isnan().all()
    assert torch.equal(o[:140], good[0][:140]) and torch.equal(lse[:140], good[1][:140])
    assert dv[40:, :d].isnan().all()  # each of these keys is seen by a query from 140 on


def test_packed_attention_malformed_lengths_stay_in_bounds():
    """Cumulative lengths out of order or range are clamped to the tensors;
    what they select is unspecified, what lies outside is untouched."""
    d, H, KV = 64, 2, 1
    q, k, v, do = _attn_inputs([100], [100], H, KV, d, "plain", 8)
    for cu in ([0, 400, 90], [-50, 30, 20], [90, 10, 1 << 30], [0, 0, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
        hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV)
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0


def test_packed_attention_malformed_lengths_of_sorted_tiles():
    d, H, KV = 64, 4, 1
    q, k, v, do = _attn_inputs([2000], [2000], H, KV, d, "plain", 13)
    for cu in ([0, 1 << 30, 90, 1 << 30, 0], [-50, 1900, 20, 2000, -1], [1 << 30, 0, 700, 0, 700],
               [0, 0, 0, 0, 0]):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
        hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV)
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0


def test_packed_attention_matches_single_sequence_entry():
    """One causal sequence of head_dim 128 agrees with decoder_attention_fwd
    within both results' tolerance."""
    T, H, KV, d = 333, 8, 2, 128
    q, k, v, _ = _attn_inputs([T], [T], H, KV, d, "plain", 9)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, _cu([T]), H, KV)
    o2, lse2 = hsnf4.attention_fwd(q, k, v, H, KV)
    _, rl, to = _attn_ref(q, k, v, [T], [T], H, KV, True, d ** -0.5)
    _within(o, o2.double(), 2 * to, "o")
    assert (lse - lse2).abs().max() < 2 ** -11


def test_packed_attention_repeats_bit_for_bit():
    lens = [200, 31, 1, 300]
    q, k, v, do = _attn_inputs(lens, lens, 8, 2, 128, "fused", 10)
    cu = _cu(lens)
    outs = []
    for fill in (0x00, 0xFF):
        ws = torch.full((hsnf4.attention_packed_workspace_bytes(532, 532, 4, 8, 2, 128),), fill,
                        dtype=torch.uint8, device="cuda")
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, 8, 2)
        outs.append((o, lse) + hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, 8, 2,
                                                          workspace=ws))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_packed_attention_gradient_differences():
    """Directional derivatives of <do, o> in 64 bits against the gradients."""
    lens, H, KV, d = [40, 65], 4, 2, 64
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 11)
    cu, scale = _cu(lens), d ** -0.5
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
    grads = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV)
    loss = lambda *x: (_attn_ref(*x, lens, lens, H, KV, True, scale)[0] * do.double()).sum()
    refs = _attn_ref(q, k, v, lens, lens, H, KV, True, scale, o, lse, do)
    x = [t.double() for t in (q, k, v)]
    g = _gen(12)
    # o enters D rounded to bf16: another u of |do| |o| per row, which P spreads
    for i in range(3):
        e = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up = [t + 1e-5 * e if j == i else t for j, t in enumerate(x)]
        dn = [t - 1e-5 * e if j == i else t for j, t in enumerate(x)]
        slope = (loss(*up) - loss(*dn)) / 2e-5
        got = (grads[i].double() * e).sum()
        # independent errors add in squares; ten deviations
        tol = 10 * float(((2 * refs[i][1] * e) ** 2).sum().sqrt())
        assert abs(float(got - slope)) <= tol, (i, float(got), float(slope), tol)


# ---------------------------------------------------------------- gradient norm

def _clip_ref(gs, limit):
    norm = torch.sqrt(sum(g.double().square().sum() for g in gs))
    c = min(1.0, limit / (float(norm) + 1e-6)) if limit != float("inf") else 1.0
    return norm, [g.double() * c for g in gs]


GRAD_SIZES = [[1], [3, 0, 5], [4096], [4097, 1, 8191], [0], [10 ** 6 + 7], [17] * 1000,
              [57344, 57344, 16 * 512, 512 * 16, 303104, 57344, 0, 2]]


@pytest.mark.parametrize("sizes", GRAD_SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, None])
@pytest.mark.parametrize("place", ["in_place", "out", "unaligned"])
def test_grad_clip(sizes, dtype, place):
    g = _gen(sum(sizes) + 1)
    types = [dtype or (torch.float32, torch.bfloat16, torch.float16)[i % 3]
             for i in range(len(sizes))]
    lead = 1 if place == "unaligned" else 0

    def new(n, t):  # a tensor, or one that starts off 16-byte alignment
        return torch.empty(n + lead, dtype=t, device="cuda")[lead:]

    grads = []
    for n, t in zip(sizes, types):
        x = new(n, t)
        x.copy_(torch.randn(n, generator=g, device="cuda"))
        grads.append(x)
    outs = None if place == "in_place" else [new(n, t) for n, t in zip(sizes, types)]
    gs = hsnf4.GradSet(grads, outs=outs)
    norm0, _ = _clip_ref(grads, 1.0)
    assert abs(float(hsnf4.grad_norm(gs)) - float(norm0)) <= 2.0 ** -22 * float(norm0)
    for limit in (float("inf"), 2.0 * float(norm0) + 1.0, 0.5 * float(norm0)):
        _, refs = _clip_ref(grads, limit)
        norm = hsnf4.grad_clip(gs, limit)
        torch.cuda.synchronize()
        # squares added in fp32 within a load (at most 8: 8 * 2^-24), doubles beyond, one rounding
        assert abs(float(norm) - float(norm0)) <= 2.0 ** -22 * float(norm0)
        for got, ref, t in zip(gs.outs, refs, types):
            half = torch.finfo(t).eps / 2
            tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps
            err = (got.double() - ref).abs()
            assert (err <= (half + 2.0 ** -21) * ref.abs() + tiny).all()
        if limit > float(norm0):  # a factor of one changes no bit
            assert all(torch.equal(a, b) for a, b in zip(gs.outs, grads))


def test_grad_norm_extremes():
    """No overflow or underflow of the squares; zeros; NaN and infinity."""
    one = lambda *v: hsnf4.GradSet([torch.tensor(v, dtype=torch.float32, device="cuda")])
    assert float(hsnf4.grad_norm(one(3e30, 4e30))) == pytest.approx(5e30, rel=2 ** -22)
    assert float(hsnf4.grad_norm(one(3e-30, 4e-30))) == pytest.approx(5e-30, rel=2 ** -22)
    assert float(hsnf4.grad_norm(one(0.0, -0.0, 0.0))) == 0.0
    assert float(hsnf4.grad_norm(one(1.0, float("-inf")))) == float("inf")
    assert np.isnan(float(hsnf4.grad_norm(one(1.0, NAN, 1.0, 1.0, 1.0))))
    g = one(1.0, float("inf"), 2.0)
    hsnf4.grad_clip(g, 1.0)  # a factor of 0: infinity becomes NaN, as 0 * inf does
    assert g.tensors[0].tolist()[0] == 0.0 and np.isnan(g.tensors[0].tolist()[1])
    g = one(1.0, NAN)
    hsnf4.grad_clip(g, 1.0)
    assert np.isnan(g.tensors[0].tolist()).all()
    g = one(*[3.0, 4.0] * 8)
    hsnf4.grad_clip(g, 0.0)
    assert g.tensors[0].abs().max() == 0
    g = one(3.0, 4.0)
    hsnf4.grad_clip(g, float("inf"))
    assert g.tensors[0].tolist() == [3.0, 4.0]


def test_grad_clip_many_small_and_repeats():
    g = _gen(20)
    ts = [torch.randn(1 + i % 37, generator=g, device="cuda") for i in range(5000)]
    gs = hsnf4.GradSet(ts)
    ref = float(torch.sqrt(sum(t.double().square().sum() for t in ts)))
    a, b = hsnf4.grad_norm(gs), hsnf4.grad_norm(gs, workspace=gs.new_workspace().fill_(0xFF))
    assert torch.equal(a, b) and abs(float(a) - ref) <= 2.0 ** -22 * ref


# ---------------------------------------------------------------- streams and graphs

def test_offsets_beyond_32_bits():
    """Rope, attention with its gradients and clipping at the end of tensors
    of more than 2^31 elements: the last sequence against 64 bits, rows
    before it zero."""
    H, KV, d, n = 64, 1, 128, 128
    lens = [n] * 2100 + [77]
    T, a = sum(lens), n * 2100
    assert a * H * d > 2 ** 31
    g = _gen(40)
    q, do = (torch.zeros(T, H * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k, v = (torch.zeros(T, KV * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (q, k, v, do):
        t[a:] = _normal((77, t.shape[1]), g)
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(d, 1e4))
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    ref, mag = _rope_ref(rope, pos[a:].contiguous(), q[a:], H, 1)
    hsnf4.rope_fwd(rope, pos, q, k, q, k)
    _within(q[a:], ref, U * ref.abs() + ROPE_W * mag, "rope")
    cu = _cu(lens)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
    args = ([77], [77], H, KV, True, d ** -0.5)
    ro, rl, to = _attn_ref(q[a:], k[a:], v[a:], *args)
    _within(o[a:], ro, to + 1e-30, "o")
    _lse_within(lse[:, a:], rl, "lse")
    dq, dk, dv = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV)
    refs = _attn_ref(q[a:], k[a:], v[a:], *args, o[a:], lse[:, a:].contiguous(), do[a:])
    for got, (r, tol), name in zip((dq, dk, dv), refs, ("dq", "dk", "dv")):
        _within(got[a:], r, tol, name)
    for t in (q, o, dq, dk, dv):
        assert not t[:a].any()
    gs = hsnf4.GradSet([dq])
    want = dq[a:].double().norm()
    before = dq[a:].clone()
    norm = hsnf4.grad_clip(gs, 0.5 * float(want))
    assert abs(float(norm) - float(want)) <= 2.0 ** -22 * float(want)
    c = 0.5 * float(want) / (float(norm) + 1e-6)
    assert ((dq[a:].double() - before.double() * c).abs()
            <= (U + 2.0 ** -20) * before.double().abs() * c + 1e-38).all()


def test_calls_at_once():
    """Steps of different sizes and head dimensions on three streams at once,
    each with its own workspaces, repeat what they give alone."""
    steps = []
    for lens, H, KV, d, causal in (([512] * 8, 28, 4, 128, True), ([64] * 40, 16, 16, 64, False),
                                   ([900, 3, 700], 40, 20, 64, True)):
        q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "fused", 50 + d)
        cu, pos = _cu(lens), torch.arange(sum(lens), dtype=torch.int32, device="cuda")
        rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(d, 1e4))
        o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV, causal=causal)
        g = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV, causal=causal)
        ws = torch.empty(hsnf4.attention_packed_workspace_bytes(sum(lens), sum(lens), len(lens),
                                                                H, KV, d),
                         dtype=torch.uint8, device="cuda")
        q1, k1 = torch.empty_like(do), torch.empty_like(g[1])
        out = [torch.empty_like(t) for t in g]
        gs = hsnf4.GradSet(g, outs=out)

        def step(stream=None, a=(q, k, v, do, cu, H, KV, causal, pos, rope, ws, o, lse, g, gs, q1,
                                 k1)):
            q, k, v, do, cu, H, KV, causal, pos, rope, ws, o, lse, g, gs, q1, k1 = a
            hsnf4.rope_fwd(rope, pos, q, k, q1, k1, stream=stream)
            hsnf4.attention_packed_fwd(q1, k1, v, cu, H, KV, causal=causal, o=o, lse=lse,
                                       stream=stream)
            hsnf4.attention_packed_bwd(q1, k1, v, o, lse, do, cu, H, KV, causal=causal, dq=g[0],
                                       dk=g[1], dv=g[2], workspace=ws, stream=stream)
            hsnf4.grad_clip(gs, 1.0, stream=stream)

        step()
        torch.cuda.synchronize()
        outs = [q1, k1, o, lse, *g, *out]
        steps.append((step, outs, [t.clone() for t in outs], torch.cuda.Stream()))
    for _ in range(20):
        for step, *_, stream in steps:
            step(stream)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    for _, outs, want, _ in steps:
        assert all(torch.equal(x, y) for x, y in zip(outs, want))


def test_outputs_made_by_a_call_on_a_side_stream():
    """Outputs and workspaces that a call makes belong to its stream: the
    current stream, busy meanwhile, neither fills them late nor reuses them."""
    lens, H, KV, d = [100, 33, 128], 4, 2, 128
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 33)
    cu, pos = _cu(lens), torch.arange(261, dtype=torch.int32, device="cuda")
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(d, 1e4))

    def step(stream):
        q1, k1 = hsnf4.rope_fwd(rope, pos, q, k, stream=stream)
        o, lse = hsnf4.attention_packed_fwd(q1, k1, v, cu, H, KV, stream=stream)
        g = hsnf4.attention_packed_bwd(q1, k1, v, o, lse, do, cu, H, KV, stream=stream)
        gs = hsnf4.GradSet(g, stream=stream)
        return [q1, k1, o, lse, hsnf4.grad_clip(gs, 1.0, stream=stream), *g]

    ref = step(None)
    x = torch.zeros(4096, 4096, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):  # some milliseconds of work
        x = x @ x
    got = step(side)
    junk = [torch.full_like(t, 3.0) for t in ref for _ in range(3)]
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0 and junk
    for a, b in zip(ref, got):
        assert torch.equal(a, b)


def test_ops_on_a_side_stream_and_in_a_graph():
    lens, H, KV, d = [100, 33, 128], 4, 2, 128
    q, k, v, do = _attn_inputs(lens, lens, H, KV, d, "plain", 30)
    cu = _cu(lens)
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(d, 1e4), [16, 24, 24])
    pos = torch.arange(3 * 261, dtype=torch.int32, device="cuda").view(3, 261) % 97
    b = {n: torch.zeros_like(t) for n, t in dict(q=q, k=k, o=q, dq=q, dk=k, dv=v, gq=q,
                                                 gk=k).items()}
    lse = torch.zeros(H, 261, device="cuda")
    ws = torch.empty(hsnf4.attention_packed_workspace_bytes(261, 261, 3, H, KV, d),
                     dtype=torch.uint8, device="cuda")
    gs = hsnf4.GradSet([b["gq"], b["gk"], b["dv"]],
                       outs=[torch.zeros_like(b[n]) for n in ("gq", "gk", "dv")])
    norm = torch.zeros((), device="cuda")

    def step(stream=None):
        hsnf4.rope_fwd(rope, pos, q, k, b["q"], b["k"], stream=stream)
        hsnf4.attention_packed_fwd(b["q"], b["k"], v, cu, H, KV, o=b["o"], lse=lse, stream=stream)
        hsnf4.attention_packed_bwd(b["q"], b["k"], v, b["o"], lse, do, cu, H, KV, dq=b["dq"],
                                   dk=b["dk"], dv=b["dv"], workspace=ws, stream=stream)
        hsnf4.rope_bwd(rope, pos, b["dq"], b["dk"], b["gq"], b["gk"], stream=stream)
        hsnf4.grad_clip(gs, 1.0, norm=norm, stream=stream)

    def outs():
        torch.cuda.synchronize()
        return [t.clone() for t in list(b.values()) + [lse, norm] + gs.outs]

    step()
    ref = outs()
    for t in list(b.values()) + [lse, norm] + gs.outs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    assert all(torch.equal(x, y) for x, y in zip(ref, outs()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
        with pytest.raises(hsnf4.HsNf4Error) as e:  # the table's copy is refused
            hsnf4.GradSet([q])
        assert e.value.status == hsnf4.ERR_STATE
    for seed in (31, 32):  # new inputs in the same buffers, new lengths too
        for t, new in zip((q, k, v, do), _attn_inputs(lens, lens, H, KV, d, "plain", seed)):
            t.copy_(new)
        cu.copy_(_cu([5, 200, 56]) if seed == 32 else _cu(lens))
        graph.replay()
        got = outs()
        step()
        assert all(torch.equal(x, y) for x, y in zip(outs(), got))
