"""Rotary positions, packed attention and gradient clipping in calls at the
edges of what the header allows: two query tiles per CTA, queries without a
key beside values that are not finite, memory around the tensors, streams.

Tolerances are those of the operators' other tests, with their reasons."""
import pytest
import torch

import test_gpu_train_ops as ops
from host_streamed_nf4_b200 import hsnf4

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- packed attention

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lq,lk", [(6400, 100), (7000, 900), (8192, 7000)])
def test_first_query_tile_of_a_pair_without_keys(d, lq, lk):
    """One long sequence (two query tiles per CTA) whose queries outnumber the
    keys so that the causal mask leaves a pair's first tile nothing and its
    second one something: the first one's rows are 0, -inf."""
    H, KV = 2, 1
    assert 128 < (lq - lk) % 256 < 256
    q, k, v, do = ops._attn_inputs([lq], [lk], H, KV, d, "padded", lk)
    o = torch.full_like(do, 7.0)
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    cu_q, cu_k = ops._cu([lq]), ops._cu([lk])
    ref, rl, tol = ops._attn_ref(q[:lq], k[:lk], v[:lk], [lq], [lk], H, KV, True, d ** -0.5)
    for _ in range(8):
        hsnf4.attention_packed_fwd(q, k, v, cu_q, H, KV, cu_k=cu_k, o=o, lse=lse)
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0
        assert not o[:lq - lk].any() and torch.isneginf(lse[:, :lq - lk]).all()
        ops._within(o[:lq], ref, tol + 1e-30, "o")
        ops._lse_within(lse[:, :lq], rl, "lse")
        assert (o[lq:] == 7.0).all() and (lse[:, lq:] == 7.0).all()


@pytest.mark.parametrize("d,H,KV,lq,lk", [
    (64, 2, 1, 200, 30), (128, 2, 1, 200, 30), (64, 2, 1, 6300, 30), (128, 2, 1, 6300, 30),
    (64, 1000, 2, 200, 30)])  # (so many heads take 64 keys a step)
@pytest.mark.parametrize("value", [ops.NAN, float("inf")])
def test_queries_without_keys_beside_values_that_are_not_finite(d, H, KV, lq, lk, value):
    """A query that sees no key gives 0, -inf and no gradient whatever its
    sequence's keys and values hold, in the tile of queries that see some too."""
    q, k, v, do = ops._attn_inputs([lq], [lk], H, KV, d, "plain", d)
    k[3, 5], v[7, 9] = value, value
    cu_q, cu_k, none = ops._cu([lq]), ops._cu([lk]), lq - lk
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu_q, H, KV, cu_k=cu_k)
    dq, _, _ = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu_q, H, KV, cu_k=cu_k)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    assert not o[:none].any() and torch.isneginf(lse[:, :none]).all() and not dq[:none].any()
    assert torch.isfinite(lse[:, none:none + 3]).all()  # these see finite keys alone


@pytest.mark.parametrize("d,H,KV,lq", [(64, 2, 1, 150), (128, 2, 1, 150), (64, 2, 1, 6200),
                                       (128, 2, 1, 6200), (64, 1000, 2, 150)])
def test_first_keys_with_scores_of_minus_infinity(d, H, KV, lq):
    """130 keys whose scores are -inf in every query, then keys with scores
    near -256: the softmax of those, as without the first ones.  Whole numbers, so that
    the scores are exact."""
    lk, g = 300, ops._gen(lq + d)
    small = lambda t, n: torch.randint(-1, 2, (t, n, d), generator=g, device="cuda").bfloat16()
    q, k = small(lq, H), small(lk, KV)
    q[..., 0], q[..., 1], k[..., 1] = 1, 32, -32
    k[:130, :, 0] = -float("inf")
    q, k, v = q.flatten(1), k.flatten(1), ops._normal((lk, KV * d), g)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, ops._cu([lq]), H, KV, causal=False,
                                        cu_k=ops._cu([lk]), scale=0.25)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    ref, rl, tol = ops._attn_ref(q, k, v, [lq], [lk], H, KV, False, 0.25)
    ops._within(o, ref, tol + 1e-30, "o")
    ops._lse_within(lse, rl, "lse")


@pytest.mark.parametrize("lq,lk,causal", [
    # (6144 queries a sequence and more: two query tiles per CTA)
    ([6144], None, True), ([6145], None, True), ([6273], None, False),  # a last pair of 1, of 129
    ([6200], [6500], True), ([6300], [4000], True), ([6300], [133], False),
    ([12200, 150], None, True)])
@pytest.mark.parametrize("d", [64, 128])
def test_two_query_tiles_per_cta(lq, lk, causal, d):
    ops.test_packed_attention(lq, lk, 2, 1, causal, d, "padded")


@pytest.mark.parametrize("d,causal", [(64, True), (128, True), (64, False), (128, False)])
def test_two_query_tiles_and_a_maximum_that_moves(d, causal):
    """Keys that grow along the sequence: late tiles pass the maximum so far
    by far, and the sums are scaled anew."""
    n, H, KV = 6500, 2, 1
    q, k, v, do = ops._attn_inputs([n], [n], H, KV, d, "fused", 60 + d)
    k *= torch.linspace(0.02, 3.0, n, device="cuda")[:, None].bfloat16()
    cu, scale = ops._cu([n]), d ** -0.5
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV, causal=causal)
    grads = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV, causal=causal)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0
    args = ([n], [n], H, KV, causal, scale)
    ref, rl, tol = ops._attn_ref(q, k, v, *args)
    ops._within(o, ref, tol + 1e-30, "o")
    ops._lse_within(lse, rl, "lse")
    for got, (r, t), name in zip(grads, ops._attn_ref(q, k, v, *args, o, lse, do),
                                 ("dq", "dk", "dv")):
        ops._within(got, r, t, name)


@pytest.mark.parametrize("H,KV,d,causal", [(4, 2, 128, True), (7, 1, 64, True),
                                           (16, 16, 64, False)])
def test_one_long_sequence_among_short_ones(H, KV, d, causal):
    """The kernels are chosen by the mean length, which hides it."""
    ops.test_packed_attention([50] * 20 + [3000] + [50] * 20, None, H, KV, causal, d, "padded")


@pytest.mark.parametrize("d,H,KV,lens", [(128, 28, 4, [300, 1, 211]), (64, 6, 6, [40] * 9),
                                         (64, 8, 2, [700])])
def test_every_tensor_a_part_of_wider_rows(d, H, KV, lens):
    """q, k, v and their gradients as columns of one tensor each, turned in
    place there, o and its gradient in rows with room beside them: bit for
    bit what separate tensors give, and the rest stays as it was."""
    T, g, w = sum(lens), ops._gen(d + H), (H + 2 * KV) * d
    cu, pos = ops._cu(lens), torch.arange(T, dtype=torch.int32, device="cuda")
    rope = hsnf4.Rope(d, hsnf4.rope_inv_freq(d, 1e4))

    def parts(buf):
        return buf[:, :H * d], buf[:, H * d:(H + KV) * d], buf[:, (H + KV) * d:w]

    x, do = ops._normal((T, w), g), ops._normal((T, H * d), g)
    q, k, v = (t.contiguous() for t in parts(x))
    q, k = hsnf4.rope_fwd(rope, pos, q, k)
    o, lse = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV)
    dq, dk, dv = hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV)
    want = [q, k, v, o, *hsnf4.rope_bwd(rope, pos, dq, dk), dv]

    wide = torch.full((T, w + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :w] = x
    grad = torch.full((T, w + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((T, 2 * H * d + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    o, dout = out[:, 8:8 + H * d], out[:, 16 + H * d:]
    dout.copy_(do)
    q, k, v = parts(wide)
    dq, dk, dv = parts(grad)
    hsnf4.rope_fwd(rope, pos, q, k, q, k)
    _, lse2 = hsnf4.attention_packed_fwd(q, k, v, cu, H, KV, o=o)
    hsnf4.attention_packed_bwd(q, k, v, o, lse2, dout, cu, H, KV, dq=dq, dk=dk, dv=dv)
    hsnf4.rope_bwd(rope, pos, dq, dk, dq, dk)
    torch.cuda.synchronize()
    assert hsnf4.device_status() == 0 and torch.equal(lse, lse2)
    for got, ref in zip((q, k, v, o, dq, dk, dv), want):
        assert torch.equal(got, ref)
    assert torch.equal(dout, do) and (wide[:, w:] == 7).all() and (grad[:, w:] == 7).all()
    assert (out[:, :8] == 7).all() and (out[:, 8 + H * d:16 + H * d] == 7).all()


def _guarded(rows, cols, mark, lead=8):
    """A [rows, cols] bf16 tensor inside a larger one, and that."""
    whole = torch.full((rows + 2 * lead, cols), mark, dtype=torch.bfloat16, device="cuda")
    return whole[lead:lead + rows], whole


MALFORMED = [[0, 400, 90], [-50, 30, 20], [90, 10, 1 << 30], [0, 0, 0], [0, 1 << 30, 90, 1 << 30, 0],
             [-50, 1900, 20, 2000, -1], [1 << 30, 0, 700, 0, 700], [0, 0, 0, 0, 0],
             [-(1 << 31), (1 << 31) - 1], [(1 << 31) - 1, -(1 << 31)]]


@pytest.mark.parametrize("T", [100, 2000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_malformed_lengths_write_nothing_outside(T, d, causal):
    """Every tensor lies inside a larger one whose values stay as they are;
    sequences that are all empty change nothing at all."""
    H, KV, mark = 4, 1, 7.0
    g = ops._gen(T + d)
    ins = [_guarded(T, n * d, ops.NAN) for n in (H, KV, KV, H)]
    for t, _ in ins:
        t.copy_(ops._normal(t.shape, g))
    q, k, v, do = (t for t, _ in ins)
    for cu in MALFORMED:
        n_seq = len(cu) - 1
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        outs = [_guarded(T, n * d, mark) for n in (H, H, KV, KV)]
        flat = torch.full((H * T + 128,), mark, device="cuda")
        lse = flat[64:64 + H * T].view(H, T)
        need = hsnf4.attention_packed_workspace_bytes(T, T, n_seq, H, KV, d)
        scratch = torch.full((need + 1024,), 0x5A, dtype=torch.uint8, device="cuda")
        o, dq, dk, dv = (t for t, _ in outs)
        hsnf4.attention_packed_fwd(q, k, v, cu, H, KV, causal=causal, o=o, lse=lse)
        hsnf4.attention_packed_bwd(q, k, v, o, lse, do, cu, H, KV, causal=causal, dq=dq, dk=dk,
                                   dv=dv, workspace=scratch[512:512 + need])
        torch.cuda.synchronize()
        assert hsnf4.device_status() == 0
        for t, whole in outs:
            assert (whole[:8] == mark).all() and (whole[8 + T:] == mark).all()
            if not cu.any():
                assert (t == mark).all()
        assert (flat[:64] == mark).all() and (flat[64 + H * T:] == mark).all()
        assert (scratch[:512] == 0x5A).all() and (scratch[512 + need:] == 0x5A).all()
        if not cu.any():
            assert (lse == mark).all()


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("T,H,KV,d,half,sections,pairing", [
    # a token's heads in two and four passes of the threads, also uneven ones
    (37, 32, 8, 128, 64, None, "half"), (64, 40, 8, 128, 64, [16, 24, 24], "half"),
    (33, 33, 2, 128, 64, None, "half"), (50, 28, 4, 128, 64, [16, 24, 24], "adjacent"),
    (29, 56, 8, 128, 64, None, "adjacent"), (41, 31, 2, 128, 64, None, "adjacent"),
    (9001, 32, 8, 128, 64, [16, 24, 24], "half"), (70, 17, 8, 256, 64, None, "half")])
@pytest.mark.parametrize("way", ["fwd", "bwd"])
@pytest.mark.parametrize("form", ["plain", "fused", "in_place"])
def test_rope_of_more_heads_than_threads(T, H, KV, d, half, sections, pairing, way, form):
    ops.test_rope(T, H, KV, d, half, sections, pairing, way, form)


# ---------------------------------------------------------------- gradient norm

@pytest.mark.parametrize("given", [True, False])
def test_set_dropped_while_another_stream_uses_it(given):
    """The table of addresses and the workspace stay the set's until a call
    on another stream has ended, though nothing refers to the set any more."""
    grads = [torch.ones(n, device="cuda") for n in (5, 4096, 77)]
    norm, x = torch.zeros((), device="cuda"), torch.zeros(4096, 4096, device="cuda")
    side, done = torch.cuda.Stream(), torch.cuda.Event()
    hsnf4.grad_clip(hsnf4.GradSet(grads), 1.0, norm=norm)  # (loading code waits for the device)
    x = x @ x
    gs = hsnf4.GradSet(grads)
    mine = {gs.table.data_ptr(), gs.workspace.data_ptr()}
    sizes = (gs.table.nbytes, gs.workspace.nbytes)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):  # some tens of milliseconds
            x = x @ x
    if given:
        hsnf4.grad_clip(gs, 1.0, norm=norm, stream=side)
    else:
        with torch.cuda.stream(side):
            hsnf4.grad_clip(gs, 1.0, norm=norm)
    done.record(side)
    del gs
    later = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    assert not done.query()  # the call is still to come
    assert not mine & {t.data_ptr() for t in later}
    torch.cuda.synchronize()
    # the call before left a norm of 1 / (1 + 1e-6 / norm)
    assert abs(float(norm) - 1.0) <= 2.0 ** -20


def test_streams_and_graphs_of_one_set_have_a_workspace_each():
    """Norms of one set on two streams and in two graphs at once: none of
    them writes where another one's sums are."""
    g = ops._gen(70)
    grads = [ops._normal((n,), g, torch.float32) for n in (5, 3_000_000, 4097)]
    gs = hsnf4.GradSet(grads)
    want = hsnf4.grad_norm(gs)
    graphs, norms = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norms.append([hsnf4.grad_norm(gs) for _ in range(20)])
        graphs.append(graph)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    gs.workspace.fill_(0xFF)  # of the calls on this stream: no other may touch it
    torch.cuda.synchronize()
    eager = []
    for graph, stream in zip(graphs, side):
        with torch.cuda.stream(stream):
            graph.replay()
            eager += [hsnf4.grad_norm(gs) for _ in range(20)]
        eager += [hsnf4.grad_norm(gs, stream=stream) for _ in range(20)]
    torch.cuda.synchronize()
    assert (gs.workspace == 0xFF).all()
    for got in eager + norms[0] + norms[1]:
        assert torch.equal(got, want)
    assert torch.equal(hsnf4.grad_norm(gs), want)
