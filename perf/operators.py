"""Cases of the operators that a decoder layer's training step adds around
the LoRA projections: rotary positions with several axes, attention over
packed sequences with its backward pass, and the global gradient norm with
clipping.

`listed()` and `draw()` give cases (dicts of plain values); `prepare()` makes
a case's inputs on the GPU, `run()` computes one pass (with `own` through the
library, without it in elementary torch operations) and `exact()` computes
the same in 64 bits; `work()` counts the bytes and operations a pass cannot
do without.
"""
import random

import torch

own = False

# Head layouts (query heads, key/value heads) of the decoder families the
# repository is sized for, its test stack, and a tower with one KV head per
# query head.
LAYOUTS = {"2:1": (2, 1), "16:16": (16, 16), "28:4": (28, 4), "32:8": (32, 8), "40:8": (40, 8),
           "64:8": (64, 8)}
# (hidden, inter, heads, kv heads) of the same families, head_dim 128.
SHAPES = {"tiny": (256, 640, 2, 1), "7b": (3584, 18944, 28, 4), "8b": (4096, 14336, 32, 8),
          "32b": (5120, 27648, 40, 8), "72b": (8192, 29568, 64, 8)}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # rotary: the test stack's smallest call; a 7B layer's q and k out of
        # one fused projection buffer with (time, height, width) positions;
        # the gradient's way back at a 72B layer's heads and an odd length
        dict(name="rope fwd 64 tokens", op="rope", way="fwd", tokens=64, layout="2:1", dim=128,
             rot=128, axes=1, fused=False, pairing="half"),
        dict(name="rope fwd 7B 3 axes fused", op="rope", way="fwd", tokens=512, layout="28:4",
             dim=128, rot=128, axes=3, fused=True, pairing="half"),
        dict(name="rope bwd 72B 8191 tokens", op="rope", way="bwd", tokens=8191, layout="64:8",
             dim=128, rot=128, axes=3, fused=False, pairing="half"),
        # attention: one short sequence (latency), the 7B layer's 512 tokens
        # of the benchmark's step as nine packed samples, a long document, and
        # a tower's images as ragged windows without a causal mask
        dict(name="attn fwd 7B 9 packed", op="attn", way="fwd", tokens=512, seqs=9, cut=1,
             layout="28:4", dim=128, causal=True, fused=True, pad=0, extra=0),
        dict(name="attn fwd 64-wide windows", op="attn", way="fwd", tokens=4100, seqs=23, cut=2,
             layout="16:16", dim=64, causal=False, fused=True, pad=60, extra=0),
        dict(name="attn fwd 8B 16384 tokens", op="attn", way="fwd", tokens=16384, seqs=1, cut=3,
             layout="32:8", dim=128, causal=True, fused=False, pad=0, extra=0),
        # its backward pass: the 72B layer's 512 tokens as one sequence, a
        # packed 7B batch of ragged samples, and the long document
        dict(name="attn bwd 72B 512 tokens", op="attn", way="bwd", tokens=512, seqs=1, cut=4,
             layout="64:8", dim=128, causal=True, fused=False, pad=0, extra=0),
        dict(name="attn bwd 7B 17 packed", op="attn", way="bwd", tokens=8150, seqs=17, cut=5,
             layout="28:4", dim=128, causal=True, fused=True, pad=42, extra=0),
        dict(name="attn bwd 8B 16384 tokens", op="attn", way="bwd", tokens=16384, seqs=1, cut=6,
             layout="32:8", dim=128, causal=True, fused=False, pad=0, extra=0),
        # clipping: one 7B layer's 14 adapter gradients, the 72B stack's 1120
        # (where the norm is above the limit), and 16-bit gradients of odd
        # sizes under the limit
        dict(name="clip 7B layer", op="clip", shape="7b", layers=1, rank=16, dtype="f32",
             odd=0, limit=0.5),
        dict(name="clip 72B stack", op="clip", shape="72b", layers=80, rank=16, dtype="f32",
             odd=0, limit=0.5),
        dict(name="clip 8B stack bf16 odd", op="clip", shape="8b", layers=32, rank=16,
             dtype="bf16", odd=1, limit=2.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(("rope", "attn", "attn", "clip"))
    way = rng.choice(("fwd", "bwd"))
    layout = rng.choice(sorted(LAYOUTS))
    if op == "rope":
        dim = rng.choice((64, 80, 96, 128, 256))
        rot = rng.choice((dim, dim, dim // 2))
        rot -= rot % 16
        heads = sum(LAYOUTS[layout])
        return dict(op=op, way=way, tokens=log(1, max(2, 8191 * 72 * 128 // (heads * dim))),
                    layout=layout, dim=dim, rot=rot, axes=rng.choice((1, 2, 3)),
                    fused=rng.random() < 0.5, pairing=rng.choice(("half", "half", "adjacent")))
    if op == "attn":
        # a drawn case costs no more than the 16384-token ones with 32 heads
        # (and in the backward a sequence has more than one key: one key alone
        # gives its query and itself a gradient of zero)
        heads = LAYOUTS[layout][0]
        few = 1 if way == "fwd" else 16
        tokens = log(few, int(16000 * min(1.0, (32 / heads) ** 0.5)))
        return dict(op=op, way=way, tokens=tokens, seqs=min(max(1, 2 * tokens // few), log(1, 64)),
                    cut=rng.randrange(1 << 30), layout=layout, dim=rng.choice((64, 128)),
                    causal=rng.random() < 0.6, fused=rng.random() < 0.5,
                    pad=rng.choice((0, 0, log(1, 200))),
                    extra=rng.choice((0, 0, 0, log(1, 300))) if tokens < 8000 else 0)
    return dict(op=op, shape=rng.choice(sorted(SHAPES)), layers=log(1, 28),
                rank=rng.choice((8, 16, 24, 32)), dtype=rng.choice(sorted(DTYPES)),
                odd=rng.choice((0, 0, 1, 3)), limit=rng.choice((0.1, 0.5, 1.0, 2.0)))


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((seed * 1_000_003 + salt) % (1 << 62))


def _normal(shape, g, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _lens(case):
    """Lengths of a case's sequences (queries, keys): a random partition of
    its tokens; `extra` more keys than queries are spread over them (queries
    that continue earlier keys)."""
    r = random.Random(case["cut"])
    n = case["seqs"]
    cuts = sorted(r.randrange(case["tokens"] + 1) for _ in range(n - 1))
    cuts = [0] + cuts + [case["tokens"]]
    q = [b - a for a, b in zip(cuts, cuts[1:])]
    k = list(q)
    for _ in range(n):
        k[r.randrange(n)] += case["extra"] // n
    return q, k


def _cu(lens):
    out = [0]
    for x in lens:
        out.append(out[-1] + x)
    return out


def _axis_of(case):
    """The axis each frequency follows: contiguous sections, the first the
    smallest (16, 24, 24 of 64 for three axes)."""
    half, axes = case["rot"] // 2, case["axes"]
    first = half // 4 if axes == 3 else half // axes
    rest = half - first
    sections = [first] if axes == 1 else [first, rest] if axes == 2 else \
        [first, rest // 2, rest - rest // 2]
    if axes == 1:
        sections = [half]
    return sections


def _grad_sizes(case):
    hidden, inter, heads, kv = SHAPES[case["shape"]]
    q, c = heads * 128, kv * 128
    r = case["rank"]
    one = []
    for n, k in ((q, hidden), (c, hidden), (c, hidden), (hidden, q), (inter, hidden),
                 (inter, hidden), (hidden, inter)):
        one += [r * k + case["odd"], n * r]
    return one * case["layers"]


def prepare(case, seed):
    op = case["op"]
    if op == "rope":
        H, KV = LAYOUTS[case["layout"]]
        T, d = case["tokens"], case["dim"]
        g = _gen(seed, 11)
        if case["fused"]:
            buf = _normal((T, (H + 2 * KV) * d), g)
            q, k = buf[:, :H * d], buf[:, H * d:(H + KV) * d]
        else:
            q, k = _normal((T, H * d), g), _normal((T, KV * d), g)
        # positions: time runs on, height and width come from a 32-wide grid,
        # somewhere inside a long context
        start = int(torch.randint(0, 100_000, (1,), generator=g, device="cuda"))
        t = torch.arange(T, device="cuda")
        pos = torch.stack([t + start, t // 32 + start, t % 32 + start])[:case["axes"]]
        pos = pos.to(torch.int32).contiguous()
        i = torch.arange(case["rot"] // 2, dtype=torch.float64)
        inv_freq = (1_000_000.0 ** (-2.0 * i / case["rot"])).to(torch.float32)
        st = dict(case=case, q=q, k=k, pos=pos, H=H, KV=KV, inv_freq=inv_freq.cuda(),
                  axis=torch.repeat_interleave(torch.arange(case["axes"]),
                                               torch.tensor(_axis_of(case))).cuda(),
                  q_out=torch.zeros(T, H * d, dtype=torch.bfloat16, device="cuda"),
                  k_out=torch.zeros(T, KV * d, dtype=torch.bfloat16, device="cuda"))
        if own:
            from host_streamed_nf4_b200 import hsnf4
            st["rope"] = hsnf4.Rope(d, inv_freq, sections=_axis_of(case), pairing=case["pairing"])
        return st
    if op == "attn":
        H, KV = LAYOUTS[case["layout"]]
        d = case["dim"]
        lq, lk = _lens(case)
        cq, ck = _cu(lq), _cu(lk)
        Tq, Tk = cq[-1] + case["pad"], ck[-1] + case["pad"]
        g = _gen(seed, 12)
        if case["fused"] and Tq == Tk:
            buf = _normal((Tq, (H + 2 * KV) * d), g)
            q, k, v = buf[:, :H * d], buf[:, H * d:(H + KV) * d], buf[:, (H + KV) * d:]
        else:
            q, k, v = _normal((Tq, H * d), g), _normal((Tk, KV * d), g), _normal((Tk, KV * d), g)
        st = dict(case=case, q=q, k=k, v=v, H=H, KV=KV, cq=cq, ck=ck, scale=d ** -0.5,
                  cu_q=torch.tensor(cq, dtype=torch.int32, device="cuda"),
                  cu_k=torch.tensor(ck, dtype=torch.int32, device="cuda"),
                  o=torch.zeros(Tq, H * d, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.zeros(H, Tq, dtype=torch.float32, device="cuda"))
        if case["way"] == "bwd":
            # what the forward left behind, and the gradient arriving
            st["o"], st["lse"] = _attn_fwd(st)
            st["do"] = _normal((Tq, H * d), g)
            st["dq"], st["dk"], st["dv"] = (
                torch.zeros(t, n * d, dtype=torch.bfloat16, device="cuda")
                for t, n in ((Tq, H), (Tk, KV), (Tk, KV)))
            if own:
                from host_streamed_nf4_b200 import hsnf4
                st["ws"] = torch.empty(
                    hsnf4.attention_packed_workspace_bytes(Tq, Tk, len(lq), H, KV, d),
                    dtype=torch.uint8, device="cuda")
        return st
    sizes = _grad_sizes(case)
    total = sum(sizes)
    g = _gen(seed, 13)
    flat = torch.randn(total, generator=g, device="cuda")
    # a norm of 1: some limits clip, others do not
    flat = (flat * float(total) ** -0.5).to(DTYPES[case["dtype"]])
    st = dict(case=case, flat=flat, out=torch.zeros_like(flat))
    if own:
        from host_streamed_nf4_b200 import hsnf4
        st["set"] = hsnf4.GradSet(flat.split(sizes), outs=st["out"].split(sizes))
        st["norm"] = torch.zeros((), dtype=torch.float32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _turn(x, heads, d, rot, cos, sin, pairing):
    """x [T, heads * d] with each head's first `rot` values turned by the
    angles (cos, sin [T, rot / 2])."""
    T = x.shape[0]
    x = x.to(cos.dtype).view(T, heads, d)
    cos, sin = cos[:, None, :], sin[:, None, :]
    out = x.clone()
    if pairing == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return out.reshape(T, heads * d)


def _rope(st):
    case = st["case"]
    angle = st["pos"].double()[st["axis"]].T * st["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    if case["way"] == "bwd":
        sin = -sin
    return [_turn(x, n, case["dim"], case["rot"], cos, sin, case["pairing"]).to(torch.bfloat16)
            for x, n in ((st["q"], st["H"]), (st["k"], st["KV"]))]


def _heads(x, n, d):
    """[t, n * d] -> [n, t, d] in 32 bits"""
    return x.float().view(x.shape[0], n, d).transpose(0, 1)


def _scores(qh, kh, r0, r1, lq, lk, causal, scale):
    """scale q k^T of query rows r0..r1 (kv heads, group, rows, keys), -inf
    where the mask (causal, the last query on the last key) is."""
    s = (qh[:, :, r0:r1] @ kh.transpose(-1, -2)[:, None]) * scale
    if causal:
        row = torch.arange(r0, r1, device=s.device)[:, None] + (lk - lq)
        s = s.masked_fill(torch.arange(lk, device=s.device) > row, float("-inf"))
    return s


def _pieces(st):
    """(query range, key range, rows at a time) of each sequence with queries"""
    for q0, q1, k0, k1 in zip(st["cq"], st["cq"][1:], st["ck"], st["ck"][1:]):
        if q1 > q0:
            yield q0, q1, k0, k1, max(1, (1 << 28) // max(1, st["H"] * (k1 - k0)))


def _attn_fwd(st):
    case, H, KV = st["case"], st["H"], st["KV"]
    d = case["dim"]
    o = torch.zeros(st["q"].shape, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(H, st["q"].shape[0], device="cuda")
    for q0, q1, k0, k1, step in _pieces(st):
        lq, lk = q1 - q0, k1 - k0
        if lk == 0:
            lse[:, q0:q1] = float("-inf")
            continue
        qh = _heads(st["q"][q0:q1], H, d).reshape(KV, H // KV, lq, d)
        kh, vh = _heads(st["k"][k0:k1], KV, d), _heads(st["v"][k0:k1], KV, d)
        for r0 in range(0, lq, step):
            r1 = min(lq, r0 + step)
            s = _scores(qh, kh, r0, r1, lq, lk, case["causal"], st["scale"])
            m = s.amax(-1, keepdim=True).clamp_min(-3e38)
            p = (s - m).exp()
            l = p.sum(-1, keepdim=True)
            out = (p @ vh[:, None]) / l.clamp_min(1e-38)
            o[q0 + r0:q0 + r1] = out.reshape(H, r1 - r0, d).transpose(0, 1).reshape(r1 - r0, H * d)
            lse[:, q0 + r0:q0 + r1] = torch.where(l > 0, m + l.log(), float("-inf")).reshape(H, -1)
    return o, lse


def _attn_bwd(st):
    case, H, KV = st["case"], st["H"], st["KV"]
    d, G = case["dim"], H // KV
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.bfloat16, device="cuda")
                  for x in (st["q"], st["k"], st["v"]))
    for q0, q1, k0, k1, step in _pieces(st):
        lq, lk = q1 - q0, k1 - k0
        if lk == 0:
            continue
        qh = _heads(st["q"][q0:q1], H, d).reshape(KV, G, lq, d)
        oh = _heads(st["o"][q0:q1], H, d).reshape(KV, G, lq, d)
        gh = _heads(st["do"][q0:q1], H, d).reshape(KV, G, lq, d)
        kh, vh = _heads(st["k"][k0:k1], KV, d), _heads(st["v"][k0:k1], KV, d)
        lse = st["lse"][:, q0:q1].reshape(KV, G, lq, 1)
        D = (gh * oh).sum(-1, keepdim=True)
        gk, gv = torch.zeros_like(kh), torch.zeros_like(vh)
        for r0 in range(0, lq, step):
            r1 = min(lq, r0 + step)
            s = _scores(qh, kh, r0, r1, lq, lk, case["causal"], st["scale"])
            p = torch.where(s == float("-inf"), 0.0, (s - lse[:, :, r0:r1]).exp())
            g = gh[:, :, r0:r1]
            gv += (p.transpose(-1, -2) @ g).sum(1)
            ds = p * (g @ vh.transpose(-1, -2)[:, None] - D[:, :, r0:r1]) * st["scale"]
            gk += (ds.transpose(-1, -2) @ qh[:, :, r0:r1]).sum(1)
            gq = ds @ kh[:, None]
            dq[q0 + r0:q0 + r1] = gq.reshape(H, r1 - r0, d).transpose(0, 1).reshape(r1 - r0, H * d)
        dk[k0:k1] = gk.transpose(0, 1).reshape(lk, KV * d)
        dv[k0:k1] = gv.transpose(0, 1).reshape(lk, KV * d)
    return dq, dk, dv


def _clip(st):
    x = st["flat"].float()
    norm = x.double().square().sum().sqrt().float()
    coef = (st["case"]["limit"] / (norm + 1e-6)).clamp_max(1.0)
    return norm, (x * coef).to(st["flat"].dtype)


def run(st):
    case = st["case"]
    op, fwd = case["op"], case.get("way") == "fwd"
    if own:
        from host_streamed_nf4_b200 import hsnf4
        if op == "rope":
            f = hsnf4.rope_fwd if fwd else hsnf4.rope_bwd
            return f(st["rope"], st["pos"], st["q"], st["k"], st["q_out"], st["k_out"])
        if op == "attn" and fwd:
            return hsnf4.attention_packed_fwd(st["q"], st["k"], st["v"], st["cu_q"], st["H"],
                                              st["KV"], causal=case["causal"], cu_k=st["cu_k"],
                                              o=st["o"], lse=st["lse"])
        if op == "attn":
            return hsnf4.attention_packed_bwd(st["q"], st["k"], st["v"], st["o"], st["lse"],
                                              st["do"], st["cu_q"], st["H"], st["KV"],
                                              causal=case["causal"], cu_k=st["cu_k"],
                                              dq=st["dq"], dk=st["dk"], dv=st["dv"],
                                              workspace=st["ws"])
        norm = hsnf4.grad_clip(st["set"], case["limit"], norm=st["norm"])
        return norm, st["out"]
    if op == "rope":
        return _rope(st)
    if op == "attn":
        return _attn_fwd(st) if fwd else _attn_bwd(st)
    return _clip(st)


# ------------------------------------------------------------------ work

def _pairs(case):
    """query-key pairs that the masks leave, of one head"""
    n = 0
    for a, b in zip(*_lens(case)):
        if not case["causal"]:
            n += a * b
        else:  # row i sees keys 0 .. i + b - a
            n += sum(min(b, max(0, i + b - a + 1)) for i in range(a))
    return n


def work(case):
    if case["op"] == "rope":
        H, KV = LAYOUTS[case["layout"]]
        n = case["tokens"] * (H + KV) * case["dim"]
        return {"bytes": 4 * n + 4 * case["axes"] * case["tokens"],
                "flops": 3 * case["tokens"] * (H + KV) * case["rot"]}
    if case["op"] == "attn":
        H, KV = LAYOUTS[case["layout"]]
        d = case["dim"]
        lq, lk = (sum(x) for x in _lens(case))
        p = _pairs(case) * H * d
        if case["way"] == "fwd":  # q, k, v read, o and lse written; two products
            return {"bytes": 2 * d * (2 * lq * H + 2 * lk * KV) + 4 * H * lq, "flops": 4 * p}
        # q, k, v, o, do, lse read, dq, dk, dv written; five products
        return {"bytes": 2 * d * (4 * lq * H + 4 * lk * KV) + 4 * H * lq, "flops": 10 * p}
    n = sum(_grad_sizes(case))
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": 2 * n * size, "flops": 3 * n}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        T, d, half = case["tokens"], case["dim"], case["rot"] // 2
        where = torch.stack([st["pos"][a].double() for a in st["axis"].tolist()], 1)
        z = torch.polar(torch.ones(T, half, dtype=torch.float64, device="cuda"),
                        where * st["inv_freq"].double())
        if case["way"] == "bwd":
            z = z.conj()
        outs = []
        for x, n in ((st["q"], st["H"]), (st["k"], st["KV"])):
            x = x.double().reshape(T, n, d).clone()
            if case["pairing"] == "half":
                c = torch.complex(x[..., :half], x[..., half:2 * half].contiguous()) * z[:, None]
                x[..., :half], x[..., half:2 * half] = c.real, c.imag
            else:
                c = torch.view_as_complex(x[..., :2 * half].reshape(T, n, half, 2)) * z[:, None]
                x[..., :2 * half] = torch.view_as_real(c).reshape(T, n, 2 * half)
            outs.append(x.reshape(T, n * d))
        return outs
    if case["op"] == "clip":
        parts = st["flat"].double()
        norm = torch.linalg.vector_norm(parts)
        return norm, parts * min(1.0, case["limit"] / (float(norm) + 1e-6))
    H, KV, d = st["H"], st["KV"], case["dim"]
    f64 = dict(dtype=torch.float64, device="cuda")
    q, k, v = (st[n].double().unflatten(1, (-1, d)) for n in "qkv")
    out, lse = torch.zeros(q.shape, **f64), torch.zeros(H, q.shape[0], **f64)
    dq, dk, dv = torch.zeros(q.shape, **f64), torch.zeros(k.shape, **f64), torch.zeros(v.shape, **f64)
    if case["way"] == "bwd":
        o, do = (st[n].double().unflatten(1, (-1, d)) for n in ("o", "do"))
    for b in range(case["seqs"]):
        (qa, qb), (ka, kb) = st["cq"][b:b + 2], st["ck"][b:b + 2]
        for h in range(H):
            c = h // (H // KV)
            for ra in range(qa, qb, 4096):
                rb = min(qb, ra + 4096)
                e = torch.einsum("qd,kd->qk", q[ra:rb, h], k[ka:kb, c]) * st["scale"]
                if case["causal"]:
                    gap = (kb - ka) - (qb - qa)
                    keep = torch.ones(rb - ra, kb - ka, dtype=torch.bool, device="cuda").tril(
                        ra - qa + gap)
                    e = torch.where(keep, e, -torch.inf)
                if case["way"] == "fwd":
                    z = torch.logsumexp(e, 1)
                    w = torch.where(torch.isneginf(z)[:, None], 0.0, torch.exp(e - z[:, None]))
                    lse[h, ra:rb] = z
                    out[ra:rb, h] = w @ v[ka:kb, c]
                    continue
                z = st["lse"][h, ra:rb].double()[:, None]
                w = torch.where(torch.isneginf(e), 0.0, torch.exp(e - z))
                g = do[ra:rb, h]
                dv[ka:kb, c] += w.T @ g
                w *= g @ v[ka:kb, c].T - (g * o[ra:rb, h]).sum(1, keepdim=True)
                dk[ka:kb, c] += st["scale"] * (w.T @ q[ra:rb, h])
                dq[ra:rb, h] = st["scale"] * (w @ k[ka:kb, c])
    flat = [x.flatten(1) for x in (out, dq, dk, dv)]
    return (flat[0], lse) if case["way"] == "fwd" else tuple(flat[1:])
