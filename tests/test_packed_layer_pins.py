"""The oracle's decoder layer with rotary positions and packed sequences in
exact arithmetic: its gradients match central differences, its sequences do
not see each other, and rotary positions act through their differences only."""
import numpy as np
import pytest

from oracle import decoder as dec


def _layer(rng, T, lens, angles):
    H, KV, d, hid, inter, r = 2, 1, 8, 12, 10, 4
    shapes = {"q": (H * d, hid), "k": (KV * d, hid), "v": (KV * d, hid), "o": (hid, H * d),
              "gate": (inter, hid), "up": (inter, hid), "down": (hid, inter)}
    lin = {n: dec.Linear(o, i, A=0.3 * rng.standard_normal((r, i)),
                         B=0.3 * rng.standard_normal((o, r)),
                         W=0.3 * rng.standard_normal((o, i))) for n, (o, i) in shapes.items()}
    return dec.Layer(H=H, KV=KV, d=d, g1=1 + 0.1 * rng.standard_normal(hid),
                     g2=1 + 0.1 * rng.standard_normal(hid), lin=lin, alpha=4.0, angles=angles,
                     lens=lens), hid


IDENT = staticmethod(lambda x: x).__func__


@pytest.mark.parametrize("lens", [None, [3, 1, 4]])
def test_layer_gradients_match_differences(orc, lens):
    rng = np.random.default_rng(5)
    T = 8
    layer, hid = _layer(rng, T, lens, rng.uniform(-3, 3, (T, 4)))
    h0, G = rng.standard_normal((T, hid)), rng.standard_normal((T, hid))
    s = dec.layer_forward(layer, h0, rnd=IDENT)
    dh0, grads = dec.layer_backward(layer, s, G, rnd=IDENT)
    loss = lambda h: float(np.sum(G * dec.layer_forward(layer, h, rnd=IDENT)["h2"]))
    eps = 1e-6
    for _ in range(6):
        e = rng.standard_normal(h0.shape)
        slope = (loss(h0 + eps * e) - loss(h0 - eps * e)) / (2 * eps)
        assert abs(slope - np.sum(dh0 * e)) <= 1e-7 * max(1.0, abs(slope))
    for name in ("q", "k", "v"):
        L = layer.lin[name]
        for M, g in zip((L.A, L.B), grads[name]):
            e = rng.standard_normal(M.shape)
            base = M.copy()
            M[...] = base + eps * e
            up = loss(h0)
            M[...] = base - eps * e
            dn = loss(h0)
            M[...] = base
            slope = (up - dn) / (2 * eps)
            assert abs(slope - np.sum(g * e)) <= 1e-6 * max(1.0, abs(slope))


def test_sequences_are_independent(orc):
    rng = np.random.default_rng(6)
    layer, hid = _layer(rng, 8, [3, 5], rng.uniform(-3, 3, (8, 4)))
    h0 = rng.standard_normal((8, hid))
    ref = dec.layer_forward(layer, h0, rnd=IDENT)["h2"]
    h0[:3] += 1.0
    assert np.array_equal(dec.layer_forward(layer, h0, rnd=IDENT)["h2"][3:], ref[3:])


def test_rotation_depends_on_differences(orc):
    rng = np.random.default_rng(7)
    T, freq = 9, np.array([1.0, 0.3, 0.07, 0.01])
    layer, hid = _layer(rng, T, None, np.arange(T)[:, None] * freq)
    h0 = rng.standard_normal((T, hid))
    ref = dec.layer_forward(layer, h0, rnd=IDENT)["h2"]
    layer.angles = (np.arange(T)[:, None] + 1000) * freq
    assert np.allclose(dec.layer_forward(layer, h0, rnd=IDENT)["h2"], ref, rtol=0, atol=1e-10)
    x = rng.standard_normal((T, 16))
    back = dec.rotate(dec.rotate(x, 2, layer.angles), 2, layer.angles, -1)
    assert np.allclose(back, x, rtol=0, atol=1e-12)
