"""Pins of the sequence oracle (oracle/sequence.py): hand-worked values, and its
gradients against central differences of its forward functions.

Differences: with step d the truncation error is d^2/6 times a third derivative
of order 1 and the rounding error 2^-53 |f| / d; d = 1e-5 keeps both under 1e-9
times the loss, so gradients agree to 1e-6 of their scale.
"""
import numpy as np
import pytest

from oracle import sequence as seq

STEP, NEAR = 1e-5, 1e-6


def differences(loss, arrays, name):
    v = arrays[name]
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        kept = v[i]
        v[i] = kept + STEP
        up = loss(arrays)
        v[i] = kept - STEP
        g[i] = (up - loss(arrays)) / (2 * STEP)
        v[i] = kept
    return g


def agree(a, b):
    assert np.abs(a - b).max() <= NEAR * max(1.0, np.abs(b).max())


def test_conv_by_hand():
    x = np.array([[[1.0, 2.0, 3.0]]])
    w = np.array([[10.0, 1.0]])
    y, new, S = seq.causal_conv(x, w, np.array([0.5]), silu=False, state=np.array([[[4.0]]]))
    assert y.tolist() == [[[41.5, 12.5, 23.5]]]
    assert new.tolist() == [[[3.0]]] and S.tolist() == y.tolist()
    # shorter than the state: what it held moves up; an empty sequence keeps it
    y, new, _ = seq.causal_conv(x, np.ones((1, 4)), silu=False, state=np.array([[[7.0, 8.0, 9.0]]]),
                                lengths=[1])
    assert y.tolist() == [[[25.0, 0.0, 0.0]]] and new.tolist() == [[[8.0, 9.0, 1.0]]]
    _, new, _ = seq.causal_conv(x, np.ones((1, 4)), state=np.array([[[7.0, 8.0, 9.0]]]), lengths=[0])
    assert new.tolist() == [[[7.0, 8.0, 9.0]]]


def test_scan_by_hand():
    """One state, A = -log 2 and steps of 1: the state halves and takes x B."""
    x = np.array([[[1.0, 2.0, 4.0]]])
    one = np.ones((1, 1, 1, 3))
    A = np.array([[-np.log(2.0)]])
    y, h, S, H = seq.state_scan(x, np.ones((1, 1, 3)), A, one, 2 * one, skip=np.array([10.0]),
                                soft=False, state=np.array([[[8.0]]]))
    assert np.allclose(y, [[[2 * 5 + 10, 2 * 4.5 + 20, 2 * 6.25 + 40]]], atol=1e-12)
    assert np.allclose(h, 6.25) and np.allclose(S, y) and np.allclose(H, h)
    y, h, _, _ = seq.state_scan(x, np.ones((1, 1, 3)), A, one, one, soft=False, lengths=[1])
    assert np.allclose(y, [[[1.0, 0.0, 0.0]]]) and np.allclose(h, 1.0)


def test_norm_by_hand():
    y, r = np.array([[[3.0], [4.0]]]), np.array([[[1.0], [1.0]]])
    out, u, _, _ = seq.block_norm(y, r, np.ones(2), np.array([1.0, 2.0]), eps=0.0,
                                  gate=np.zeros((1, 2, 1)), scale=np.array([2.0, 4.0]))
    n = np.array([3.0, 4.0]) / np.sqrt(12.5)
    want = 1 + np.array([1.0, 2.0]) * n
    assert np.allclose(out[0, :, 0], want)
    assert np.allclose(u[0, :, 0], want / np.sqrt((want ** 2).mean()) * [1, 2])


@pytest.mark.parametrize("silu", [True, False])
def test_conv_grads_against_differences(silu):
    rng = np.random.default_rng(1)
    v = {"x": rng.normal(size=(2, 3, 5)), "w": rng.normal(size=(3, 4)), "b": rng.normal(size=3)}
    gy = rng.normal(size=(2, 3, 5))
    n = [5, 3]

    def loss(a):
        return (seq.causal_conv(a["x"], a["w"], a["b"], silu, lengths=n)[0] * gy).sum()

    g = seq.causal_conv_grads(gy, v["x"], v["w"], v["b"], silu, lengths=n)
    for name, key in (("x", "dx"), ("w", "dw"), ("b", "db")):
        agree(g[key], differences(loss, v, name))


@pytest.mark.parametrize("soft,gate", [(True, True), (False, False)])
def test_scan_grads_against_differences(soft, gate):
    rng = np.random.default_rng(2)
    B, D, L, N, G = 2, 4, 5, 3, 2
    v = {"x": rng.normal(size=(B, D, L)), "dt": rng.normal(size=(B, D, L)) * 0.3,
         "A": -rng.uniform(0.2, 2, (D, N)), "B": rng.normal(size=(B, G, N, L)),
         "C": rng.normal(size=(B, G, N, L)), "D": rng.normal(size=D), "bias": rng.normal(size=D),
         "state": rng.normal(size=(B, D, N))}
    if gate:
        v["z"] = rng.normal(size=(B, D, L))
    gout, gstate = rng.normal(size=(B, D, L)), rng.normal(size=(B, D, N))
    n = [5, 2]

    def args(a):
        return (a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a.get("z"), a["bias"], soft, a["state"], n)

    def loss(a):
        y, h, _, _ = seq.state_scan(*args(a))
        return (y * gout).sum() + (h * gstate).sum()

    g = seq.state_scan_grads(gout, *args(v), gstate)
    names = {"x": "dx", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "bias": "ddt_bias",
             "state": "dstate"}
    if gate:
        names["z"] = "dz"
    for name, key in names.items():
        agree(g[key], differences(loss, v, name))


@pytest.mark.parametrize("parts", ["all", "pre", "post", "none"])
def test_norm_grads_against_differences(parts):
    rng = np.random.default_rng(3)
    B, D, L = 2, 4, 3
    v = {"y": rng.normal(size=(B, D, L)), "r": rng.normal(size=(B, D, L))}
    if parts in ("all", "post"):
        v["w_post"] = rng.normal(size=D)
    if parts in ("all", "pre"):
        v["w_pre"] = rng.normal(size=D)
    if parts == "all":
        v["gate"], v["scale"] = rng.normal(size=(B, D, L)), rng.normal(size=D)
    gr, gu = rng.normal(size=(B, D, L)), rng.normal(size=(B, D, L))
    n = [3, 1]

    def forward(a):
        return seq.block_norm(a["y"], a["r"], a.get("w_post"), a.get("w_pre"), a.get("gate"),
                              a.get("scale"), 0.1, n)

    def loss(a):
        out, u, _, _ = forward(a)
        return (out * gr).sum() + (0 if u is None else (u * gu).sum())

    g = seq.block_norm_grads(gr, gu if "w_pre" in v else None, v["y"], forward(v)[0], v.get("w_post"),
                             v.get("w_pre"), v.get("gate"), v.get("scale"), 0.1, n)
    names = {"y": "dy", "r": "dresidual", "gate": "dgate", "scale": "dscale", "w_post": "dweight_post",
             "w_pre": "dweight_pre"}
    for name in v:
        agree(g[names[name]], differences(loss, v, name))
