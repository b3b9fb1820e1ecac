"""Pins of the oracle of the gated recurrence and of the 8-bit projections
(oracle/sequence.py): hand-worked values, and gradients against central differences.

Differences: with step d = 1e-5 truncation (d^2/6 times a third derivative of order 1)
and rounding (2^-53 |f| / d) are both under 1e-9 of the loss: gradients agree to 1e-6.
"""
import numpy as np
import pytest

from oracle import sequence as seq
from test_oracle_sequence import agree, differences


def test_gated_scan_by_hand():
    """Gates of 1/2 and A = 2 log(3/5): a = 3/5, the normaliser 4/5."""
    x = np.array([[[10.0, 0.0, 20.0]]])
    A, none = np.array([2 * np.log(0.6)]), np.zeros((1, 1, 3))
    y, h, S, H, marks = seq.gated_scan(x, none, none, A, state=np.array([[5.0]]), every=2)
    # 3 + 4 = 7, 4.2, 2.52 + 8
    assert np.allclose(y, [[[7.0, 4.2, 10.52]]]) and np.allclose(h, 10.52)
    assert np.allclose(S, y) and np.allclose(H, h) and np.allclose(marks, [[[5.0, 4.2]]])
    y, h, _, _ = seq.gated_scan(x, none, none, A, z=none, lengths=[1])
    assert np.allclose(y, 0) and np.allclose(h, 4.0)
    _, h, _, _ = seq.gated_scan(x, none, none, A, state=np.array([[5.0]]), lengths=[0])
    assert np.allclose(h, 5.0)
    # biases move the gates: sigmoid(log 3) = 3/4
    y, _, _, _ = seq.gated_scan(x, none, none, np.array([4 / 3 * np.log(0.6)]), None,
                                np.array([np.log(3.0)]), np.array([np.log(3.0)]))
    assert np.allclose(y[0, 0, 0], 0.8 * 0.75 * 10)


@pytest.mark.parametrize("gate", [True, False])
def test_gated_scan_grads_against_differences(gate):
    rng = np.random.default_rng(4)
    B, D, L = 2, 3, 5
    v = {k: rng.normal(size=(B, D, L)) for k in ("x", "r", "i") + (("z",) if gate else ())}
    v.update(A=-rng.uniform(0.2, 2, D), r_bias=rng.normal(size=D), i_bias=rng.normal(size=D),
             state=rng.normal(size=(B, D)))
    gout, gstate = rng.normal(size=(B, D, L)), rng.normal(size=(B, D))
    n = [5, 2]

    def args(a):
        return (a["x"], a["r"], a["i"], a["A"], a.get("z"), a["r_bias"], a["i_bias"], a["state"], n)

    def loss(a):
        y, h, _, _ = seq.gated_scan(*args(a))
        return (y * gout).sum() + (h * gstate).sum()

    g = seq.gated_scan_grads(gout, *args(v), gstate)
    for name in v:
        agree(g["d" + name], differences(loss, v, name))


def test_codes_by_hand():
    """Borders go to the even code, rows of zeros and of no numbers have codes 0."""
    rows = np.array([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0], [1, np.inf, 0, 0, 0],
                     [254, 1, 3, -3, 5]])
    codes, scales = seq.int8_codes(rows, 8)
    assert codes.tolist() == [[127, 0, 2, -2, -127, 0, 0, 0], [0] * 8, [0] * 8, [127, 0, 2, -2, 2, 0, 0, 0]]
    assert scales[0] == 1 and scales[1] == 0 and np.isnan(scales[2]) and scales[3] == 2


def test_product_by_hand():
    y, S = seq.int8_product([[1, 2], [-3, 0]], [0.5, 2.0], [[4, 5]], [10.0], [1.0])
    assert y.tolist() == [[71.0, -239.0]] and S.tolist() == [[71.0, 241.0]]
