"""state_scan by every way its work is dealt to waves, forward and backward, against the
float64 oracle: more states than one stage holds, odd numbers of them, partly filled
tiles of channels, ragged batches with an empty row, every type.

Each case names the plan it is there for, and a test without a GPU
(test_sequence_plans.py) holds that it gets it and that no plan is left out.
Groups of channels have nothing to do with each other, so the oracle follows a few
of them; tolerances are those of test_gpu_sequence.py.
"""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
from test_gpu_sequence import TYPES, Scan, check, num  # noqa: E402

import conv2d_backward_amd as gi  # noqa: E402

FORWARD = [  # plan; B, D, L, N, G
    ("waves=8 lanes=64 positions=16 shares=1 staged=4", (7, 320, 1540, 9, 64)),
    ("waves=8 lanes=64 positions=16 shares=2 staged=4", (4, 192, 1540, 18, 64)),
    ("waves=8 lanes=64 positions=16 shares=4 staged=4", (4, 192, 1540, 33, 64)),
    ("waves=8 lanes=64 positions=8 shares=1 staged=16", (7, 320, 2050, 18, 64)),
    ("waves=8 lanes=64 positions=8 shares=2 staged=16", (7, 192, 1030, 33, 64)),
    ("waves=8 lanes=64 positions=8 shares=4 staged=16", (4, 12, 1030, 18, 4)),
    ("waves=4 lanes=16 positions=16 shares=1 staged=16", (4, 3200, 390, 18, 64)),
    ("waves=4 lanes=16 positions=4 shares=1 staged=64", (7, 3200, 140, 70, 64)),
    ("waves=8 lanes=16 positions=8 shares=2 staged=32", (7, 832, 140, 33, 64)),
    ("waves=8 lanes=16 positions=8 shares=4 staged=32", (4, 320, 140, 38, 64)),
]
BACKWARD = [  # plan, rows whole or cut into segments; B, D, L, N, G
    ("waves=8 positions=16 joined=2", "whole", (4, 1280, 250, 33, 32)),
    ("waves=8 positions=16 joined=2", "cut", (4, 560, 500, 24, 16)),
    ("waves=8 positions=16 joined=1", "whole", (4, 192, 150, 192, 64)),
    ("waves=8 positions=16 joined=1", "cut", (4, 96, 390, 192, 32)),
    ("waves=8 positions=8 joined=4", "whole", (4, 1280, 100, 33, 32)),
    ("waves=8 positions=8 joined=4", "cut", (4, 640, 140, 24, 16)),
    ("waves=8 positions=8 joined=2", "whole", (4, 192, 25, 255, 64)),
    ("waves=8 positions=8 joined=2", "cut", (4, 96, 140, 255, 32)),
    ("waves=4 positions=8 joined=4", "whole", (4, 72, 25, 33, 4)),
    ("waves=4 positions=8 joined=4", "cut", (7, 72, 390, 33, 4)),
    ("waves=4 positions=8 joined=4", "cut", (4, 6, 140, 255, 2)),
]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


class Groups:
    """A ragged scan, and a few of its groups of channels."""

    def __init__(self, sizes, dtype):
        self.s = Scan((*sizes, "ragged", "dense"), dtype)
        B, D, L, N, G = sizes
        self.groups = sorted({0, G // 2, G - 1})
        self.channels = (torch.tensor(self.groups)[:, None] * (D // G) + torch.arange(D // G)).flatten().cuda()

    def of(self, t, axis=1):
        return None if t is None else t.index_select(axis, self.channels)

    def numbers(self):
        s = self.s
        return num(self.of(s.x), self.of(s.dt), self.of(s.A, 0), s.B[:, self.groups], s.C[:, self.groups],
                   self.of(s.skip, 0), self.of(s.z), self.of(s.bias, 0))


def same(a, b):
    return all(p is q is None or torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("plan,sizes", FORWARD, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(plan, sizes, dtype):
    c, L = Groups(sizes, dtype), sizes[2]
    out = c.s.forward(want_state=True, want_checkpoints=True)
    y, h, marks = (c.of(v) for v in out)
    ry, rh, S, H, rmarks = oracle.state_scan(*c.numbers(), True, *num(c.of(c.s.state)), c.s.n, every=gi.SCAN_CHECKPOINT)
    check(y, ry, S, 32 * L + 64, "y")
    check(h, rh, H, 32 * L + 64, "state")
    check(marks, rmarks, np.abs(rmarks) + np.abs(H)[:, :, None], 32 * L + 64, "checkpoints")
    assert torch.equal(out[1][0], c.s.state[0]) and bool((out[0][0] == 0).all())   # the empty row
    assert same(out, c.s.forward(want_state=True, want_checkpoints=True))


@pytest.mark.parametrize("plan,rows,sizes", BACKWARD, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(plan, rows, sizes, dtype):
    B, D, L, N, G = sizes
    c = Groups(sizes, dtype)
    s = c.s
    marks = s.forward(want_checkpoints=True)[2]
    g = s.backward(marks, want_dstate=True)
    ref = oracle.state_scan_grads(*num(c.of(s.gout)), *c.numbers(), True, *num(c.of(s.state)), s.n, *num(c.of(s.gstate)))
    more = {"dA": B * L, "dD": B * L, "ddt_bias": B * L, "dB": D // G, "dC": D // G}
    for name, got in g._asdict().items():
        if name in ("dB", "dC"):
            got = got[:, c.groups]
        else:
            got = c.of(got, 0 if name in ("dA", "dD", "ddt_bias") else 1)
        check(got, ref[name], ref["S" + name], 64 * L + 128 + more.get(name, 0), name)
    assert torch.equal(g.dstate[0], s.gstate[0])                                   # the empty row
    assert same(g, s.backward(marks, want_dstate=True))
