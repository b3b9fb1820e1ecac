"""gated_scan, its gradients and its single positions against the float64 oracle.

Tolerances (u = 2^-24, h half a step of the output's type, S the oracle's sum of
magnitudes), with |gate| <= 6 and |A| <= 2: a sigmoid is good to |v| + 5 u (12 u), so the
exponent A sigmoid(r) is good to 14 u of itself and a to (14 |A| + 2) u <= 30 u.  1 - a^2
moves by at most as much as its exponent does (14 u), its series or the difference from
a below exp(-0.3) adds 18 u, and the root halves that: 18 u; with the other gate and x an
input is good to 32 u.  So a position adds at most 32 u to a path, and a path of L positions
is good to 32 L u; silu and the stores are within 64 u more.  Gradients have two chains and
1 / m (18 u): twice that, and sums over n more terms add n u.  `check` holds the 2-norm to
the square root of the count.
"""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_sequence import TYPES, Inputs, check, lengths_of, num, poison  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


CASES = [  # B, D, L, lengths, layout
    (1, 1, 1, None, "dense"), (1, 1, 2, None, "dense"), (2, 3, 7, None, "padded"), (7, 5, 9, "ragged", "dense"),
    (3, 6, 8, "none", "dense"), (1, 17, 127, None, "padded"), (1, 33, 128, None, "slice"), (2, 5, 129, None, "swapped"),
    (7, 3, 256, "ragged", "slice"), (7, 3, 257, "ragged", "padded"), (2, 9, 511, None, "dense"), (1, 5, 513, None, "slice"),
    (3, 4, 1030, "ragged", "swapped"), (1, 3, 2049, None, "padded"), (4, 2, 4100, "ragged", "dense"),
    (2, 1, 9001, None, "dense"), (9, 21, 33, None, "dense"), (20, 7, 5, None, "slice"), (5, 35, 31, "ragged", "padded"),
    (7, 18, 100, "ragged", "dense"), (4, 3, 4500, "ragged", "dense"), (10, 5, 1300, None, "dense"),
]


class Gated:
    def __init__(self, case, dtype, gate=True, extras=True):
        B, D, L, kind, layout = case
        i = Inputs(B * 1000 + D * 10 + L, dtype)
        self.case, self.inputs, self.n = case, i, lengths_of(kind, B, L)

        def act(**k):
            return poison(i.normal(B, D, L, layout=layout, **k), self.n)

        self.x, self.r, self.i, self.gout = act(), act(), act(), act()
        self.z = act() if gate else None
        # Rates of long memory and of short, decays of 0.999 and of 0.13 at an open gate.
        self.A = -torch.exp(i.params(D, low=-7, high=0.69))
        self.r_bias, self.i_bias = (i.params(D, scale=0.5) if extras else None for _ in range(2))
        self.state = i.params(B, D) if extras else None
        self.gstate = i.params(B, D) if extras else None

    def forward(self, **k):
        return gi.gated_scan(self.x, self.r, self.i, self.A, self.z, self.r_bias, self.i_bias, state=self.state,
                             lengths=self.n, **k)

    def backward(self, marks, **k):
        return gi.gated_scan_backward(self.gout, self.x, self.r, self.i, self.A, marks, self.z, self.r_bias,
                                      self.i_bias, lengths=self.n, grad_state=self.gstate, **k)

    def numbers(self):
        return num(self.x, self.r, self.i, self.A, self.z, self.r_bias, self.i_bias, self.state)

    def check_forward(self):
        L = self.case[2]
        y, h, marks = self.forward(want_state=True, want_checkpoints=True)
        ry, rh, S, H, rmarks = oracle.gated_scan(*self.numbers(), self.n, every=gi.SCAN_CHECKPOINT)
        check(y, ry, S, 32 * L + 64, "y")
        check(h, rh, H, 32 * L + 64, "state")
        check(marks, rmarks, np.abs(rmarks) + np.abs(H)[:, :, None], 32 * L + 64, "checkpoints")
        plain = self.forward()
        assert torch.equal(plain[0], y) and plain[1] is None and plain[2] is None
        return marks

    def check_backward(self, marks):
        B, D, L, _, _ = self.case
        g = self.backward(marks, want_dstate=True)
        ref = oracle.gated_scan_grads(*num(self.gout), *self.numbers(), self.n, *num(self.gstate))
        for name, got in g._asdict().items():
            if got is not None:
                more = B * L if got.dim() == 1 else 0
                check(got, ref[name], ref["S" + name], 64 * L + 128 + more, name)
        assert (g.dz is None) == (self.z is None) and (g.dr_bias is None) == (self.r_bias is None)
        again = self.backward(marks, want_dstate=True)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(g, again))


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(case, dtype):
    Gated(case, dtype).check_forward()


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(case, dtype):
    s = Gated(case, dtype)
    s.check_backward(s.forward(want_checkpoints=True)[2])


@pytest.mark.parametrize("case", [
    # Enough rows for every way they are dealt that few rows do not have.
    (3, 1400, 150, None, "dense"), (1, 4100, 520, None, "dense"), (2, 2100, 300, None, "padded"), (1, 1100, 4200, None, "dense")],
    ids=str)
def test_many_rows(case):
    s = Gated(case, "bf16")
    s.check_backward(s.check_forward())


@pytest.mark.parametrize("gate,extras", [(False, True), (True, False), (False, False)])
def test_options(gate, extras):
    s = Gated((2, 18, 600, None, "dense"), "f32", gate, extras)
    s.check_backward(s.check_forward())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D", [(1, 1), (1, 300), (5, 258), (9, 64), (70, 1001)])
def test_step(B, D, dtype):
    i = Inputs(B + D, dtype)
    A, r_bias, i_bias = -torch.exp(i.params(D, low=-7, high=0.69)), i.params(D), i.params(D)
    for strided in (False, True):
        # Contiguous channels, and columns of a wider tensor.
        x, r, g, z = ((i.normal(B, 2 * D + 1)[:, 1::2] if strided else i.normal(B, D)) for _ in range(4))
        state = i.params(B + 3, D)
        slots = torch.from_numpy(i.rng.permutation(B + 3)[:B].astype(np.int32)).cuda()
        for at, bad in ((1, -1), (3, B + 3), (4, 2 ** 31 - 1), (5, -2 ** 31)):
            if at < B:
                slots[at] = bad
        before = state.clone()
        y = gi.gated_scan_step(x, r, g, A, state, z, r_bias, i_bias, slots=slots)
        lines = slots.tolist()
        live = [b for b in range(B) if 0 <= lines[b] < B + 3]
        at = [lines[b] for b in live]
        rows = [num(v)[0][live][..., None] for v in (x, r, g)]
        ry, rh, S, H = oracle.gated_scan(*rows, *num(A), num(z)[0][live][..., None], *num(r_bias, i_bias),
                                         num(before)[0][at])
        check(y[live], ry[..., 0], S[..., 0], 96, "y")
        check(state[at], rh, H, 96, "state")
        rest = [k for k in range(B + 3) if k not in at]
        assert torch.equal(state[rest], before[rest])
        assert (y[[b for b in range(B) if b not in live]] == 0).all()
        state = before.clone()
        y = gi.gated_scan_step(x, r, g, A, state)
        rows = [num(v)[0][..., None] for v in (x, r, g)]
        ry, rh, S, H = oracle.gated_scan(*rows, *num(A), None, None, None, num(before)[0][:B])
        check(y, ry[..., 0], S[..., 0], 96, "y")
        assert torch.equal(state[B:], before[B:])


def test_in_pieces():
    """A prompt in two calls, then tokens, against one call."""
    s = Gated((2, 20, 700, None, "dense"), "f32")
    ry, rh, S, H = oracle.gated_scan(*s.numbers())
    h, ys = s.state, []
    for lo, hi in ((0, 577), (577, 690)):
        x, r, i, z = (v[..., lo:hi] for v in (s.x, s.r, s.i, s.z))
        y, h, _ = gi.gated_scan(x, r, i, s.A, z, s.r_bias, s.i_bias, state=h, want_state=True)
        ys.append(y)
    for t in range(690, 700):
        x, r, i, z = (v[..., t] for v in (s.x, s.r, s.i, s.z))
        ys.append(gi.gated_scan_step(x, r, i, s.A, h, z, s.r_bias, s.i_bias)[..., None])
    check(torch.cat(ys, -1), ry, S, 32 * 700 + 64, "y")
    check(h, rh, H, 32 * 700 + 64, "state")


def test_gradient_against_differences():
    """dA and dstate of a float32 call against differences of the oracle's loss."""
    s = Gated((1, 2, 40, None, "dense"), "f32")
    v = dict(zip("x r i A z r_bias i_bias state".split(), s.numbers()))
    gout, gstate = num(s.gout, s.gstate)

    def loss():
        y, h, _, _ = oracle.gated_scan(*v.values())
        return (y * gout).sum() + (h * gstate).sum()

    g = s.backward(s.forward(want_checkpoints=True)[2], want_dstate=True)
    for name in ("A", "state", "r_bias"):
        at, got = v[name], num(getattr(g, "d" + name))[0]
        for k in np.ndindex(at.shape):
            kept, d = at[k], 1e-5 * abs(at[k])
            at[k] = kept + d
            up = loss()
            at[k] = kept - d
            assert abs(got[k] - (up - loss()) / (2 * d)) <= 2e-4 * (1 + np.abs(got).max()), name
            at[k] = kept


def test_later_trouble_keeps_from_earlier_positions():
    """NaN at one position reaches that and later ones of its channel, nothing else."""
    for L in (200, 1500):
        s = Gated((1, 20, L, None, "dense"), "f32")
        clean = s.forward()[0]
        s.x[0, 3, 100] = float("nan")
        y = s.forward()[0]
        bad = torch.isnan(y)
        assert bad[0, 3, 100:].all() and int(bad.sum()) == L - 100
        assert torch.equal(y[~bad], clean[~bad])


def test_ends_of_the_gates():
    """Closed gates keep the state, a rate of 0 does too, one of -inf forgets it; gradients stay numbers."""
    s = Gated((1, 6, 300, None, "dense"), "f32", gate=False, extras=False)
    s.state = torch.full((1, 6), 3.0, device="cuda")
    s.r[0, 0], s.r[0, 1] = -1e4, -float("inf")
    s.i[0, 2] = -float("inf")
    s.A[3], s.A[4], s.A[5] = 0.0, -float("inf"), -1e-38
    y, h, marks = s.forward(want_state=True, want_checkpoints=True)
    assert (y[0, [0, 1, 3]] == 3).all() and (h[0, [0, 1, 3]] == 3).all()
    assert torch.allclose(y[0, 4], torch.sigmoid(s.i[0, 4]) * s.x[0, 4], rtol=1e-6, atol=1e-7)
    assert (y[0, 5] - 3).abs().max() < 1e-15
    g = s.backward(marks)
    for t in (g.dx, g.dr, g.di):
        assert torch.isfinite(t).all()
    assert torch.isfinite(g.dA[[0, 1, 2, 3, 4]]).all()


def test_no_trace_beyond_a_length():
    """Weights that are no numbers leave 0 beyond the lengths."""
    s = Gated((5, 4, 700, "ragged", "dense"), "f32")
    s.A[1] = float("nan")
    s.r_bias[2] = float("inf")
    y, _, marks = s.forward(want_checkpoints=True)
    g = s.backward(marks)
    n = s.n.clamp(0, 700)
    for b in range(5):
        for t in (y, g.dx, g.dr, g.di, g.dz):
            assert (t[b, :, int(n[b]):] == 0).all()


def test_outputs_of_the_caller():
    s = Gated((2, 10, 300, None, "dense"), "bf16")
    y, _, marks = s.forward(want_checkpoints=True)
    wide = torch.full((2, 24, 300), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 3:13]
    assert s.forward(out=out)[0] is out and torch.equal(out, y)
    g = s.backward(marks)
    outs = {k: torch.full((2, 14, 301), 7.0, dtype=torch.bfloat16, device="cuda")[:, 2:12, 1:] for k in ("dx", "dr", "di", "dz")}
    h = s.backward(marks, **outs)
    for k, v in outs.items():
        assert getattr(h, k) is v and torch.equal(v, getattr(g, k))
        assert (v._base[:, :2] == 7).all() and (v._base[:, 12:] == 7).all() and (v._base[:, :, 0] == 7).all()
    assert (wide[:, :3] == 7).all() and (wide[:, 13:] == 7).all()


@pytest.mark.parametrize("L", [3, 100, 700, 3000])
def test_rate_of_minus_infinity(L):
    """Forgets as a rate does whose decays are 0 in fp32, with the same gradients."""
    s = Gated((2, 36, L, None, "dense"), "f32")
    got = []
    for rate in (-float("inf"), -1e30):
        s.A[::3] = rate
        y, h, marks = s.forward(want_state=True, want_checkpoints=True)
        got.append([y, h, marks, *s.backward(marks, want_dstate=True)])
    assert all(torch.equal(p, q) and torch.isfinite(p).all() for p, q in zip(*got))


def test_graph_replays():
    """Captured once, replayed with eager work in between: each replay equals the eager pass."""
    s = Gated((2, 36, 700, None, "dense"), "bf16")
    cache = s.inputs.params(2, 36)

    def everything(state):
        y, h, marks = s.forward(want_state=True, want_checkpoints=True)
        x, r, i = (v[..., 3] for v in (s.x, s.r, s.i))
        return [y, h, marks, *s.backward(marks, want_dstate=True), gi.gated_scan_step(x, r, i, s.A, state)]

    kept, eager = cache.clone(), cache.clone()
    everything(cache.clone())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = everything(cache)
    cache.copy_(kept)
    for _ in range(4):
        graph.replay()
        want = everything(eager)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)) and torch.equal(cache, eager)


def test_on_a_named_stream():
    s = Gated((2, 36, 700, None, "dense"), "bf16")
    want = s.forward(want_state=True, want_checkpoints=True)
    grads = s.backward(want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.forward(want_state=True, want_checkpoints=True, stream=side)
    got_grads = s.backward(got[2], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all(p is q is None or torch.equal(p, q) for p, q in zip(got_grads, grads))


def test_offsets_beyond_32_bits():
    i = Inputs(4, "bf16")
    B, D = 2, 64
    lines = 2 ** 31 // D + 10
    state = torch.empty(lines, D, device="cuda")
    slots = torch.tensor([lines - 1, 5], dtype=torch.int32, device="cuda")
    start = i.params(B, D)
    state[slots.long()] = start
    x, r, g, A = i.normal(B, D), i.normal(B, D), i.normal(B, D), i.params(D, low=-2, high=-0.1)
    y = gi.gated_scan_step(x, r, g, A, state, slots=slots)
    want_state = start.clone()
    assert torch.equal(y, gi.gated_scan_step(x, r, g, A, want_state))
    assert torch.equal(state[slots.long()], want_state)
    del state
    far = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    near, r, g, A = i.normal(2, 8, 100), i.normal(2, 8, 100), i.normal(2, 8, 100), i.params(8, low=-2, high=-0.1)
    wide = far.as_strided((2, 8, 100), (2 ** 31 + 100, 100, 1))
    wide.copy_(near)
    assert torch.equal(gi.gated_scan(wide, r, g, A)[0], gi.gated_scan(near, r, g, A)[0])


def test_refusals():
    i = Inputs(1, "bf16")
    x, A, state = i.normal(2, 6, 10), i.params(6, low=-2, high=-1), i.params(2, 6)
    marks = i.params(2, 6, 1)
    bad = [
        lambda: gi.gated_scan(x[0], x, x, A), lambda: gi.gated_scan(x.double(), x, x, A),
        lambda: gi.gated_scan(x, x.float(), x, A), lambda: gi.gated_scan(x, x, x[:, :5], A),
        lambda: gi.gated_scan(x, x, x, A.bfloat16()), lambda: gi.gated_scan(x, x, x, A[:5]),
        lambda: gi.gated_scan(x, x, x, A.cpu()), lambda: gi.gated_scan(x.transpose(1, 2), x, x, A),
        lambda: gi.gated_scan(x, x, x, A, state=state[:1]), lambda: gi.gated_scan(x, x, None, A),
        lambda: gi.gated_scan(x, x, x, A, lengths=torch.zeros(2, device="cuda", dtype=torch.int64)),
        lambda: gi.gated_scan(x, x, x, A, out=x.float()), lambda: gi.gated_scan(None, x, x, A),
        lambda: gi.gated_scan_backward(x, x, x, x, A, i.params(2, 6, 2)),
        lambda: gi.gated_scan_backward(x, x, x, x, A, None),
        lambda: gi.gated_scan_backward(x, x, x, x, A, marks, dz=x),
        lambda: gi.gated_scan_step(x, x, x, A, state),
        lambda: gi.gated_scan_step(x[..., 0], x[..., 0], x[..., 0], A, state.bfloat16()),
        lambda: gi.gated_scan_step(x[..., 0], x[..., 0], x[..., 0], A, state[:, :5]),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % k)
    for f in (lambda: gi.gated_scan(x[..., :0], x[..., :0], x[..., :0], A),
              lambda: gi.gated_scan(x, x, x, A, out=x[:1].expand(2, 6, 10)),
              lambda: gi.gated_scan_backward(x, x, x, x, A, marks, dx=x[:1].expand(2, 6, 10)),
              lambda: gi.gated_scan_step(x[..., 0], x[..., 0], x[..., 0], A, i.params(1, 6))):
        with pytest.raises(gi.Conv2dGiError):
            f()
