"""The sequence kernels where a position, a length or a part is missing, and where
values are infinite, zero or tiny, against the float64 oracle.

Tolerances and their counts are those of test_gpu_sequence.py.  The oracle sees
each sequence cut to its length, so that nothing beyond one enters a sum.
"""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import test_gpu_sequence as base  # noqa: E402
from test_gpu_sequence import TYPES, Inputs, check, num, poison  # noqa: E402

import conv2d_backward_amd as gi  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def ends(lengths, B, L):
    return [L] * B if lengths is None else [min(max(n, 0), L) for n in lengths.tolist()]


def beyond(t, lengths):
    """The values of t [B, D, L] beyond the lengths, in one row."""
    return torch.cat([t[b, :, n:].flatten() for b, n in enumerate(ends(lengths, t.shape[0], t.shape[-1]))])


# ---- block_norm ----------------------------------------------------------------------------------


class Norm:
    def __init__(self, B, D, L, dtype, lengths=None, parts="post pre gate scale", eps=0.0, size=1.0):
        i = Inputs(B + D + L, dtype)
        self.eps, self.n = eps, None if lengths is None else ints(*lengths)

        def act(dtype=None, scale=1.0):
            return poison(i.normal(B, D, L, dtype=dtype, scale=scale), self.n)

        parts = parts.split()
        self.y, self.r, self.gr = act(scale=size), act(torch.float32, size), act(torch.float32)
        self.post = i.params(D) if "post" in parts else None
        self.pre = i.params(D) if "pre" in parts else None
        self.gate = act() if "gate" in parts else None
        self.scale = i.params(D) if "scale" in parts else None
        self.gu = act() if "pre" in parts else None

    def forward(self):
        return gi.block_norm(self.y, self.r, self.post, self.pre, gate=self.gate, scale=self.scale, eps=self.eps,
                             lengths=self.n)

    def backward(self, r):
        return gi.block_norm_backward(self.gr, self.gu, self.y, r, self.post, self.pre, gate=self.gate,
                                      scale=self.scale, eps=self.eps, lengths=self.n)

    def by_sequence(self, function, acts):
        """function(activations of one sequence, weights) of each sequence that has positions: [(b, length, result)]."""
        B, _, L = self.y.shape
        weights = num(self.post, self.pre)
        out = []
        for b, n in enumerate(ends(self.n, B, L)):
            if n:
                cut = [None if v is None else v[b:b + 1, :, :n] for v in num(*acts, self.gate)]
                out.append((b, n, function(*cut[:-1], *weights, cut[-1], *num(self.scale), self.eps)))
        return out

    def check_forward(self):
        B, D, L = self.y.shape
        r, u = self.forward()
        for b, n, (rr, ru, Sr, Su) in self.by_sequence(oracle.block_norm, (self.y, self.r)):
            check(r[b:b + 1, :, :n], rr, Sr, D + 32, "residual")
            if u is not None:
                check(u[b:b + 1, :, :n], ru, Su, 2 * D + 64, "u")
        for v in (r, u):
            assert v is None or bool((beyond(v, self.n) == 0).all())
        return r

    def check_backward(self, r):
        B, D, L = self.y.shape
        g = self.backward(r)._asdict()
        whole = {}
        for b, n, ref in self.by_sequence(oracle.block_norm_grads, (self.gr, self.gu, self.y, r)):
            for name, v in ref.items():
                if v.ndim == 1:
                    whole[name] = whole.get(name, 0) + v
                elif not name.startswith("S"):
                    check(g[name][b:b + 1, :, :n], v, ref["S" + name], 4 * D + 128, name)
        for name, got in g.items():
            if got is not None and got.dim() == 1:
                check(got, whole[name], whole["S" + name], 4 * D + 128 + B * L, name)
            elif got is not None:
                assert bool((beyond(got, self.n) == 0).all()), name


AT_ZERO = [  # B, D, L, lengths
    (1, 20, 9, None), (4, 20, 9, (9, 0, 3, 8)), (3, 70, 1, (1, 0, 1)), (2, 4200, 1, (0, 1)), (3, 130, 70, (70, 64, 1)),
    (2, 2060, 33, (0, 20)), (1, 4200, 21, None), (130, 33, 40, tuple(range(130))),
]


@pytest.mark.parametrize("case", AT_ZERO, ids=lambda c: "x".join(map(str, c[:3])))
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_without_eps(case, dtype):
    """Positions that nothing is added to have no root of zero in them: 0 where the contract says 0."""
    B, D, L, lengths = case
    Norm(B, D, L, dtype, lengths).check_forward()


@pytest.mark.parametrize("D,L", [(20, 9), (20, 1), (4200, 12)])
def test_norm_is_zero_beyond_lengths_whatever_the_weight(D, L):
    s = Norm(2, D, L, "bf16", (L // 2, 0), eps=1e-6)
    s.pre[3], s.pre[4] = float("inf"), float("nan")
    for v in s.forward():
        assert bool((beyond(v, s.n) == 0).all())


@pytest.mark.parametrize("case", AT_ZERO, ids=lambda c: "x".join(map(str, c[:3])))
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_gradients_without_eps(case, dtype):
    """Columns without a position add nothing to the parameters' gradients."""
    B, D, L, lengths = case
    s = Norm(B, D, L, dtype, lengths)
    s.check_backward(s.forward()[0])


@pytest.mark.parametrize("parts", ["post pre gate scale", "pre", "post"])
@pytest.mark.parametrize("size", [2.0 ** -50, 2.0 ** -60, 2.0 ** 50])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_gradients_of_tiny_and_huge_values(parts, size, dtype):
    """The inverse root's cube is beyond float32 for values under 2^-42, the gradients are not."""
    s = Norm(2, 40, 13, dtype, (13, 6), parts, size=size)
    s.check_backward(s.check_forward())


def test_norm_gradients_of_norms_that_are_not_there():
    """Without a norm its input has no part in the gradients: no mean, no root of zero, no NaN of its own."""
    s = Norm(2, 20, 9, "f32", parts="post gate scale")
    r, _ = s.forward()
    want = s.backward(r)
    for value in (0.0, float("nan"), float("inf"), 1e30):
        r[0, :, 4] = value
        got = s.backward(r)
        assert torch.equal(got.dresidual, s.gr)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(got, want)), value
    s = Norm(2, 20, 9, "f32", parts="pre gate scale")
    r, _ = s.forward()
    want = s.backward(r)
    for value in (0.0, float("nan"), float("inf")):
        s.y[1, 3, 7] = value
        assert torch.equal(s.backward(r).dy, want.dy) and torch.equal(s.backward(r).dresidual, want.dresidual)


# ---- causal_conv ---------------------------------------------------------------------------------


@pytest.mark.parametrize("L,lengths", [(13, None), (21, (21, 5, 18)), (700, (699, 0, 130)), (2077, (2077, 2049, 2050))])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_conv_taps_take_only_positions_they_meet(L, lengths, value):
    """x[len-1] meets the last tap alone."""
    i = Inputs(L, "f32")
    n = None if lengths is None else ints(*lengths)
    x, gy, w = i.normal(3, 5, L), i.normal(3, 5, L), i.params(5, 4)
    at = L if n is None else ends(n, 3, L)[0]
    x[0, 2, at - 1] = value
    dx, dw, db = gi.causal_conv_backward(poison(gy, n), poison(x, n), w, silu=False, lengths=n, want_db=True)
    bad = ~torch.isfinite(dw)
    assert bad[2].tolist() == [False, False, False, True] and int(bad.sum()) == 1
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(db).all())
    if value == float("inf"):
        assert float(dw[2, 3]) == value * float(torch.sign(gy[0, 2, at - 1]))


@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradient_is_zero_beyond_lengths_whatever_the_weight(silu):
    i = Inputs(3, "bf16")
    n = ints(21, 0, 5, 600)
    x, gy, w = poison(i.normal(4, 5, 700), n), poison(i.normal(4, 5, 700), n), i.params(5, 4)
    w[1, 0], w[2, 3], w[3, 2] = float("inf"), float("nan"), -float("inf")
    dx = gi.causal_conv_backward(gy, x, w, silu=silu, lengths=n)[0]
    assert bool((beyond(dx, n) == 0).all())


# ---- state_scan ----------------------------------------------------------------------------------


@pytest.mark.parametrize("case", [(4, 20, 45, 5, 1), (4, 36, 300, 16, 2), (4, 2000, 600, 4, 2)], ids=str)
def test_scan_gradients_are_zero_beyond_lengths_whatever_the_skip(case):
    s = base.Scan((*case, None, "dense"), "bf16")
    s.n = ints(case[2], 0, 7, 30)
    for v in (s.x, s.dt, s.z, s.gout, s.B, s.C):
        poison(v, s.n)
    s.skip[1], s.skip[2] = float("inf"), float("nan")
    g = s.backward(s.forward(want_checkpoints=True)[2])
    for v in (g.dx, g.ddt, g.dz):
        assert bool((beyond(v, s.n) == 0).all())


SCAN_FORGETS = [(4, 20, 45, 5, 1), (4, 36, 300, 16, 2), (4, 1024, 1030, 4, 1), (4, 2000, 600, 4, 2)]


@pytest.mark.parametrize("case", SCAN_FORGETS, ids=str)
def test_scan_of_infinite_rates(case):
    """A = -inf forgets the state at each position (exp(-inf) = 0); beyond a length the state still passes."""
    B, D, L, N, G = case
    s = base.Scan((*case, None, "dense"), "f32")
    s.n = ints(L, 0, 7, 30)
    for v in (s.x, s.dt, s.z, s.gout, s.B, s.C):
        poison(v, s.n)
    s.A[2, 0] = s.A[5, N - 1] = -float("inf")
    y, h, marks = s.forward(want_state=True, want_checkpoints=True)
    some = [0, 2, 5, D - 1]                          # (rows of channels do not meet: a few do for the oracle)
    of = torch.tensor(some, device="cuda") // (D // G)
    x, dt, z = (v[:, some] for v in (s.x, s.dt, s.z))
    Bm, Cm = s.B[:, of], s.C[:, of]
    args = num(x, dt, s.A[some], Bm, Cm, s.skip[some], z, s.bias[some])
    ry, rh, S, H, rmarks = oracle.state_scan(*args, True, *num(s.state[:, some]), s.n, every=gi.SCAN_CHECKPOINT)
    check(y[:, some], ry, S, 32 * L + 64, "y")
    check(h[:, some], rh, H, 32 * L + 64, "state")
    check(marks[:, some], rmarks, np.abs(rmarks) + np.abs(H)[:, :, None], 32 * L + 64, "checkpoints")


@pytest.mark.parametrize("case", SCAN_FORGETS, ids=str)
def test_scan_gradients_of_infinite_rates(case):
    """The gradients at A = -inf are those at a rate whose decay is 0 in float32."""
    B, D, L, N, G = case
    s = base.Scan((*case, None, "dense"), "f32")
    s.n = ints(L, 0, 7, 30)
    for v in (s.x, s.dt, s.z, s.gout, s.B, s.C):
        poison(v, s.n)
    got = {}
    for rate in (-1e30, -float("inf")):
        s.A[2, 0] = s.A[5, N - 1] = rate
        got[rate] = s.backward(s.forward(want_checkpoints=True)[2], want_dstate=True)
    for name, p, q in zip(got[-1e30]._fields, *got.values()):
        assert bool(torch.isfinite(p).all()) and torch.equal(p, q), name


def test_scan_of_more_states_and_positions_than_gradients_have():
    """B*G*N*(L+256) beyond 2^30: a prompt of equal rows (batch stride 0) and a large generation step."""
    B, D, L, N, G = 64, 8, 16640, 128, 8
    i = Inputs(8, "bf16")
    x, dt, Bm, Cm = i.normal(1, D, L), i.normal(1, D, L, scale=0.3), i.normal(1, G, N, L), i.normal(1, G, N, L)
    A, bias = i.params(D, N, low=-4, high=-0.05), i.params(D, low=-5, high=-3)
    every = [v.expand(B, *v.shape[1:]) for v in (x, dt, Bm, Cm)]
    y, h, _ = gi.state_scan(*every[:2], A, *every[2:], dt_bias=bias, want_state=True)
    ry, rh, S, H = oracle.state_scan(*num(x, dt, A, Bm, Cm), None, None, *num(bias), True)
    check(y[:1], ry, S, 32 * L + 64, "y")
    check(h[:1], rh, H, 32 * L + 64, "state")
    assert all(torch.equal(v, v[:1].expand_as(v)) for v in (y, h))
    B = 4200
    rows = [v[..., 5].expand(B, *v.shape[1:-1]) for v in (x, dt, Bm, Cm)]
    state = i.params(1, D, N).repeat(B, 1, 1)
    before = state[:1].clone()
    y = gi.state_scan_step(*rows[:2], A, *rows[2:], state, dt_bias=bias)
    ry, rh, S, H = oracle.state_scan(*num(*[v[..., 5:6] for v in (x, dt)], A, *[v[..., 5:6] for v in (Bm, Cm)]),
                                     None, None, *num(bias), True, *num(before))
    check(y[:1], ry[..., 0], S[..., 0], 96 + 8 * N, "y")
    check(state[:1], rh, H, 96, "state")
    assert torch.equal(y, y[:1].expand_as(y)) and torch.equal(state, state[:1].expand_as(state))


@pytest.mark.parametrize("B,D", [(4200, 4096), (2048, 8200)])
def test_generation_steps_of_large_batches(B, D):
    """B*D beyond 2^24: rows of two kinds in turn, so that one of each tells all."""
    i = Inputs(B, "bf16")
    kinds = torch.arange(B, device="cuda") % 2
    x, dt, Bm, Cm = i.normal(2, D), i.normal(2, D, scale=0.3), i.normal(2, 1, 4), i.normal(2, 1, 4)
    w, A, bias = i.params(D, 4, scale=0.5), i.params(D, 4, low=-4, high=-0.05), i.params(D, low=-5, high=-3)
    lines, states = i.normal(2, D, 3), i.params(2, D, 4)
    line, state = lines[kinds], states[kinds]
    y = gi.causal_conv_step(x[kinds], line, w)
    ry, rline, S = oracle.causal_conv(num(x)[0][..., None], *num(w), None, True, *num(lines))
    check(y[:2], ry[..., 0], S[..., 0], 18 + S.max(), "y")
    assert torch.equal(y, y[kinds]) and torch.equal(line, line[kinds]) and (num(line[:2])[0] == rline).all()
    y = gi.state_scan_step(x[kinds], dt[kinds], A, Bm[kinds], Cm[kinds], state, dt_bias=bias)
    ry, rh, S, H = oracle.state_scan(*[v[..., None] for v in num(x, dt)], *num(A), *[v[..., None] for v in num(Bm, Cm)],
                                     None, None, *num(bias), True, *num(states))
    check(y[:2], ry[..., 0], S[..., 0], 96 + 8 * 4, "y")
    check(state[:2], rh, H, 96, "state")
    assert torch.equal(y, y[kinds]) and torch.equal(state, state[kinds])


# ---- streams -------------------------------------------------------------------------------------


def test_stream_of_another_device_is_refused():
    """Its kernels would run there, on memory that is here."""
    class Elsewhere:
        device_index, cuda_stream = 1, 0

    i = Inputs(1, "bf16")
    x = i.normal(2, 6, 10)
    for f in (lambda: gi.causal_conv(x, i.params(6, 4), stream=Elsewhere()),
              lambda: gi.block_norm(x, x.float(), stream=Elsewhere())):
        with pytest.raises(ValueError, match="cuda:1"):
            f()


@pytest.mark.parametrize("case,plans", [
    ((7, 192, 1030, 33, 64), ("waves=8 lanes=64 positions=8", "waves=8 positions=8")),
    ((4, 12, 1030, 18, 4), ("waves=8 lanes=64 positions=8", "waves=4 positions=8")),
    ((4, 560, 500, 24, 16), ("waves=", "waves=8 positions=16"))], ids=str)
def test_graph_replays_of_large_work_groups(case, plans):
    """Work-groups with more than 64 KB of LDS, captured: each replay equals the eager pass."""
    assert all(gi.state_scan_plan(*case, backward=k).startswith(p) for k, p in enumerate(plans))
    s = base.Scan((*case, "ragged", "dense"), "bf16")

    def both():
        y, h, marks = s.forward(want_state=True, want_checkpoints=True)
        return [y, h, marks, *s.backward(marks, want_dstate=True)]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both()
    for _ in range(3):
        for v in got:
            v.fill_(7)
        graph.replay()
        again = both()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) and torch.equal(p, r) for p, q, r in zip(got, want, again))
