"""The sequence kernels against the float64 oracle, through the binding.

Tolerances (u = 2^-24, half a float32 step; h = half a step of the output's
type, 0 for float32, whose rounding is among the sums').  S is the oracle's sum
of magnitudes.  Element by element:

* causal_conv: K+1 roundings of the sum; sigmoid costs |p| + 7 (its argument's
  rounding is a relative |p| of the exponential): h |y| + (2K + 10 + S) u S.
* state_scan: the inputs keep s |A| <= 1 a step.  s itself is good to 25 u (the
  logarithm, reciprocal and exponential are 2 u each, the exponential's argument
  |raw| u), so a step's factor exp(s A) is good to (25 + 3) u, and with the
  multiply-adds of both passes 32 u a position covers a path: (32 L + 64) u S for
  y and the states, twice that for gradients, whose path has both chains; sums
  over n more terms (batch and positions, or channels) add n u.
* block_norm: the means run over D terms: (D + 32) u S, twice that for gradients.

These grow with the length as if every rounding went the same way.  The 2-norm
of the error is held to what independent roundings give: the square root of that
count, times 8 u, and h, of the result's norm.
"""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


def half(dtype):
    return 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2


def check(got, ref, S, count, what):
    """Element by element against (count) u S and the rounding; the 2-norm against the root of count."""
    h = half(got.dtype)
    x = got.detach().double().cpu().numpy()
    assert x.shape == ref.shape, what
    assert np.isfinite(x).all(), "%s: not finite" % what
    err = np.abs(x - ref)
    # (1e-30: results below the normal range become 0; a 16-bit one below its own, h of its smallest normal)
    tiny = 1e-30 if h == 0 else float(torch.finfo(got.dtype).tiny) * h * 2
    limit = h * np.abs(ref) + count * U * S * (1 + h) + tiny
    assert (err <= limit).all(), "%s: %d of %d beyond, worst %.3g of the limit" % (
        what, int((err > limit).sum()), err.size, float((err / limit).max()))
    norm = np.linalg.norm(S)
    assert np.linalg.norm(err) <= h * np.linalg.norm(ref) + 8 * np.sqrt(count) * U * norm + tiny * x.size, (
        "%s: 2-norm %.3g of S's" % (what, np.linalg.norm(err) / max(norm, 1e-300)))


class Inputs:
    """Seeded inputs on the GPU in a type, and the float64 values they hold."""

    def __init__(self, seed, dtype):
        self.rng = np.random.default_rng(seed)
        self.dtype = TYPES[dtype]

    def normal(self, *shape, scale=1.0, layout="dense", dtype=None):
        v = torch.from_numpy(self.rng.normal(size=shape) * scale).to(dtype or self.dtype).cuda()
        return arrange(v, layout)

    def params(self, *shape, low=None, high=None, scale=1.0):
        v = self.rng.normal(size=shape) * scale if low is None else self.rng.uniform(low, high, shape)
        return torch.from_numpy(v).float().cuda()


def arrange(v, layout):
    """The values of v [B, D, ...] at other strides and alignments."""
    if layout == "dense":
        return v.contiguous()
    B, D = v.shape[:2]
    if layout == "slice":       # channels 1 .. D of a wider tensor, odd row starts
        wide = torch.full((B, D + 3, *v.shape[2:]), float("nan"), dtype=v.dtype, device=v.device)
        wide[:, 1:D + 1] = v
        return wide[:, 1:D + 1]
    if layout == "swapped":     # channels outside the batch
        return v.transpose(0, 1).contiguous().transpose(0, 1)
    assert layout == "padded"   # rows of L + 5 positions, one element off the start
    flat = torch.full((B * D * (v.shape[2] + 5) + 1,), float("nan"), dtype=v.dtype, device=v.device)
    out = flat[1:].view(B, D, -1)[:, :, :v.shape[2]]
    out.copy_(v)
    return out


def num(*ts):
    return [None if t is None else t.double().cpu().numpy() for t in ts]


def lengths_of(kind, B, L):
    if kind is None:
        return None
    # empty, whole, one position, and out of range on both sides (clamped)
    v = [0, L, 1, L + 7, -3, max(L - 2, 0), L // 2][:B] if kind == "ragged" else [0] * B
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def poison(t, lengths):
    """NaN in every position beyond the lengths."""
    if lengths is not None:
        at = torch.arange(t.shape[-1], device="cuda") >= lengths.clamp(0, t.shape[-1])[:, None]
        t.masked_fill_(at.view(at.shape[0], *[1] * (t.dim() - 2), -1), float("nan"))
    return t


# ---- causal_conv ---------------------------------------------------------------------------------

CONV = [  # B, D, L, K, lengths, layout
    (1, 1, 1, 1, None, "dense"), (1, 1, 1, 4, None, "dense"), (2, 3, 2, 4, None, "dense"),
    (7, 5, 9, 4, "ragged", "dense"), (7, 3, 8, 8, "ragged", "slice"), (2, 4, 7, 3, "none", "dense"),
    (3, 6, 257, 4, None, "padded"), (5, 2, 1001, 2, "ragged", "swapped"), (2, 3, 2049, 4, None, "slice"),
    (2, 1, 4100, 5, None, "dense"), (1, 70, 64, 6, None, "padded"), (40, 2, 17, 7, None, "swapped"),
]


def conv_inputs(case, dtype):
    B, D, L, K, kind, layout = case
    i = Inputs(B * 1000 + L * 10 + K, dtype)
    n = lengths_of(kind, B, L)
    x = poison(i.normal(B, D, L, layout=layout), n)
    return i, n, x, i.params(D, K, scale=K ** -0.5), i.params(D, scale=0.2)


@pytest.mark.parametrize("case", CONV, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_conv_forward(case, dtype):
    B, D, L, K, _, _ = case
    i, n, x, w, bias = conv_inputs(case, dtype)
    state = i.normal(B, D, K - 1)
    for silu, b, st in ((True, bias, state), (False, None, None)):
        y, new = gi.causal_conv(x, w, b, silu=silu, state=st, lengths=n, want_state=True)
        ry, rnew, S = oracle.causal_conv(*num(x, w, b), silu, *num(st), n)
        check(y, ry, S, 2 * K + 10 + S.max(initial=0), "y")
        assert np.array_equal(new.double().cpu().numpy(), rnew)


@pytest.mark.parametrize("case", CONV, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_conv_backward(case, dtype):
    B, D, L, K, _, layout = case
    i, n, x, w, bias = conv_inputs(case, dtype)
    gy = poison(i.normal(B, D, L, layout=layout), n)
    for silu, b in ((True, bias), (False, None)):
        dx, dw, db = gi.causal_conv_backward(gy, x, w, b, silu=silu, lengths=n, want_db=True)
        ref = oracle.causal_conv_grads(*num(gy, x, w, b), silu, n)
        # The scale: gradients with every factor by magnitude and slope 1 (silu's is at most 1.1).
        clean = [np.nan_to_num(v) for v in num(gy, x)]
        S = oracle.causal_conv_grads(*np.abs(clean), np.abs(num(w)[0]), None, False, n)
        Sp = oracle.causal_conv(*num(x, w, b), silu, None, n)[2].max(initial=0)
        count = 1.1 * (2 * K + 14 + 2 * Sp)
        check(dx, ref["dx"], S["dx"], count, "dx")
        check(dw, ref["dw"], S["dw"], count + B * L, "dw")
        check(db, ref["db"], S["db"], count + B * L, "db")
        again = gi.causal_conv_backward(gy, x, w, b, silu=silu, lengths=n, want_db=True)
        assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    dx, dw, db = gi.causal_conv_backward(gy, x, w, bias, lengths=n, want_dx=False)
    assert dx is None and dw is not None and db is not None
    dx, dw, db = gi.causal_conv_backward(gy, x, w, lengths=n, want_dw=False)
    assert dx is not None and dw is None and db is None


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,K", [(1, 1, 1), (1, 300, 4), (5, 257, 2), (9, 64, 8), (300, 33, 3)])
def test_conv_step(B, D, K, dtype):
    """Lines in any order, padding rows (slots outside on both sides), untouched lines."""
    i = Inputs(B + D + K, dtype)
    x = i.normal(B, 2 * D)[:, 1:2 * D:2]          # element stride 2
    w, bias = i.params(D, K, scale=K ** -0.5), i.params(D, scale=0.2)
    state = i.normal(B + 3, D, K - 1)
    slots = torch.from_numpy(i.rng.permutation(B + 3)[:B].astype(np.int32)).cuda()
    for at, bad in ((1, -1), (3, B + 3), (4, 2 ** 31 - 1), (5, -2 ** 31)):
        if at < B:
            slots[at] = bad
    before = state.clone()
    y = gi.causal_conv_step(x, state, w, bias, slots=slots)
    lines = slots.tolist()
    live = [b for b in range(B) if 0 <= lines[b] < B + 3]
    at = [lines[b] for b in live]
    ry, rnew, S = oracle.causal_conv(num(x)[0][live][..., None], *num(w, bias), True, num(before)[0][at])
    check(y[live], ry[..., 0], S[..., 0], 2 * K + 10 + S.max(), "y")
    want = num(before)[0]
    want[at] = rnew
    assert np.array_equal(num(state)[0], want)
    dead = [b for b in range(B) if b not in live]
    assert (y[dead] == 0).all()
    # Without slots row b has line b.
    state = before.clone()
    y = gi.causal_conv_step(x, state, w, None, silu=False)
    ry, rnew, S = oracle.causal_conv(num(x)[0][..., None], *num(w), None, False, num(before)[0][:B])
    check(y, ry[..., 0], S[..., 0], 2 * K + 10, "y")
    assert np.array_equal(num(state)[0], np.concatenate([rnew, num(before)[0][B:]]))


def test_conv_in_pieces():
    """A prompt in two calls and then tokens gives what one call gives."""
    i = Inputs(5, "bf16")
    x, w, bias = i.normal(3, 10, 40), i.params(10, 4, scale=0.5), i.params(10)
    whole, state = gi.causal_conv(x, w, bias, want_state=True)
    a, s = gi.causal_conv(x[..., :21], w, bias, want_state=True)
    b, s = gi.causal_conv(x[..., 21:30], w, bias, state=s, want_state=True)
    tokens = [gi.causal_conv_step(x[..., t], s, w, bias) for t in range(30, 40)]
    assert torch.equal(torch.cat([a, b, torch.stack(tokens, -1)], -1), whole)
    assert torch.equal(s, state)


# ---- state_scan ----------------------------------------------------------------------------------

SCAN = [  # B, D, L, N, G, lengths, layout
    (1, 1, 1, 1, 1, None, "dense"), (1, 1, 2, 16, 1, None, "dense"), (2, 3, 5, 3, 1, None, "dense"),
    (7, 6, 9, 16, 2, "ragged", "dense"), (2, 4, 7, 4, 4, "none", "dense"), (1, 17, 127, 16, 1, None, "padded"),
    (1, 33, 128, 16, 1, None, "slice"), (2, 40, 129, 5, 2, None, "swapped"),
    (5, 20, 300, 24, 1, "ragged", "padded"), (2, 35, 257, 33, 1, None, "slice"),
    (1, 2, 1500, 16, 1, None, "dense"), (1, 3, 140, 256, 1, None, "dense"), (3, 70, 20, 8, 2, "ragged", "swapped"),
]


class Scan:
    def __init__(self, case, dtype, soft=True, gate=True, extras=True):
        B, D, L, N, G, kind, layout = case
        i = Inputs(B * 100 + L + N, dtype)
        self.case, self.inputs, self.soft = case, i, soft
        self.n = lengths_of(kind, B, L)

        def act(*shape, **k):
            return poison(i.normal(*shape, layout=layout, **k), self.n)

        self.x, self.gout = act(B, D, L), act(B, D, L)
        self.z = act(B, D, L) if gate else None
        if soft:
            self.dt, self.bias = act(B, D, L, scale=0.3), i.params(D, low=-5, high=-3) if extras else None
        else:
            v = torch.from_numpy(i.rng.uniform(0.01, 0.2, (B, D, L))).to(i.dtype).cuda()
            self.dt, self.bias = poison(arrange(v, layout), self.n), None
        if soft and not extras:
            self.dt = poison(arrange((i.normal(B, D, L) - 4), layout), self.n)
        bc = poison(i.normal(B, 2 * G * N + 1, L), self.n)
        self.B, self.C = (bc[:, k * G * N:(k + 1) * G * N].unflatten(1, (G, N)) for k in (0, 1))
        self.A = i.params(D, N, low=-4, high=-0.05)
        self.skip = i.params(D) if extras else None
        self.state = i.params(B, D, N) if extras else None
        self.gstate = i.params(B, D, N) if extras else None

    def forward(self, **k):
        return gi.state_scan(self.x, self.dt, self.A, self.B, self.C, self.skip, self.z, self.bias,
                             softplus=self.soft, state=self.state, lengths=self.n, **k)

    def backward(self, marks, **k):
        return gi.state_scan_backward(self.gout, self.x, self.dt, self.A, self.B, self.C, marks, self.skip,
                                      self.z, self.bias, softplus=self.soft, lengths=self.n,
                                      grad_state=self.gstate, **k)

    def numbers(self):
        return num(self.x, self.dt, self.A, self.B, self.C, self.skip, self.z, self.bias)

    def check_forward(self):
        L = self.case[2]
        y, h, marks = self.forward(want_state=True, want_checkpoints=True)
        ry, rh, S, H, rmarks = oracle.state_scan(*self.numbers(), self.soft, *num(self.state), self.n,
                                                 every=gi.SCAN_CHECKPOINT)
        check(y, ry, S, 32 * L + 64, "y")
        check(h, rh, H, 32 * L + 64, "state")
        check(marks, rmarks, np.abs(rmarks) + np.abs(H)[:, :, None], 32 * L + 64, "checkpoints")
        plain = self.forward()
        assert torch.equal(plain[0], y) and plain[1] is None and plain[2] is None
        return marks

    def check_backward(self, marks):
        B, D, L, N, G, _, _ = self.case
        g = self.backward(marks, want_dstate=True)
        ref = oracle.state_scan_grads(*num(self.gout), *self.numbers(), self.soft, *num(self.state), self.n,
                                      *num(self.gstate))
        more = {"dA": B * L, "dD": B * L, "ddt_bias": B * L, "dB": D // G, "dC": D // G}
        for name, got in g._asdict().items():
            if got is not None:
                check(got, ref[name], ref["S" + name], 64 * L + 128 + more.get(name, 0), name)
        assert (g.dz is None) == (self.z is None) and (g.dD is None) == (self.skip is None)
        again = self.backward(marks, want_dstate=True)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(g, again))


@pytest.mark.parametrize("case", SCAN, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_forward(case, dtype):
    Scan(case, dtype).check_forward()


@pytest.mark.parametrize("case", SCAN, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_scan_backward(case, dtype):
    s = Scan(case, dtype)
    s.check_backward(s.forward(want_checkpoints=True)[2])


@pytest.mark.parametrize("case", [
    # Sizes for which the work is dealt to waves in every way there is (two chunks at least).
    (1, 4096, 1030, 16, 1), (1, 1024, 1030, 16, 1), (1, 256, 1030, 16, 1), (1, 1024, 600, 16, 1),
    (8, 4096, 260, 16, 1), (8, 2048, 150, 16, 1), (16, 1024, 70, 16, 1), (1, 1536, 140, 16, 1), (5, 1000, 301, 16, 1),
    (3, 700, 150, 18, 2)], ids=str)
def test_scan_sizes(case):
    Scan((*case, None, "dense"), "bf16").check_forward()


@pytest.mark.parametrize("case", [(8, 1040, 300, 16, 1), (260, 2, 140, 3, 2), (2, 600, 777, 24, 2)], ids=str)
def test_scan_backward_sizes(case):
    """Whole rows a work-group and cut ones, lanes of 16 and of 8 positions."""
    s = Scan((*case, None, "dense"), "f32")
    s.check_backward(s.forward(want_checkpoints=True)[2])


@pytest.mark.parametrize("case", [(1, 2000, 2045, 4, 2), (1, 1030, 2045, 5, 1), (1, 260, 2050, 4, 2), (2, 1024, 1030, 4, 1),
                                  (2, 4096, 250, 4, 1), (1, 1024, 2040, 4, 1)], ids=str)
def test_scan_sizes_of_few_states(case):
    """Rows of 64 lanes dealt in every way; backward by work-groups of 8 waves, whole rows and cut ones."""
    s = Scan((*case, None, "dense"), "bf16")
    s.check_backward(s.check_forward())


@pytest.mark.parametrize("soft,gate,extras", [(True, False, True), (False, True, False), (True, True, False)])
def test_scan_options(soft, gate, extras):
    s = Scan((2, 18, 150, 16, 1, None, "dense"), "f32", soft, gate, extras)
    s.check_backward(s.check_forward())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,N,G", [(1, 1, 1, 1), (1, 300, 16, 1), (5, 258, 24, 2), (9, 64, 7, 4), (3, 40, 256, 1),
                                     (70, 33, 16, 1)])
def test_scan_step(B, D, N, G, dtype):
    i = Inputs(B + D + N, dtype)
    x, dt, z = i.normal(B, 2 * D)[:, 1:2 * D:2], i.normal(B, D, scale=0.3), i.normal(B, D)
    A, skip, bias = i.params(D, N, low=-4, high=-0.05), i.params(D), i.params(D, low=-5, high=-3)
    bc = i.normal(B, 2 * G * N + 1)
    for Bm, Cm in ((bc[:, :G * N].unflatten(1, (G, N)), bc[:, G * N:2 * G * N].unflatten(1, (G, N))),
                   (i.normal(B, G, N, 3)[..., 1], i.normal(B, G, N, 3)[..., 2])):   # strided states
        state = i.params(B + 3, D, N)
        slots = torch.from_numpy(i.rng.permutation(B + 3)[:B].astype(np.int32)).cuda()
        for at, bad in ((1, -1), (3, B + 3), (4, 2 ** 31 - 1), (5, -2 ** 31)):
            if at < B:
                slots[at] = bad
        before = state.clone()
        y = gi.state_scan_step(x, dt, A, Bm, Cm, state, skip, z, bias, slots=slots)
        lines = slots.tolist()
        live = [b for b in range(B) if 0 <= lines[b] < B + 3]
        at = [lines[b] for b in live]

        def row(t):
            return num(t)[0][live][..., None]

        ry, rh, S, H = oracle.state_scan(row(x), row(dt), *num(A), row(Bm), row(Cm), *num(skip), row(z), *num(bias),
                                         True, num(before)[0][at])
        check(y[live], ry[..., 0], S[..., 0], 96, "y")
        check(state[at], rh, H, 96, "state")
        rest = [k for k in range(B + 3) if k not in at]
        assert torch.equal(state[rest], before[rest])
        dead = [b for b in range(B) if b not in live]
        assert (y[dead] == 0).all()
    state = before.clone()
    y = gi.state_scan_step(x, dt, A, Bm, Cm, state)
    ry, rh, S, H = oracle.state_scan(*[num(v)[0][..., None] for v in (x, dt)], *num(A),
                                     *[num(v)[0][..., None] for v in (Bm, Cm)], None, None, None, True,
                                     num(before)[0][:B])
    check(y, ry[..., 0], S[..., 0], 96 + 8 * N, "y")
    assert torch.equal(state[B:], before[B:])


def test_scan_in_pieces():
    """A prompt in two calls, then tokens, against one call."""
    s = Scan((2, 20, 200, 16, 1, None, "dense"), "f32")
    ry, rh, S, H = oracle.state_scan(*s.numbers(), True, *num(s.state))
    h, ys = s.state, []
    for lo, hi in ((0, 77), (77, 190)):
        part = [v[..., lo:hi] for v in (s.x, s.dt, s.B, s.C, s.z)]
        y, h, _ = gi.state_scan(part[0], part[1], s.A, part[2], part[3], s.skip, part[4], s.bias, state=h,
                                want_state=True)
        ys.append(y)
    for t in range(190, 200):
        x, dt, B, C, z = (v[..., t] for v in (s.x, s.dt, s.B, s.C, s.z))
        ys.append(gi.state_scan_step(x, dt, s.A, B, C, h, s.skip, z, s.bias)[..., None])
    check(torch.cat(ys, -1), ry, S, 32 * 200 + 64, "y")
    check(h, rh, H, 32 * 200 + 64, "state")


def test_scan_keeps_later_trouble_from_earlier_positions():
    """NaN at one position reaches that and later ones of its channel, nothing else."""
    s = Scan((1, 20, 200, 16, 1, None, "dense"), "f32")
    clean = s.forward()[0]
    s.x[0, 3, 100] = float("nan")
    y = s.forward()[0]
    bad = torch.isnan(y)
    assert bad[0, 3, 100:].all() and int(bad.sum()) == 100
    assert torch.equal(y[~bad], clean[~bad])


# ---- block_norm ----------------------------------------------------------------------------------

NORM = [  # B, D, L, lengths, layout
    (1, 1, 1, None, "dense"), (1, 64, 1, None, "dense"), (3, 1000, 1, None, "slice"), (2, 4100, 1, None, "swapped"),
    (2, 9, 3, None, "dense"), (7, 130, 9, "ragged", "dense"), (2, 33, 8, "none", "dense"), (2, 257, 33, None, "padded"),
    (1, 96, 130, None, "slice"), (5, 40, 300, "ragged", "swapped"), (1, 2050, 40, None, "dense"),
]


class Norm:
    def __init__(self, case, dtype, parts="all"):
        B, D, L, kind, layout = case
        i = Inputs(B + D + L, dtype)
        self.case, self.n = case, lengths_of(kind, B, L)

        def act(dtype=None):
            return poison(i.normal(B, D, L, layout=layout, dtype=dtype), self.n)

        self.y, self.r, self.gu, self.gr = act(), act(torch.float32), act(), act(torch.float32)
        self.post = i.params(D) if parts in ("all", "post") else None
        self.pre = i.params(D) if parts in ("all", "pre") else None
        self.gate = act() if parts in ("all", "gate") else None
        self.scale = i.params(D) if parts in ("all", "scale") else None
        if self.pre is None:
            self.gu = None

    def forward(self, **k):
        return gi.block_norm(self.y, self.r, self.post, self.pre, gate=self.gate, scale=self.scale, eps=1e-3,
                             lengths=self.n, **k)

    def check(self):
        B, D, L, _, _ = self.case
        r, u = self.forward()
        rest = num(self.post, self.pre, self.gate, self.scale)
        rr, ru, Sr, Su = oracle.block_norm(*num(self.y, self.r), *rest, 1e-3, self.n)
        check(r, rr, Sr, D + 32, "residual")
        assert (u is None) == (self.pre is None)
        if u is not None:
            check(u, ru, Su, 2 * D + 64, "u")
        r2, u2 = self.forward(residual_out=self.r.clone())
        assert torch.equal(r2, r) and (u is None or torch.equal(u2, u))
        g = self.backward(r)
        ref = oracle.block_norm_grads(*num(self.gr, self.gu, self.y, r), *rest, 1e-3, self.n)
        for name, got in g._asdict().items():
            assert (got is None) == (name not in ref), name
            if got is not None:
                more = B * L if got.dim() == 1 else 0
                check(got, ref[name], ref["S" + name], 4 * D + 128 + more, name)
        again = self.backward(r)
        assert all(p is q is None or torch.equal(p, q) for p, q in zip(g, again))

    def backward(self, r):
        return gi.block_norm_backward(self.gr, self.gu, self.y, poison(r.clone(), self.n), self.post, self.pre,
                                      gate=self.gate, scale=self.scale, eps=1e-3, lengths=self.n)


@pytest.mark.parametrize("case", NORM, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(case, dtype):
    Norm(case, dtype).check()


@pytest.mark.parametrize("case", [
    # Tiles of 32, 16 and 8 columns, kept and read again.
    (16, 33, 250, None, "dense"), (6, 70, 250, "ragged", "dense"), (6, 1030, 250, None, "padded"),
    (1, 1100, 30, None, "dense"), (3, 2060, 100, "ragged", "slice"), (1, 4100, 20, None, "dense"),
    (32, 2060, 250, None, "dense")], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_sizes(case, dtype):
    Norm(case, dtype).check()


@pytest.mark.parametrize("parts", ["post", "pre", "gate", "scale", "none"])
def test_norm_options(parts):
    Norm((2, 50, 20, None, "dense"), "f32", parts).check()


def test_norm_missing_gradients_are_zeros():
    s = Norm((2, 50, 20, None, "dense"), "f32")
    r, _ = s.forward()
    for gr, gu in ((None, s.gu), (s.gr, None), (None, None)):
        g = gi.block_norm_backward(gr, gu, s.y, r, s.post, s.pre, gate=s.gate, scale=s.scale, eps=1e-3)
        zr, zu = (torch.zeros_like(a) if b is None else b for a, b in ((s.gr, gr), (s.gu, gu)))
        want = gi.block_norm_backward(zr, zu, s.y, r, s.post, s.pre, gate=s.gate, scale=s.scale, eps=1e-3)
        assert all(torch.equal(p, q) for p, q in zip(g, want))


def test_norm_in_place():
    """The new residual may be written over the old one."""
    s = Norm((2, 70, 50, None, "dense"), "bf16")
    r, u = s.forward()
    kept = s.r.clone()
    s.r = kept
    r2, u2 = s.forward(residual_out=kept)
    assert r2 is kept and torch.equal(r2, r) and torch.equal(u2, u)


# ---- streams, graphs, long caches, refusals -------------------------------------------------------


def everything(s, c, m, conv_state, scan_state):
    """One pass through every entry point; the two caches are updated in place."""
    out = list(s.forward(want_state=True, want_checkpoints=True))
    out += s.backward(out[2])
    x, w, b, gy = c
    out += gi.causal_conv(x, w, b, want_state=True) + gi.causal_conv_backward(gy, x, w, b)
    r, u = m.forward()
    out += [r, u, *m.backward(r)]
    t = 3
    out.append(gi.causal_conv_step(x[..., t], conv_state, w, b))
    out.append(gi.state_scan_step(s.x[..., t], s.dt[..., t], s.A, s.B[..., t], s.C[..., t], scan_state))
    return [v for v in out if v is not None]


def parts_of_everything():
    s = Scan((2, 36, 300, 16, 1, None, "dense"), "bf16")
    i = Inputs(9, "bf16")
    c = (i.normal(2, 30, 500), i.params(30, 4), i.params(30), i.normal(2, 30, 500))
    m = Norm((2, 70, 50, None, "dense"), "bf16")
    return s, c, m, i.normal(2, 30, 3), i.params(2, 36, 16)


def test_graph_replays():
    """Captured once, replayed with eager work in between: each replay equals the eager pass."""
    parts = parts_of_everything()
    caches = [v.clone() for v in parts[3:]]
    everything(*parts)                       # loads the kernels before the capture
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = everything(*parts)
    eager_caches = [v.clone() for v in caches]
    for v, kept in zip(parts[3:], caches):
        v.copy_(kept)
    for _ in range(4):
        graph.replay()
        want = everything(*parts[:3], *eager_caches)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert all(torch.equal(p, q) for p, q in zip(parts[3:], eager_caches))


def test_on_a_named_stream():
    """Outputs of a call on another stream are good once that stream is done."""
    s = Scan((2, 36, 300, 16, 1, None, "dense"), "bf16")
    want = s.forward(want_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.forward(want_state=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_offsets_beyond_32_bits():
    """A cache and an activation whose far elements are past 2^32 bytes and 2^31 elements."""
    i = Inputs(4, "bf16")
    B, D, N = 2, 64, 16
    lines = 2 ** 31 // (D * N) + 10
    state = torch.empty(lines, D, N, device="cuda")
    slots = torch.tensor([lines - 1, 5], dtype=torch.int32, device="cuda")
    start = i.params(B, D, N)
    state[slots.long()] = start
    x, dt, Bm, Cm = i.normal(B, D), i.normal(B, D), i.normal(B, 1, N), i.normal(B, 1, N)
    A = i.params(D, N, low=-4, high=-0.05)
    y = gi.state_scan_step(x, dt, A, Bm, Cm, state, slots=slots)
    want_state = start.clone()
    want = gi.state_scan_step(x, dt, A, Bm, Cm, want_state)
    assert torch.equal(y, want) and torch.equal(state[slots.long()], want_state)
    del state
    far = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    near = i.normal(2, 8, 100)
    wide = far.as_strided((2, 8, 100), (2 ** 31 + 100, 100, 1))
    wide.copy_(near)
    w = i.params(8, 4)
    assert torch.equal(gi.causal_conv(wide, w)[0], gi.causal_conv(near, w)[0])
    r = i.normal(2, 8, 100, dtype=torch.float32)
    assert torch.equal(gi.block_norm(wide, r, w[:, 0].contiguous())[0], gi.block_norm(near, r, w[:, 0].contiguous())[0])


def test_refusals():
    i = Inputs(1, "bf16")
    x, w = i.normal(2, 6, 10), i.params(6, 4)
    A, B, C = i.params(6, 3), i.normal(2, 1, 3, 10), i.normal(2, 1, 3, 10)
    r = i.normal(2, 6, 10, dtype=torch.float32)
    bad = [
        lambda: gi.causal_conv(x[0], w), lambda: gi.causal_conv(x.double(), w),
        lambda: gi.causal_conv(x, w.bfloat16()), lambda: gi.causal_conv(x, w[:5]),
        lambda: gi.causal_conv(x, w.cpu()), lambda: gi.causal_conv(x.transpose(1, 2), i.params(10, 4)),
        lambda: gi.causal_conv(x, w, state=i.normal(2, 6, 4)),
        lambda: gi.causal_conv(x, w, lengths=torch.zeros(2, device="cuda", dtype=torch.int64)),
        lambda: gi.causal_conv(x, w, out=x.float()),
        lambda: gi.causal_conv(x, None), lambda: gi.causal_conv(None, w),
        lambda: gi.causal_conv_backward(x.float(), x, w),
        lambda: gi.causal_conv_step(x[..., 0], i.normal(2, 6, 2), w),
        lambda: gi.causal_conv_step(x, i.normal(2, 6, 3), w),
        lambda: gi.state_scan(x, x, A, B[:, :, :2], C), lambda: gi.state_scan(x, x.float(), A, B, C),
        lambda: gi.state_scan(x, x, A.T, B, C), lambda: gi.state_scan(x, x, A, B[..., :9], C),
        lambda: gi.state_scan(x, x, A, B, C, state=i.params(2, 6, 4)),
        lambda: gi.state_scan(x, x, A, i.normal(2, 3, 3, 10)[:, ::2], i.normal(2, 2, 3, 10)),
        lambda: gi.state_scan_backward(x, x, x, A, B, C, i.params(2, 6, 2, 3)),
        lambda: gi.state_scan_backward(x, x, x, A, B, C, i.params(2, 6, 1, 3), dz=x),
        lambda: gi.state_scan_step(x[..., 0], x[..., 0], A, B[..., 0], C[..., 0], i.params(2, 6, 3).bfloat16()),
        lambda: gi.block_norm(x, x), lambda: gi.block_norm(x, r, out=x), lambda: gi.block_norm(x, r[:1]),
        lambda: gi.block_norm(x, r, gate=r), lambda: gi.block_norm_backward(r, None, x, r, dgate=x),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % k)
    for f in (lambda: gi.causal_conv(x, i.params(6, 9)),                      # beyond the taps
              lambda: gi.causal_conv(x[..., :0], w),                          # no positions
              lambda: gi.causal_conv(x, w, out=x[:1].expand(2, 6, 10)),       # an output that shares elements
              lambda: gi.state_scan(x, x, i.params(6, 3), i.normal(2, 4, 3, 10), i.normal(2, 4, 3, 10)),
              lambda: gi.state_scan_step(x[..., 0], x[..., 0], A, B[..., 0], C[..., 0], i.params(1, 6, 3)),
              lambda: gi.block_norm(x, r, eps=-1.0)):
        with pytest.raises(gi.Conv2dGiError):
            f()
