"""gated_scan_step of large batches, four channels a thread, against the oracle and against one
channel a thread on the same numbers.

Tolerances as in test_gpu_gated_scan.py: one position is good to 32 u, the stores and silu to 64 more."""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_sequence import TYPES, Inputs, check, num  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


def spread(t):
    """The same numbers as every second column of a wider tensor, one element off its start."""
    wide = torch.full((t.shape[0], 2 * t.shape[1] + 1), 7.0, dtype=t.dtype, device=t.device)
    wide[:, 1::2] = t
    return wide[:, 1::2]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gate,extras", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("B,D", [(256, 1024), (70, 4004), (300, 1020), (3, 100000), (1, 262144)])
def test_step(B, D, gate, extras, dtype):
    i = Inputs(B + D, dtype)
    A = -torch.exp(i.params(D, low=-7, high=0.69))
    r_bias, i_bias = (i.params(D, scale=0.5) if extras else None for _ in range(2))
    x, r, g = (i.normal(B, D) for _ in range(3))
    z = i.normal(B, D) if gate else None
    lines = B + 3
    state = i.params(lines, D)
    slots = torch.from_numpy(i.rng.permutation(lines)[:B].astype(np.int32)).cuda()
    for at, bad in ((1, -1), (3, lines), (4, 2 ** 31 - 1), (5, -2 ** 31), (68, -7)):
        if at < B:
            slots[at] = bad
    before, at = state.clone(), slots.tolist()
    # Rows of a wider tensor, as a projection leaves them.
    xs = torch.cat([x, r, g], 1)
    y = gi.gated_scan_step(xs[:, :D], xs[:, D:2 * D], xs[:, 2 * D:], A, state, z, r_bias, i_bias, slots=slots)
    live = [b for b in range(B) if 0 <= at[b] < lines]
    used = [at[b] for b in live]
    rows = [None if v is None else num(v)[0][live][..., None] for v in (x, r, g, z)]
    ry, rh, S, H = oracle.gated_scan(*rows[:3], *num(A), rows[3], *num(r_bias, i_bias), num(before)[0][used])
    check(y[live], ry[..., 0], S[..., 0], 96, "y")
    check(state[used], rh, H, 96, "state")
    rest = [k for k in range(lines) if k not in set(used)]
    assert torch.equal(state[rest], before[rest])
    assert (y[[b for b in range(B) if b not in set(live)]] == 0).all()
    # One channel a thread.
    single, out = before.clone(), spread(torch.zeros_like(x))
    got = gi.gated_scan_step(spread(x), spread(r), spread(g), A, single, None if z is None else spread(z), r_bias,
                             i_bias, slots=slots, out=out)
    assert got is out and torch.equal(got, y) and torch.equal(single, state)
    assert (out._base[:, ::2] == 7).all()
    # Without slots: row b uses line b.
    state = before.clone()
    y = gi.gated_scan_step(x, r, g, A, state, z, r_bias, i_bias)
    single = before.clone()
    assert torch.equal(gi.gated_scan_step(spread(x), r, g, A, single, z, r_bias, i_bias), y)
    assert torch.equal(single, state) and torch.equal(state[B:], before[B:]) and not torch.equal(state[:B], before[:B])


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_rows_on_any_alignment(offset):
    """Dense channels that start anywhere, states and parameters too."""
    i = Inputs(offset, "bf16")
    B, D = 256, 1024

    def shifted(t):
        flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:]
        return flat.copy_(t.flatten()).view(t.shape)

    A = -torch.exp(i.params(D, low=-7, high=0.69))
    b1, b2, state = i.params(D), i.params(D), i.params(B, D)
    x, r, g, z = (i.normal(B, D) for _ in range(4))
    want_state, got_state = state.clone(), shifted(state)
    want = gi.gated_scan_step(x, r, g, A, want_state, z, b1, b2)
    got = gi.gated_scan_step(shifted(x), shifted(r), shifted(g), shifted(A), got_state, shifted(z), shifted(b1),
                             shifted(b2))
    assert torch.equal(got, want) and torch.equal(got_state, want_state)


def test_cache_beyond_32_bits():
    i = Inputs(4, "bf16")
    B, D = 256, 1024
    lines = 2 ** 31 // D + 300
    state = torch.empty(lines, D, device="cuda")
    slots = torch.arange(B, dtype=torch.int32, device="cuda") * 2
    slots[1::2] = lines - 1 - slots[1::2]
    start = i.params(B, D)
    state[slots.long()] = start
    x, r, g, z, A = *(i.normal(B, D) for _ in range(4)), i.params(D, low=-2, high=-0.1)
    want_state = start.clone()
    want = gi.gated_scan_step(spread(x), r, g, A, want_state, z)      # (one channel a thread)
    assert torch.equal(gi.gated_scan_step(x, r, g, A, state, z, slots=slots), want)
    assert torch.equal(state[slots.long()], want_state)


def test_graph_replays():
    i = Inputs(5, "f16")
    B, D = 300, 1024
    A, start = i.params(D, low=-2, high=-0.1), i.params(B, D)
    x, r, g, z = (i.normal(B, D) for _ in range(4))
    cache, eager = start.clone(), start.clone()
    gi.gated_scan_step(x, r, g, A, start.clone(), z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = gi.gated_scan_step(x, r, g, A, cache, z)
    cache.copy_(start)
    for _ in range(4):
        x.mul_(-0.9)
        graph.replay()
        want = gi.gated_scan_step(x, r, g, A, eager, z)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(cache, eager)
