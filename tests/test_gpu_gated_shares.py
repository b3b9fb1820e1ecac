"""gated_scan_backward by every plan with all batch items in a work-group and with one, at
test_gpu_gated_scan.py's tolerances; and long rows held to the positions that they remember."""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_gated_scan import Gated  # noqa: E402
from test_gpu_sequence import TYPES, U, half, num  # noqa: E402

# (plan, all batch items in a work-group), case
SHARES = [
    (("lanes=4 waves=1", True), (6, 21, 30, "ragged", "dense")),
    (("lanes=4 waves=1", False), (11, 40, 17, None, "padded")),
    (("lanes=16 waves=1", True), (8, 700, 100, None, "dense")),
    (("lanes=16 waves=1", False), (8, 1100, 100, None, "slice")),
    (("lanes=64 waves=1", True), (7, 11, 1000, "ragged", "slice")),
    (("lanes=64 waves=1", False), (9, 5, 300, None, "dense")),
    (("lanes=64 waves=1", False), (6, 400, 300, "ragged", "dense")),
    (("lanes=64 waves=2", True), (4, 5, 1030, "ragged", "padded")),
    (("lanes=64 waves=2", False), (7, 5, 2000, "ragged", "dense")),
    (("lanes=64 waves=4", True), (2, 3, 3000, "ragged", "dense")),
    (("lanes=64 waves=4", False), (3, 3, 3000, "ragged", "swapped")),
    (("lanes=64 waves=8", True), (1, 3, 4100, None, "padded")),
    (("lanes=64 waves=8", False), (6, 2, 5000, "ragged", "dense")),
    (("lanes=64 waves=16", True), (1, 5, 9001, None, "dense")),
    (("lanes=64 waves=16", False), (6, 3, 8200, "ragged", "dense")),
]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


@pytest.mark.parametrize("plan,case", SHARES, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_shares(plan, case, dtype):
    s = Gated(case, dtype)
    s.check_backward(s.check_forward())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [700, 2100, 9001])
def test_long_rows_with_a_short_memory(L, dtype):
    """Each position's roundings count for as long as it is remembered.

    What entered k positions ago has been multiplied by k decays, each good to 30 u, and by k sums' roundings, 1 u: with
    the gates' 32 u it is good to 32 (k + 1) u of its own magnitude.  V below is the sum of (k + 1) times these
    magnitudes; silu and the stores are within 64 u of the whole."""
    s = Gated((2, 12, L, None, "dense"), dtype)
    s.A = -torch.exp(torch.linspace(-4, 0.69, 12, device="cuda"))
    x, r, i, A, z, r_bias, i_bias, state = s.numbers()
    y, h, _ = s.forward(want_state=True)
    ry, rh, S, H = oracle.gated_scan(x, r, i, A, z, r_bias, i_bias, state)
    u = A[:, None] * oracle.sigmoid(r + r_bias[:, None])
    a, enter = np.exp(u), np.sqrt(-np.expm1(2 * u)) * np.abs(x) * oracle.sigmoid(i + i_bias[:, None])
    V, size = np.abs(state), np.abs(state)     # by the positions that each has seen, and once
    Vs = np.zeros_like(ry)
    for t in range(L):
        V = a[:, :, t] * (V + size) + enter[:, :, t]
        size = a[:, :, t] * size + enter[:, :, t]
        Vs[:, :, t] = V * np.abs(z[:, :, t]) * oracle.sigmoid(z[:, :, t])
    hb = half(y.dtype)
    tiny = 1e-30 if hb == 0 else float(torch.finfo(y.dtype).tiny) * hb * 2
    err = np.abs(num(y)[0] - ry)
    limit = hb * np.abs(ry) + U * (32 * Vs + 64 * S) * (1 + hb) + tiny
    assert (err <= limit).all(), float((err / limit).max())
    err = np.abs(num(h)[0] - rh)
    assert (err <= U * (32 * V + 64 * H)).all(), float((err / (U * (32 * V + 64 * H))).max())
