"""gated_scan at rates and gates at the ends of what it takes, forward and backward."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_gated_scan import Gated  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


@pytest.mark.parametrize("L", [3, 100, 700, 3000])
@pytest.mark.parametrize("gate", [True, False])
def test_rate_above_zero(L, gate):
    """1 - a^2 is negative: its root is NaN, and so is what the root enters; other channels do not change."""
    s = Gated((6, 36, L, "ragged", "dense"), "f32", gate=gate)

    def everything():
        y, h, marks = s.forward(want_state=True, want_checkpoints=True)
        return y, h, s.backward(marks, want_dstate=True)

    clean_y, clean_h, clean = everything()
    s.A[5], s.A[17] = 0.3, 1e-3
    y, h, g = everything()
    bad, good = [5, 17], [d for d in range(36) if d not in (5, 17)]
    for b in range(6):
        n = int(s.n[b].clamp(0, L))
        for name, t in [("y", y), ("dx", g.dx), ("dr", g.dr), ("di", g.di)] + ([("dz", g.dz)] if gate else []):
            assert torch.isnan(t[b, bad, :n]).all(), name
            assert (t[b, :, n:] == 0).all(), name
    for name in ("dA", "dr_bias", "di_bias"):
        assert torch.isnan(getattr(g, name)[bad]).all(), name
    for p, q in zip((y, h, *g), (clean_y, clean_h, *clean)):
        if p is not None:
            assert torch.equal(*((v[:, good] if v.dim() > 1 else v[good]) for v in (p, q)))
