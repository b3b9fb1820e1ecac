"""Products in 8 bits whose scales, or the scales' product, are near the ends of fp32's range.

The bound is test_gpu_int8.py's, 4 u of the terms' magnitudes: a sum as a float, the scales'
product, the product and the addition.  A result beyond the type's range is an infinity.
"""
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


SIZES = [  # B, E, L, K: every kernel of the product, along positions and along channels
    (1, 40, 9, 128), (1, 4200, 12, 256), (1, 300, 20, 128), (1, 4200, 30, 128), (2, 1000, 40, 128), (1, 2100, 60, 128),
    (3, 1000, 301, 128), (2, 1700, 700, 256), (2, 4200, 2000, 256),
    (9, 40, 1, 128), (16, 5000, 1, 256), (30, 200, 1, 128), (30, 5000, 1, 128), (60, 8000, 1, 128), (60, 9000, 1, 128), (900, 1500, 1, 128),
    (2100, 1800, 1, 128), (4000, 4200, 1, 256),
]


def rows(case, scales, w_scales, dtype, bias):
    B, E, L, K = case
    i = Inputs(E + L, "f32")
    codes = torch.from_numpy(i.rng.integers(-127, 128, (B, L, K)).astype(np.int8)).cuda()
    w = torch.from_numpy(i.rng.integers(-127, 128, (E, K)).astype(np.int8)).cuda()
    (codes if L == 1 else codes.transpose(0, 1))[::3] = 0     # positions, and channels, whose sums are 0
    w[::5] = 0

    def pick(values, *shape):
        at = torch.from_numpy(i.rng.integers(len(values), size=shape))
        return torch.tensor(values, dtype=torch.float32)[at].cuda()

    s, ws = pick(scales, B, L), pick(w_scales, E)
    b = i.params(E) * bias if bias else None
    y = gi.project_int8(codes, s, w, ws, b, dtype=TYPES[dtype])
    ref, S = oracle.int8_product(codes.view(B * L, K).cpu().numpy(), num(s.view(-1))[0], w.cpu().numpy(), *num(ws, b))
    return y, ref.reshape(E, B, L).transpose(1, 0, 2), S.reshape(E, B, L).transpose(1, 0, 2)


def check_ends(y, ref, S):
    """Infinities where the result is beyond the type's range; the others as `check` has them."""
    top = float(torch.finfo(y.dtype).max)
    got = y.double().cpu().numpy()
    beyond, within = np.abs(ref) > top * 1.02, np.abs(ref) < top * 0.98
    assert (got[beyond] == np.sign(ref[beyond]) * np.inf).all()
    assert not np.isnan(got).any()
    keep = torch.from_numpy(within.copy()).cuda()
    zero = torch.zeros((), dtype=y.dtype, device="cuda")
    check(torch.where(keep, y, zero), np.where(within, ref, 0), np.where(within, S, 0), 4, "y")


@pytest.mark.parametrize("case", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_products_beyond_the_range(case, dtype):
    """Products of the scales past 2^128: a sum of 0 leaves the bias, others are infinite; and ones inside the range."""
    check_ends(*rows(case, [2e36, 1e-2, 1.0, 1e20], [1e30, 200.0, 1e-3, 1e-35], dtype, 1.0))


@pytest.mark.parametrize("case", SIZES, ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_products_below_the_range(case, dtype):
    """Products of the scales of 1e-40 to 1e-34 whose sums, some 1e4 to 1e6, are normal numbers."""
    y, ref, S = rows(case, [3e-25, 7e-21, 1.3e-19], [1e-15, 2.7e-16, 3.3e-15], dtype, 0.0)
    err = np.abs(y.double().cpu().numpy() - ref)
    # (by itself: `check` allows 1e-30 for what is lost below the normal range, which starts at 2^-126)
    h = 0.0 if dtype == "f32" else 2.0 ** -8
    limit = h * np.abs(ref) + 4 * 2.0 ** -24 * S * (1 + h)
    normal = np.abs(ref) > 2.0 ** -125
    assert (err <= limit)[normal].all() and normal.mean() > 0.3
    assert (err <= 2.0 ** -124)[~normal].all()


@pytest.mark.parametrize("dtype", TYPES)
def test_ordinary_results_have_the_same_bits_beside_extreme_ones(dtype):
    """One position or channel of extreme scale changes no other's result."""
    for B, E, L, K in SIZES:
        i = Inputs(B + E, dtype)
        codes = torch.from_numpy(i.rng.integers(-127, 128, (B, L, K)).astype(np.int8)).cuda()
        w = torch.from_numpy(i.rng.integers(-127, 128, (E, K)).astype(np.int8)).cuda()
        s, ws, b = i.params(B, L, low=1e-3, high=2e-3), i.params(E, low=1e-3, high=2e-3), i.params(E)
        clean = gi.project_int8(codes, s, w, ws, b, dtype=i.dtype)
        far = s.clone()
        far.view(-1)[:: 7], keep = 1e30, torch.ones(B * L, dtype=torch.bool, device="cuda")
        keep[::7] = False
        got = gi.project_int8(codes, far, w, ws, b, dtype=i.dtype)
        p, q = (t.transpose(1, 2).reshape(B * L, E)[keep] for t in (got, clean))
        assert torch.equal(p, q)
        far = ws.clone()
        far[::7] = 1e-30
        got = gi.project_int8(codes, s, w, far, b, dtype=i.dtype)
        keep = torch.ones(E, dtype=torch.bool, device="cuda")
        keep[::7] = False
        assert torch.equal(got[:, keep], clean[:, keep])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,E", [(3, 130, 70), (16, 500, 5000), (70, 300, 200)])
def test_step_of_extreme_rows(B, D, E, dtype):
    """Rows of the largest and the smallest numbers, with weights of 1e4 and of 1e-6: one call is the two calls, and
    each result the formula's."""
    i = Inputs(B + D, dtype)
    x = i.normal(B, D)
    x[::3] *= 2.5e37
    x[1::3] *= 1e-31
    x[1, :] = 0
    weight = i.normal(E, D, dtype=torch.float32)
    weight[::2] *= 1e4
    weight[1::2] *= 1e-6
    weight[4] = 0
    w, ws = gi.quantize_weight(weight)
    bias = i.params(E)
    y = gi.project_int8_step(x, w, ws, bias)
    codes, scales = gi.quantize_tokens(x.unsqueeze(2))
    assert torch.equal(y, gi.project_int8(codes, scales, w, ws, bias, dtype=i.dtype)[..., 0])
    ref, S = oracle.int8_product(codes[:, 0].cpu().numpy(), *num(scales[:, 0]), w.cpu().numpy(), *num(ws, bias))
    check_ends(y, ref.T, S.T)
    assert torch.equal(y[1], bias.to(y.dtype)) and torch.equal(y[:, 4], bias[4].to(y.dtype).expand(B))
