"""A product's result does not depend on the call that it is part of: the sum turns to fp32, meets
scales and bias in one fused operation, and is rounded once more to a 16-bit type, in every
kernel alike."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_sequence import TYPES, Inputs  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,K", [(4200, 1024), (1030, 256)])
def test_rows_alone_and_among_others(E, K, dtype):
    i = Inputs(E, dtype)
    N = 4100
    codes = torch.from_numpy(i.rng.integers(-127, 128, (N, K)).astype(np.int8)).cuda()
    w = torch.from_numpy(i.rng.integers(-127, 128, (E, K)).astype(np.int8)).cuda()
    s, ws, bias = i.params(N, low=1e-3, high=2e-3), i.params(E, low=1e-3, high=2e-3), i.params(E)
    # As one long sequence: tiles.
    want = gi.project_int8(codes[None], s[None], w, ws, bias, dtype=i.dtype)[0].t()
    # The formula, with numpy's float32 and its exact products and sums of float64.
    sums = (codes.double() @ w.double().t()).cpu().numpy().astype(np.float32)
    f = s.cpu().numpy()[:, None] * ws.cpu().numpy()
    # (a product of 24 by 24 bits is exact, the sum with the bias takes more: differs by a rounding at most where
    # float64's 53 bits end half way between two of float32; left out by what lies next to such a border)
    exact = sums.astype(np.float64) * f + bias.double().cpu().numpy()
    once = torch.from_numpy(exact.astype(np.float32)).cuda().to(i.dtype)
    assert (want != once).float().mean() < 1e-6
    for count in (1, 2, 8, 16, 17, 30, 40, 64, 100, 300, 1000, 2100):
        part = codes[:count].contiguous()
        for prompt in (False, True):
            if prompt:
                y = gi.project_int8(part[None], s[None, :count].contiguous(), w, ws, bias, dtype=i.dtype)[0].t()
            else:
                y = gi.project_int8(part[:, None], s[:count, None].contiguous(), w, ws, bias, dtype=i.dtype)[..., 0]
            assert torch.equal(y, want[:count]), (count, prompt, int((y != want[:count]).sum()))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,E", [(2048, 4096), (300, 4100)])
def test_tokens_alone_and_among_others(D, E, dtype):
    i = Inputs(E, dtype)
    x, (w, ws), bias = i.normal(2100, D), gi.quantize_weight(i.normal(E, D, dtype=torch.float32)), i.params(E)
    want = gi.project_int8_step(x, w, ws, bias)
    for count in (1, 3, 8, 16, 17, 40, 300):
        assert torch.equal(gi.project_int8_step(x[:count], w, ws, bias), want[:count]), count
