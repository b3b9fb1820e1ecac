"""project_int8_step on both sides of the borders between codes made inside the product and
before it: one call is the two calls, bit for bit, and the formula's result.

The bound is test_gpu_int8.py's: 4 u of the terms' magnitudes, and the type's rounding."""
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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,E", [
    (16, 1024, 300), (16, 1025, 300), (16, 2048, 40), (16, 2047, 40), (9, 1024, 33), (9, 1100, 33), (9, 2049, 33),
    (8, 2048, 70), (7, 2049, 70), (8, 4096, 50), (5, 4097, 50), (5, 6500, 20), (4, 4096, 30), (3, 4097, 30),
    (3, 10922, 20), (3, 10923, 20), (4, 8192, 20), (2, 16384, 10), (2, 16385, 10), (1, 32768, 10), (1, 32769, 10),
    (9, 3640, 20), (16, 70, 16384), (16, 70, 16385), (5, 130, 16400), (1, 130, 16384), (2, 130, 16387), (4, 70, 33000)])
def test_either_side_of_a_border(B, D, E, dtype):
    i = Inputs(B + D + E, dtype)
    w, ws = gi.quantize_weight(i.normal(E, D, dtype=torch.float32))
    bias, x = i.params(E), i.normal(B, D)
    codes, scales = gi.quantize_tokens(x.unsqueeze(2))
    want = gi.project_int8(codes, scales, w, ws, bias, dtype=i.dtype)[..., 0]
    ref, S = oracle.int8_product(codes[:, 0].cpu().numpy(), *num(scales[:, 0]), w.cpu().numpy(), *num(ws, bias))
    check(want, ref.T, S.T, 4, "y")
    assert torch.equal(gi.project_int8_step(x, w, ws, bias), want)
    wide = i.normal(B, 2 * D + 1)
    wide[:, 1::2] = x
    assert torch.equal(gi.project_int8_step(wide[:, 1::2], w, ws, bias), want)
