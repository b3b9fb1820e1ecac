"""quantize_tokens by every share of positions and channels, in every type, and the products of
short prompts into wide layers.

Codes and scales have to be equal; products keep test_gpu_int8.py's bound.  A work-group of a
quantization has 1, 2 or 4 times 16 bytes of positions, by how many there are in all, 4, 8 or 16
waves, and keeps 1, 2 or 4 rounds of channels in registers, beyond which it reads them again."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_int8 import Product, check_codes  # noqa: E402
from test_gpu_sequence import TYPES, Inputs, lengths_of, poison  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


# Positions of a float32 call (16-bit ones have twice as many), channels.
SHARES = [
    # 4 times 16 bytes: 1024 or more of them.
    ((1, 4100), (130, 512, 900, 1500, 2048, 2100, 4200)),
    ((7, 601), (500, 2500)),
    # Twice: 256 or more, or rows of up to 32 bytes.
    ((1, 1030), (70, 1000, 2000, 2500, 4000, 5000, 9000)),
    ((7, 201), (600, 1300, 2049, 4097)),
    ((600, 7), (300, 2300)),
    # Rows of up to 16 bytes.
    ((257, 4), (90, 1000, 2000, 3000, 5000, 9000)),
    ((300, 3), (1025, 2049)),
]
SHARES = [(B, L, D) for (B, L), Ds in SHARES for D in Ds]


@pytest.mark.parametrize("B,L,D", SHARES)
@pytest.mark.parametrize("dtype", TYPES)
def test_codes(B, L, D, dtype):
    L = L if dtype == "f32" else 2 * L - L % 2
    i = Inputs(B + L + D, dtype)
    n = lengths_of("ragged", 7, L) if B == 7 else None
    layout = ("dense", "padded", "slice", "swapped")[(D + L) % 4]
    x = poison(i.normal(B, D, L, layout=layout), n)
    codes, scales = gi.quantize_tokens(x, lengths=n)
    check_codes(x, codes, scales, n)


def borders(dtype, D, L, rng):
    """[3, D, L]: numbers half way between two codes and a step of the type to either side, in rows from the smallest
    to the largest."""
    T = TYPES[dtype]
    top = {"f32": 3e38, "bf16": 3e38, "f16": 6e4}[dtype]
    low = {"f32": 1e-44, "bf16": 1e-39, "f16": 1e-7}[dtype]
    most = np.exp(rng.uniform(np.log(low), np.log(top), (3, 1, L)))
    most[0], most[1, :, 0] = rng.uniform(0.5, 2, (1, L)), top
    x = (rng.integers(-127, 127, (3, D, L)) + 0.5) / 127 * most
    x[:, 0] = most[:, 0]
    x = torch.from_numpy(x).to(T)
    words = x.view(torch.int32 if dtype == "f32" else torch.int16)
    step = torch.from_numpy(rng.integers(-2, 3, (3, D, L))).to(words.dtype)
    step[:, 0] = 0
    size = words & (0x7fffffff if dtype == "f32" else 0x7fff)
    x = torch.where(size > 4, words + step, words).view(T)
    return x.clamp(-torch.finfo(T).max, torch.finfo(T).max).cuda()


@pytest.mark.parametrize("D,L", [(700, 1501), (1100, 1400), (300, 400), (2600, 350)])
@pytest.mark.parametrize("dtype", TYPES)
def test_codes_at_the_borders(D, L, dtype):
    L = L if dtype == "f32" else 2 * L
    x = borders(dtype, D, L, np.random.default_rng(D + L))
    check_codes(x, *gi.quantize_tokens(x))


@pytest.mark.parametrize("B,L,D", [(1, 4100, 600), (1, 4100, 4200), (1, 1030, 1000), (1, 1030, 9000), (257, 4, 1000),
                                   (257, 4, 9000)])
@pytest.mark.parametrize("dtype", TYPES)
def test_positions_that_are_no_numbers(B, L, D, dtype):
    L = L if dtype == "f32" else 2 * L
    x = Inputs(B + D, dtype).normal(B, D, L)
    x[0, 7, 3], x[B - 1, :, 2] = float("nan"), 0
    x[B - 1, D - 1, L - 1], x[B // 2, D // 2, 1] = -float("inf"), float("inf")
    codes, scales = gi.quantize_tokens(x)
    check_codes(x, codes, scales)
    assert int(torch.isnan(scales).sum()) == 3 and scales[B - 1, 2] == 0


@pytest.mark.parametrize("case", [   # few positions along a wide layer: k shared by the waves of a work-group
    (1, 4097, 2, 128, None, "dense"), (1, 4200, 9, 640, None, "padded"), (7, 5000, 2, 1152, "ragged", "slice"),
    (16, 70000, 1, 256, None, "dense"), (1, 5000, 17, 128, None, "swapped"), (1, 8300, 30, 1408, None, "dense"),
    (7, 4500, 4, 384, "ragged", "padded"), (2, 515, 150, 256, None, "dense"), (3, 300, 130, 1024, "none", "dense"),
    (7, 400, 60, 2048, "ragged", "slice"), (1, 1000, 500, 384, None, "padded"), (5, 1000, 100, 256, "ragged", "dense"),
    (1, 60, 900, 128, None, "dense"), (60, 8000, 1, 384, None, "dense"), (40, 4200, 1, 128, None, "swapped")], ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_products_of_few_positions(case, dtype):
    s = Product(case, dtype)
    y = s.check()
    assert torch.equal(s.run(), y)


@pytest.mark.parametrize("case", [   # single positions of which some are empty
    (7, 40, 1, 256, "ragged", "dense"), (30, 5000, 1, 128, "ragged", "slice"), (60, 8000, 1, 128, "ragged", "dense"),
    (900, 1500, 1, 384, "ragged", "swapped"), (2100, 1800, 1, 128, "ragged", "dense"),
    (4000, 4200, 1, 256, "ragged", "dense"), (3, 70, 1, 128, "none", "dense")], ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_products_of_single_positions_with_lengths(case, dtype):
    s = Product(case, dtype)
    y = s.check()
    assert torch.equal(s.run(), y)


@pytest.mark.parametrize("dtype", TYPES)
def test_codes_of_single_positions_with_lengths(dtype):
    for layout in ("dense", "slice", "swapped"):
        n = lengths_of("ragged", 7, 1)
        x = poison(Inputs(3, dtype).normal(7, 700, 1, layout=layout), n)
        codes, scales = gi.quantize_tokens(x, lengths=n)
        check_codes(x, codes, scales, n)
