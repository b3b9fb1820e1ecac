"""quantize_tokens, project_int8 and project_int8_step against the oracle.

Codes and scales are decided exactly and have to be equal.  The sums are exact; y has
roundings of the sum as a float, of the scales' product, of the product and of the
addition (u = 2^-24 each), and its own (h): |y - ref| <= h |ref| + 4 u (1 + h) S with S =
|scaled sum| + |bias|.
"""
import numpy as np
import pytest

from oracle import sequence as oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import conv2d_backward_amd as gi  # noqa: E402
from test_gpu_sequence import TYPES, Inputs, check, half, lengths_of, num, poison  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gi.load_library()


def clamped(n, B, L):
    return [L] * B if n is None else n.clamp(0, L).tolist()


def check_codes(x, codes, scales, n=None):
    B, D, L = x.shape
    rows = num(x)[0].transpose(0, 2, 1)
    for b, m in enumerate(clamped(n, B, L)):
        want, want_scales = oracle.int8_codes(rows[b, :m]) if m else (np.zeros((0, codes.shape[2])), np.zeros(0))
        got = codes[b].cpu().numpy()
        assert (got[:m] == want).all(), "batch item %d: %d codes differ" % (b, int((got[:m] != want).sum()))
        assert (got[m:] == 0).all()
        s = scales[b].cpu().numpy()
        assert np.array_equal(s[:m], want_scales, equal_nan=True) and (s[m:] == 0).all()


QUANT = [  # B, D, L, lengths, layout
    (1, 1, 1, None, "dense"), (1, 5, 3, None, "dense"), (2, 128, 8, None, "padded"), (7, 129, 9, "ragged", "dense"),
    (3, 40, 31, "none", "dense"), (2, 300, 33, None, "slice"), (5, 1001, 70, "ragged", "padded"),
    (1, 260, 257, None, "swapped"), (4, 300, 1, None, "dense"), (4, 300, 1, None, "slice"), (7, 2050, 1, "ragged", "swapped"),
    (1, 4100, 40, None, "dense"), (2, 9000, 5, None, "slice"), (1, 2000, 64, None, "padded"),
    (1, 2561, 33, None, "dense"), (3, 4100, 70, "ragged", "padded"), (1, 16384, 40, None, "slice"), (1, 16385, 40, None, "dense"),
    (2, 8000, 100, "none", "swapped"),
]


@pytest.mark.parametrize("case", QUANT, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_codes(case, dtype):
    B, D, L, kind, layout = case
    i = Inputs(B + D + L, dtype)
    n = lengths_of(kind, B, L)
    x = poison(i.normal(B, D, L, layout=layout), n)
    codes, scales = gi.quantize_tokens(x, lengths=n)
    check_codes(x, codes, scales, n)


@pytest.mark.parametrize("case", [
    # Enough positions for every way they are shared out, with channels for every number of rounds kept and beyond.
    (1, 1500, 3000, None, "dense"), (1, 3000, 2500, None, "slice"), (1, 4500, 2100, None, "padded"),
    (1, 8300, 2100, None, "dense"), (7, 600, 620, "ragged", "padded"), (4, 900, 2101, None, "dense"),
    (8, 1100, 1030, None, "dense"), (8, 2100, 1030, None, "swapped"), (8, 4200, 1030, None, "dense")], ids=str)
def test_codes_of_many_positions(case):
    test_codes(case, "bf16")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 40])
def test_codes_at_the_borders(dtype, L):
    """Numbers half way between two codes, just beside that, and rows from the smallest to the largest."""
    i = Inputs(L, dtype)
    D = 700
    top = {"f32": 3e38, "bf16": 3e38, "f16": 6e4}[dtype]
    low = {"f32": 1e-44, "bf16": 1e-39, "f16": 1e-7}[dtype]
    rows = np.exp(i.rng.uniform(np.log(low), np.log(top), (3, 1, L)))
    rows[0], rows[1, :, 0] = i.rng.uniform(0.5, 2, (1, L)), top
    k = i.rng.integers(-127, 127, (3, D, L))
    x = (k + 0.5) / 127 * rows
    x[:, 0] = rows[:, 0]
    x = torch.from_numpy(x).to(i.dtype)
    if dtype == "f32":   # a step of the type to either side
        step = torch.from_numpy(i.rng.integers(-2, 3, (3, D, L)).astype(np.int32))
        step[:, 0] = 0
        v = x.view(torch.int32)
        x = torch.where(v & 0x7fffffff > 4, v + step, v).view(torch.float32)
    x = x.clamp(-torch.finfo(i.dtype).max, torch.finfo(i.dtype).max).cuda()
    check_codes(x, *gi.quantize_tokens(x))


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_that_are_no_numbers(dtype):
    for shape, row in (((4, 300, 1), lambda t, b: t[b, :, 0]), ((1, 300, 40), lambda t, b: t[0, :, b])):
        x = Inputs(3, dtype).normal(*shape)
        row(x, 0)[7], row(x, 1)[299], row(x, 2)[:] = float("nan"), -float("inf"), 0
        codes, scales = gi.quantize_tokens(x)
        check_codes(x, codes, scales)
        w, ws = gi.quantize_weight(Inputs(4, "f32").normal(5, 300))
        y = gi.project_int8(codes, scales, w, ws)
        bad = torch.isnan(y).all(1) if shape[2] == 1 else torch.isnan(y).all(1)
        assert bad.flatten().tolist()[:3] == [True, True, False] and int(torch.isnan(y).sum()) == 10


def test_weights():
    w = Inputs(5, "bf16").normal(70, 301)
    codes, scales = gi.quantize_weight(w)
    want, want_scales = oracle.int8_codes(num(w)[0])
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(scales.cpu().numpy(), want_scales)
    wide = Inputs(6, "f32").normal(70, 400)[:, 17:318]     # a slice of its columns, a transpose
    for v in (wide, wide.t()):
        codes, scales = gi.quantize_weight(v)
        assert np.array_equal(codes.cpu().numpy(), oracle.int8_codes(num(v)[0])[0])


PRODUCT = [  # B, E, L, K, lengths, layout of the result
    (1, 1, 1, 128, None, "dense"), (1, 3, 2, 128, None, "dense"), (2, 33, 31, 256, None, "padded"),
    (7, 64, 9, 384, "ragged", "dense"), (3, 65, 64, 128, "none", "dense"), (1, 100, 257, 640, None, "slice"),
    (5, 130, 75, 256, "ragged", "swapped"), (40, 70, 1, 512, None, "dense"), (3, 257, 300, 128, "ragged", "padded"),
    (1, 1000, 2100, 128, None, "dense"), (2, 2200, 700, 256, "ragged", "dense"), (1, 4000, 3300, 128, None, "slice"),
    (16, 3, 17, 1024, "ragged", "slice"), (33, 515, 1, 1152, None, "swapped"),
]


class Product:
    def __init__(self, case, dtype, bias=True):
        B, E, L, K, kind, layout = case
        i = Inputs(B + E + L + K, dtype)
        self.case, self.i, self.dtype = case, i, i.dtype
        self.codes = torch.from_numpy(i.rng.integers(-127, 128, (B, L, K)).astype(np.int8)).cuda()
        self.w = torch.from_numpy(i.rng.integers(-127, 128, (E, K)).astype(np.int8)).cuda()
        self.scales, self.w_scales = i.params(B, L, low=1e-3, high=2e-3), i.params(E, low=1e-3, high=2e-3)
        self.bias = i.params(E) if bias else None
        self.n = lengths_of(kind, min(B, 7), L)
        if self.n is not None and B > 7:
            self.n = self.n.repeat(-(-B // 7))[:B].contiguous()
        if self.n is not None:   # what lies beyond is not used
            beyond = torch.arange(L, device="cuda") >= self.n.clamp(0, L)[:, None]
            self.scales.masked_fill_(beyond, float("nan"))
        self.out = i.normal(B, E, L, layout=layout) if layout != "dense" else None

    def run(self, **k):
        return gi.project_int8(self.codes, self.scales, self.w, self.w_scales, self.bias, dtype=self.dtype,
                               lengths=self.n, out=self.out, **k)

    def check(self):
        B, E, L, K, _, _ = self.case
        y = self.run()
        ref, S = np.zeros((B, E, L)), np.zeros((B, E, L))
        for b, m in enumerate(clamped(self.n, B, L)):
            if m:
                ref[b, :, :m], S[b, :, :m] = oracle.int8_product(
                    self.codes[b, :m].cpu().numpy(), *num(self.scales[b, :m]), self.w.cpu().numpy(),
                    *num(self.w_scales, self.bias))
        check(y, ref, S, 4, "y")
        return y


@pytest.mark.parametrize("case", PRODUCT, ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_product(case, dtype):
    Product(case, dtype).check()


@pytest.mark.parametrize("case", [
    # Tiles of 256 for every compute unit, and more; 2, 3 and 5 steps of k; items that end inside a tile.
    (1, 3500, 3400, 256, None, "padded"), (1, 5000, 4200, 256, None, "dense"), (7, 6500, 300, 384, "ragged", "dense"),
    (2, 3333, 1900, 640, None, "slice"), (1, 5120, 5120, 384, None, "dense"), (3, 8200, 1000, 256, "none", "dense")], ids=str)
@pytest.mark.parametrize("dtype", TYPES)
def test_product_of_many_tiles(case, dtype):
    s = Product(case, dtype)
    y = s.check()
    assert torch.equal(s.run(), y)


def test_product_without_bias():
    Product((2, 70, 90, 256, None, "dense"), "f32", bias=False).check()


def test_largest_sums():
    """Sums of 65536 products of -128 by -128 and of 127 by 127."""
    for v in (-128, 127):
        codes = torch.full((1, 40, 65536), v, dtype=torch.int8, device="cuda")
        w = torch.full((50, 65536), v, dtype=torch.int8, device="cuda")
        one = torch.ones(50, device="cuda")
        y = gi.project_int8(codes, one[None, :40].contiguous(), w, one)
        assert (y == float(v * v * 65536)).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,E", [(1, 1, 1), (1, 64, 70), (3, 130, 33), (8, 2048, 300), (16, 1000, 515), (17, 300, 64),
                                   (33, 515, 100), (64, 128, 2000), (65, 700, 130), (130, 260, 400), (2, 4100, 1030),
                                   (16, 9000, 20), (300, 260, 2100), (1100, 128, 1500), (2100, 300, 6300),
                                   (500, 64, 3300), (2100, 128, 1800), (40, 130, 8500), (32, 256, 8300)])
def test_step(B, D, E, dtype):
    """One call is the two calls, bit for bit, whatever the strides."""
    i = Inputs(B + D + E, dtype)
    w, ws = gi.quantize_weight(i.normal(E, D, dtype=torch.float32))
    bias = i.params(E)
    x = i.normal(B, D)
    codes, scales = gi.quantize_tokens(x.unsqueeze(2))
    check_codes(x.unsqueeze(2), codes, scales)
    want = gi.project_int8(codes, scales, w, ws, bias, dtype=i.dtype)[..., 0]
    ref, S = oracle.int8_product(codes[:, 0].cpu().numpy(), *num(scales[:, 0]), w.cpu().numpy(), *num(ws, bias))
    check(want, ref.T, S.T, 4, "y")
    assert torch.equal(gi.project_int8_step(x, w, ws, bias), want)
    wide = i.normal(B, 2 * D + 1)
    wide[:, 1::2] = x
    out = torch.full((B, 2 * E + 1), 7.0, dtype=i.dtype, device="cuda")
    got = gi.project_int8_step(wide[:, 1::2], w, ws, bias, out=out[:, 1::2])
    assert torch.equal(got, want) and (out[:, ::2] == 7).all()
    assert torch.equal(gi.project_int8_step(x, w, ws), gi.project_int8(codes, scales, w, ws, dtype=i.dtype)[..., 0])


@pytest.mark.parametrize("B,D,E", [(1, 8192, 5000), (4, 8192, 300), (1, 8150, 9), (3, 10900, 4100), (2, 16384, 4097),
                                   (1, 32768, 600), (1, 32769, 40), (16, 2048, 4099), (5, 6500, 70)])
def test_step_of_few_long_rows(B, D, E):
    """Codes of all channels of a few rows, made inside the product or before it."""
    i = Inputs(B + D + E, "bf16")
    w, ws = gi.quantize_weight(i.normal(E, D))
    x = i.normal(B, D)
    want = gi.project_int8(*gi.quantize_tokens(x.unsqueeze(2)), w, ws, dtype=i.dtype)[..., 0]
    assert torch.equal(gi.project_int8_step(x, w, ws), want)
    wide = i.normal(B, 2 * D + 1)
    wide[:, 1::2] = x
    assert torch.equal(gi.project_int8_step(wide[:, 1::2], w, ws), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [300, 4000])
def test_positions_that_are_no_numbers(D, dtype):
    i = Inputs(6, dtype)
    x = i.normal(1, D, 50)
    x[0, 7, 3], x[0, :, 4], x[0, D - 1, 40] = float("nan"), 0, -float("inf")
    codes, scales = gi.quantize_tokens(x)
    check_codes(x, codes, scales)
    assert torch.isnan(scales[0, [3, 40]]).all() and scales[0, 4] == 0 and torch.isfinite(scales).sum() == 48


def test_step_with_rows_that_are_no_numbers():
    i = Inputs(2, "bf16")
    w, ws = gi.quantize_weight(i.normal(40, 300))
    x = i.normal(9, 300)
    clean = gi.project_int8_step(x, w, ws)
    x[3, 5], x[4], x[7, 299] = float("nan"), 0, float("inf")
    y = gi.project_int8_step(x, w, ws)
    assert torch.isnan(y[[3, 7]]).all() and (y[4] == 0).all()
    rest = [0, 1, 2, 5, 6, 8]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dtype", TYPES)
def test_against_a_convolution(dtype):
    """The library's fp32 1x1 convolution of the numbers that the codes stand for.

    Both sum the same terms; the convolution's bound is 1e-5 of the sum of their magnitudes."""
    i = Inputs(8, dtype)
    B, D, E, L = 2, 200, 90, 48
    x, weight = i.normal(B, D, L), i.normal(E, D, dtype=torch.float32)
    codes, scales = gi.quantize_tokens(x)
    w, ws = gi.quantize_weight(weight)
    y = gi.project_int8(codes, scales, w, ws, dtype=i.dtype)
    xs = (codes[..., :D].float() * scales[..., None]).transpose(1, 2).contiguous()
    wide = w[:, :D].float() * ws[:, None]
    conv = gi.forward(xs.view(B, D, 6, 8), wide.view(E, D, 1, 1), stride=1, padding=0).view(B, E, L)
    S = torch.matmul(wide.abs(), xs.abs())
    assert ((y.float() - conv).abs() <= half(i.dtype) * conv.abs() + 1e-5 * S * (1 + half(i.dtype)) + 1e-6).all()


def test_graph_replays_and_streams():
    i = Inputs(7, "bf16")
    x, w, ws = i.normal(3, 300, 70), *gi.quantize_weight(i.normal(200, 300))

    def everything(**k):
        codes, scales = gi.quantize_tokens(x, **k)
        return [codes, scales, gi.project_int8(codes, scales, w, ws, dtype=torch.bfloat16, **k),
                gi.project_int8_step(x[..., 5], w, ws, **k)]

    want = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    named = everything(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(named, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = everything()
    for k in range(4):
        x.add_(0.25 * k)
        graph.replay()
        want = everything()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("B,D,E,L", [(1, 600, 4096, 3000), (2, 300, 2100, 1000), (3, 1000, 515, 301), (1, 900, 1000, 90),
                                     (900, 128, 1500, 1), (5, 6500, 70, 1), (3000, 300, 4097, 1),
                                     (1, 4096, 300, 90)])
def test_every_size_of_tiles_replays_and_runs_beside_another(B, D, E, L):
    """Captured and replayed, and on two streams at once."""
    i = Inputs(B + D + E, "bf16")
    x, w, ws = i.normal(B, D, L), *gi.quantize_weight(i.normal(E, D))
    other = i.normal(B, D, L)

    def everything(x, **k):
        y = gi.project_int8(*gi.quantize_tokens(x, **k), w, ws, dtype=torch.bfloat16, **k)
        return [y] + ([gi.project_int8_step(x[..., 0], w, ws, **k)] if L == 1 else [])

    want, want_other = everything(x), everything(other)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    for side in sides:
        side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got, got_other = everything(x, stream=sides[0]), everything(other, stream=sides[1])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got + got_other, want + want_other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sides[0]):
        got = everything(x)
    for _ in range(3):
        x.copy_(other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want_other))
        other.mul_(-0.5)
        want_other = everything(other)


@pytest.mark.parametrize("E,L", [(40, 70), (300, 1000), (4096, 1600)])
def test_results_beyond_32_bits(E, L):
    i = Inputs(5, "bf16")
    codes, scales = gi.quantize_tokens(i.normal(2, 300, L))
    w, ws = gi.quantize_weight(i.normal(E, 300))
    want = gi.project_int8(codes, scales, w, ws, dtype=torch.bfloat16)
    far = torch.empty(2 ** 31 + 2 * E * L, dtype=torch.bfloat16, device="cuda")
    out = far.as_strided((2, E, L), (2 ** 31 + 100, L, 1))
    gi.project_int8(codes, scales, w, ws, out=out)
    assert torch.equal(out, want)


def test_offsets_beyond_32_bits():
    """Codes and a result whose far elements are past 2^32 bytes."""
    i = Inputs(4, "f32")
    K, L = 65536, 70000
    w = torch.from_numpy(i.rng.integers(-127, 128, (3, K)).astype(np.int8)).cuda()
    codes = torch.zeros(1, L, K, dtype=torch.int8, device="cuda")
    codes[0, -5:] = torch.from_numpy(i.rng.integers(-127, 128, (5, K)).astype(np.int8)).cuda()
    one = torch.ones(L, device="cuda")
    y = gi.project_int8(codes, one[None], w, one[:3].contiguous())
    near = gi.project_int8(codes[:, -5:].contiguous(), one[None, :5].contiguous(), w, one[:3].contiguous())
    assert torch.equal(y[..., -5:], near) and (y[..., :-5] == 0).all()
    del codes
    far = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    x = i.normal(2, 8, 100, dtype=torch.bfloat16)
    wide = far.as_strided((2, 8, 100), (2 ** 31 + 100, 100, 1))
    wide.copy_(x)
    assert all(torch.equal(p, q) for p, q in zip(gi.quantize_tokens(wide), gi.quantize_tokens(x)))


def test_refusals():
    i = Inputs(1, "bf16")
    x = i.normal(2, 6, 10)
    codes, scales = gi.quantize_tokens(x)
    w, ws = gi.quantize_weight(i.normal(5, 6))
    bad = [
        lambda: gi.quantize_tokens(x[0]), lambda: gi.quantize_tokens(x.double()), lambda: gi.quantize_tokens(None),
        lambda: gi.quantize_tokens(x.cpu()), lambda: gi.quantize_tokens(x, codes=codes[..., :64]),
        lambda: gi.quantize_tokens(x, codes=codes.float()), lambda: gi.quantize_tokens(x.transpose(1, 2)),
        lambda: gi.quantize_weight(x), lambda: gi.quantize_weight(w),
        lambda: gi.project_int8(codes, scales, w, ws, dtype=torch.int8),
        lambda: gi.project_int8(codes, scales, w, ws, dtype=torch.float64),
        lambda: gi.project_int8(codes.float(), scales, w, ws), lambda: gi.project_int8(codes, scales[:1], w, ws),
        lambda: gi.project_int8(codes, scales, w[:, :64], ws), lambda: gi.project_int8(codes, scales, w, ws[:4]),
        lambda: gi.project_int8(codes, scales, w.cpu(), ws), lambda: gi.project_int8(codes, scales, w, ws, ws.half()),
        lambda: gi.project_int8(codes[0], scales, w, ws), lambda: gi.project_int8(None, scales, w, ws),
        lambda: gi.project_int8(codes, scales, w, ws, dtype=torch.float16, out=i.normal(2, 5, 10)),
        lambda: gi.project_int8_step(x, w, ws), lambda: gi.project_int8_step(x[..., 0], w[:, :64], ws),
        lambda: gi.project_int8_step(i.normal(2, 200), w, ws),
    ]
    for k, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was not refused" % k)
    for f in (lambda: gi.quantize_tokens(x[..., :0]),
              lambda: gi.project_int8(codes, scales, w, ws, dtype=torch.bfloat16, out=i.normal(1, 5, 10).expand(2, 5, 10)),
              lambda: gi.project_int8(torch.zeros(2, 10, 64, dtype=torch.int8, device="cuda"), scales,
                                      torch.zeros(5, 64, dtype=torch.int8, device="cuda"), ws)):
        with pytest.raises(gi.Conv2dGiError):
            f()
