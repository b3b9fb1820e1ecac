"""The example block (examples/recurrent_block.py): its gradients against float64 automatic
differentiation of the same formulas, and the block served in 8 bits."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("recurrent_block",
                                                  os.path.join(ROOT, "examples", "recurrent_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_block(p, r, D):
    """The block in elementary operations on the CPU, position by position."""
    def rms(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w[:, None]

    silu = torch.nn.functional.silu
    xz = torch.matmul(p["in"], rms(r, p["w_pre"]))
    K, L = p["conv"].shape[1], r.shape[2]
    x = torch.nn.functional.pad(xz[:, :D], (K - 1, 0))
    x = silu(sum(p["conv"][:, k, None] * x[:, :, k:k + L] for k in range(K)) + p["conv_bias"][:, None])
    ae = torch.matmul(p["gates"], x)
    a = torch.exp(-torch.exp(p["A_log"])[:, None] * torch.sigmoid(ae[:, :D] + p["r_bias"][:, None]))
    enter = (1 - a * a).sqrt() * torch.sigmoid(ae[:, D:] + p["i_bias"][:, None]) * x
    h, ys = 0, []
    for t in range(L):
        h = a[:, :, t] * h + enter[:, :, t]
        ys.append(h)
    og = torch.matmul(p["out"], torch.stack(ys, -1) * silu(xz[:, D:]))
    o, gate = og.chunk(2, dim=1)
    return rms(r + p["scale"][:, None] * torch.sigmoid(gate) * rms(o, p["w_post"]), p["w_out_norm"])


def test_gradients(example):
    """float32 sums of a few hundred terms through some ten operators: 2^-24 * 10 * sqrt(300) is
    1e-5 of the 2-norm; 1e-4 leaves room for cancellation in the norms' gradients."""
    block = example.Block(channels=16, inner=24)
    g = torch.Generator().manual_seed(3)
    r, gout = (torch.randn(3, 16, 150, generator=g) for _ in range(2))
    out, saved, _ = block.forward(r.cuda())
    grads = block.backward(gout.cuda(), saved)
    p = {k: v.double().cpu().requires_grad_() for k, v in block.p.items()}
    want = plain_block(p, r.double(), 24)
    assert float((out.double().cpu() - want.detach()).norm() / want.detach().norm()) < 1e-5
    for k, v in zip(p, torch.autograd.grad((want * gout.double()).sum(), list(p.values()))):
        assert float((grads[k].double().cpu() - v).norm() / v.norm()) < 1e-4, k


def test_trains(example):
    block = example.Block(channels=32, inner=64)
    before = {k: v.clone() for k, v in block.p.items()}
    losses = example.train(block, steps=3)
    assert len(losses) == 3 and all(v == v for v in losses)
    assert all(torch.isfinite(v).all() and not torch.equal(v, before[k]) for k, v in block.p.items())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_served(example, dtype):
    """Numbers of a normal distribution in rows of 32 or 64 have their largest at some 2.4 of their
    spread, so a code is off by 2.4 / 127 / sqrt(12) = 0.6% of it, and so is a weight's: 0.8% a
    projection, 1.4% for the three, 16-bit roundings 2^-9 at most in some ten places: under 2%, and
    the gates' slopes at most 1; 5% for both figures.  (Tokens and whole sequences differ where the
    last bits move a code over its border.)"""
    apart, off = example.serve(example.Block(channels=32, inner=64), dtype=dtype)
    assert apart < 0.05 and off < 0.05
