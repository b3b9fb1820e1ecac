"""The example block (examples/mixer_block.py): its gradients against float64 automatic
differentiation of the same formulas, training, and tokens against whole sequences."""
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
    spec = importlib.util.spec_from_file_location("mixer_block",
                                                  os.path.join(ROOT, "examples", "mixer_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_block(p, r, D, R, N):
    """The block in elementary operations on the CPU, position by position."""
    def rms(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w[:, None]

    silu = torch.nn.functional.silu
    xz = torch.matmul(p["in"], rms(r, p["w_pre"]))
    K, L = p["conv"].shape[1], r.shape[2]
    x = torch.nn.functional.pad(xz[:, :D], (K - 1, 0))
    x = silu(sum(p["conv"][:, k, None] * x[:, :, k:k + L] for k in range(K)) + p["conv_bias"][:, None])
    xp = torch.matmul(p["x"], x)
    s = torch.nn.functional.softplus(torch.matmul(p["dt"], xp[:, :R]) + p["dt_bias"][:, None])
    A, h, ys = -torch.exp(p["A_log"]), 0, []
    for t in range(L):
        h = torch.exp(s[:, :, t, None] * A) * h + (s * x)[:, :, t, None] * xp[:, None, R:R + N, t]
        ys.append((h * xp[:, None, R + N:, t]).sum(-1) + p["skip"] * x[:, :, t])
    og = torch.matmul(p["out"], torch.stack(ys, -1) * silu(xz[:, D:]))
    o, gate = og.chunk(2, dim=1)
    return rms(r + p["scale"][:, None] * torch.sigmoid(gate) * rms(o, p["w_post"]), p["w_out_norm"])


def test_gradients(example):
    """float32 sums of a few hundred terms through some ten operators: 2^-24 * 10 * sqrt(300) is
    1e-5 of the 2-norm; 1e-4 leaves room for cancellation in the norms' gradients."""
    block = example.Block(channels=16, inner=24, states=8, rank=4)
    g = torch.Generator().manual_seed(3)
    r, gout = (torch.randn(3, 16, 150, generator=g) for _ in range(2))
    out, saved, _ = block.forward(r.cuda())
    grads = block.backward(gout.cuda(), saved)
    p = {k: v.double().cpu().requires_grad_() for k, v in block.p.items()}
    want = plain_block(p, r.double(), 24, 4, 8)
    assert float((out.double().cpu() - want.detach()).norm() / want.detach().norm()) < 1e-5
    for k, v in zip(p, torch.autograd.grad((want * gout.double()).sum(), list(p.values()))):
        assert float((grads[k].double().cpu() - v).norm() / v.norm()) < 1e-4, k


def test_trains_and_generates(example):
    block = example.Block(channels=32, inner=64)
    losses = example.train(block, steps=80)
    assert losses[-1] < 0.5 * losses[0]
    assert example.generate(block) < 1e-4
