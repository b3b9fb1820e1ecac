"""A gated state space block from the library's operators: trained, then run token by token.

    python examples/mixer_block.py

The block, channel-first [batch, channel, time], in float32:

    u  = rms(r) w_pre                       norm before       block_norm (of the block before)
    x, z = W_in u                           1x1 convolution   forward / backward
    x  = silu(causal convolution of x)      4 taps            causal_conv
    d, B, C = W_x x;  dt = W_dt d           1x1 convolutions  forward / backward
    y  = silu(z) * scan(x, dt, A, B, C)                       state_scan
    o, gate = W_out y                       1x1 convolution   forward / backward
    r' = r + scale * sigmoid(gate) * rms(o) w_post            block_norm

It learns to add to each position the input of two positions before; then the
same weights run over prompts of different lengths in one call and on, one token
a call, from the caches that call leaves.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv2d_backward_amd as gi  # noqa: E402


def plane(L):
    """Height and width of a plane of L positions (a 1x1 convolution sees them one by one)."""
    W = next(w for w in range(min(L, 128), 0, -1) if L % w == 0)
    return L // W, W


def project(x, w):
    """W x for every position: x [B, Ci, L], w [Co, Ci]."""
    B, Ci, L = x.shape
    y = gi.forward(x.contiguous().view(B, Ci, *plane(L)), w.view(*w.shape, 1, 1), stride=1, padding=0)
    return y.view(B, w.shape[0], L)


def project_backward(gy, x, w):
    """The gradients (of x, of w) of ``project``."""
    B, Ci, L = x.shape
    hw = plane(L)
    dx, dw, _ = gi.backward(gy.contiguous().view(B, w.shape[0], *hw), x.contiguous().view(B, Ci, *hw),
                            w.view(*w.shape, 1, 1), stride=1, padding=0)
    return dx.view(B, Ci, L), dw.view(w.shape)


class Block:
    """The block's weights, its passes over whole sequences, and single tokens."""

    def __init__(self, channels, inner, states=16, rank=8, taps=4, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).cuda()

        step = torch.exp(torch.rand(inner, generator=g) * 4.6 - 6.9)  # 1e-3 .. 1e-1
        self.inner, self.states, self.rank = inner, states, rank
        self.p = {
            "w_pre": torch.ones(channels).cuda(), "w_post": torch.ones(channels).cuda(),
            "w_out_norm": torch.ones(channels).cuda(), "scale": torch.ones(channels).cuda(),
            "in": rand(2 * inner, channels, scale=channels ** -0.5),
            "conv": rand(inner, taps, scale=taps ** -0.5), "conv_bias": torch.zeros(inner).cuda(),
            "x": rand(rank + 2 * states, inner, scale=inner ** -0.5),
            "dt": rand(inner, rank, scale=rank ** -0.5),
            "dt_bias": (step + torch.log(-torch.expm1(-step))).cuda(),
            "A_log": torch.log(torch.arange(1., states + 1)).repeat(inner, 1).cuda(),
            "skip": torch.ones(inner).cuda(),
            "out": rand(2 * channels, inner, scale=inner ** -0.5),
        }

    def rows(self, xp):
        """The rows of W_x x: the low-rank step, B and C."""
        R, N = self.rank, self.states
        return xp[:, :R], xp[:, R:R + N], xp[:, R + N:]

    def forward(self, r, lengths=None, want_caches=False):
        """(output of the norm after the block, saved values, caches) from the residual r [B, C, L]."""
        p, s, D = self.p, {"r": r}, self.inner
        # The norm before: block_norm of a block that added nothing.
        _, s["u"] = gi.block_norm(torch.zeros_like(r), r, weight_pre=p["w_pre"], lengths=lengths)
        s["xz"] = project(s["u"], p["in"])
        s["xc"], conv_cache = gi.causal_conv(s["xz"][:, :D], p["conv"], p["conv_bias"], lengths=lengths,
                                             want_state=want_caches)
        s["xp"] = project(s["xc"], p["x"])
        d, B, C = self.rows(s["xp"])
        s["dt"] = project(d, p["dt"])
        s["A"] = -torch.exp(p["A_log"])
        s["y"], scan_cache, s["marks"] = gi.state_scan(
            s["xc"], s["dt"], s["A"], B, C, p["skip"], s["xz"][:, D:], p["dt_bias"], lengths=lengths,
            want_state=want_caches, want_checkpoints=not want_caches)
        s["og"] = project(s["y"], p["out"])
        o, gate = s["og"].chunk(2, dim=1)
        s["r2"], out = gi.block_norm(o, r, p["w_post"], p["w_out_norm"], gate=gate, scale=p["scale"],
                                     lengths=lengths)
        return out, s, (conv_cache, scan_cache)

    def backward(self, gout, s):
        """The gradients of the parameters, given that of the output."""
        p, D, g = self.p, self.inner, {}
        dog, dxz = torch.empty_like(s["og"]), torch.empty_like(s["xz"])
        C = s["r"].shape[1]
        o, gate = s["og"].chunk(2, dim=1)
        n = gi.block_norm_backward(None, gout, o, s["r2"], p["w_post"], p["w_out_norm"], gate=gate,
                                   scale=p["scale"], dy=dog[:, :C], dgate=dog[:, C:])
        g["scale"], g["w_post"], g["w_out_norm"] = n.dscale, n.dweight_post, n.dweight_pre
        dy, g["out"] = project_backward(dog, s["y"], p["out"])
        d, B, Cm = self.rows(s["xp"])
        k = gi.state_scan_backward(dy, s["xc"], s["dt"], s["A"], B, Cm, s["marks"], p["skip"], s["xz"][:, D:],
                                   p["dt_bias"], dz=dxz[:, D:])
        g["skip"], g["dt_bias"], g["A_log"] = k.dD, k.ddt_bias, k.dA * s["A"]
        dd, g["dt"] = project_backward(k.ddt, d, p["dt"])
        dxc, g["x"] = project_backward(torch.cat([dd, k.dB, k.dC], 1), s["xc"], p["x"])
        _, g["conv"], g["conv_bias"] = gi.causal_conv_backward(dxc + k.dx, s["xz"][:, :D], p["conv"],
                                                               p["conv_bias"], dx=dxz[:, :D])
        du, g["in"] = project_backward(dxz, s["u"], p["in"])
        g["w_pre"] = gi.block_norm_backward(None, du, torch.zeros_like(du), s["r"],
                                            weight_pre=p["w_pre"]).dweight_pre
        return g

    def token(self, r, caches, slots=None):
        """One position for every row of r [B, C]: the output; the caches are updated."""
        p, D = self.p, self.inner
        conv_cache, scan_cache = caches
        r = r[..., None]
        _, u = gi.block_norm(torch.zeros_like(r), r, weight_pre=p["w_pre"])
        xz = project(u, p["in"])[..., 0]
        xc = gi.causal_conv_step(xz[:, :D], conv_cache, p["conv"], p["conv_bias"], slots=slots)
        xp = project(xc[..., None], p["x"])
        d, B, C = self.rows(xp)
        dt = project(d, p["dt"])[..., 0]
        y = gi.state_scan_step(xc, dt, -torch.exp(p["A_log"]), B[..., 0], C[..., 0], scan_cache, p["skip"],
                               xz[:, D:], p["dt_bias"], slots=slots)
        o, gate = project(y[..., None], p["out"]).chunk(2, dim=1)
        return gi.block_norm(o, r, p["w_post"], p["w_out_norm"], gate=gate, scale=p["scale"])[1][..., 0]


def train(block, steps=150, batch=8, channels=32, length=96, delay=2, rate=1e-2, seed=1):
    """Learns to add the input of `delay` positions before; the losses."""
    g = torch.Generator().manual_seed(seed)
    moments = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in block.p.items()}
    losses = []
    for step in range(1, steps + 1):
        r = torch.randn(batch, channels, length, generator=g).cuda()
        want = (r + torch.roll(r, delay, dims=2)) * 0.5 ** 0.5
        out, saved, _ = block.forward(r)
        diff = out - want
        diff[:, :, :delay] = 0
        losses.append(float(diff.square().mean()))
        for k, grad in block.backward(diff * (2 / diff.numel()), saved).items():
            m, v = moments[k]
            m.lerp_(grad, 0.1)
            v.lerp_(grad.square(), 0.01)
            block.p[k] -= rate * (m / (1 - 0.9 ** step)) / ((v / (1 - 0.99 ** step)).sqrt() + 1e-8)
    return losses


def generate(block, channels=32, batch=4, length=40, tokens=12, seed=2):
    """Prompts of different lengths in one call, then tokens from the caches: the largest
    difference from one call over the whole sequences."""
    g = torch.Generator().manual_seed(seed)
    r = torch.randn(batch, channels, length + tokens, generator=g).cuda()
    lengths = torch.tensor([length, 1, length // 2, 0][:batch], dtype=torch.int32).cuda()
    _, _, caches = block.forward(r[:, :, :length].contiguous(), lengths=lengths, want_caches=True)
    whole = block.forward(r)[0]
    worst = 0.0
    rows = torch.arange(batch, device="cuda")
    for t in range(tokens):
        at = lengths.long() + t
        out = block.token(r[rows, :, at].contiguous(), caches)
        worst = max(worst, float((out - whole[rows, :, at]).abs().max()))
    return worst


def main():
    block = Block(channels=32, inner=64)
    losses = train(block)
    print("loss %.3f -> %.3f in %d steps" % (losses[0], losses[-1], len(losses)))
    print("tokens from caches against whole sequences: at most %.2g apart" % generate(block))


if __name__ == "__main__":
    main()
