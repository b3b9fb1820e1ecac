"""A gated recurrent block from the library's operators: trained in float32, then served in 8 bits.

    python examples/recurrent_block.py

The block, channel-first [batch, channel, time]:

    u  = rms(r) w_pre                       norm before       block_norm (of the block before)
    x, z = W_in u                           1x1 convolution   forward / backward
    x  = silu(causal convolution of x)      4 taps            causal_conv
    a, e = W_gates x                        1x1 convolution   forward / backward
    y  = silu(z) * recurrence(x, a, e, A)                     gated_scan
    o, gate = W_out y                       1x1 convolution   forward / backward
    r' = r + scale * sigmoid(gate) * rms(o) w_post            block_norm

It learns to add to each position the input of two positions before.  Served, its three
convolutions are products in 8-bit integers (quantize_tokens, project_int8): prompts of
different lengths in one call, then one token a call from the caches which that call leaves.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import conv2d_backward_amd as gi  # noqa: E402
from mixer_block import project, project_backward, train  # noqa: E402


class Block:
    """The block's weights and its passes over whole sequences."""

    def __init__(self, channels, inner, taps=4, seed=0):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape, scale):
            return (torch.randn(*shape, generator=g) * scale).cuda()

        self.inner = inner
        self.p = {
            "w_pre": torch.ones(channels).cuda(), "w_post": torch.ones(channels).cuda(),
            "w_out_norm": torch.ones(channels).cuda(), "scale": torch.ones(channels).cuda(),
            "in": rand(2 * inner, channels, scale=channels ** -0.5),
            "conv": rand(inner, taps, scale=taps ** -0.5), "conv_bias": torch.zeros(inner).cuda(),
            "gates": rand(2 * inner, inner, scale=inner ** -0.5),
            "r_bias": torch.zeros(inner).cuda(), "i_bias": torch.zeros(inner).cuda(),
            # Decays between 0.2 and 0.999 a position at an open gate.
            "A_log": torch.log(-torch.log(0.2 + 0.799 * torch.rand(inner, generator=g))).cuda(),
            "out": rand(2 * channels, inner, scale=inner ** -0.5),
        }

    def forward(self, r):
        """(output of the norm after the block, saved values, no caches) from the residual r [B, C, L]."""
        p, s, D = self.p, {"r": r}, self.inner
        _, s["u"] = gi.block_norm(torch.zeros_like(r), r, weight_pre=p["w_pre"])
        s["xz"] = project(s["u"], p["in"])
        s["xc"], _ = gi.causal_conv(s["xz"][:, :D], p["conv"], p["conv_bias"])
        s["ae"] = project(s["xc"], p["gates"])
        s["A"] = -torch.exp(p["A_log"])
        s["y"], _, s["marks"] = gi.gated_scan(s["xc"], s["ae"][:, :D], s["ae"][:, D:], s["A"], s["xz"][:, D:],
                                              p["r_bias"], p["i_bias"], want_checkpoints=True)
        s["og"] = project(s["y"], p["out"])
        o, gate = s["og"].chunk(2, dim=1)
        s["r2"], out = gi.block_norm(o, r, p["w_post"], p["w_out_norm"], gate=gate, scale=p["scale"])
        return out, s, None

    def backward(self, gout, s):
        """The gradients of the parameters, given that of the output."""
        p, D, g = self.p, self.inner, {}
        dog, dxz, dae = (torch.empty_like(s[k]) for k in ("og", "xz", "ae"))
        C = s["r"].shape[1]
        o, gate = s["og"].chunk(2, dim=1)
        n = gi.block_norm_backward(None, gout, o, s["r2"], p["w_post"], p["w_out_norm"], gate=gate,
                                   scale=p["scale"], dy=dog[:, :C], dgate=dog[:, C:])
        g["scale"], g["w_post"], g["w_out_norm"] = n.dscale, n.dweight_post, n.dweight_pre
        dy, g["out"] = project_backward(dog, s["y"], p["out"])
        k = gi.gated_scan_backward(dy, s["xc"], s["ae"][:, :D], s["ae"][:, D:], s["A"], s["marks"], s["xz"][:, D:],
                                   p["r_bias"], p["i_bias"], dr=dae[:, :D], di=dae[:, D:], dz=dxz[:, D:])
        g["r_bias"], g["i_bias"], g["A_log"] = k.dr_bias, k.di_bias, k.dA * s["A"]
        dxc, g["gates"] = project_backward(dae, s["xc"], p["gates"])
        _, g["conv"], g["conv_bias"] = gi.causal_conv_backward(dxc + k.dx, s["xz"][:, :D], p["conv"],
                                                               p["conv_bias"], dx=dxz[:, :D])
        du, g["in"] = project_backward(dxz, s["u"], p["in"])
        g["w_pre"] = gi.block_norm_backward(None, du, torch.zeros_like(du), s["r"],
                                            weight_pre=p["w_pre"]).dweight_pre
        return g


class Served:
    """A block with its projections in 8 bits, for prompts and single tokens of a 16-bit type."""

    def __init__(self, block, dtype=torch.bfloat16):
        self.p, self.inner, self.dtype = block.p, block.inner, dtype
        self.w = {k: gi.quantize_weight(block.p[k]) for k in ("in", "gates", "out")}
        self.A = -torch.exp(block.p["A_log"])

    def project(self, x, name, lengths):
        codes, scales = gi.quantize_tokens(x, lengths=lengths)
        return gi.project_int8(codes, scales, *self.w[name], dtype=self.dtype, lengths=lengths)

    def prompt(self, r, lengths=None):
        """(output, caches) of whole sequences r [B, C, L] float32."""
        p, D = self.p, self.inner
        _, u = gi.block_norm(torch.zeros_like(r, dtype=self.dtype), r, weight_pre=p["w_pre"], lengths=lengths)
        xz = self.project(u, "in", lengths)
        x, conv_cache = gi.causal_conv(xz[:, :D], p["conv"], p["conv_bias"], lengths=lengths, want_state=True)
        ae = self.project(x, "gates", lengths)
        y, scan_cache, _ = gi.gated_scan(x, ae[:, :D], ae[:, D:], self.A, xz[:, D:], p["r_bias"], p["i_bias"],
                                         lengths=lengths, want_state=True)
        o, gate = self.project(y, "out", lengths).chunk(2, dim=1)
        out = gi.block_norm(o, r, p["w_post"], p["w_out_norm"], gate=gate, scale=p["scale"], lengths=lengths)[1]
        return out, (conv_cache, scan_cache)

    def token(self, r, caches, slots=None):
        """One position for every row of r [B, C]: the output; the caches are updated."""
        p, D = self.p, self.inner
        conv_cache, scan_cache = caches
        r = r[..., None]
        _, u = gi.block_norm(torch.zeros_like(r, dtype=self.dtype), r, weight_pre=p["w_pre"])
        xz = gi.project_int8_step(u[..., 0], *self.w["in"])
        x = gi.causal_conv_step(xz[:, :D], conv_cache, p["conv"], p["conv_bias"], slots=slots)
        ae = gi.project_int8_step(x, *self.w["gates"])
        y = gi.gated_scan_step(x, ae[:, :D], ae[:, D:], self.A, scan_cache, xz[:, D:], p["r_bias"], p["i_bias"],
                               slots=slots)
        o, gate = gi.project_int8_step(y, *self.w["out"])[..., None].chunk(2, dim=1)
        return gi.block_norm(o, r, p["w_post"], p["w_out_norm"], gate=gate, scale=p["scale"])[1][..., 0]


def serve(block, channels=32, batch=4, length=40, tokens=12, seed=2, dtype=torch.bfloat16):
    """Prompts of different lengths in one call, then tokens from the caches: how far that is, relative
    to its 2-norm, from one call over the whole sequences, and that call from the float32 block."""
    g = torch.Generator().manual_seed(seed)
    r = torch.randn(batch, channels, length + tokens, generator=g).cuda()
    served = Served(block, dtype)
    lengths = torch.tensor([length, 1, length // 2, 0][:batch], dtype=torch.int32).cuda()
    _, caches = served.prompt(r[:, :, :length].contiguous(), lengths)
    whole = served.prompt(r)[0].float()
    rows = torch.arange(batch, device="cuda")
    out, want = [], []
    for t in range(tokens):
        at = lengths.long() + t
        out.append(served.token(r[rows, :, at].contiguous(), caches).float())
        want.append(whole[rows, :, at])
    out, want, exact = torch.stack(out), torch.stack(want), block.forward(r)[0]
    return float((out - want).norm() / want.norm()), float((whole - exact).norm() / exact.norm())


def main():
    block = Block(channels=32, inner=64)
    losses = train(block)
    print("loss %.3f -> %.3f in %d steps" % (losses[0], losses[-1], len(losses)))
    print("8 bits: tokens from caches against whole sequences %.2g, those against float32 %.2g" % serve(block))


if __name__ == "__main__":
    main()
