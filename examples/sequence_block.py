"""A sequence block made of this library's operators: 1x1 convolutions around linear attention
with a decay for each head, the gated norms, and orthogonalised updates of the convolutions'
weights. Trains it to answer random tokens as another block of the kind does, and then decodes
token by token from the state that a prompt left.

    python examples/sequence_block.py [--steps 100]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import grouped_convolution_amd as G  # noqa: E402


class Block:
    """y = x + scale * rmsnorm(conv_out(gated_norm(attention(conv_in(rmsnorm(x)))))), and rmsnorm(y)."""

    def __init__(self, dim=64, heads=4, kv_heads=2, dk=16, dv=32, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.dk, self.dv = heads, kv_heads, dk, dv
        self.cuts = [heads * dk, kv_heads * dk, kv_heads * dv, heads * dv]  # q, k, v and the gate
        wide = sum(self.cuts)
        self.w_in = (torch.randn(wide, dim, 1, 1, generator=gen) * dim ** -0.5).cuda()
        self.w_out = (torch.randn(dim, heads * dv, 1, 1, generator=gen) * (heads * dv) ** -0.5).cuda()
        self.log_decay = (-0.5 * torch.exp(-4.0 * torch.arange(heads) / heads)).cuda()
        self.w_first, self.w_head = torch.ones(dim).cuda(), torch.ones(dv).cuda()
        self.w_post, self.w_pre = torch.ones(dim).cuda(), torch.ones(dim).cuda()
        self.scale = torch.ones(dim).cuda()

    def parts(self, p):
        """Slices of the first convolution's result [.., wide] as heads."""
        q, k, v, z = p.split(self.cuts, -1)
        return (q.unflatten(-1, (self.heads, self.dk)), k.unflatten(-1, (self.kv_heads, self.dk)),
                v.unflatten(-1, (self.kv_heads, self.dv)), z.unflatten(-1, (self.heads, self.dv)))

    @staticmethod
    def conv(x, w):
        """A 1x1 convolution of tokens [N, T, C], which are a channels-last image one pixel high."""
        return G.gconv_fwd(x.unsqueeze(1), w, None, layout="nhwc").squeeze(1)

    def forward(self, x, state=None):
        n, t, _ = x.shape
        h, _ = G.gconv_normgate_fwd(None, x, w_post=self.w_first)
        p = self.conv(h, self.w_in)
        q, k, v, z = self.parts(p)
        o, state = G.gconv_linattn_fwd(q, k, v, self.log_decay, initial_state=state)
        # a norm for each head's values: every token is a "sequence" of its heads
        rows = lambda a: a.reshape(n * t, self.heads, self.dv) if a.is_contiguous() else a.flatten(0, 1)  # noqa: E731
        g, _ = G.gconv_normgate_fwd(None, rows(o), gate=rows(z), w_post=self.w_head)
        g = g.view(n, t, -1)
        m = self.conv(g, self.w_out)
        y, out = G.gconv_normgate_fwd(x, m, w_post=self.w_post, scale=self.scale, w_pre=self.w_pre)
        self.saved = (x, h, q, k, v, z, o, g, m)
        return y, out, state

    def step(self, x, state):
        """One token [N, dim] of each sequence, on `state` in place."""
        h, _ = G.gconv_normgate_fwd(None, x, w_post=self.w_first)
        q, k, v, z = self.parts(self.conv(h[:, None], self.w_in)[:, 0])
        o = G.gconv_linattn_step(q, k, v, self.log_decay, state)
        g, _ = G.gconv_normgate_fwd(None, o, gate=z, w_post=self.w_head)
        m = self.conv(g.flatten(1)[:, None], self.w_out)[:, 0]
        return G.gconv_normgate_fwd(x, m, w_post=self.w_post, scale=self.scale, w_pre=self.w_pre)

    def backward(self, dy, dout):
        """Gradients of x, the convolutions' weights and the scales, by the last forward pass."""
        x, h, q, k, v, z, o, g, m = self.saved
        n, t, dim = x.shape
        image = lambda a: a.unsqueeze(1)  # noqa: E731
        dx, dm, _, dw_post, dscale, dw_pre = G.gconv_normgate_bwd(dy, dout, x, m, w_post=self.w_post, scale=self.scale, w_pre=self.w_pre)
        dg = G.gconv_bwd_data(image(dm), self.w_out, (n, 1, t, g.shape[2]), layout="nhwc").view(n * t, self.heads, self.dv)
        dw_out = G.gconv_bwd_filter(image(g), image(dm), self.w_out.shape, layout="nhwc")
        _, do, dz, dw_head, _, _ = G.gconv_normgate_bwd(dg, None, None, o.flatten(0, 1), gate=z.flatten(0, 1), w_post=self.w_head)
        dq, dk, dv, _ = G.gconv_linattn_bwd(do.view(o.shape), q, k, v, self.log_decay)
        dp = torch.cat([a.reshape(n, t, -1) for a in (dq, dk, dv, dz)], -1)
        dh = G.gconv_bwd_data(image(dp), self.w_in, (n, 1, t, dim), layout="nhwc").squeeze(1)
        dw_in = G.gconv_bwd_filter(image(h), image(dp), self.w_in.shape, layout="nhwc")
        _, dx_first, _, dw_first, _, _ = G.gconv_normgate_bwd(dh, None, None, x, w_post=self.w_first)
        vectors = {"w_first": dw_first, "w_head": dw_head, "w_post": dw_post, "w_pre": dw_pre, "scale": dscale}
        return dx + dx_first, {"w_in": dw_in, "w_out": dw_out}, vectors

    def update(self, matrices, vectors, rate):
        """Orthogonalised steps of the convolutions' weights, plain ones of the scales."""
        for name, grad in matrices.items():
            w = getattr(self, name)
            w.add_(G.gconv_orthogonalize(grad).float(), alpha=-rate * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
        for name, grad in vectors.items():
            getattr(self, name).add_(grad, alpha=-rate)


def tokens(gen, n, t, dim):
    return torch.randn(n, t, dim, generator=gen).cuda()


def train(block, steps, n=8, t=96, dim=64, rate=0.1, say=print):
    gen = torch.Generator().manual_seed(1)
    teacher = Block(seed=7)
    losses = []
    for i in range(steps):
        x = tokens(gen, n, t, dim)
        _, want, _ = teacher.forward(x)
        _, out, _ = block.forward(x)
        off = out - want
        losses.append(float(off.square().mean()))
        _, matrices, vectors = block.backward(torch.zeros_like(x), off * (2.0 / off.numel()))
        block.update(matrices, vectors, rate * (1 - i / steps))
        if i % 10 == 0 or i == steps - 1:
            say("step %3d  loss %.4f" % (i, losses[-1]))
    return losses


def decode(block, n=3, t=50, more=6, dim=64):
    """How far answers token by token, from a prompt's state, are from those of the whole sequence."""
    x = tokens(torch.Generator().manual_seed(2), n, t + more, dim)
    _, whole, _ = block.forward(x)
    _, _, state = block.forward(x[:, :t].contiguous())
    worst = 0.0
    for i in range(t, t + more):
        _, out = block.step(x[:, i].contiguous(), state)
        worst = max(worst, float((out - whole[:, i]).abs().max()))
    return worst


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=100)
    block = Block()
    train(block, args.parse_args().steps)
    print("decoding differs from the whole sequence by at most %.2g" % decode(block))
