"""A token model made of this library's operators: an embedding, blocks of a 1x1 convolution, a short
causal convolution, a selective scan and a second 1x1 convolution with the norms around them, and the
cross entropy of the next token against the vocabulary. Trains it on repeating texts, with its own
gradients and orthogonalised updates of the convolutions, and then decodes token by token.

    python examples/token_model.py [--steps 60]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import grouped_convolution_amd as G  # noqa: E402


def conv(x, w):
    """A 1x1 convolution of tokens [N, T, C], which are a channels-last image one pixel high."""
    return G.gconv_fwd(x.unsqueeze(1).contiguous(), w[:, :, None, None], None, layout="nhwc").squeeze(1)


def conv_bwd(dy, x, w):
    """Gradients of conv's input and weights."""
    n, t, c = x.shape
    dy, x = dy.unsqueeze(1).contiguous(), x.unsqueeze(1).contiguous()
    dx = G.gconv_bwd_data(dy, w[:, :, None, None], (n, 1, t, c), layout="nhwc").squeeze(1)
    return dx, G.gconv_bwd_filter(x, dy, tuple(w.shape) + (1, 1), layout="nhwc")[:, :, 0, 0]


class Model:
    """Parameters by name in `p`; a block's names end in its number."""

    def __init__(self, vocab=61, dim=32, inner=64, states=8, groups=2, taps=4, blocks=2, seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.vocab, self.dim, self.inner, self.states, self.groups, self.taps, self.blocks = vocab, dim, inner, states, groups, taps, blocks
        n = lambda *s, std: torch.randn(*s, generator=gen) * std  # noqa: E731
        p = {"table": n(vocab, dim, std=1.0), "head": n(vocab, dim, std=dim ** -0.5), "first": torch.ones(dim)}
        for i in range(blocks):
            p["w_in%d" % i] = n(2 * inner, dim, std=dim ** -0.5)
            p["taps%d" % i] = n(inner, taps, std=taps ** -0.5)
            p["bias%d" % i] = torch.zeros(inner)
            p["w_scan%d" % i] = n(inner + 2 * groups * states, inner, std=inner ** -0.5)
            p["a%d" % i] = -torch.arange(1.0, states + 1).repeat(inner, 1)
            p["skip%d" % i] = torch.ones(inner)
            p["dt_bias%d" % i] = torch.log(torch.expm1(torch.exp(torch.empty(inner).uniform_(-6.0, -2.0, generator=gen))))
            p["w_out%d" % i] = n(dim, inner, std=inner ** -0.5)
            p["post%d" % i], p["pre%d" % i] = torch.ones(dim), torch.ones(dim)
        self.p = {k: v.cuda() for k, v in p.items()}

    def cuts(self, s):
        """Slices of what the scan's projection gives: its steps, and inputs and outputs of the states."""
        gs = self.groups * self.states
        dt, b, c = s.split([self.inner, gs, gs], -1)
        heads = lambda v: v.unflatten(-1, (self.groups, self.states))  # noqa: E731
        return dt, heads(b), heads(c)

    def forward(self, ids, state=None):
        """h of tokens ids [N, T], going on from `state` (None: a text's start), and the state after them."""
        p = self.p
        x = G.gconv_embed_fwd(p["table"], ids)
        h, _ = G.gconv_normgate_fwd(None, x, w_post=p["first"])
        self.saved, after = [(ids, x)], []
        for i in range(self.blocks):
            q = lambda k: p["%s%d" % (k, i)]  # noqa: E731
            held = state[i] if state is not None else (None, None)
            xz = conv(h, q("w_in"))
            xi, z = xz.split(self.inner, -1)
            u, left = G.gconv_shortconv_fwd(xi, q("taps"), q("bias"), initial_state=held[0])
            s = conv(u, q("w_scan"))
            dt, b, c = self.cuts(s)
            y, scanned = G.gconv_scan_fwd(u, dt, q("a"), b, c, skip=q("skip"), gate=z, dt_bias=q("dt_bias"), initial_state=held[1])
            m = conv(y, q("w_out"))
            out, h2 = G.gconv_normgate_fwd(x, m, w_post=q("post"), w_pre=q("pre"))
            self.saved.append((h, x, xz, u, s, y, m))
            after.append((left, scanned))
            x, h = out, h2
        return h, after

    def loss(self, ids, targets, state=None):
        h, after = self.forward(ids, state)
        loss, lse = G.gconv_xent_fwd(h, self.p["head"], targets)
        self.last = (h, targets, lse)
        return loss, after

    def backward(self, dloss):
        """Gradients of all parameters for dloss of the last loss (from a text's start)."""
        p, g = self.p, {}
        h, targets, lse = self.last
        dh, g["head"] = G.gconv_xent_bwd(dloss, h, p["head"], targets, lse)
        dx = torch.zeros_like(dh)
        for i in reversed(range(self.blocks)):
            q = lambda k: p["%s%d" % (k, i)]  # noqa: E731
            put = lambda k, v: g.__setitem__("%s%d" % (k, i), v)  # noqa: E731
            h_in, x, xz, u, s, y, m = self.saved[i + 1]
            xi, z = xz.split(self.inner, -1)
            dx, dm, _, dpost, _, dpre = G.gconv_normgate_bwd(dx, dh, x, m, w_post=q("post"), w_pre=q("pre"))
            put("post", dpost)
            put("pre", dpre)
            dy, dw = conv_bwd(dm, y, q("w_out"))
            put("w_out", dw)
            dt, b, c = self.cuts(s)
            du, ddt, da, db, dc, dskip, dz, dbias, _ = G.gconv_scan_bwd(dy, u, dt, q("a"), b, c, skip=q("skip"), gate=z, dt_bias=q("dt_bias"))
            for k, v in (("a", da), ("skip", dskip), ("dt_bias", dbias)):
                put(k, v)
            ds = torch.cat([ddt, db.flatten(-2), dc.flatten(-2)], -1)
            du2, dw = conv_bwd(ds, u, q("w_scan"))
            put("w_scan", dw)
            dxi, dtaps, db_, _ = G.gconv_shortconv_bwd(du + du2, xi, q("taps"), q("bias"))
            put("taps", dtaps)
            put("bias", db_)
            dh, dw = conv_bwd(torch.cat([dxi, dz], -1), h_in, q("w_in"))
            put("w_in", dw)
        ids, x = self.saved[0]
        _, dx0, _, g["first"], _, _ = G.gconv_normgate_bwd(dh, None, None, x, w_post=p["first"])
        g["table"] = G.gconv_embed_bwd(dx + dx0, ids, self.vocab)
        return g

    def step(self, ids, state, slots):
        """Logits' argument h of one token of each sequence, on the pools of states in place."""
        p = self.p
        x = G.gconv_embed_fwd(p["table"], ids)
        h, _ = G.gconv_normgate_fwd(None, x, w_post=p["first"])
        for i in range(self.blocks):
            q = lambda k: p["%s%d" % (k, i)]  # noqa: E731
            left, scanned = state[i]
            xi, z = conv(h[:, None], q("w_in"))[:, 0].split(self.inner, -1)
            u = G.gconv_shortconv_step(xi, q("taps"), left, q("bias"), slots=slots)
            dt, b, c = self.cuts(conv(u[:, None], q("w_scan"))[:, 0])
            y = G.gconv_scan_step(u, dt, q("a"), b, c, scanned, skip=q("skip"), gate=z, dt_bias=q("dt_bias"), slots=slots)
            x, h = G.gconv_normgate_fwd(x, conv(y[:, None], q("w_out"))[:, 0], w_post=q("post"), w_pre=q("pre"))
        return h

    def update(self, grads, rate):
        """Orthogonalised steps of the convolutions' weights, plain ones of the rest."""
        for name, g in grads.items():
            w = self.p[name]
            if name.startswith("w_"):
                w.add_(G.gconv_orthogonalize(g.contiguous()).float(), alpha=-rate * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
            else:
                w.add_(g, alpha=-rate * (20 if name in ("table", "head") else 1))


def texts(gen, n, t, vocab):
    """Texts that repeat a few random tokens: what comes next can be told from what came before."""
    period = torch.randint(0, vocab, (n, 7), generator=gen)
    return period.repeat(1, t // 7 + 2)[:, :t + 1].cuda()


def train(model, steps, n=8, t=70, rate=0.05, say=print):
    gen = torch.Generator().manual_seed(1)
    for i in range(steps):
        ids = texts(gen, n, t, model.vocab)
        targets = ids[:, 1:].clone()
        targets[:, :7] = -1  # nothing tells the first of them
        loss, _ = model.loss(ids[:, :-1].contiguous(), targets)
        count = int((targets >= 0).sum())
        if i % 10 == 0 or i == steps - 1:
            say("step %3d  loss %.4f" % (i, float(loss.sum()) / count))
        model.update(model.backward(torch.full_like(loss, 1.0 / count)), rate * (1 - i / steps))


def decode(model, n=3, t=40, more=6):
    """How far h token by token, from a prompt's state in a pool, is from h of the whole text."""
    ids = texts(torch.Generator().manual_seed(2), n, t + more, model.vocab)[:, :t + more].contiguous()
    whole, _ = model.forward(ids)
    _, state = model.forward(ids[:, :t].contiguous())
    slots = torch.tensor([4, 0, 3], dtype=torch.int32, device="cuda")
    pools = []
    for left, scanned in state:
        pool = [v.new_zeros((6,) + v.shape[1:]) for v in (left, scanned)]
        for to, v in zip(pool, (left, scanned)):
            to[slots.long()] = v
        pools.append(pool)
    return max(float((model.step(ids[:, i].contiguous(), pools, slots) - whole[:, i]).abs().max()) for i in range(t, t + more))


if __name__ == "__main__":
    args = argparse.ArgumentParser()
    args.add_argument("--steps", type=int, default=60)
    model = Model()
    train(model, args.parse_args().steps)
    print("decoding differs from the whole text by at most %.2g" % decode(model))
