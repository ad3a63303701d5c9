"""The token operators run together, as the example uses them: gradients of every parameter against those of
the same model written out in 64 bits, a prompt taken in two parts, and decoding."""
from __future__ import annotations

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import token_model as M  # noqa: E402


def norm(v, w):
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w


def plain(m, p, ids, targets):
    """The model's losses in 64 bits (CPU)."""
    x = p["table"][ids]
    h = norm(x, p["first"])
    for i in range(m.blocks):
        q = lambda k: p["%s%d" % (k, i)]  # noqa: E731
        xi, z = (h @ q("w_in").T).split(m.inner, -1)
        pad = torch.cat([xi.new_zeros(xi.shape[0], m.taps - 1, m.inner), xi], 1)
        u = torch.nn.functional.silu(q("bias") + sum(pad[:, j:j + xi.shape[1]] * q("taps")[:, j] for j in range(m.taps)))
        dt, b, c = m.cuts(u @ q("w_scan").T)
        dt = torch.nn.functional.softplus(dt + q("dt_bias"), threshold=100.0)
        b, c = (v.repeat_interleave(m.inner // m.groups, 2) for v in (b, c))
        s, y = x.new_zeros(x.shape[0], m.inner, m.states), []
        for t in range(x.shape[1]):
            s = torch.exp(dt[:, t, :, None] * q("a")) * s + (dt[:, t] * u[:, t])[..., None] * b[:, t]
            y.append((s * c[:, t]).sum(-1) + q("skip") * u[:, t])
        y = torch.stack(y, 1) * torch.nn.functional.silu(z)
        x = x + norm(y @ q("w_out").T, q("post"))
        h = norm(x, q("pre"))
    z = h @ p["head"].T
    at = targets.clamp(min=0)
    loss = torch.logsumexp(z, -1) - z.gather(-1, at[..., None])[..., 0]
    return torch.where(targets >= 0, loss, 0.0)


def test_gradients_of_the_whole():
    m = M.Model()
    ids = M.texts(torch.Generator().manual_seed(4), 3, 41, m.vocab)
    targets = ids[:, 1:].clone()
    targets[:, :5] = -1
    ids = ids[:, :-1].contiguous()
    loss, _ = m.loss(ids, targets)
    weight = torch.rand(loss.shape, generator=torch.Generator().manual_seed(1))
    got = m.backward(weight.cuda())
    p = {k: v.cpu().double().requires_grad_() for k, v in m.p.items()}
    want = plain(m, p, ids.cpu(), targets.cpu())
    grads = dict(zip(p, torch.autograd.grad((want * weight.double()).sum(), list(p.values()))))
    # float32 throughout: some 10 operators one after another, forward and back, each off by a few times 2^-24 of
    # sums of up to 123 x 64 terms, 2^-24 sqrt(8000) = 5e-6 at worst each
    assert (loss.cpu().double() - want).abs().max() <= 1e-4 * want.abs().max()
    assert set(got) == set(grads)
    for name, g in grads.items():
        off = float((got[name].cpu().double() - g).norm() / g.norm())
        assert off <= 1e-4, (name, off)


def test_a_text_in_two_parts():
    """The state after the first part carries on: the second's losses are those within the whole."""
    m = M.Model(seed=3)
    ids = M.texts(torch.Generator().manual_seed(5), 4, 60, m.vocab)
    whole, end = m.loss(ids[:, :-1].contiguous(), ids[:, 1:].contiguous())
    _, state = m.loss(ids[:, :23].contiguous(), ids[:, 1:24].contiguous())
    rest, end2 = m.loss(ids[:, 23:-1].contiguous(), ids[:, 24:].contiguous(), state)
    assert (rest - whole[:, 23:]).abs().max() <= 1e-4 * whole.abs().max()
    for (a, b), (c, d) in zip(end, end2):
        assert (a - c).abs().max() <= 1e-4 * a.abs().max() and (b - d).abs().max() <= 1e-4 * b.abs().max()


def test_training_runs_and_decoding_goes_on_as_the_whole():
    m = M.Model(seed=1)
    said = []
    M.train(m, 12, say=said.append)
    assert said and all(torch.isfinite(v).all() for v in m.p.values())
    # h is a norm's output, of size 1
    assert M.decode(m) <= 1e-4
