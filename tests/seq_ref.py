"""Plain 64-bit definitions (CPU) of the sequence operators, written from their formulas, and the
comparison the tests use: an error bound for each element from the sum of its terms' magnitudes."""
from __future__ import annotations

import torch

F64 = torch.float64


def linattn(q, k, v, g, scale, init=None):
    """Linear attention of one sequence, by its recurrence: q [T, H, dk], k [T, Hk, dk], v [T, Hk, dv],
    g [H], init [H, dk, dv] or None. Returns o, the final state, all in 64 bits."""
    q, k, v, g = q.to(F64), k.to(F64), v.to(F64), g.to(F64)
    T, H, dk = q.shape
    rep = H // k.shape[1]
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    s = torch.zeros(H, dk, v.shape[2], dtype=F64) if init is None else init.to(F64)
    lam = torch.exp(g)[:, None, None]
    o = []
    for t in range(T):
        s = lam * s + k[t, :, :, None] * v[t, :, None, :]
        o.append(scale * (q[t, :, None, :] @ s)[:, 0])
    return (torch.stack(o) if o else torch.zeros(0, H, v.shape[2], dtype=F64)), s


def check_mag(name, got, want, mag, rtol, atol=0.0):
    """|got - want| <= rtol mag + atol, element by element; mag: the sum of the element's terms' magnitudes."""
    got, want, mag = got.detach().cpu().to(F64), want.detach().cpu().to(F64), mag.detach().cpu().to(F64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return 0.0
    assert torch.isfinite(got).all(), "%s: not finite" % name
    ratio = (got - want).abs() / (rtol * mag + atol + 1e-300)
    i = int(ratio.argmax())
    assert ratio.flatten()[i] <= 1, "%s: element %d got %r want %r mag %r: %.3g of the bound" % (
        name, i, got.flatten()[i].item(), want.flatten()[i].item(), mag.flatten()[i].item(), ratio.flatten()[i].item())
    return float(ratio.flatten()[i])


def _act(z, act):
    """act(z), its derivative, and the magnitude of the derivative's terms."""
    s = 1 / (1 + torch.exp(-z))
    if act == "none":
        return z, torch.ones_like(z), torch.ones_like(z)
    if act == "sigmoid":
        return s, s * (1 - s), s * (1 - s)
    return z * s, s + z * s * (1 - s), s + z.abs() * s * (1 - s)


def normgate(x, b, gate, act, w_post, scale, w_pre, eps, dy=None, dh=None):
    """The norms around a block and their gradients in 64 bits, [N, T, D]; {name: (value, magnitude of
    its terms)}, from the formulas (not by autograd)."""
    b = b.to(F64)
    one = torch.ones(b.shape[-1], dtype=F64)
    z = gate.to(F64).expand_as(b) if gate is not None else None
    wp, sc = w_post.to(F64), scale.to(F64) if scale is not None else one
    rb = (b.square().mean(-1, keepdim=True) + eps) ** -0.5
    bn = b * rb
    n = bn * wp
    a, da, da_m = _act(z, act) if z is not None else (torch.ones_like(b),) * 3
    t = sc * a * n
    y = t + (x.to(F64) if x is not None else 0)
    y_m = t.abs() + (x.to(F64).abs() if x is not None else 0)
    out = {"y": (y, y_m)}
    if w_pre is not None:
        wq = w_pre.to(F64)
        ry = (y.square().mean(-1, keepdim=True) + eps) ** -0.5
        yn, yn_m = y * ry, y_m * ry
        out["h"] = (yn * wq, yn_m * wq.abs())
    if dy is None:
        return out
    d = dy.to(F64)
    d_m = d.abs()
    if w_pre is not None:
        e = dh.to(F64) * wq
        d = d + ry * (e - yn * (e * yn).mean(-1, keepdim=True))
        d_m = d_m + ry * (e.abs() + yn_m * (e.abs() * yn_m).mean(-1, keepdim=True))
        out["dw_pre"] = ((dh.to(F64) * yn).sum((0, 1)), (dh.to(F64).abs() * yn_m).sum((0, 1)))
    if x is not None:
        out["dx"] = (d, d_m)
    f, f_m = d * sc * a * wp, d_m * (sc * a * wp).abs()
    out["db"] = (rb * (f - bn * (f * bn).mean(-1, keepdim=True)), rb * (f_m + bn.abs() * (f_m * bn.abs()).mean(-1, keepdim=True)))
    if z is not None:
        g, g_m = d * sc * n * da, d_m * (sc * n).abs() * da_m
        if gate.shape != b.shape:
            g, g_m = g.sum(1, keepdim=True), g_m.sum(1, keepdim=True)
        out["dgate"] = (g, g_m)
    out["dw_post"] = ((d * sc * a * bn).sum((0, 1)), (d_m * (sc * a * bn).abs()).sum((0, 1)))
    if scale is not None:
        out["dscale"] = ((d * a * n).sum((0, 1)), (d_m * (a * n).abs()).sum((0, 1)))
    return out


def orthogonalize(u, groups, steps, eps):
    """Newton-Schulz rounds of each group's matrix, scaled to norm 1, in 64 bits; u [K, D]."""
    a, b, c = 3.4445, -4.7750, 2.0315
    out = []
    for x in u.to(F64).chunk(groups):
        tall = x.shape[0] > x.shape[1]
        x = x.T if tall else x
        x = x / (x.square().sum().sqrt() + eps)
        for _ in range(steps):
            g = x @ x.T
            x = a * x + (b * g + c * (g @ g)) @ x
        out.append(x.T if tall else x)
    return torch.cat(out)
