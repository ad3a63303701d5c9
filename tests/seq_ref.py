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
