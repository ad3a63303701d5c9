"""Plain 64-bit definitions (CPU) of the token operators, written from their formulas, each value with a
bound on a float32 implementation's error, and the comparison the tests use.

U is half a float32 step. A bound is derived along with the value: every operation adds its own
rounding (U times the magnitude of its result; a hardware exponential, logarithm or reciprocal two of
them, an exponential also its argument's rounding) to what its operands bring. The sum of n terms adds
n U of the terms' magnitudes, whatever its order."""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    """A rounding to dtype, relative to the value."""
    return torch.finfo(dtype).eps / 2


def check(name, got, want, bound, dtype=None):
    """|got - want| <= bound + a rounding to got's type, element by element (and a rounding of values near 0)."""
    dtype = got.dtype
    got, want, bound = got.detach().cpu().to(F64), want.detach().cpu().to(F64), bound.detach().cpu().to(F64)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.numel() == 0:
        return
    assert torch.isfinite(got).all(), "%s: not finite" % name
    room = bound + half_step(dtype) * (want.abs() + bound) + 1e-37
    ratio = (got - want).abs() / room
    i = int(ratio.argmax())
    assert ratio.flatten()[i] <= 1, "%s: element %d got %r want %r room %r: %.3g of the bound" % (
        name, i, got.flatten()[i].item(), want.flatten()[i].item(), room.flatten()[i].item(), ratio.flatten()[i].item())


def _act(p, ep, act):
    """act(p) and act'(p), with bounds for an error ep of p. |act''| is at most 0.5."""
    s = torch.sigmoid(p)
    es = s * (1 - s) * (4 * p.abs() + 8) * U + 4 * U * s
    if act == "none":
        return p, ep, torch.ones_like(p), torch.zeros_like(p)
    if act == "sigmoid":
        return s, ep + es, s * (1 - s), ep + 2 * es + 4 * U * s
    d = s * (1 + p * (1 - s))
    return p * s, 1.1 * ep + p.abs() * es + 2 * U * (p * s).abs(), d, 0.5 * ep + es * (1 + 2 * p.abs()) + 4 * U * s * (1 + p.abs())


def shortconv(x, w, bias, act, init=None, dy=None, dfinal=None):
    """One sequence: x, dy [T, D], w [D, K], init, dfinal [K - 1, D]. {name: (value, bound)}."""
    x, w = x.to(F64), w.to(F64)
    T, D = x.shape
    K = w.shape[1]
    b = bias.to(F64) if bias is not None else torch.zeros(D, dtype=F64)
    seq = torch.cat([init.to(F64) if init is not None else torch.zeros(K - 1, D, dtype=F64), x])
    p = b + sum(seq[j:j + T] * w[:, j] for j in range(K))
    mag = b.abs() + sum((seq[j:j + T] * w[:, j]).abs() for j in range(K))
    y, ey, d, ed = _act(p, (K + 1) * U * mag, act)
    out = {"y": (y, ey), "final": (seq[T:], torch.zeros_like(seq[T:]))}
    if dy is None:
        return out
    dy = dy.to(F64)
    dp, edp = dy * d, dy.abs() * ed + U * (dy * d).abs()
    ds, eds, mds = (torch.zeros_like(seq) for _ in range(3))
    dw, edw = [], []
    n = T + 300  # a sum over the tokens and over the kernels' parts
    for j in range(K):
        ds[j:j + T] += dp * w[:, j]
        mds[j:j + T] += (dp * w[:, j]).abs()
        eds[j:j + T] += edp * w[:, j].abs()
        dw.append((dp * seq[j:j + T]).sum(0))
        edw.append((edp * seq[j:j + T].abs() + n * U * (dp * seq[j:j + T]).abs()).sum(0))
    if dfinal is not None:
        ds[T:] += dfinal.to(F64)
        mds[T:] += dfinal.to(F64).abs()
    eds = eds + (K + 2) * U * mds
    out.update(dx=(ds[K - 1:], eds[K - 1:]), dinit=(ds[:K - 1], eds[:K - 1]), dw=(torch.stack(dw, 1), torch.stack(edw, 1)),
               dbias=(dp.sum(0), (edp + n * U * dp.abs()).sum(0)))
    return out


def _silu(z):
    s = torch.sigmoid(z)
    es = s * (1 - s) * (4 * z.abs() + 8) * U + 4 * U * s
    return z * s, z.abs() * es + 2 * U * (z * s).abs(), s * (1 + z * (1 - s)), es * (1 + 2 * z.abs()) + 4 * U * s * (1 + z.abs())


def scan(u, dt, a, b, c, skip, gate, dt_bias, softplus, init=None, dy=None, dfinal=None):
    """One sequence: u, dt, gate, dy [T, D], a [D, S], b, c [T, G, S], init, dfinal [D, S]. {name: (value, bound)}."""
    u, a = u.to(F64), a.to(F64)
    T, D = u.shape
    S, G = a.shape[1], b.shape[1]
    rep = D // G
    b, c = (v.to(F64).repeat_interleave(rep, 1) for v in (b, c))  # [T, D, S]
    zero = torch.zeros(D, dtype=F64)
    skip_ = skip.to(F64) if skip is not None else zero
    raw = dt.to(F64) + (dt_bias.to(F64) if dt_bias is not None else zero)
    if softplus:
        s = torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs()))
        rs = (4 * raw.abs() + 10) * U  # relative error of s
        slope = torch.sigmoid(raw)
    else:
        s, slope = raw, torch.ones_like(raw)
        rs = U + 2 * U * ((raw - dt.to(F64)).abs() + dt.to(F64).abs()) / (raw.abs() + 1e-300)
    h = init.to(F64) if init is not None else torch.zeros(D, S, dtype=F64)
    M, E = h.abs(), torch.zeros_like(h)
    y, ey = torch.zeros(T, D, dtype=F64), torch.zeros(T, D, dtype=F64)
    hist = []
    for t in range(T):
        arg = s[t, :, None] * a
        e = torch.exp(arg)
        re = arg.abs() * (rs[t, :, None] + 3 * U) + 2 * U
        x = (s[t] * u[t])[:, None] * b[t]
        hist.append((h, M, E, e, re))
        h = e * h + x
        E = e * E + (re + 2 * U) * e * M + (rs[t, :, None] + 3 * U) * x.abs()
        M = e * M + x.abs()
        y[t] = (c[t] * h).sum(1) + skip_ * u[t]
        ey[t] = (c[t].abs() * (E + (S + 4) * U * M)).sum(1) + 4 * U * (skip_ * u[t]).abs()
        hist[-1] += (h, M, E)
    out = {"final": (h, 4 * E + 2 * U * M)}
    z = gate.to(F64) if gate is not None else None
    if z is None:
        out["y"] = (y, 4 * ey)
        sz = torch.ones_like(y)
        esz = torch.zeros_like(y)
    else:
        sz, esz, dz, edz = _silu(z)
        out["y"] = (y * sz, 4 * (ey * sz.abs() + y.abs() * esz) + 2 * U * (y * sz).abs())
    if dy is None:
        return out
    dyo = dy.to(F64)
    d, ed = dyo * sz, dyo.abs() * esz + 2 * U * (dyo * sz).abs()
    if z is not None:
        out["dgate"] = (dyo * y * dz, 4 * dyo.abs() * (ey * dz.abs() + y.abs() * edz) + 4 * U * (dyo * y * dz).abs())
    g = dfinal.to(F64) if dfinal is not None else torch.zeros(D, S, dtype=F64)
    MG, EG = g.abs(), torch.zeros_like(g)
    n = T + 300
    du, ddt, edu, eddt = (torch.zeros(T, D, dtype=F64) for _ in range(4))
    db, dc, edb, edc = (torch.zeros(T, D, S, dtype=F64) for _ in range(4))
    da, eda = torch.zeros(D, S, dtype=F64), torch.zeros(D, S, dtype=F64)
    for t in reversed(range(T)):
        h0, M0, E0, e, re, h1, M1, E1 = hist[t]
        x = c[t] * d[t][:, None]
        g = g + x
        EG = EG + c[t].abs() * ed[t][:, None] + 2 * U * (MG + x.abs())
        MG = MG + x.abs()
        st, ut = s[t][:, None], u[t][:, None]
        dc[t], edc[t] = d[t][:, None] * h1, ed[t][:, None] * M1 + d[t].abs()[:, None] * (E1 + (D + 20) * U * M1)
        db[t] = g * st * ut
        edb[t] = (st * ut).abs() * (EG + (rs[t][:, None] + (D + 20) * U) * MG)
        fed, efed = (g * b[t]).sum(1), (b[t].abs() * (EG + (S + 4) * U * MG)).sum(1)
        m, Mm = e * h0 * g, e * M0 * MG
        Em = e * (E0 * MG + M0 * EG) + (re + 4 * U) * Mm
        da += st * m
        eda += st.abs() * (Em + (rs[t][:, None] + n * U) * Mm)
        du[t] = s[t] * fed + skip_ * d[t]
        edu[t] = s[t].abs() * (efed + (rs[t] + 3 * U) * (b[t].abs() * MG).sum(1)) + skip_.abs() * (ed[t] + 3 * U * d[t].abs())
        ddt[t] = u[t] * fed + (a * m).sum(1)
        mag = u[t].abs() * (b[t].abs() * MG).sum(1) + (a.abs() * Mm).sum(1)
        eddt[t] = u[t].abs() * efed + (a.abs() * Em).sum(1) + (S + 6) * U * mag
        eddt[t] = slope[t] * eddt[t] + ((4 * raw[t].abs() + 12) * U * slope[t]) * mag
        ddt[t] *= slope[t]
        g = e * g
        EG = e * EG + (re + U) * e * MG
        MG = e * MG
    out.update(du=(du, 4 * edu), ddt=(ddt, 4 * eddt), da=(da, 4 * eda), dinit=(g, 4 * EG + 2 * U * MG),
               dskip=((d * u).sum(0), ((ed + n * U * d.abs()) * u.abs()).sum(0)),
               ddt_bias=(ddt.sum(0), (4 * eddt + n * U * ddt.abs()).sum(0)))
    for name, v, ev in (("db", db, edb), ("dc", dc, edc)):
        out[name] = (v.unflatten(1, (G, rep)).sum(2), 4 * ev.unflatten(1, (G, rep)).sum(2))
    return out


def sequences(one, lens, parts, states, shared):
    """Packed sequences: `one` of each, its results joined. parts: tensors over tokens, states: over sequences (either may
    hold None); shared: the names of results that are summed over the sequences."""
    first, got = 0, []
    for i, n in enumerate(lens):
        kw = {k: (v[first:first + n] if v is not None else None) for k, v in parts.items()}
        kw.update({k: (v[i] if v is not None else None) for k, v in states.items()})
        got.append(one(**kw))
        first += n
    out = {}
    for name in got[0]:
        vals, errs = [g[name][0] for g in got], [g[name][1] for g in got]
        if name in shared:
            # (sums over all tokens: as many more roundings as the other sequences' tokens)
            out[name] = (sum(vals), sum(errs) * (1 + len(lens)))
        elif name in ("final", "dinit"):
            out[name] = (torch.stack(vals), torch.stack(errs))
        else:
            out[name] = (torch.cat(vals), torch.cat(errs))
    return out


def embed_grad(dy, ids, rows, scale):
    """dtable and its bound; dy [T, D], ids [T]."""
    dy = dy.to(F64)
    out, mag, count = torch.zeros(rows, dy.shape[1], dtype=F64), torch.zeros(rows, dy.shape[1], dtype=F64), torch.zeros(rows, 1, dtype=F64)
    for t, i in enumerate(ids.tolist()):
        if 0 <= i < rows:
            out[i] += dy[t] * scale
            mag[i] += (dy[t] * scale).abs()
            count[i] += 1
    return out, (count + 3) * U * mag


def xent(h, w, targets, scale, dloss=None, dlse=None):
    """loss, lse and gradients with bounds; h [T, D], w [V, D], targets [T]. Products of float32 inputs are
    sums of six times as many terms."""
    f32 = h.dtype == torch.float32
    h, w = h.to(F64), w.to(F64)
    T, D = h.shape
    V = w.shape[0]
    n = (6 if f32 else 1) * D + 8
    z = scale * (h @ w.T)
    ez = n * U * abs(scale) * (h.abs() @ w.abs().T) + U * z.abs()
    lse = torch.logsumexp(z, 1)
    counts = (targets >= 0) & (targets < V)
    at = torch.where(counts, targets, 0).long()[:, None]
    # the exponentials' arguments are off by z's error and the roundings of z and the maximum; V of them are added up
    elz = ez.amax(1) + (4 * z.abs().amax(1) + 4) * U
    elz = elz + (40 + V ** 0.5) * U
    zt, ezt = z.gather(1, at)[:, 0], ez.gather(1, at)[:, 0]
    loss = torch.where(counts, lse - zt, 0.0)
    out = {"lse": (lse, elz), "loss": (loss, elz + ezt + 2 * U * (lse.abs() + zt.abs()))}
    if dloss is None:
        return out
    dl = torch.where(counts, dloss.to(F64), 0.0)[:, None]
    de = torch.where(counts, dlse.to(F64), 0.0)[:, None] if dlse is not None else torch.zeros_like(dl)
    p = torch.exp(z - lse[:, None])
    one = torch.zeros_like(z).scatter_(1, at, 1.0)
    dz = scale * ((dl + de) * p - dl * one)
    ep = p * (ez + 2 * elz[:, None] + (8 + 4 * (z.abs() + lse.abs()[:, None])) * U)
    edz = abs(scale) * ((dl + de).abs() * ep + 4 * U * ((dl + de).abs() * p + dl.abs() * one))
    # the second products' operand is rounded to bfloat16: 8 significant bits, a last place of 2^-7 of a value in [1, 2),
    # so off by 2^-8 of it at most. Of three such parts each leaves 2^-8 of what it takes, 2^-24 after the third, and the
    # products of parts that are left out, second x third (2^-8 x 2^-16) twice and third x third, are 2^-23 + 2^-32.
    edz = edz + (2 ** -22 if f32 else half_step(torch.bfloat16)) * dz.abs()
    nv, nt = (6 if f32 else 1) * V + 300, (6 if f32 else 1) * T + 300
    hk = torch.where(counts[:, None], h, 0.0)
    out["dh"] = (dz @ w, edz @ w.abs() + nv * U * (dz.abs() @ w.abs()))
    out["dw"] = (dz.T @ hk, edz.T @ hk.abs() + nt * U * (dz.abs().T @ hk.abs()))
    return out
