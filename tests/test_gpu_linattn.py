"""Linear attention with a decay for each head on the GPU, against its recurrence in 64 bits.

Tolerances, from the roundings: in float32 each sum of n terms is off by at most n 2^-24 of the
sum of their magnitudes (n: dk for a product of a query and a key, the tokens for the sum over
them, some for the weights). With bf16 operands a weight or a state is rounded to bf16 before its
product (2^-8), a value with its weight (2^-8), and the output (2^-8). States come back with the
float32 bound in both types. Over many random elements the roundings are independent and have a
standard deviation of at most 2^-8 / sqrt(3) each, so three of them stay under 2^-8 in the 2-norm."""
from __future__ import annotations

import pytest

from seq_ref import F64, check_mag, linattn

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def make(seed, type_, lens, H, Hk, dk, dv, packed, decay=None, state=True):
    """Inputs on the CPU, in the type the kernel gets: q, k, v slices of one projection."""
    gen = torch.Generator().manual_seed(seed)
    T = sum(lens)
    qkv = torch.randn(T, H * dk + Hk * (dk + dv), generator=gen).to(TYPES[type_])
    q = qkv[:, :H * dk].unflatten(-1, (H, dk))
    k = qkv[:, H * dk:(H + Hk) * dk].unflatten(-1, (Hk, dk))
    v = qkv[:, (H + Hk) * dk:].unflatten(-1, (Hk, dv))
    g = -0.4 * torch.rand(H, generator=gen) if decay is None else torch.tensor(decay, dtype=torch.float32)
    s0 = torch.randn(len(lens), H, dk, dv, generator=gen) if state else None
    do = torch.randn(T, H, dv, generator=gen).to(TYPES[type_])
    ds = torch.randn(len(lens), H, dk, dv, generator=gen) if state else None
    return dict(qkv=qkv, q=q, k=k, v=v, g=g, s0=s0, do=do, ds=ds, lens=lens, packed=packed)


def on_gpu(c, stride="slices"):
    """The tensors a call takes; unpacked sequences of one length as [N, T, ...]."""
    H, dk = c["q"].shape[1:]
    Hk, dv = c["v"].shape[1:]
    if stride == "slices":
        p = c["qkv"].cuda()
        q, k, v = (p[:, a:b].unflatten(-1, (h, d)) for a, b, h, d in (
            (0, H * dk, H, dk), (H * dk, (H + Hk) * dk, Hk, dk), ((H + Hk) * dk, p.shape[1], Hk, dv)))
    elif stride == "heads first":
        q, k, v = (c[n].transpose(0, 1).contiguous().cuda().transpose(0, 1) for n in "qkv")
    elif stride == "odd":  # no row on 16 bytes, gaps between the rows
        def odd(t):
            b = torch.full((t.shape[0], t.shape[1], t.shape[2] + 3), float("nan"), dtype=t.dtype, device="cuda")
            b[..., 1:-2] = t.cuda()
            return b[..., 1:-2]
        q, k, v = (odd(c[n]) for n in "qkv")
    else:
        q, k, v = (c[n].contiguous().cuda() for n in "qkv")
    do = c["do"].cuda()
    cu = None
    if c["packed"]:
        cu = torch.tensor([0] + c["lens"]).cumsum(0).to(torch.int32).cuda()
    else:
        q, k, v, do = (t.unflatten(0, (len(c["lens"]), c["lens"][0])) for t in (q, k, v, do))
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    return q, k, v, c["g"].cuda(), dict(cu_seqlens=cu, initial_state=up(c["s0"])), do, up(c["ds"])


def reference(c, scale, grads=False, absolute=False):
    """o, final (and dq, dk, dv, dstate) over all sequences; of the magnitudes if `absolute`."""
    f = (lambda t: None if t is None else t.to(F64).abs()) if absolute else (lambda t: None if t is None else t.to(F64))
    q, k, v, s0, do, ds = (f(c[n]) for n in ("q", "k", "v", "s0", "do", "ds"))
    leaves = [t.clone().requires_grad_(grads) for t in (q, k, v)] + ([s0.clone().requires_grad_(grads)] if s0 is not None else [])
    outs, fins, at = [], [], 0
    for n, L in enumerate(c["lens"]):
        o, s = linattn(*(t[at:at + L] for t in leaves[:3]), c["g"], abs(scale), leaves[3][n] if s0 is not None else None)
        outs.append(o)
        fins.append(s)
        at += L
    o, fin = torch.cat(outs), torch.stack(fins)
    if not grads:
        return {"o": o, "final": fin}
    loss = (o * do).sum() + ((fin * ds).sum() if ds is not None else 0) + 0 * sum(t.sum() for t in leaves)
    got = torch.autograd.grad(loss, leaves)
    return dict(zip(("dq", "dk", "dv", "dstate"), got), o=o.detach(), final=fin.detach())


def bounds(c, name):
    """rtol on the terms' magnitudes."""
    dk, dv = c["q"].shape[2], c["v"].shape[2]
    f32 = (max(dk, dv) + max(c["lens"], default=0) + 64) * 2.0 ** -24
    if name in ("final", "dstate") or c["q"].dtype == torch.float32:
        return f32
    # P (or the state) and the weighted value, the output, the sums; dk and dv of shared heads
    # are summed in float32 before their one rounding
    return 3 * 2.0 ** -8 + f32


def compare(tag, c, got, scale, grads):
    want = reference(c, scale, grads)
    mag = reference(c, scale, grads, absolute=True)
    for name in got:
        w, m = want[name], mag[name]
        t = got[name].reshape(w.shape)
        check_mag("%s %s" % (tag, name), t, w, m, bounds(c, name), 1e-37)
        if t.numel() > 2000 and c["q"].dtype == torch.bfloat16 and t.dtype == torch.bfloat16:
            rel = float((t.cpu().to(F64) - w).norm() / w.norm())
            assert rel <= 2.0 ** -8, (tag, name, rel)


def run(tag, c, stride="slices", grads=True, scale=None):
    scale = c["q"].shape[2] ** -0.5 if scale is None else scale
    q, k, v, g, kw, do, ds = on_gpu(c, stride)
    print("linattn", tag, tuple(q.shape), tuple(v.shape), q.dtype, flush=True)
    o, fin = G.gconv_linattn_fwd(q, k, v, g, scale=scale, **kw)
    got = {"o": o, "final": fin}
    if grads:
        dq, dk, dv, dst = G.gconv_linattn_bwd(do, q, k, v, g, scale=scale, d_final_state=ds, **kw)
        assert (dst is None) == (c["s0"] is None)
        got.update(dq=dq, dk=dk, dv=dv)
        if dst is not None:
            got["dstate"] = dst
        for t, like in ((dq, q), (dk, k), (dv, v)):
            assert t.shape == like.shape and t.dtype == like.dtype
    torch.cuda.synchronize()
    compare(tag, c, got, scale, grads)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 200])
def test_lengths(type_, T):
    run("T=%d" % T, make(T, type_, [T, T], 4, 2, 32, 48, False, state=T % 2 == 0))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(1, 1, 1, 1), (3, 1, 17, 33), (2, 2, 64, 64), (6, 3, 72, 96), (4, 1, 128, 128),
                                        (2, 1, 128, 64), (2, 2, 64, 128), (5, 5, 16, 127), (8, 2, 100, 20), (2, 1, 65, 63)])
def test_head_layouts(type_, H, Hk, dk, dv):
    run("heads", make(7 * dk + dv, type_, [150], H, Hk, dk, dv, False))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("stride", ["dense", "heads first", "odd"])
def test_strides(type_, stride):
    run(stride, make(5, type_, [90, 90], 4, 2, 64, 32, False), stride)
    run(stride + " packed", make(6, type_, [70, 0, 20, 131], 4, 2, 64, 32, True), stride)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[0], [0, 0, 1], [1, 1, 1], [64, 0, 65, 1, 0], [3, 200, 0, 64, 128, 17]])
def test_packed(type_, lens):
    run("packed", make(sum(lens), type_, lens, 4, 2, 48, 64, True))
    run("packed, no state", make(sum(lens), type_, lens, 2, 2, 16, 16, True, state=False))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_many_segments(type_):
    # sequences of several segments (H x T over 512 x 64) whose last segment and chunk are short
    run("segments", make(1, type_, [2500], 16, 4, 24, 40, False))
    run("segments packed", make(2, type_, [1, 1300, 0, 64, 900, 333], 16, 16, 32, 16, True))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_decays(type_):
    c = make(3, type_, [140], 6, 2, 32, 32, False, decay=[0.0, -float("inf"), -30.0, 0.02, -1e-4, -1.0])
    q, k, v, g, kw, do, ds = on_gpu(c)
    o, fin = G.gconv_linattn_fwd(q, k, v, g, scale=0.2, **kw)
    grads = G.gconv_linattn_bwd(do, q, k, v, g, scale=0.2, d_final_state=ds, **kw)
    compare("decays", c, dict(zip(("o", "final", "dq", "dk", "dv", "dstate"), (o, fin) + grads)), 0.2, True)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_later_tokens_reach_no_earlier_ones(type_, value):
    lens = [150, 40, 100]
    c = make(11, type_, lens, 4, 2, 32, 48, True)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    o, fin = G.gconv_linattn_fwd(q, k, v, g, **kw)
    spots = {"q": (70, 1, 3), "k": (85, 0, 5), "v": (71, 1, 7)}
    for name, spot in spots.items():
        bad = {"q": q.clone(), "k": k.clone(), "v": v.clone()}
        bad[name][spot] = value
        ob, fb = G.gconv_linattn_fwd(bad["q"], bad["k"], bad["v"], g, **kw)
        t = spot[0]
        assert torch.equal(ob[150:], o[150:]) and torch.equal(fb[1:], fin[1:]), name   # other sequences
        if name == "q":
            keep = torch.ones(o.shape[0], dtype=torch.bool, device="cuda")
            keep[t] = False
            assert torch.equal(ob[keep], o[keep]) and not torch.isfinite(ob[t, spot[1]]).all()
            continue
        # earlier tokens: the same terms (the spot's chunk may add them in another order)
        check_mag(name, ob[:t], o[:t].cpu().to(F64), reference(c, 32 ** -0.5, absolute=True)["o"][:t], 2 * bounds(c, "o"))
        assert (~torch.isfinite(ob[t:150, 2 * spot[1]])).any(-1).all()
        assert not torch.isfinite(fb[0]).all()
        # backwards in time: what comes before a gradient that is not a number keeps its own,
        # and the later tokens' gradients do not see it
    dob = do.clone()
    dob[75, 2, 9] = value
    a = G.gconv_linattn_bwd(do, q, k, v, g, d_final_state=ds, **kw)
    b = G.gconv_linattn_bwd(dob, q, k, v, g, d_final_state=ds, **kw)
    mag = reference(c, 32 ** -0.5, True, absolute=True)
    for n, x, y in zip(("dq", "dk", "dv"), a, b):
        if n == "dq":
            keep = torch.ones(o.shape[0], dtype=torch.bool, device="cuda")
            keep[75] = False
            assert torch.equal(x[keep], y[keep])
        else:
            assert torch.equal(x[150:], y[150:])
            check_mag(n, y[76:150], x[76:150].cpu().to(F64), mag[n][76:150], 2 * bounds(c, n))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("B,H,Hk,dk,dv", [(1, 16, 16, 128, 128), (5, 4, 2, 64, 64), (3, 3, 1, 17, 33), (40, 16, 4, 128, 128),
                                          (2, 1, 1, 1, 1), (60, 12, 3, 72, 96), (4, 2, 2, 33, 128)])
def test_step(type_, B, H, Hk, dk, dv):
    c = make(B + dk, type_, [1] * B, H, Hk, dk, dv, True)
    slots = torch.randperm(B + 3, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    pool = torch.randn(B + 3, H, dk, dv, generator=torch.Generator().manual_seed(1))
    c["s0"] = pool[slots.long()]
    state = pool.cuda()
    p = c["qkv"].cuda()
    q, k, v = (p[:, a:b].unflatten(-1, (h, d)) for a, b, h, d in (
        (0, H * dk, H, dk), (H * dk, (H + Hk) * dk, Hk, dk), ((H + Hk) * dk, p.shape[1], Hk, dv)))
    print("step", type_, B, H, Hk, dk, dv, flush=True)
    o = G.gconv_linattn_step(q, k, v, c["g"].cuda(), state, scale=0.3, slots=slots.cuda())
    want, mag = reference(c, 0.3), reference(c, 0.3, absolute=True)
    out_tol = 2.0 ** -8 if type_ == "bf16" else 0.0
    check_mag("o", o, want["o"], mag["o"], out_tol + (dk + 8) * 2.0 ** -24, 1e-37)
    check_mag("state", state[slots.cuda().long()], want["final"], mag["final"], 8 * 2.0 ** -24)
    other = torch.ones(B + 3, dtype=torch.bool)
    other[slots.long()] = False
    assert torch.equal(state.cpu()[other], pool[other])


def test_step_slots_out_of_range():
    c = make(9, "bf16", [1] * 4, 4, 2, 32, 32, True)
    q, k, v, g, _, _, _ = on_gpu(c, "dense")
    pool = torch.randn(3, 4, 32, 32).cuda()
    state = pool.clone()
    slots = torch.tensor([2, -1, 3, 0], dtype=torch.int32).cuda()
    o = G.gconv_linattn_step(q, k, v, g, state, slots=slots)
    assert torch.equal(o[1:3], torch.zeros_like(o[1:3])) and torch.equal(state[1], pool[1])
    assert (o[0] != 0).any() and (o[3] != 0).any() and not torch.equal(state[2], pool[2])
    one = pool.clone()
    o0 = G.gconv_linattn_step(q[:1], k[:1], v[:1], g, one, slots=slots[:1])
    assert torch.equal(o0[0], o[0]) and torch.equal(one[2], state[2])


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_prompt_then_tokens(type_):
    """A prompt in two calls and then single tokens give what one call over all of it gives."""
    c = make(21, type_, [100], 4, 2, 64, 64, False)
    q, k, v, g, kw, _, _ = on_gpu(c)
    scale = 64 ** -0.5
    o1, s = G.gconv_linattn_fwd(q[:, :70], k[:, :70], v[:, :70], g, **kw)
    o2, s = G.gconv_linattn_fwd(q[:, 70:95], k[:, 70:95], v[:, 70:95], g, initial_state=s)
    outs = [o1, o2]
    for t in range(95, 100):
        outs.append(G.gconv_linattn_step(q[:, t], k[:, t], v[:, t], g, s)[:, None])
    compare("parts", c, {"o": torch.cat(outs, 1), "final": s}, scale, False)


def test_gradient_against_differences():
    """The pass is linear in each argument, so a central difference over a whole step is exact but
    for float32's rounding."""
    c = make(31, "fp32", [90, 33], 4, 2, 24, 40, True)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    s0 = kw["initial_state"]

    def loss(q, k, v, s0):
        o, fin = G.gconv_linattn_fwd(q, k, v, g, scale=0.2, cu_seqlens=kw["cu_seqlens"], initial_state=s0)
        return (o.double() * do.double()).sum() + (fin.double() * ds.double()).sum(), \
            float((o * do).abs().sum() + (fin * ds).abs().sum())

    grads = G.gconv_linattn_bwd(do, q, k, v, g, scale=0.2, d_final_state=ds, **kw)
    args = [q, k, v, s0]
    for i, gr in enumerate(grads):
        d = torch.randn_like(args[i])
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + d, args[i] - d
        (a, ma), (b, mb) = loss(*up), loss(*down)
        want = float((gr.double() * d.double()).sum())
        # each o is off by at most (dk + T + 64) 2^-24 of its terms, some ten times its size here
        assert abs(float(a - b) / 2 - want) <= 10 * (40 + 90 + 64) * 2.0 ** -24 * (ma + mb), (i, float(a - b) / 2, want)


def test_same_bits_every_time_and_other_streams():
    c = make(41, "bf16", [700, 64, 300], 8, 2, 64, 128, True)
    q, k, v, g, kw, do, ds = on_gpu(c)
    call = lambda: G.gconv_linattn_fwd(q, k, v, g, **kw) + G.gconv_linattn_bwd(do, q, k, v, g, d_final_state=ds, **kw)  # noqa: E731
    first = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            again = call()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_graph_capture():
    c = make(43, "bf16", [200, 200], 4, 2, 64, 64, False)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    call = lambda: G.gconv_linattn_fwd(q, k, v, g, **kw) + G.gconv_linattn_bwd(do, q, k, v, g, d_final_state=ds, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(3):
        q.copy_(torch.randn(q.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


# Segments of five chunks of 64 tokens (64 heads x T over 512 workgroups) whose last chunk is short, so
# that a chunk's state, its flags and its loads meet those of several others.
LONG = [([2500], False), ([1250, 1250], False), ([900, 1, 0, 700, 640, 259], True)]


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("Hk,dk,dv", [(4, 128, 128), (1, 24, 40), (2, 33, 65)])
@pytest.mark.parametrize("lens,packed", LONG)
def test_segments_of_many_chunks(type_, Hk, dk, dv, lens, packed):
    """Four heads sixteen times over (the reference takes them once): the copies have the same bits."""
    c = make(51, type_, lens, 4, Hk, dk, dv, packed)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    many = lambda t, axis: torch.cat([t] * 16, axis)  # noqa: E731
    kw["initial_state"] = many(kw["initial_state"], 1)
    q, k, v, do = (many(t, -2) for t in (q, k, v, do))
    g, ds, scale = many(g, 0), many(ds, 1), dk ** -0.5
    print("linattn many chunks", tuple(q.shape), tuple(v.shape), q.dtype, flush=True)
    o, fin = G.gconv_linattn_fwd(q, k, v, g, scale=scale, **kw)
    grads = G.gconv_linattn_bwd(do, q, k, v, g, scale=scale, d_final_state=ds, **kw)
    got = dict(zip(("o", "final", "dq", "dk", "dv", "dstate"), (o, fin) + grads))
    for name, t in got.items():
        axis = 1 if name in ("final", "dstate") else t.dim() - 2
        parts = t.split(t.shape[axis] // 16, axis)
        assert all(torch.equal(parts[0], p) for p in parts), name
        got[name] = parts[0]
    compare("many chunks", c, got, scale, True)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("spot", [70, 140, 300, 319, 330])
def test_not_finite_in_a_segment_of_many_chunks(type_, value, spot):
    """A value of token `spot` that is not finite: earlier tokens keep their outputs, whichever chunk of
    a segment it lies in and whatever comes after; every later one sees it; gradients likewise."""
    c = make(61, type_, [2500], 64, 16, 16, 16, False)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    o, fin = G.gconv_linattn_fwd(q, k, v, g, **kw)
    mag = reference(c, 16 ** -0.5, absolute=True)["o"]
    bad = v.clone()
    bad[0, spot, 3, 5] = value
    ob, fb = G.gconv_linattn_fwd(q, k, bad, g, **kw)
    check_mag("v", ob[0, :spot], o[0, :spot].cpu().to(F64), mag[:spot], 2 * bounds(c, "o"))
    mine = torch.zeros(64, 16, dtype=torch.bool, device="cuda")
    mine[12:16, 5] = True  # the four heads that share it, the column that it is in
    assert (~torch.isfinite(ob[0, spot:][:, mine])).all() and not torch.isfinite(fb[0, 12:16, :, 5]).any()
    check_mag("v, others", ob[0, spot:][:, ~mine], o[0, spot:][:, ~mine].cpu().to(F64), mag[spot:][:, ~mine.cpu()], 2 * bounds(c, "o"))
    dob = do.clone()
    dob[0, spot, 12, 5] = value
    a = G.gconv_linattn_bwd(do, q, k, v, g, d_final_state=ds, **kw)
    b = G.gconv_linattn_bwd(dob, q, k, v, g, d_final_state=ds, **kw)
    keep = torch.ones(2500, dtype=torch.bool, device="cuda")
    keep[spot] = False
    assert torch.equal(a[0][0, keep], b[0][0, keep])
    gmag = reference(c, 16 ** -0.5, True, absolute=True)
    for n, x, y in zip(("dk", "dv"), a[1:3], b[1:3]):
        check_mag(n, y[0, spot + 1:], x[0, spot + 1:].cpu().to(F64), gmag[n][spot + 1:], 2 * bounds(c, n))
        assert not torch.isfinite(y[0, :spot + 1, 3]).all(-1).any(), n


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("H,Hk", [(4, 2), (64, 64)])
@pytest.mark.parametrize("cu,T", [([0, 70, 70, 200], 300), ([5, 70, 140], 140), ([130, 130, 400, 1000], 1500), ([40, 40], 77),
                                  ([0, 0], 200), ([64, 128], 192), ([700, 701, 701], 1000)])
def test_tokens_of_no_sequence(type_, H, Hk, cu, T):
    """Rows before the first and after the last sequence (a buffer's padding): 0, and the others as without them."""
    lens = [b - a for a, b in zip(cu, cu[1:])]
    c = make(71, type_, lens, H, Hk, 16, 24, True)
    q, k, v, g, kw, do, ds = on_gpu(c, "dense")
    scale = 0.25
    print("linattn padding", type_, H, cu, T, flush=True)

    def padded(t):
        out = torch.full((T,) + t.shape[1:], float("nan"), dtype=t.dtype, device="cuda")
        out[cu[0]:cu[-1]] = t
        return out

    want = G.gconv_linattn_fwd(q, k, v, g, scale=scale, **kw) + \
        G.gconv_linattn_bwd(do, q, k, v, g, scale=scale, d_final_state=ds, **kw)
    kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32).cuda()
    q, k, v, do = (padded(t) for t in (q, k, v, do))
    dirty = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
    del dirty  # what the allocator hands out next is not 0 by chance
    got = G.gconv_linattn_fwd(q, k, v, g, scale=scale, **kw) + \
        G.gconv_linattn_bwd(do, q, k, v, g, scale=scale, d_final_state=ds, **kw)
    names = ("o", "final", "dq", "dk", "dv", "dstate")
    mag = reference(c, scale, True, absolute=True)
    for name, a, b in zip(names, got, want):
        if name not in ("final", "dstate"):
            assert not a[:cu[0]].any() and not a[cu[-1]:].any(), name
            a = a[cu[0]:cu[-1]]
        # the same terms, in segments that may begin elsewhere
        check_mag(name, a, b.cpu().to(F64), mag[name], 2 * bounds(c, name), 1e-37)
