"""The norms around a block on the GPU against their formulas in 64 bits.

Tolerances: a value is off by at most 512 2^-24 of the magnitude of its terms (a row's sum of up
to 8192 squares is 8 terms a thread and a tree of ten levels; the exponential and the reciprocals
a few units each; a sum over the rows is at most some 300 additions deep), and a bf16 output by
half a step (2^-8 of it) more."""
from __future__ import annotations

import pytest

from seq_ref import F64, check_mag, normgate

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("dx", "db", "dgate", "dw_post", "dscale", "dw_pre")


def make(seed, type_, N, T, D, gate="full", residual=True, pre=True, scale=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std).to(TYPES[type_])  # noqa: E731
    c = dict(x=r(N, T, D, std=2.0) if residual else None, b=r(N, T, D, std=0.7),
             gate=r(N, T, D) if gate == "full" else r(N, 1, D) if gate == "sequence" else None,
             w_post=1 + r(D, std=0.2), scale=r(D, std=0.3) if scale else None, w_pre=1 + r(D, std=0.2) if pre else None)
    c["dy"] = r(N, T, D)
    c["dh"] = r(N, T, D) if pre else None
    return c


def up(t):
    return None if t is None else t.cuda()


def call(c, act, eps, move=up):
    x, b, gate, dy, dh = (move(c[n]) for n in ("x", "b", "gate", "dy", "dh"))
    kw = dict(gate=gate, act=act, w_post=up(c["w_post"]), scale=up(c["scale"]), w_pre=up(c["w_pre"]), eps=eps)
    y, h = G.gconv_normgate_fwd(x, b, **kw)
    return dict(zip(("y", "h") + NAMES, (y, h) + tuple(G.gconv_normgate_bwd(dy, dh, x, b, **kw))))


def run(tag, c, act="silu", eps=1e-6, move=up):
    print("normgate", tag, tuple(c["b"].shape), c["b"].dtype, act, flush=True)
    got = call(c, act, eps, move)
    torch.cuda.synchronize()
    want = normgate(c["x"], c["b"], c["gate"], act, c["w_post"], c["scale"], c["w_pre"], eps, c["dy"], c["dh"])
    half = 2.0 ** -8 if c["b"].dtype == torch.bfloat16 else 0.0
    for name in ("y", "h") + NAMES:
        assert (got[name] is None) == (name not in want), name
        if got[name] is not None:
            w, m = want[name]
            assert got[name].dtype == c["b"].dtype
            check_mag("%s %s" % (tag, name), got[name], w, 512 * 2.0 ** -24 * m + half * w.abs(), 1.0, 1e-37)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [1, 3, 8, 31, 64, 127, 128, 129, 256, 500, 512, 1001, 1024, 2000, 2048, 2049, 4096, 5000, 8192])
def test_widths(type_, D):
    run("D", make(D, type_, 2, 5, D))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", ["none", "full", "sequence"])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
@pytest.mark.parametrize("residual,pre,scale", [(True, True, True), (False, False, False), (True, False, True), (False, True, False)])
def test_variants(type_, gate, act, residual, pre, scale):
    run("variant", make(5, type_, 3, 37, 160, gate, residual, pre, scale), act)


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("N,T,D,gate", [(1, 1, 64, "full"), (1, 3000, 72, "full"), (600, 2, 96, "sequence"), (1030, 3, 33, "sequence"),
                                        (3, 1111, 40, "sequence"), (2, 700, 1000, "sequence"), (5, 1, 4096, "sequence")])
def test_rows(type_, N, T, D, gate):
    run("rows", make(N + T, type_, N, T, D, gate))


@pytest.mark.parametrize("N,T", [(0, 5), (4, 0)])
@pytest.mark.parametrize("gate", ["full", "sequence"])
def test_no_rows(N, T, gate):
    c = make(1, "bf16", N, T, 64, gate)
    got = call(c, "silu", 1e-6)
    torch.cuda.synchronize()
    for n in ("dw_post", "dscale", "dw_pre"):
        assert torch.equal(got[n], torch.zeros_like(got[n])), n
    if gate == "sequence":
        assert torch.equal(got["dgate"], torch.zeros_like(got["dgate"]))


@pytest.mark.parametrize("type_", ["fp32", "bf16"])
@pytest.mark.parametrize("D", [64, 250, 1001])
def test_strides(type_, D):
    def slices(t):  # an odd slice of a wider row, the token axis first in memory
        if t is None:
            return None
        wide = torch.full((t.shape[1], t.shape[0], t.shape[2] + 3), float("nan"), dtype=t.dtype, device="cuda")
        wide[..., 1:-2] = t.transpose(0, 1).cuda()
        return wide[..., 1:-2].transpose(0, 1)

    run("strides", make(D, type_, 3, 20, D, "full"), move=slices)
    run("strides", make(D, type_, 3, 20, D, "sequence"), move=slices)


def test_one_sequence_without_its_axis():
    c = make(3, "bf16", 1, 9, 96)
    flat = {n: t[0] if t is not None and t.dim() == 3 else t for n, t in c.items()}
    a, b = call(c, "silu", 1e-6), call(flat, "silu", 1e-6)
    assert all(torch.equal(a[n].reshape(b[n].shape), b[n]) for n in a)


def test_large_and_small_values():
    for std in (1e-12, 1e6):
        c = make(7, "fp32", 2, 6, 200)
        c["b"] = c["b"] * std
        run("std %g" % std, c, eps=1e-5)
    c = make(8, "fp32", 2, 6, 200)
    c["b"][0, 0] = 0  # a row of zeros: the eps alone
    run("zeros", c)


def test_a_row_that_is_not_finite_stays_alone():
    c = make(9, "bf16", 2, 30, 128)
    a = call(c, "silu", 1e-6)
    c["b"][1, 7, 3] = float("nan")
    c["gate"][0, 5, 100] = float("inf")
    b = call(c, "silu", 1e-6)
    keep = torch.ones(2, 30, dtype=torch.bool)
    keep[1, 7] = keep[0, 5] = False
    for n in ("y", "h", "dx", "db", "dgate"):
        assert torch.equal(a[n].cpu()[keep], b[n].cpu()[keep]), n
    assert torch.isnan(b["y"][1, 7]).all()


def test_gradients_against_differences():
    """Central differences of the GPU's own forward pass in float32: the second-order term is
    step^2 / 6 of a third derivative of order one, the rounding 2^-24 of the loss's terms over the step."""
    c = make(11, "fp32", 2, 9, 70, "sequence")
    got = call(c, "silu", 1e-3)

    def loss(c):
        y, h = G.gconv_normgate_fwd(up(c["x"]), up(c["b"]), gate=up(c["gate"]), act="silu", w_post=up(c["w_post"]),
                                    scale=up(c["scale"]), w_pre=up(c["w_pre"]), eps=1e-3)
        t = y.cpu().to(F64) * c["dy"].to(F64), h.cpu().to(F64) * c["dh"].to(F64)
        return float(t[0].sum() + t[1].sum()), float(t[0].abs().sum() + t[1].abs().sum())

    step = 2.0 ** -7
    for name in ("x", "b", "gate", "w_post", "scale", "w_pre"):
        d = torch.randn(c[name].shape, generator=torch.Generator().manual_seed(1))
        (a, m), (b, _) = loss(dict(c, **{name: c[name] + step * d})), loss(dict(c, **{name: c[name] - step * d}))
        want = float((got["d" + name].cpu().to(F64) * d.to(F64)).sum())
        assert abs((a - b) / (2 * step) - want) <= m * (step ** 2 * 4 + 64 * 2.0 ** -24 / step), (name, (a - b) / (2 * step), want)


def test_same_bits_other_streams_and_graph():
    c = make(13, "bf16", 4, 600, 256, "sequence")
    x, b, gate, dy, dh = (up(c[n]) for n in ("x", "b", "gate", "dy", "dh"))
    kw = dict(gate=gate, act="silu", w_post=up(c["w_post"]), scale=up(c["scale"]), w_pre=up(c["w_pre"]))
    both = lambda: G.gconv_normgate_fwd(x, b, **kw) + tuple(G.gconv_normgate_bwd(dy, dh, x, b, **kw))  # noqa: E731
    first = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = both()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for i in range(3):
        b.copy_(torch.randn(b.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, both())), i
