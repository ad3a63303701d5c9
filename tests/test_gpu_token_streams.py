"""The token operators on two streams at once, and in two graphs that share a workspace."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

BF = torch.bfloat16


def randn(gen, *shape, dtype=BF):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def conv(gen):
    x, dy, w = randn(gen, 2, 500, 264), randn(gen, 2, 500, 264), randn(gen, 264, 4)
    return lambda ws: [t for t in G.gconv_shortconv_bwd(dy, x, w, workspace=ws) if t is not None]


def scan(gen):
    u, dt, z, dy = (randn(gen, 2, 300, 130) for _ in range(4))
    b, c = randn(gen, 2, 300, 1, 16), randn(gen, 2, 300, 1, 16)
    a = -torch.rand(130, 16, generator=gen, device="cuda")
    return lambda ws: [t for t in G.gconv_scan_bwd(dy, u, dt, a, b, c, gate=z, workspace=ws) if t is not None]


def embed(gen):
    ids = torch.randint(100, (3000,), generator=gen, device="cuda")
    dy = randn(gen, 3000, 72)
    return lambda ws: [G.gconv_embed_bwd(dy, ids, 100, workspace=ws)]


def xent(gen):
    h, w = randn(gen, 300, 128), randn(gen, 1000, 128)
    t = torch.randint(1000, (300,), generator=gen, device="cuda")
    dl = torch.rand(300, generator=gen, device="cuda")
    _, lse = G.gconv_xent_fwd(h, w, t)
    return lambda ws: list(G.gconv_xent_bwd(dl, h, w, t, lse, workspace=ws))


def two(make):
    return [make(torch.Generator(device="cuda").manual_seed(s)) for s in (1, 2)]


@pytest.mark.parametrize("make", [conv, scan, embed, xent])
def test_two_streams_at_once(make):
    calls = two(make)
    want = [f(None) for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls[i](None))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


@pytest.mark.parametrize("make", [conv, scan, embed, xent])
def test_two_graphs_share_a_workspace(make):
    calls = two(make)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = [f(ws) for f in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f(ws))
        graphs.append(g)
    for turn in range(4):
        for o in outs:
            for t in o:
                t.zero_()
        for g in graphs if turn % 2 else reversed(graphs):
            g.replay()
        calls[0](ws)
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(a, b) for a, b in zip(w, o))
