"""Packed sequences of the selective scan keep to themselves: what is not finite in one of them changes no bit
of another's outputs, states and gradients, wherever the cuts into chunks and tiles lie."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit")


def inputs(dtype, lens, dim, states, groups, seed):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    n = lambda *s, t=F32: torch.randn(*s, generator=gen).to(t).cuda()  # noqa: E731
    s = {k: n(T, dim, t=dtype) for k in ("u", "dt", "gate", "dy")}
    s.update({k: n(T, groups, states, t=dtype) for k in ("b", "c")})
    s.update(a=-torch.exp(0.5 * n(dim, states)), skip=n(dim), dt_bias=0.5 * n(dim) - 2, init=n(N, dim, states), dfinal=n(N, dim, states))
    return s


def both(s, cu):
    kw = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"], cu_seqlens=cu, initial_state=s["init"])
    args = [s[k] for k in ("u", "dt", "a", "b", "c")]
    y, final = G.gconv_scan_fwd(*args, **kw)
    out = dict(zip(NAMES, G.gconv_scan_bwd(s["dy"], *args, d_final_state=s["dfinal"], **kw)))
    out.update(y=y, final=final)
    return out


# Chunks are 32 tokens here: the second sequence begins inside one in which the first, of several chunks, ends, and
# (70, 60) holds whole tiles of that chunk without a sequence's first or last token.
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,states", [([40, 10, 90], 16), ([70, 60, 5, 40], 16), ([35, 0, 3, 30, 33], 3), ([33, 200], 64)])
@pytest.mark.parametrize("what", ["dy", "gate", "c", "b", "dt", "u", "init", "dfinal"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_sequence(dtype, lens, states, what, value):
    s = inputs(dtype, lens, 72, states, 2, sum(lens))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    clean = both(s, cu)
    starts = cu.tolist()
    for n, length in enumerate(lens):
        places = [n] if what in ("init", "dfinal") else sorted({starts[n] + i for i in (0, 5, length // 2, length - 1) if 0 <= i < length})
        for at in places:
            bad = dict(s)
            bad[what] = s[what].clone()
            bad[what][at] = value
            got = both(bad, cu)
            other = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
            other[starts[n]:starts[n + 1]] = False
            rest = [i for i in range(len(lens)) if i != n]
            for k in ("y", "du", "ddt", "db", "dc", "dgate"):
                assert torch.equal(got[k][other], clean[k][other]), (n, at, k)
            for k in ("final", "dinit"):
                assert torch.equal(got[k][rest], clean[k][rest]), (n, at, k)
