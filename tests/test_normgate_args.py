"""What the gated norm's entry points refuse, on the host (no GPU: nothing here launches)."""
from __future__ import annotations

import ctypes

import pytest

from grouped_convolution_amd import binding as B

P = ctypes.c_void_p
I2 = ctypes.c_int64 * 2


def desc(**kw):
    d = dict(dtype=B.BF16, sequences=2, tokens=10, dim=256, gate=B.GATE_FULL, act=B.ACTS["silu"], eps=1e-6)
    d.update(kw)
    out = B.gconv_normgate_desc(**d)
    for n in ("x_stride", "b_stride", "gate_stride", "dy_stride", "dh_stride"):
        setattr(out, n, I2(d["tokens"] * d["dim"], d["dim"]))
    return out


def at(i):
    """A made-up device address, far from every other."""
    return P(0x100000000 * (i + 1))


FWD = ("x", "b", "gate", "w_post", "scale", "w_pre", "y", "h")
BWD = ("dy", "dh", "x", "b", "gate", "w_post", "scale", "w_pre", "dx", "db", "dgate", "dw_post", "dscale", "dw_pre")


def fwd(d, **swap):
    a = {n: at(i) for i, n in enumerate(FWD)}
    a.update(swap)
    return B.load().gconv_normgate_fwd(ctypes.byref(d), *(a[n] for n in FWD), None)


def bwd(d, ws=at(30), nws=1 << 40, **swap):
    a = {n: at(i) for i, n in enumerate(BWD)}
    a.update(swap)
    return B.load().gconv_normgate_bwd(ctypes.byref(d), *(a[n] for n in BWD), ws, nws, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=5), 7), (dict(gate=3), 7), (dict(gate=-1), 7), (dict(act=3), 7), (dict(sequences=-1), 2), (dict(tokens=-2), 2),
    (dict(dim=0), 2), (dict(dim=8193), 6), (dict(sequences=1 << 25, tokens=1 << 25), 6), (dict(eps=-1.0), 7),
    (dict(eps=float("nan")), 7),
])
def test_bad_descriptors(bad, status):
    d = desc(**bad)
    assert B.load().gconv_normgate_workspace_size(ctypes.byref(d), ctypes.byref(ctypes.c_size_t())) == status
    assert fwd(d) == status and bwd(d) == status
    assert B.load().gconv_last_error() != b""


def test_what_goes_together():
    d = desc()
    for name in ("b", "w_post", "y", "gate", "w_pre", "h"):
        assert fwd(d, **{name: None}) == 1, name
    for name in ("dy", "dh", "b", "gate", "w_post", "scale", "w_pre", "db", "dgate", "dw_post", "dscale", "dw_pre", "x"):
        assert bwd(d, **{name: None}) == 1, name
    assert fwd(desc(gate=B.GATE_NONE)) == 1           # a gate where there is none
    assert bwd(desc(gate=B.GATE_NONE)) == 1


def test_workspace_and_overlaps():
    d = desc()
    n = ctypes.c_size_t()
    assert B.load().gconv_normgate_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(d, nws=n.value - 1) == 4
    assert bwd(d, ws=None) == 4
    assert bwd(d, ws=P(at(30).value + 8), nws=n.value) == 4
    assert fwd(d, y=at(0)) == 7
    assert fwd(d, h=at(6)) == 7
    assert bwd(d, dx=P(at(0).value + 16)) == 7
    assert bwd(d, dscale=at(11)) == 7


def test_python_checks():
    torch = pytest.importorskip("torch")
    import grouped_convolution_amd as G
    b = torch.zeros(2, 3, 8)
    with pytest.raises(ValueError, match="GPU"):
        G.gconv_normgate_fwd(None, b, w_post=torch.ones(8))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G.gconv_normgate_fwd(None, b.double(), w_post=torch.ones(8))


def test_gradient_of_a_sequence_gate_without_tokens():
    """The sums over no tokens are still written: [sequences, dim] zeros, so there has to be a place for them."""
    d = desc(gate=B.GATE_SEQUENCE, tokens=0)
    assert bwd(d, dgate=None) == 1
    assert bwd(d, gate=None, dgate=None) == 1
