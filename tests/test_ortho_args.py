"""What the orthogonalised update's entry points refuse, on the host (no GPU: nothing here launches)."""
from __future__ import annotations

import ctypes

import pytest

from grouped_convolution_amd import binding as B

P = ctypes.c_void_p


def desc(**kw):
    d = dict(dtype=B.F32, filters=256, inner=1200, groups=2, steps=5, eps=1e-7)
    d.update(kw)
    return B.gconv_ortho_desc(**d)


def size(d):
    n = ctypes.c_size_t()
    return B.load().gconv_orthogonalize_workspace_size(ctypes.byref(d), ctypes.byref(n)), n.value


def call(d, u=P(0x100000000), out=P(0x200000000), ws=P(0x300000000), nws=1 << 40):
    return B.load().gconv_orthogonalize(ctypes.byref(d), u, out, ws, nws, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(filters=0), 2), (dict(inner=0), 2), (dict(groups=0), 2), (dict(groups=3), 3), (dict(steps=0), 7),
    (dict(steps=1001), 7), (dict(eps=-1.0), 7), (dict(eps=float("nan")), 7), (dict(filters=1 << 15, inner=1 << 15, groups=1), 6),
    (dict(filters=2, inner=(1 << 24) + 1), 6), (dict(filters=1 << 21, groups=1 << 21), 6),
])
def test_bad_descriptors(bad, status):
    d = desc(**bad)
    assert size(d)[0] == status and call(d) == status
    assert B.load().gconv_last_error() != b""


def test_pointers_workspace_and_overlaps():
    d = desc()
    st, n = size(d)
    assert st == 0 and n > 0
    assert call(d, u=None) == 1 and call(d, out=None) == 1
    assert call(d, ws=None) == 4 and call(d, nws=n - 1) == 4 and call(d, ws=P(0x300000008)) == 4
    assert call(d, out=P(0x200000004)) == 7
    assert call(d, out=P(0x100000000 + 256 * 1200 * 4 - 8)) == 7
    assert B.load().gconv_orthogonalize_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert B.load().gconv_orthogonalize_workspace_size(ctypes.byref(d), None) == 1


def test_python_checks():
    torch = pytest.importorskip("torch")
    import grouped_convolution_amd as G
    with pytest.raises(ValueError, match="GPU"):
        G.gconv_orthogonalize(torch.zeros(4, 4))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G.gconv_orthogonalize(torch.zeros(4, 4).half())


def test_more_workgroups_than_a_launch_takes():
    """A launch takes fewer than 2^32 threads: many groups of several workgroups each are refused beforehand."""
    for bad, good in ((dict(filters=1 << 20, inner=1024, groups=1 << 20), dict(filters=1 << 19, inner=1024, groups=1 << 19)),
                      (dict(filters=200 << 20, inner=200, groups=1 << 20), dict(filters=200 << 19, inner=200, groups=1 << 19))):
        d = desc(**bad)
        assert size(d)[0] == 6 and call(d) == 6
        assert size(desc(**good))[0] == 0
