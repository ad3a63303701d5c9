"""What the linear-attention entry points refuse, on the host (no GPU: nothing here launches)."""
from __future__ import annotations

import ctypes

import pytest

from grouped_convolution_amd import binding as B

P = ctypes.c_void_p
I3 = ctypes.c_int64 * 3


def desc(**kw):
    d = dict(dtype=B.BF16, packed=0, sequences=2, tokens=100, heads=4, kv_heads=2, dk=64, dv=64, scale=0.125)
    strides = {n: kw.pop(n, None) for n in ("q_stride", "k_stride", "v_stride", "do_stride")}
    d.update(kw)
    h, hk = d["heads"], d["kv_heads"]
    T = d["tokens"]
    full = dict(q_stride=(T * h * d["dk"], h * d["dk"], d["dk"]), k_stride=(T * hk * d["dk"], hk * d["dk"], d["dk"]),
                v_stride=(T * hk * d["dv"], hk * d["dv"], d["dv"]), do_stride=(T * h * d["dv"], h * d["dv"], d["dv"]))
    out = B.gconv_linattn_desc(**d)
    for n, s in full.items():
        setattr(out, n, I3(*(strides[n] or s)))
    return out


def at(i):
    """A made-up device address, far from every other."""
    return P(0x100000000 * (i + 1))


def fwd(d, cu=None, ws=at(8), nws=1 << 40, **swap):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), s0=None, o=at(4), fin=at(5))
    a.update(swap)
    return B.load().gconv_linattn_fwd(ctypes.byref(d), a["q"], a["k"], a["v"], a["g"], cu, a["s0"], a["o"], a["fin"], ws, nws,
                                      None)


def bwd(d, cu=None, ws=at(18), nws=1 << 40, **swap):
    a = dict(do=at(9), q=at(0), k=at(1), v=at(2), g=at(3), s0=None, df=None, dq=at(10), dk=at(11), dv=at(12), ds=None)
    a.update(swap)
    return B.load().gconv_linattn_bwd(ctypes.byref(d), a["do"], a["q"], a["k"], a["v"], a["g"], cu, a["s0"], a["df"], a["dq"],
                                      a["dk"], a["dv"], a["ds"], ws, nws, None)


def step(d, slots=None, num=8, **swap):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), state=at(4), o=at(5))
    a.update(swap)
    return B.load().gconv_linattn_step(ctypes.byref(d), a["q"], a["k"], a["v"], a["g"], a["state"], slots, num, a["o"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(sequences=-1), 2), (dict(tokens=-1), 2), (dict(heads=0), 2), (dict(kv_heads=0), 2),
    (dict(heads=4, kv_heads=3), 3), (dict(dk=0), 2), (dict(dv=0), 2), (dict(dk=129), 6), (dict(dv=200), 6),
    (dict(tokens=1 << 31), 6), (dict(sequences=1 << 20, tokens=1 << 20), 6), (dict(heads=1 << 17, kv_heads=1), 6),
])
def test_bad_descriptors(bad, status):
    d = desc(**bad)
    with pytest.raises(B.GconvError) as e:
        B.gconv_linattn_workspace_size(d, B.LINATTN_FWD)
    assert e.value.status == status
    assert fwd(d) == status and bwd(d) == status
    assert B.load().gconv_last_error() != b""


def test_null_pointers_and_packing():
    d = desc()
    for name in ("q", "k", "v", "g", "o"):
        assert fwd(d, **{name: None}) == 1, name
    for name in ("do", "q", "k", "v", "g", "dq", "dk", "dv"):
        assert bwd(d, **{name: None}) == 1, name
    assert fwd(d, cu=at(7)) == 1                     # cu_seqlens without packed
    assert fwd(desc(packed=1)) == 1                  # packed without cu_seqlens
    assert fwd(desc(packed=1, sequences=0), cu=at(7)) == 2   # tokens of no sequence
    assert B.load().gconv_linattn_workspace_size(ctypes.byref(d), 5, ctypes.byref(ctypes.c_size_t())) == 7
    assert B.load().gconv_linattn_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == 1


def test_workspace():
    d = desc(tokens=4000)
    for op, run in ((B.LINATTN_FWD, fwd), (B.LINATTN_BWD, bwd)):
        n = B.gconv_linattn_workspace_size(d, op)
        assert n > 0
        assert run(d, nws=n - 1) == 4
        assert run(d, ws=None, nws=0) == 4
        assert run(d, ws=P(at(8).value + 4), nws=n) == 4
    # the shared heads' gradients need room of their own, the segment states are needed by both
    alone = B.gconv_linattn_workspace_size(desc(tokens=4000, kv_heads=4), B.LINATTN_BWD)
    assert B.gconv_linattn_workspace_size(d, B.LINATTN_BWD) >= alone + 2 * 4000 * 4 * 128 * 4


def test_overlaps():
    d = desc()
    assert fwd(d, o=P(at(0).value + 64)) == 7
    assert fwd(d, fin=at(4)) == 7
    assert fwd(d, s0=at(5)) == 7
    assert bwd(d, dq=at(9)) == 7
    assert bwd(d, dk=at(12)) == 7
    s = desc(tokens=0, sequences=4)
    assert step(s, state=at(0)) == 7
    assert step(s, o=at(4)) == 7


def test_step_arguments():
    s = desc(tokens=0, sequences=4)
    for name in ("q", "k", "v", "g", "state", "o"):
        assert step(s, **{name: None}) == 1, name
    assert step(s, num=-1) == 2
    assert step(s, num=3) == 2                     # four sequences, three states, no slots
    assert step(desc(tokens=5)) == 7
    assert step(desc(tokens=0, packed=1)) == 7
    assert step(desc(tokens=0, sequences=0)) == 0 or not __import__("torch").cuda.is_available()


def test_python_checks():
    torch = pytest.importorskip("torch")
    import grouped_convolution_amd as G
    q = torch.zeros(1, 4, 2, 16)
    with pytest.raises(ValueError, match="GPU"):
        G.gconv_linattn_fwd(q, q, q, torch.zeros(2))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        G.gconv_linattn_fwd(q.half(), q.half(), q.half(), torch.zeros(2))
    with pytest.raises(ValueError, match="torch.Tensor"):
        G.gconv_linattn_step(None, q, q, torch.zeros(2), q)


def test_more_workgroups_than_a_launch_takes():
    """A launch takes fewer than 2^32 threads, 256 a workgroup: what would need more is refused beforehand."""
    size = B.gconv_linattn_workspace_size
    # the scan over segments: 16 workgroups a state of 128 x 128, 4 of 64 x 64
    for sequences, dim, ok in ((1 << 16, 128, False), ((1 << 16) - 1, 128, True), (1 << 17, 64, True), (1 << 18, 64, False),
                               (1 << 24, 128, False)):
        d = desc(sequences=sequences, tokens=1, heads=16, kv_heads=16, dk=dim, dv=dim)
        if ok:
            assert size(d, B.LINATTN_FWD) > 0 and size(d, B.LINATTN_BWD) > 0
            continue
        assert fwd(d) == 6 and bwd(d) == 6
        with pytest.raises(B.GconvError) as e:
            size(d, B.LINATTN_FWD)
        assert e.value.status == 6
    # the sum over shared heads: an element a thread in odd head sizes, four in others
    odd = desc(sequences=1, tokens=1 << 23, heads=16, kv_heads=8, dk=127, dv=64)
    assert size(odd, B.LINATTN_FWD) > 0 and bwd(odd) == 6
    assert size(desc(sequences=1, tokens=1 << 23, heads=16, kv_heads=8, dk=128, dv=64), B.LINATTN_BWD) > 0
    # the single-token step: a workgroup a head here
    assert step(desc(tokens=0, sequences=1 << 20, heads=16, kv_heads=16, dk=1, dv=1), num=1 << 20) == 6


def test_cu_seqlens_has_to_be_a_tensor():
    """(Shapes and types come before the device, so host tensors that say they are on the GPU suffice.)"""
    torch = pytest.importorskip("torch")

    class OnGpu(torch.Tensor):
        is_cuda = True

    def t(*shape):
        return torch.zeros(*shape).as_subclass(OnGpu)

    q = t(4, 2, 16)
    for bad in ([0, 4], (0, 4), 4):
        with pytest.raises(ValueError, match="cu_seqlens must be a torch.Tensor"):
            B.gconv_linattn_fwd(q, q, q, t(2), cu_seqlens=bad)
        with pytest.raises(ValueError, match="cu_seqlens must be a torch.Tensor"):
            B.gconv_linattn_bwd(q, q, q, q, t(2), cu_seqlens=bad)
    with pytest.raises(ValueError, match=r"cu_seqlens must be \[sequences \+ 1\]"):
        B.gconv_linattn_fwd(q, q, q, t(2), cu_seqlens=torch.zeros(2, 2, dtype=torch.int32))
