"""What the token operators' entry points refuse, on the host (no GPU: nothing here launches), and that the
binding's signatures are the header's."""
from __future__ import annotations

import ctypes
import os
import re

import pytest

from grouped_convolution_amd import binding as B

P = ctypes.c_void_p
I2, I3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3
HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gconv.h")


def at(i):
    """A made-up device address, far from every other."""
    return P(0x100000000000 * (i + 1))


def test_signatures_are_the_headers():
    """As many arguments as the header's prototypes have, whole numbers and pointers where it has them."""
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    found = 0
    for name, args in re.findall(r"^(?:int|const char\*) (gconv_\w+)\((.*?)\);", text, re.S | re.M):
        declared = [a.strip() for a in args.split(",")] if args.strip() != "void" else []
        have = getattr(B.load(), name).argtypes
        assert len(have) == len(declared), name
        for a, t in zip(declared, have):
            want = ("*" in a, a.startswith("size_t"), a.startswith("int64_t"))
            is_pointer = t is P or hasattr(t, "_type_") and not isinstance(t._type_, str)
            assert is_pointer == want[0], (name, a)
            assert want[0] or (t is ctypes.c_size_t) == want[1] and (t is ctypes.c_int64) == want[2], (name, a)
        found += 1
    assert found == len(B.EXPORTS)


# ---- the short convolution

def conv_desc(**kw):
    d = dict(dtype=B.BF16, packed=0, sequences=2, tokens=50, dim=64, taps=4, act=2)
    d.update(kw)
    n = d["dim"]
    return B.gconv_shortconv_desc(*[d[k] for k in ("dtype", "packed", "sequences", "tokens", "dim", "taps", "act")], I2(d["tokens"] * n, n),
                                  I2(d["tokens"] * n, n))


def conv_fwd(d, **swap):
    a = dict(x=at(0), w=at(1), bias=at(2), cu=None, init=None, y=at(3), final=at(4))
    a.update(swap)
    return B.load().gconv_shortconv_fwd(ctypes.byref(d), *[a[k] for k in ("x", "w", "bias", "cu", "init", "y", "final")], None)


def conv_bwd(d, ws=at(20), nws=1 << 40, **swap):
    a = dict(dy=at(5), x=at(0), w=at(1), bias=at(2), cu=None, init=None, dfinal=None, dx=at(6), dw=at(7), dbias=at(8), dinit=None)
    a.update(swap)
    keys = ("dy", "x", "w", "bias", "cu", "init", "dfinal", "dx", "dw", "dbias", "dinit")
    return B.load().gconv_shortconv_bwd(ctypes.byref(d), *[a[k] for k in keys], ws, nws, None)


def conv_step(d, num=8, **swap):
    a = dict(x=at(0), w=at(1), bias=at(2), state=at(3), slots=None, y=at(4))
    a.update(swap)
    return B.load().gconv_shortconv_step(ctypes.byref(d), *[a[k] for k in ("x", "w", "bias", "state", "slots")], num, a["y"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(act=3), 7), (dict(act=-1), 7), (dict(sequences=-1), 2), (dict(tokens=-1), 2), (dict(dim=0), 2),
    (dict(taps=0), 2), (dict(taps=9), 6), (dict(dim=(1 << 24) + 1), 6), (dict(tokens=1 << 31), 6), (dict(sequences=1 << 20, tokens=1 << 21), 6),
    (dict(sequences=1 << 30, tokens=4), 6)])
def test_shortconv_descriptors(bad, status):
    d = conv_desc(**bad)
    assert conv_fwd(d) == status and conv_bwd(d) == status
    assert B.load().gconv_last_error() != b""


def test_shortconv_pointers():
    d = conv_desc()
    for name in ("x", "w", "y"):
        assert conv_fwd(d, **{name: None}) == 1, name
    for name in ("dy", "x", "w", "dx", "dw", "dbias", "bias"):
        assert conv_bwd(d, **{name: None}) == 1, name
    assert conv_fwd(d, cu=at(9)) == 1 and conv_fwd(conv_desc(packed=1)) == 1
    assert conv_fwd(conv_desc(packed=1, sequences=0), cu=at(9)) == 2
    assert conv_fwd(d, y=at(0)) == 7 and conv_fwd(d, final=at(1)) == 7 and conv_bwd(d, dx=at(5)) == 7 and conv_bwd(d, dw=at(6)) == 7
    assert conv_bwd(d, ws=None) == 4 and conv_bwd(d, nws=16) == 4 and conv_bwd(d, ws=P(0x123456789)) == 4
    n = ctypes.c_size_t()
    assert B.load().gconv_shortconv_workspace_size(ctypes.byref(d), None) == 1
    assert B.load().gconv_shortconv_workspace_size(None, ctypes.byref(n)) == 1


def test_shortconv_step():
    assert conv_step(conv_desc()) == 7
    d = conv_desc(tokens=0)
    for name in ("x", "w", "state", "y"):
        assert conv_step(d, **{name: None}) == 1, name
    assert conv_step(d, num=-1) == 2 and conv_step(d, num=1) == 2 and conv_step(d, y=at(3)) == 7 and conv_step(d, state=at(1)) == 7


# ---- the scan

def scan_desc(**kw):
    d = dict(dtype=B.BF16, packed=0, sequences=2, tokens=50, dim=64, states=16, groups=2, softplus=1)
    d.update(kw)
    n, gs = d["dim"], d["groups"] * d["states"]
    wide, narrow = I2(d["tokens"] * n, n), I3(d["tokens"] * gs, gs, d["states"])
    return B.gconv_scan_desc(*[d[k] for k in ("dtype", "packed", "sequences", "tokens", "dim", "states", "groups", "softplus")], wide, wide, wide,
                             narrow, narrow, wide)


INS = ("u", "dt", "a", "b", "c", "skip", "gate", "dt_bias", "cu", "init")
OUTS = ("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit")


def scan_args(**swap):
    a = {k: at(i) for i, k in enumerate(INS[:8])}
    a.update({k: at(10 + i) for i, k in enumerate(OUTS[:8])})
    a.update(cu=None, init=None, y=at(20), final=at(21), dy=at(22), dfinal=None, dinit=None, state=at(23), slots=None)
    a.update(swap)
    return a


def scan_fwd(d, ws=at(30), nws=1 << 50, **swap):
    a = scan_args(**swap)
    return B.load().gconv_scan_fwd(ctypes.byref(d), *[a[k] for k in INS + ("y", "final")], ws, nws, None)


def scan_bwd(d, ws=at(30), nws=1 << 50, **swap):
    a = scan_args(**swap)
    return B.load().gconv_scan_bwd(ctypes.byref(d), *[a[k] for k in ("dy",) + INS + ("dfinal",) + OUTS], ws, nws, None)


def scan_step(d, num=8, **swap):
    a = scan_args(**swap)
    return B.load().gconv_scan_step(ctypes.byref(d), *[a[k] for k in INS[:8] + ("state", "slots")], num, a["y"], None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(sequences=-1), 2), (dict(tokens=-1), 2), (dict(dim=0), 2), (dict(states=0), 2), (dict(groups=0), 2),
    (dict(groups=3), 3), (dict(states=65), 6), (dict(dim=1 << 21), 6), (dict(tokens=1 << 31), 6), (dict(sequences=1 << 20, tokens=1 << 20), 6)])
def test_scan_descriptors(bad, status):
    d = scan_desc(**bad)
    for op in (B.SCAN_FWD, B.SCAN_BWD):
        with pytest.raises(B.GconvError) as e:
            B.gconv_scan_workspace_size(d, op)
        assert e.value.status == status
    assert scan_fwd(d) == status and scan_bwd(d) == status
    assert B.load().gconv_last_error() != b""


def test_scan_pointers():
    d = scan_desc()
    for name in ("u", "dt", "a", "b", "c", "y"):
        assert scan_fwd(d, **{name: None}) == 1, name
    for name in ("dy", "u", "dt", "a", "b", "c", "du", "ddt", "da", "db", "dc", "skip", "dskip", "gate", "dgate", "dt_bias", "ddt_bias"):
        assert scan_bwd(d, **{name: None}) == 1, name
    assert scan_fwd(d, cu=at(9)) == 1 and scan_fwd(scan_desc(packed=1)) == 1 and scan_bwd(scan_desc(packed=1)) == 1
    assert scan_fwd(scan_desc(packed=1, sequences=0), cu=at(9)) == 2
    assert scan_fwd(d, y=at(0)) == 7 and scan_fwd(d, final=at(2)) == 7 and scan_bwd(d, du=at(22)) == 7 and scan_bwd(d, dc=at(13)) == 7
    assert scan_fwd(d, ws=None) == 4 and scan_fwd(d, nws=16) == 4 and scan_bwd(d, ws=P(0x123456789)) == 4
    assert B.load().gconv_scan_workspace_size(ctypes.byref(d), 2, ctypes.byref(ctypes.c_size_t())) == 7
    assert B.load().gconv_scan_workspace_size(None, 0, ctypes.byref(ctypes.c_size_t())) == 1


def test_scan_step():
    assert scan_step(scan_desc()) == 7
    d = scan_desc(tokens=0)
    for name in ("u", "dt", "a", "b", "c", "state", "y"):
        assert scan_step(d, **{name: None}) == 1, name
    assert scan_step(d, num=-1) == 2 and scan_step(d, num=1) == 2 and scan_step(d, y=at(23)) == 7 and scan_step(d, state=at(0)) == 7


# ---- the embedding and the cross entropy

def embed_desc(**kw):
    d = dict(dtype=B.F32, index=B.I64, sequences=2, tokens=50, rows=1000, dim=64, scale=1.0)
    d.update(kw)
    return B.gconv_embed_desc(*[d[k] for k in ("dtype", "index", "sequences", "tokens", "rows", "dim")], I2(d["tokens"] * d["dim"], d["dim"]),
                              d["scale"])


def embed_both(d, ws=at(5), nws=1 << 50, **swap):
    a = dict(table=at(0), ids=at(1), y=at(2), dy=at(3), dtable=at(4))
    a.update(swap)
    lib = B.load()
    return (lib.gconv_embed_fwd(ctypes.byref(d), a["table"], a["ids"], a["y"], None),
            lib.gconv_embed_bwd(ctypes.byref(d), a["dy"], a["ids"], a["dtable"], ws, nws, None))


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(index=2), 7), (dict(scale=float("nan")), 7), (dict(sequences=-1), 2), (dict(tokens=-1), 2), (dict(rows=0), 2),
    (dict(dim=0), 2), (dict(rows=1 << 31), 6), (dict(dim=1 << 25), 6), (dict(tokens=1 << 31), 6), (dict(sequences=1 << 20, tokens=1 << 20), 6)])
def test_embed_descriptors(bad, status):
    assert embed_both(embed_desc(**bad)) == (status, status)


def test_embed_pointers():
    d = embed_desc()
    assert embed_both(d, ids=None) == (1, 1)
    assert embed_both(d, table=None, dtable=None) == (1, 1) and embed_both(d, y=None, dy=None) == (1, 1)
    assert embed_both(d, y=at(0), dtable=at(3)) == (7, 7) and embed_both(d, y=at(1), dtable=at(1)) == (7, 7)
    assert embed_both(d, y=at(1), ws=None)[1] == 4 and embed_both(d, y=at(1), nws=64)[1] == 4


def xent_desc(**kw):
    d = dict(dtype=B.BF16, index=B.I32, sequences=2, tokens=50, vocab=1000, dim=64, scale=1.0)
    d.update(kw)
    return B.gconv_xent_desc(*[d[k] for k in ("dtype", "index", "sequences", "tokens", "vocab", "dim")], I2(d["tokens"] * d["dim"], d["dim"]),
                             d["scale"])


def xent_both(d, ws=at(9), nws=1 << 50, **swap):
    a = dict(h=at(0), w=at(1), t=at(2), loss=at(3), lse=at(4), dloss=at(5), dlse=None, dh=at(6), dw=at(7))
    a.update(swap)
    lib = B.load()
    return (lib.gconv_xent_fwd(ctypes.byref(d), *[a[k] for k in ("h", "w", "t", "loss", "lse")], ws, nws, None),
            lib.gconv_xent_bwd(ctypes.byref(d), *[a[k] for k in ("dloss", "dlse", "h", "w", "t", "lse", "dh", "dw")], ws, nws, None))


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 7), (dict(index=-1), 7), (dict(scale=float("inf")), 7), (dict(sequences=-1), 2), (dict(tokens=-1), 2), (dict(vocab=0), 2),
    (dict(dim=0), 2), (dict(vocab=1 << 31), 6), (dict(dim=1 << 21), 6), (dict(tokens=1 << 31), 6), (dict(sequences=1 << 20, tokens=1 << 20), 6)])
def test_xent_descriptors(bad, status):
    d = xent_desc(**bad)
    assert xent_both(d) == (status, status)
    for op in (B.XENT_FWD, B.XENT_BWD):
        with pytest.raises(B.GconvError) as e:
            B.gconv_xent_workspace_size(d, op)
        assert e.value.status == status


def test_launches_that_are_too_large():
    """Refused before anything is enqueued: more tiles, or elements to pack, than one launch takes."""
    for d in (xent_desc(sequences=1, tokens=1 << 30, vocab=1 << 30, dim=64), xent_desc(sequences=1, tokens=1 << 30, dim=1 << 18)):
        assert xent_both(d, ws=P(0x7f0000000000000), nws=1 << 62, h=P(0x100000000000000), w=P(0x200000000000000), t=P(0x300000000000000),
                         loss=P(0x310000000000000), lse=P(0x320000000000000), dloss=P(0x330000000000000), dh=P(0x400000000000000),
                         dw=P(0x500000000000000)) == (6, 6)


@pytest.mark.parametrize("empty", [dict(sequences=0), dict(tokens=0), dict(sequences=0, tokens=0)])
def test_no_tokens_have_a_workspace_size(empty):
    for dtype in (B.F32, B.BF16):
        for op in (0, 1):
            assert B.gconv_xent_workspace_size(xent_desc(dtype=dtype, **empty), op) >= 0
            assert B.gconv_scan_workspace_size(scan_desc(dtype=dtype, **empty), op) >= 0
        n = ctypes.c_size_t()
        assert B.load().gconv_embed_workspace_size(ctypes.byref(embed_desc(dtype=dtype, **empty)), ctypes.byref(n)) == 0
        assert B.load().gconv_shortconv_workspace_size(ctypes.byref(conv_desc(dtype=dtype, **empty)), ctypes.byref(n)) == 0


def test_xent_pointers():
    d = xent_desc()
    for name in ("h", "w", "t"):
        assert xent_both(d, **{name: None}) == (1, 1), name
    assert xent_both(d, lse=None) == (1, 1) and xent_both(d, loss=None, dloss=None) == (1, 1)
    assert xent_both(d, loss=None, dh=None) == (1, 1) and xent_both(d, loss=None, dw=None) == (1, 1)
    assert xent_both(d, loss=at(0), dh=at(1)) == (7, 7) and xent_both(d, loss=at(4), dw=at(6)) == (7, 7)
    assert xent_both(d, ws=None) == (4, 4) and xent_both(d, nws=64) == (4, 4)
    assert xent_both(d, w=P(0x123456788)) == (7, 7)  # bfloat16 rows that the products read themselves
    assert B.load().gconv_xent_workspace_size(ctypes.byref(d), 2, ctypes.byref(ctypes.c_size_t())) == 7


# ---- the binding's own checks (CPU tensors are refused by all)

def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x, w, s = torch.zeros(1, 4, 8), torch.zeros(8, 3), torch.zeros(2, 2, 8)
    b, a, st = torch.zeros(1, 4, 1, 2), torch.zeros(8, 2), torch.zeros(2, 8, 2)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: B.gconv_shortconv_fwd(x, w), lambda: B.gconv_shortconv_bwd(x, x, w), lambda: B.gconv_shortconv_step(x[0, :2], w, s),
                 lambda: B.gconv_scan_fwd(x, x, a, b, b), lambda: B.gconv_scan_bwd(x, x, x, a, b, b),
                 lambda: B.gconv_scan_step(x[:, 0], x[:, 0], a, b[:, 0], b[:, 0], st), lambda: B.gconv_embed_fwd(w, ids),
                 lambda: B.gconv_embed_bwd(x[0], ids, 8), lambda: B.gconv_xent_fwd(x[0], torch.zeros(5, 8), ids),
                 lambda: B.gconv_xent_bwd(torch.zeros(4), x[0], torch.zeros(5, 8), ids, torch.zeros(4))):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: B.gconv_shortconv_fwd("x", w), lambda: B.gconv_scan_fwd(None, x, a, b, b), lambda: B.gconv_embed_fwd(3, ids),
                 lambda: B.gconv_xent_fwd([], w, ids)):
        with pytest.raises(ValueError, match="torch.Tensor"):
            call()
