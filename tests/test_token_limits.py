"""Limits of the token operators that hold before anything is launched (on the host: nothing here launches)."""
from __future__ import annotations

import ctypes

import pytest

from grouped_convolution_amd import binding as B
from test_token_args import at, embed_both, embed_desc, scan_bwd, scan_desc, xent_both, xent_desc

UNSUPPORTED, ARG = 6, 7


@pytest.mark.parametrize("desc", [
    # the sums of da: a workgroup of 1024 threads for every 64 states of a workgroup's lanes, tokens or none
    dict(dim=1 << 16, groups=1 << 16, states=64, tokens=0), dict(dim=1 << 16, groups=1 << 16, states=64, tokens=1),
    dict(dim=1 << 20, groups=1 << 20, states=4, tokens=0),
    # the last kernel: twice the waves of the first one
    dict(packed=1, sequences=1, tokens=1 << 28, dim=1024, groups=1, states=4)])
def test_backward_scans_that_are_too_large(desc):
    assert scan_bwd(scan_desc(**desc), cu=at(9) if desc.get("packed") else None) == UNSUPPORTED


@pytest.mark.parametrize("scale", [1e39, -1e39, 3.5e38, 1e308])
def test_scales_past_float32(scale):
    """Finite as a double, infinite as the float32 that the kernels take."""
    assert embed_both(embed_desc(scale=scale)) == (ARG, ARG)
    assert xent_both(xent_desc(scale=scale)) == (ARG, ARG)
    n = ctypes.c_size_t()
    assert B.load().gconv_embed_workspace_size(ctypes.byref(embed_desc(scale=scale)), ctypes.byref(n)) == ARG
    assert B.load().gconv_xent_workspace_size(ctypes.byref(xent_desc(scale=scale)), B.XENT_FWD, ctypes.byref(n)) == ARG
