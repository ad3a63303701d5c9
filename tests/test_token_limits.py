"""Limits of the token operators that hold before anything is launched (on the host: nothing here launches)."""
from __future__ import annotations

import pytest

from test_token_args import at, scan_bwd, scan_desc

UNSUPPORTED = 6


@pytest.mark.parametrize("desc", [
    # the sums of da: a workgroup of 1024 threads for every 64 states of a workgroup's lanes, tokens or none
    dict(dim=1 << 16, groups=1 << 16, states=64, tokens=0), dict(dim=1 << 16, groups=1 << 16, states=64, tokens=1),
    dict(dim=1 << 20, groups=1 << 20, states=4, tokens=0),
    # the last kernel: twice the waves of the first one
    dict(packed=1, sequences=1, tokens=1 << 28, dim=1024, groups=1, states=4)])
def test_backward_scans_that_are_too_large(desc):
    assert scan_bwd(scan_desc(**desc), cu=at(9) if desc.get("packed") else None) == UNSUPPORTED
