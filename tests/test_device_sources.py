"""Rules of the kernels' sources that no run shows reliably (host, text only)."""
from __future__ import annotations

import glob
import os
import re

import pytest

import grouped_convolution_amd

CSRC = os.path.join(os.path.dirname(grouped_convolution_amd.__file__), "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.h")))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_assembly_names_the_registers_it_writes(path):
    """An asm statement that writes M0 says so: the compiler keeps values there too."""
    with open(path) as f:
        text = f.read()
    for m in re.finditer(r"asm volatile\((.*?)\);", text, re.S):
        if re.search(r"\bs_mov_b32 m0\b", m.group(1)):
            assert '"m0"' in m.group(1), m.group(0)
