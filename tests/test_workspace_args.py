"""What a given workspace has to be (host: the checks come before any pointer is used)."""
from __future__ import annotations

import pytest

from grouped_convolution_amd import binding as B

torch = pytest.importorskip("torch")

DESC = B.make_desc(2, 64, 14, 14, 32, 3, 3)


def _conv_bytes():
    return next((op, n) for op in (B.OP_BWD_FILTER, B.OP_FWD, B.OP_BWD_DATA, B.OP_BWD_BIAS)
                for n in (B.gconv_workspace_size(DESC, op),) if n > 0)


def sequence(device, workspace):
    return B._scratch(4096, device, workspace)


def convolution(device, workspace):
    op, _ = _conv_bytes()
    return B._workspace(DESC, op, device, workspace)


@pytest.mark.parametrize("take,need", [(sequence, 4096), (convolution, _conv_bytes()[1])])
def test_given_workspace(take, need):
    host, gpu = torch.device("cpu"), torch.device("cuda", 0)
    fits = torch.empty(need, dtype=torch.uint8)
    got, n = take(host, fits)  # (the device here only stands for the tensors')
    assert got is fits and n == need
    with pytest.raises(ValueError, match="needed"):
        take(host, fits[:-1])
    with pytest.raises(ValueError, match="must be on cuda:0"):
        take(gpu, fits)
    for loose in (torch.empty(1, dtype=torch.uint8).expand(need), torch.empty(2 * need, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="contiguous"):
            take(host, loose)
    with pytest.raises(ValueError, match="torch.Tensor"):
        take(host, bytearray(need))
