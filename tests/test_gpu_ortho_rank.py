"""The orthogonalised update of gradients of low rank on the GPU, against its iteration in 64 bits:
in few rows (one workgroup, and several) and in the general kernels, wide and tall.

Tolerances, in the 2-norm: the bounds that include/gconv.h states for the rounds and the kind of
gradient, and the bf16 output's own rounding, at most 2^-8 of each value."""
from __future__ import annotations

import pytest

from seq_ref import F64, orthogonalize

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402


def bound(steps):
    return (5e-3 if steps <= 7 else 7e-3) + 2.0 ** -8


def off(tag, u, groups, steps):
    """How far each group's result is from its definition, relative in the 2-norm."""
    print("ortho rank", tag, tuple(u.shape), groups, steps, flush=True)
    got = G.gconv_orthogonalize(u.cuda(), groups=groups, steps=steps).cpu().to(F64)
    assert torch.isfinite(got).all()
    want = orthogonalize(u, groups, steps, 1e-7)
    return [float((g - w).norm() / w.norm()) for g, w in zip(got.chunk(groups), want.chunk(groups))]


def low_rank(m, n, r, seed):
    gen = torch.Generator().manual_seed(seed)
    if r == min(m, n):
        return torch.randn(m, n, generator=gen)
    return torch.randn(m, r, generator=gen) @ torch.randn(r, n, generator=gen)


SIZES = [(64, 200), (90, 1500), (128, 256), (300, 500), (500, 300), (130, 2000), (1100, 700)]


@pytest.mark.parametrize("steps", [3, 5, 7, 8])
@pytest.mark.parametrize("rank", [1, 2, 8])
@pytest.mark.parametrize("m,n", SIZES)
def test_low_rank(m, n, rank, steps):
    worst = off("low", low_rank(m, n, rank, m + rank), 1, steps)
    assert worst[0] <= bound(steps), worst


@pytest.mark.parametrize("m,n", SIZES)
def test_full_rank_and_many_rounds(m, n):
    u = low_rank(m, n, min(m, n), 3)
    for steps in (1, 5, 8):
        worst = off("full", u, 1, steps)
        assert worst[0] <= bound(steps), (steps, worst)
    worst = off("full", u, 1, 20)
    assert worst[0] <= 3e-2 + 2.0 ** -8, worst


def test_groups_of_different_rank():
    """Each group its own: what one holds next to nothing of does not grow in another."""
    u = torch.cat([low_rank(200, 300, r, 7) * s for r, s in ((1, 1e-8), (200, 1.0), (4, 1e6))])
    worst = off("groups", u, 3, 5)
    assert max(worst) <= bound(5), worst
    few = torch.cat([low_rank(70, 300, r, 9) * s for r, s in ((70, 1.0), (1, 1e4), (2, 1e-6))])
    worst = off("groups of few rows", few, 3, 5)
    assert max(worst) <= bound(5), worst


@pytest.mark.parametrize("m,n", [(97, 4000), (1389, 1050), (63, 407), (2, 3), (3, 2)])
def test_constant_and_tiny(m, n):
    """The worst kinds: entries that are all rounded the same way, and too few singular values to average over."""
    u = torch.ones(m, n) if min(m, n) > 3 else torch.randn(m, n, generator=torch.Generator().manual_seed(5))
    for steps, most in ((1, 1.5e-2), (5, 1.5e-2), (8, 6e-2)):
        worst = off("worst", u, 1, steps)
        assert worst[0] <= most + 2.0 ** -8, (steps, worst)
