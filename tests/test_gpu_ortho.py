"""The orthogonalised update on the GPU against its iteration in 64 bits.

Tolerance, in the 2-norm: the iterate, its Gram matrix and the polynomial are each rounded to fp16
once a round (and the iterate once before), each rounding at most 2^-11 of a value and 1 / sqrt(3)
of that over many values; a round enlarges an error by at most 3.4445, the slope of its polynomial
at 0, which is also how it enlarges the small singular values that the error is relative to; so
3 * 5 + 1 independent roundings come to sqrt(16) 2^-11 3.4445 / sqrt(3). The bf16 output adds its
own rounding, at most 2^-8 of a value. The float32 sums are far below both."""
from __future__ import annotations

import pytest

from seq_ref import F64, orthogonalize

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
REL = 4 * 2.0 ** -11 * 3.4445 / 3 ** 0.5


def make(seed, type_, *shape, std=1e-3):
    """A gradient: a few strong directions and noise."""
    gen = torch.Generator().manual_seed(seed)
    m, n = shape[0], 1
    for s in shape[1:]:
        n *= s
    r = min(m, n, 8)
    u = torch.randn(m, r, generator=gen) @ torch.randn(r, n, generator=gen) * 0.3 + torch.randn(m, n, generator=gen)
    return (u * std).to(TYPES[type_]).view(shape)


def run(tag, u, groups=1, steps=5, eps=1e-7):
    print("ortho", tag, tuple(u.shape), u.dtype, groups, flush=True)
    got = G.gconv_orthogonalize(u.cuda(), groups=groups, steps=steps, eps=eps)
    torch.cuda.synchronize()
    assert got.dtype == torch.bfloat16 and got.shape == u.shape
    # the reference runs on the GPU too where that is quicker: the products are plain 64-bit ones
    big = u.numel() > 1 << 18
    want = orthogonalize((u.cuda() if big else u).reshape(u.shape[0], -1), groups, steps, eps).cpu().view(u.shape)
    got = got.cpu().to(F64)
    assert torch.isfinite(got).all()
    for g, w in zip(got.chunk(groups), want.chunk(groups)):
        far = (g - w).abs()
        rms = w.square().mean().sqrt()
        assert far.square().mean().sqrt() <= (REL + 2.0 ** -8) * rms, (tag, float(far.square().mean().sqrt() / rms))
        # single elements: eight standard deviations
        assert (far <= 8 * REL * rms + 2.0 ** -8 * w.abs()).all(), tag
    return got


# one step of the smallest tile, its edges, odd sizes, tall and wide, each tile of the dispatcher
@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (2, 300), (5, 4), (63, 64), (64, 64), (65, 129), (100, 1001), (128, 1200),
                                 (129, 128), (300, 40), (1000, 17), (192, 577), (500, 515)])
@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_sizes(type_, m, n):
    run("size", make(m + n, type_, m, n))


# one workgroup, and several, by the rows that are kept in registers; the longest of each
@pytest.mark.parametrize("m,n", [(20, 30), (32, 704), (32, 705), (9, 5000), (40, 512), (64, 513), (50, 3000), (96, 448), (80, 449),
                                 (70, 2222), (128, 256), (128, 321), (100, 8200), (3, 70000), (110, 20000), (400, 128), (2000, 66)])
@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_few_rows(type_, m, n):
    run("few rows", make(m + n, type_, m, n))


@pytest.mark.parametrize("m,n", [(1100, 1300), (2000, 2050), (2500, 1025), (4000, 4100), (1700, 8000)])
def test_large(m, n):
    run("large", make(m + n, "fp32", m, n))


@pytest.mark.parametrize("shape,groups", [((256, 48, 5, 5), 2), ((128, 4, 3, 3), 32), ((64, 1, 3, 3), 64), ((96, 33, 1, 1), 3),
                                          ((600, 200, 1, 1), 2), ((1024, 7, 3, 3), 8), ((2048, 512, 1, 1), 4)])
@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_groups(type_, shape, groups):
    run("groups", make(3, type_, *shape), groups)


@pytest.mark.parametrize("steps", [1, 2, 9])
def test_steps(steps):
    run("steps", make(4, "fp32", 80, 90), steps=steps)


@pytest.mark.parametrize("std", [1e-30, 1e-18, 1e15])
def test_any_magnitude(std):
    run("std", make(5, "fp32", 70, 130, std=std), eps=0.0)


def test_zeros_and_eps():
    u = torch.zeros(3 * 40, 50)
    u[40:80] = make(6, "fp32", 40, 50)
    got = G.gconv_orthogonalize(u.cuda(), groups=3).cpu()
    assert not got[:40].any() and not got[80:].any() and got[40:80].any()
    run("eps", make(7, "fp32", 40, 50), eps=0.05)


def test_one_direction():
    """A matrix of rank one: one singular value, 1, goes through the iteration, and nothing else appears."""
    a, b = torch.randn(90, 1, generator=torch.Generator().manual_seed(1)), torch.randn(1, 200, generator=torch.Generator().manual_seed(2))
    run("rank one", a @ b)


def test_a_group_that_is_not_finite_stays_alone():
    u = make(8, "fp32", 192, 70)
    a = G.gconv_orthogonalize(u.cuda(), groups=3).cpu()
    u[70, 3] = float("nan")
    b = G.gconv_orthogonalize(u.cuda(), groups=3).cpu()
    u[70, 3] = float("inf")
    c = G.gconv_orthogonalize(u.cuda(), groups=3).cpu()
    for t in (b, c):
        assert torch.equal(a[:64], t[:64]) and torch.equal(a[128:], t[128:])
        assert torch.isnan(t[64:128]).any()


def test_tall_is_the_transpose_of_wide():
    u = make(9, "bf16", 70, 260)
    a = G.gconv_orthogonalize(u.cuda())
    b = G.gconv_orthogonalize(u.T.contiguous().cuda())
    assert torch.equal(a, b.T)


def test_nearly_orthogonal():
    """The rows of the result are orthogonal to within the iteration's own band (0.68 .. 1.21)."""
    got = run("band", torch.randn(128, 1024, generator=torch.Generator().manual_seed(3)))
    s = torch.linalg.svdvals(got)
    assert s.min() > 0.6 and s.max() < 1.25


def test_unaligned_and_given_buffers():
    u = make(10, "fp32", 48, 99)
    wide = torch.empty(48 * 99 + 1, device="cuda")
    v = wide[1:].view(48, 99)
    v.copy_(u)
    out = torch.empty(48, 99, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")  # NaN in every type
    assert torch.equal(G.gconv_orthogonalize(v, out=out, workspace=ws), G.gconv_orthogonalize(u.cuda()))


def test_same_bits_other_streams_and_graph():
    u = make(11, "fp32", 200, 700).cuda()
    first = G.gconv_orthogonalize(u, groups=2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = G.gconv_orthogonalize(u, groups=2)
    side.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.gconv_orthogonalize(u, groups=2)
    for i in range(3):
        u.copy_(torch.randn(u.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, G.gconv_orthogonalize(u, groups=2)), i
