"""Softmax cross entropy against a vocabulary against its 64-bit definition: loss, lse, gradients."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def inputs(dtype, tokens, vocab, dim, index=torch.int64, ignored=0.0, lse=False, seed=0, std=2.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, generator=gen) * std)  # noqa: E731
    targets = torch.randint(0, vocab, (tokens,), generator=gen).to(index)
    off = torch.rand(tokens, generator=gen) < ignored
    targets[off] = torch.tensor([-100, -1, vocab, vocab + 77]).to(index)[torch.randint(0, 4, (tokens,), generator=gen)][off]
    return dict(h=n(tokens, dim).to(dtype), w=n(vocab, dim, std=std * dim ** -0.5).to(dtype), targets=targets, dloss=n(tokens),
                dlse=n(tokens, std=0.3) if lse else None)


def compare(s, scale, h=None, lead=None):
    want = R.xent(s["h"], s["w"], s["targets"], scale, s["dloss"], s["dlse"])
    lead = lead or s["targets"].shape
    at = lambda v: v.view(lead).cuda() if v is not None else None  # noqa: E731
    h = s["h"].view(lead + s["h"].shape[1:]).cuda() if h is None else h
    w, targets = s["w"].cuda(), at(s["targets"])
    loss, lse = G.gconv_xent_fwd(h, w, targets, scale=scale)
    assert loss.shape == lead and lse.shape == lead and loss.dtype == torch.float32
    dh, dw = G.gconv_xent_bwd(at(s["dloss"]), h, w, targets, lse, dlse=at(s["dlse"]), scale=scale)
    assert dh.shape == h.shape and dw.shape == w.shape and dh.dtype == h.dtype
    R.check("lse", lse.flatten(), *want["lse"])
    R.check("loss", loss.flatten(), *want["loss"])
    R.check("dh", dh.reshape(s["h"].shape), *want["dh"])
    R.check("dw", dw, *want["dw"])


SIZES = [(1, 1, 1), (1, 2, 64), (2, 300, 65), (5, 257, 8), (63, 1000, 64), (64, 256, 128), (65, 255, 100), (130, 2049, 192), (257, 513, 63),
         (300, 5000, 320), (1, 70000, 64), (700, 50, 1000)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,vocab,dim", SIZES)
def test_sizes(dtype, tokens, vocab, dim):
    compare(inputs(dtype, tokens, vocab, dim, ignored=0.2 if tokens > 4 else 0.0, lse=tokens % 2 == 0, seed=vocab), 0.7)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_pieces_of_the_vocabulary(dtype, index):
    """Enough tokens that the vocabulary is taken in pieces (the last of them ends inside a tile), and a
    product with few tiles, whose reduction is cut."""
    compare(inputs(dtype, 45000 if dtype == F32 else 130000, 2500, 8, index, ignored=0.3, seed=2), 1.0)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_tiles(dtype):
    compare(inputs(dtype, 2100, 6000, 200, ignored=0.1, lse=True, seed=3), 1.0)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,vocab", [(500, 10007), (10007, 500)])
def test_tiles_of_192_columns(dtype, tokens, vocab):
    """Products of 79 x 3 or 4 x 53 tiles, which take one round of workgroups as such and two of smaller ones."""
    compare(inputs(dtype, tokens, vocab, 576, ignored=0.1, lse=True, seed=4), 1.0)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_token_counts(dtype):
    s = inputs(dtype, 70, 400, 96, ignored=1.1, lse=True)
    s["h"][3] = float("nan")
    s["h"][40, 7] = float("inf")
    h, w, t = s["h"].cuda(), s["w"].cuda(), s["targets"].cuda()
    loss, lse = G.gconv_xent_fwd(h, w, t)
    dh, dw = G.gconv_xent_bwd(s["dloss"].cuda(), h, w, t, lse, dlse=s["dlse"].cuda())
    assert not loss.any() and not dh.any() and not dw.any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_tokens(dtype):
    w = torch.randn(37, 24).to(dtype).cuda()
    h, t, z = torch.zeros(0, 24, dtype=dtype, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    loss, lse = G.gconv_xent_fwd(h, w, t)
    dh, dw = G.gconv_xent_bwd(z, h, w, t, lse)
    assert loss.shape == lse.shape == (0,) and dh.shape == (0, 24) and not dw.any()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_what_is_not_a_number_stays_in_its_token(dtype):
    """Tokens that do not count hold anything; one that counts and is not a number spoils its own loss alone."""
    s = inputs(dtype, 300, 700, 128, ignored=0.3, seed=5)
    off = (s["targets"] < 0) | (s["targets"] >= 700)
    clean = s["h"].clone()
    s["h"][off] = float("nan")
    h, w, t = s["h"].cuda(), s["w"].cuda(), s["targets"].cuda()
    want = R.xent(clean, s["w"], s["targets"], 1.0, s["dloss"])
    loss, lse = G.gconv_xent_fwd(h, w, t)
    dh, dw = G.gconv_xent_bwd(s["dloss"].cuda(), h, w, t, lse)
    R.check("loss", loss, *want["loss"])
    R.check("dh", dh, *want["dh"])
    R.check("dw", dw, *want["dw"])
    one = int((~off).nonzero()[0])
    s["h"][one, 5] = float("nan")
    loss, _ = G.gconv_xent_fwd(s["h"].cuda(), w, t)
    bad = ~torch.isfinite(loss.cpu())
    assert bad[one] and int(bad.sum()) == 1


@pytest.mark.parametrize("dtype", [F32, BF])
def test_large_logits(dtype):
    """Logits of hundreds: the largest decides, and nothing leaves float32's range."""
    compare(inputs(dtype, 90, 1500, 64, std=300.0, seed=6), 1.0)


def test_logits_of_minus_infinity():
    """Entries that cannot be chosen: rows of w that give -infinity (bfloat16, whose infinities are kept)."""
    s = inputs(BF, 40, 600, 64, seed=7)
    s["h"] = s["h"].abs() + 0.1
    s["w"][100:400] = -float("inf")
    s["targets"] = torch.randint(0, 100, (40,))
    loss, lse = G.gconv_xent_fwd(s["h"].cuda(), s["w"].cuda(), s["targets"].cuda())
    keep = torch.cat([s["w"][:100], s["w"][400:]])
    want = R.xent(s["h"], keep, s["targets"], 1.0)
    R.check("lse", lse, *want["lse"])
    R.check("loss", loss, *want["loss"])
    s["w"][:] = -float("inf")
    loss, lse = G.gconv_xent_fwd(s["h"].cuda(), s["w"].cuda(), s["targets"].cuda())
    assert (lse == -float("inf")).all() and torch.isnan(loss).all()
    s["w"][5] = float("inf")
    loss, lse = G.gconv_xent_fwd(s["h"].cuda(), s["w"].cuda(), torch.full((40,), 5).cuda())
    assert (lse == float("inf")).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Slices at odd places (copied), every other token, time-major ones, and w at an odd address."""
    for dim in (64, 50):
        s = inputs(dtype, 60, 310, dim, ignored=0.1, seed=dim)
        wide = torch.zeros(3, 20, dim + 9, dtype=dtype, device="cuda")
        wide[..., 3:3 + dim] = s["h"].view(3, 20, dim).cuda()
        compare(s, 1.0, h=wide[..., 3:3 + dim], lead=(3, 20))
        other = torch.zeros(120, dim, dtype=dtype, device="cuda")
        other[::2] = s["h"].cuda()
        compare(s, 1.0, h=other[::2])
        compare(s, 1.0, h=s["h"].view(3, 20, dim).transpose(0, 1).contiguous().cuda().transpose(0, 1), lead=(3, 20))
    flat = torch.zeros(310 * 50 + 1, dtype=dtype, device="cuda")
    flat[1:] = s["w"].flatten().cuda()
    loss, _ = G.gconv_xent_fwd(s["h"].cuda(), flat[1:].view(310, 50), s["targets"].cuda())
    assert torch.equal(loss, G.gconv_xent_fwd(s["h"].cuda(), s["w"].cuda(), s["targets"].cuda())[0])


@pytest.mark.parametrize("vocab", [1000, 20000])
def test_gradients_in_bfloat16_are_off_by_their_own_rounding(vocab):
    """In the norm. A rounding to bfloat16 of values whose logarithms are spread evenly is off by sqrt(2^-14 / 12 x 3 / (8 ln 2))
    = 1.66e-3 of them. The target's entry of the logits' gradient is not rounded; the others are, and weigh sqrt(sum p^2)
    against it, some sqrt(e^4 / 1000) = 0.23 for logits of deviation 2: 1.66e-3 x sqrt(1 + 0.23^2) = 1.7e-3, and a fifth
    for what random values may be off. With the target's rounded too it would be 2.35e-3."""
    s = inputs(BF, 500, vocab, 256, ignored=0.1, seed=vocab)
    s["dloss"] = torch.rand(500, generator=torch.Generator().manual_seed(2)) + 0.5
    want = R.xent(s["h"], s["w"], s["targets"], 1.0, s["dloss"])
    h, w, t = s["h"].cuda(), s["w"].cuda(), s["targets"].cuda()
    _, lse = G.gconv_xent_fwd(h, w, t)
    for name, v in zip(("dh", "dw"), G.gconv_xent_bwd(s["dloss"].cuda(), h, w, t, lse)):
        off = float((v.cpu().double() - want[name][0]).norm() / want[name][0].norm())
        assert off <= 2.0e-3, (name, off)


def test_one_target_for_all():
    """A row of dw that every token adds to: sums of thousands of roundings' rests, joined by slices."""
    s = inputs(BF, 3000, 700, 72, seed=8)
    s["targets"][:] = 5
    s["targets"][::3] = 699
    compare(s, 1.0)


def test_gradient_against_differences():
    """The loss's change along random directions of h and w."""
    s = inputs(F32, 40, 500, 48, ignored=0.2, lse=True, seed=11)
    gen = torch.Generator().manual_seed(1)
    vh, vw = torch.randn(40, 48, generator=gen), torch.randn(500, 48, generator=gen) * 0.1
    t = s["targets"].cuda()

    def value(e):
        loss, lse = G.gconv_xent_fwd((s["h"] + e * vh).cuda(), (s["w"] + e * vw).cuda(), t)
        keep = (s["targets"] >= 0) & (s["targets"] < 500)
        return float((loss.cpu().double() * s["dloss"].double()).sum() + (lse.cpu().double() * s["dlse"].double() * keep).sum())

    _, lse = G.gconv_xent_fwd(s["h"].cuda(), s["w"].cuda(), t)
    dh, dw = G.gconv_xent_bwd(s["dloss"].cuda(), s["h"].cuda(), s["w"].cuda(), t, lse, dlse=s["dlse"].cuda())
    along = float((dh.cpu().double() * vh).sum() + (dw.cpu().double() * vw).sum())
    e = 2.0 ** -9
    # 40 values of about 10 are off by 2^-21 of themselves at most, over 2 e; the third derivatives' share is e^2 of their size
    assert abs((value(e) - value(-e)) / (2 * e) - along) <= 40 * 10 * 2.0 ** -21 / (2 * e) + 100 * e * e * (1 + abs(along))


def test_two_runs_are_equal_and_a_graph_replays():
    s = inputs(BF, 500, 3000, 192, ignored=0.1, lse=True, seed=9)
    h, w, t, dl, de = (s[k].cuda() for k in ("h", "w", "targets", "dloss", "dlse"))

    def both():
        loss, lse = G.gconv_xent_fwd(h, w, t)
        return (loss, lse) + G.gconv_xent_bwd(dl, h, w, t, lse, dlse=de)

    first = both()
    with torch.cuda.stream(torch.cuda.Stream()):
        both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(3):
        for v in out:
            v.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, first))
        assert all(torch.equal(a, b) for a, b in zip(both(), first))
