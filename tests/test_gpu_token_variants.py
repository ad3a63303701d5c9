"""The token operators at the sizes that choose their other kernels: long chunks, waves of four states, several
tokens a thread, tables stored past the caches, pieces of the vocabulary with cut reductions. Against the 64-bit
definitions, where channels do not meet on some of them."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402
from test_gpu_scan import compare as compare_scan, inputs as scan_inputs  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def randn(seed, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, std=1.0, t=dtype: (torch.randn(*s, generator=gen, device="cuda") * std).to(t)


def starts(lens, first=0):
    return (torch.tensor([0] + lens).cumsum(0) + first).to(torch.int32).cuda()


# ---- the scan

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("count,length,dim,states", [(8, 600, 256, 4), (32, 520, 512, 2)])
def test_scan_backward_in_longer_chunks(dtype, count, length, dim, states):
    """64 tokens (320 workgroups of that many; 160 of 128) and 128 (1280 workgroups)."""
    lens = [length] * count
    compare_scan(scan_inputs(dtype, lens, dim, states, seed=dim), lens, False)


@pytest.mark.parametrize("lens", [[700, 0, 1, 330, 65, 900, 2, 64], [2100]])
def test_scan_backward_in_longer_chunks_packed(lens):
    """64 tokens: 5 groups of 100 channels, 10 workgroups a chunk."""
    compare_scan(scan_inputs(BF, lens, 500, 5, 5, seed=len(lens)), lens, True)


def some_channels(dim):
    """A workgroup's first and last channels, and others across the row."""
    return sorted({0, 1, 62, 63, 64, dim - 1, dim - 64, dim - 65} | set(range(7, dim, max(1, dim // 40))))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,dim,states,packed", [
    ([700, 0, 1, 17, 500, 64, 0, 300], 2048, 16, True),   # 20 chunks of 80 tokens, 640 workgroups: four states a wave, twice over
    ([600, 1, 900, 0, 40], 2000, 16, True),               # the same with a workgroup that is not full
    ([1541], 2048, 13, False),                            # one sequence in such chunks
    ([70] * 9, 2048, 16, False),                          # 288 workgroups: not cut, four states a wave
    ([100] * 4, 4096, 16, False),                         # 256 workgroups: not cut, two states a wave, six tiles and a part
    ([333] * 5, 4096, 6, False)])
@pytest.mark.parametrize("gate,held", [(True, True), (False, False)])
def test_scan_forward_of_many_workgroups(dtype, lens, dim, states, packed, gate, held):
    n = randn(sum(lens) + states, dtype)
    gap = 45 if packed else 0  # tokens of no sequence on both sides
    T, N, first = sum(lens) + 2 * gap, len(lens), gap
    u, dt, z = n(T, dim), n(T, dim), n(T, dim) if gate else None
    b, c = n(T, 1, states), n(T, 1, states)
    a = -torch.exp(n(dim, states, std=0.7, t=F32)) * torch.arange(1, states + 1, device="cuda")
    skip, bias = n(dim, t=F32), n(dim, std=0.5, t=F32) - 3
    init = n(N, dim, states, t=F32) if held else None
    lead = lambda v: v if packed or v is None else v.unflatten(0, (N, lens[0]))  # noqa: E731
    y, final = G.gconv_scan_fwd(lead(u), lead(dt), a, lead(b), lead(c), skip=skip, gate=lead(z), dt_bias=bias,
                                cu_seqlens=starts(lens, first) if packed else None, initial_state=init)
    y = y.reshape(T, dim)
    assert not y[:first].any() and not y[first + sum(lens):].any()
    ch = torch.tensor(some_channels(dim), device="cuda")
    pick = lambda v: v[first:first + sum(lens)][:, ch].cpu() if v is not None else None  # noqa: E731
    parts = {"u": pick(u), "dt": pick(dt), "gate": pick(z), "b": b[first:first + sum(lens)].cpu(), "c": c[first:first + sum(lens)].cpu()}
    one = lambda **k: R.scan(k["u"], k["dt"], a[ch].cpu(), k["b"], k["c"], skip[ch].cpu(), k["gate"], bias[ch].cpu(), True, k["init"])  # noqa: E731
    want = R.sequences(one, lens, parts, {"init": init[:, ch].cpu() if held else None}, ())
    R.check("y", pick(y), *want["y"])
    R.check("final", final[:, ch], *want["final"])


# ---- the short convolution

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("count,length,dim", [
    (2, 1030, 4096),    # backward in chunks of 16 tokens, forward of 8 and 4
    (6, 1030, 4099),    # of 32; the last piece of a row begins further left
    (16, 1030, 4096),   # of 128, forward of 32
    (10, 900, 4100)])
@pytest.mark.parametrize("taps,act", [(4, "silu"), (3, "none"), (8, "silu")])
def test_shortconv_in_longer_chunks(dtype, count, length, dim, taps, act):
    shortconv([length] * count, dim, taps, act, dtype, False)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_shortconv_in_longer_chunks_packed(dtype):
    """Sequences that begin and end anywhere in chunks of 128 tokens, and tokens of none between and after them."""
    shortconv([3000, 1, 0, 127, 128, 129, 2, 5000, 3, 640, 7000, 1], 4096, 4, "silu", dtype, True)


def shortconv(lens, dim, taps, act, dtype, packed):
    n = randn(dim + len(lens) + taps, dtype)
    gap = 150 if packed else 0
    N, total = len(lens), sum(lens)
    T = total + 2 * gap
    x, dy, w, bias = n(T, dim), n(T, dim), n(dim, taps, std=taps ** -0.5), n(dim, std=0.3)
    init, dfinal = n(N, taps - 1, dim), n(N, taps - 1, dim)
    lead = lambda v: v if packed else v.unflatten(0, (N, lens[0]))  # noqa: E731
    kw = dict(act=act, cu_seqlens=starts(lens, gap) if packed else None, initial_state=init)
    y, final = G.gconv_shortconv_fwd(lead(x), w, bias, **kw)
    dx, dw, dbias, dinit = G.gconv_shortconv_bwd(lead(dy), lead(x), w, bias, d_final_state=dfinal, **kw)
    y, dx = y.reshape(T, dim), dx.reshape(T, dim)
    for v in (y, dx):
        assert not v[:gap].any() and not v[gap + total:].any()
    ch = torch.tensor(sorted({0, 1, 7, 8, 255, 256, 511, 512, dim - 1, dim - 2, dim - 5, dim - 9} | set(range(3, dim, dim // 9))), device="cuda")
    own = slice(gap, gap + total)
    pick = lambda v: v[own][:, ch].cpu()  # noqa: E731
    one = lambda **k: R.shortconv(k["x"], w[ch].cpu(), bias[ch].cpu(), act, k["init"], k["dy"], k["dfinal"])  # noqa: E731
    want = R.sequences(one, lens, {"x": pick(x), "dy": pick(dy)}, {"init": init[..., ch].cpu(), "dfinal": dfinal[..., ch].cpu()}, ("dw", "dbias"))
    R.check("y", pick(y), *want["y"])
    R.check("dx", pick(dx), *want["dx"])
    R.check("dw", dw[ch], *want["dw"])
    R.check("dbias", dbias[ch], *want["dbias"])
    R.check("dinit", dinit[..., ch], *want["dinit"])
    assert torch.equal(final[..., ch].cpu().double(), want["final"][0])


# ---- the embedding

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,dim", [(8197, 2048), (33001, 264), (70003, 100)])
def test_embedding_of_many_tokens(dtype, tokens, dim):
    """Four tokens a thread, the last thread's not all there."""
    n = randn(tokens, dtype)
    table = n(501, dim)
    ids = torch.randint(-20, 530, (tokens,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    y = G.gconv_embed_fwd(table, ids, scale=1.3)
    known = ((ids >= 0) & (ids < 501))[:, None]
    want = torch.where(known, table.double()[ids.clamp(0, 500)] * 1.3, 0.0)
    R.check("y", y, want, 2 * R.U * want.abs())


@pytest.mark.parametrize("dtype,rows,dim", [(F32, 41000, 1030), (BF, 60000, 1401)])
def test_gradient_of_a_large_table(dtype, rows, dim):
    """Stored past the caches: 169 and 168 MB."""
    n = randn(rows, dtype)
    tokens = 5003
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids = (torch.rand(tokens, device="cuda", generator=gen) ** 4 * rows).long()
    ids[::11], ids[5::50] = -1, 77
    dy = n(tokens, dim)
    got = G.gconv_embed_bwd(dy, ids, rows, scale=0.9)
    known = ids >= 0
    want, mag = (torch.zeros(rows, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    part = dy[known].double() * 0.9
    want.index_add_(0, ids[known], part)
    mag.index_add_(0, ids[known], part.abs())
    count = torch.bincount(ids[known], minlength=rows)[:, None]
    R.check("dtable", got, want, (count + 3) * R.U * mag)


# ---- the cross entropy

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,vocab,dim", [(20000, 14000, 64), (16000, 40001, 128), (20000, 14001, 72)])
def test_pieces_of_the_vocabulary_with_cut_reductions(dtype, tokens, vocab, dim):
    """Pieces of the vocabulary, whose shares of dh are added up in each of the parts that the products with few tiles
    are cut into. (The definition on the GPU, as it takes seconds there.)"""
    gen = torch.Generator(device="cuda").manual_seed(dim)
    n = lambda *s, std=1.0: torch.randn(*s, generator=gen, device="cuda") * std  # noqa: E731
    h, w = n(tokens, dim).to(dtype), n(vocab, dim, std=2 * dim ** -0.5).to(dtype)
    targets = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
    targets[::9], targets[4::10] = -100, vocab - 1
    dloss, dlse = n(tokens), n(tokens, std=0.3)
    loss, lse = G.gconv_xent_fwd(h, w, targets, scale=0.7)
    dh, dw = G.gconv_xent_bwd(dloss, h, w, targets, lse, dlse=dlse, scale=0.7)
    want = R.xent(h, w, targets, 0.7, dloss, dlse)
    for name, v in (("loss", loss), ("lse", lse), ("dh", dh), ("dw", dw)):
        R.check(name, v, *want[name])


# ---- nothing to do

@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_sequences(dtype):
    """Batches of no sequence: empty results, and gradients of 0 for what all sequences share."""
    D, S, K = 40, 5, 4
    x, b = torch.zeros(0, 7, D, dtype=dtype, device="cuda"), torch.zeros(0, 7, 2, S, dtype=dtype, device="cuda")
    w, a, ids = torch.randn(D, K, device="cuda").to(dtype), -torch.rand(D, S, device="cuda"), torch.zeros(0, 7, dtype=torch.int64, device="cuda")
    d, held = torch.randn(D, device="cuda"), torch.zeros(0, D, S, device="cuda")
    y, final = G.gconv_shortconv_fwd(x, w, w[:, 0].contiguous(), initial_state=x.new_zeros(0, K - 1, D))
    dx, dw, dbias, dinit = G.gconv_shortconv_bwd(x, x, w, w[:, 0].contiguous(), initial_state=x.new_zeros(0, K - 1, D))
    assert y.shape == dx.shape == x.shape and final.shape == dinit.shape == (0, K - 1, D) and not dw.any() and not dbias.any()
    kw = dict(skip=d, gate=x, dt_bias=d, initial_state=held)
    y, final = G.gconv_scan_fwd(x, x, a, b, b, **kw)
    got = G.gconv_scan_bwd(x, x, x, a, b, b, d_final_state=held, **kw)
    assert y.shape == got[0].shape == x.shape and final.shape == got[8].shape == (0, D, S)
    assert not any(got[i].any() for i in (2, 5, 7)) and got[2].shape == (D, S)
    assert G.gconv_shortconv_step(x[:, 0], w, x.new_zeros(3, K - 1, D)).shape == (0, D)
    assert G.gconv_scan_step(x[:, 0], x[:, 0], a, b[:, 0], b[:, 0], held.new_zeros(3, D, S)).shape == (0, D)
    assert G.gconv_embed_fwd(w, ids).shape == (0, 7, K) and not G.gconv_embed_bwd(x, ids, 9).any()
    loss, lse = G.gconv_xent_fwd(x, w.new_ones(11, D), ids)
    dh, dw = G.gconv_xent_bwd(loss, x, w.new_ones(11, D), ids, lse)
    assert loss.shape == lse.shape == (0, 7) and dh.shape == x.shape and not dw.any()
