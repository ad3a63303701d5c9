"""The embedding and its gradient against their 64-bit definitions."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def compare(table, ids, dy, scale, shape=None, dy_gpu=None):
    rows, D = table.shape
    known = (ids >= 0) & (ids < rows)
    want = torch.where(known[:, None], table.double()[torch.where(known, ids, 0).long()] * scale, 0.0)
    on_gpu = ids.view(shape or ids.shape).cuda()
    y = G.gconv_embed_fwd(table.cuda(), on_gpu, scale=scale)
    assert y.shape == on_gpu.shape + (D,)
    R.check("y", y.view(-1, D), want, 2 * R.U * want.abs())
    dy_gpu = dy.view(on_gpu.shape + (D,)).cuda() if dy_gpu is None else dy_gpu
    dt = G.gconv_embed_bwd(dy_gpu, on_gpu, rows, scale=scale)
    assert dt.dtype == table.dtype and dt.shape == table.shape
    R.check("dtable", dt, *R.embed_grad(dy, ids, rows, scale))
    return dt


def inputs(dtype, index, tokens, rows, dim, seed=0, outside=0.0):
    gen = torch.Generator().manual_seed(seed)
    ids = (torch.rand(tokens, generator=gen) ** 3 * rows).to(index)
    off = torch.rand(tokens, generator=gen) < outside
    ids[off] = torch.tensor([-1, rows, rows + 5, -100]).to(index)[torch.randint(0, 4, (tokens,), generator=gen)][off]
    return torch.randn(rows, dim, generator=gen).to(dtype), ids, torch.randn(tokens, dim, generator=gen).to(dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,rows,dim", [(1, 1, 1), (0, 5, 8), (3, 1000, 7), (64, 3, 16), (65, 513, 33), (300, 40, 264), (2049, 600, 24),
                                             (5000, 300000, 4), (9000, 511, 8), (700, 512, 2100)])
def test_sizes(dtype, index, tokens, rows, dim):
    table, ids, dy = inputs(dtype, index, tokens, rows, dim, tokens + dim, 0.1)
    compare(table, ids, dy, 1.7)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_one_token_makes_up_the_text(dtype):
    for tokens in (64, 65, 4097, 20000):
        table, ids, dy = inputs(dtype, torch.int64, tokens, 9, 40, tokens)
        compare(table, torch.full((tokens,), 8, dtype=torch.int64), dy, 1.0)
        # ... and two that share slices of the sorted order, with others between them
        ids = torch.where(torch.arange(tokens) % 3 == 0, 2, 5)
        ids[tokens // 2] = 4
        compare(table, ids, dy, 1.0)


def test_every_id_is_outside():
    table, _, dy = inputs(F32, torch.int32, 40, 10, 12)
    dt = compare(table, torch.full((40,), -1, dtype=torch.int32), dy, 2.0)
    assert not dt.any()


def test_what_is_not_a_number_stays_in_its_row():
    table, ids, dy = inputs(F32, torch.int64, 500, 50, 20, 3, 0.2)
    dy[(ids < 0) | (ids >= 50)] = float("nan")
    compare(table, ids, dy, 1.0)
    dy[ids == 7] = float("inf")
    dt = G.gconv_embed_bwd(dy.cuda(), ids.cuda(), 50).cpu()
    assert not torch.isfinite(dt[7]).any() and torch.isfinite(dt[[i for i in range(50) if i != 7]]).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    table, ids, dy = inputs(dtype, torch.int64, 90, 30, 21, 5)
    wide = torch.zeros(3, 30, 50, dtype=dtype, device="cuda")
    wide[..., 9:30] = dy.view(3, 30, 21).cuda()
    compare(table, ids, dy, 0.5, shape=(3, 30), dy_gpu=wide[..., 9:30])
    swapped = dy.view(3, 30, 21).transpose(0, 1).contiguous().cuda().transpose(0, 1)
    compare(table, ids, dy, 0.5, shape=(3, 30), dy_gpu=swapped)
    # one gradient for every token
    compare(table, ids, dy[:1].expand(90, 21).contiguous(), 0.5, dy_gpu=dy[:1].cuda().expand(90, 21))


def test_two_runs_are_equal_and_a_graph_replays():
    table, ids, dy = inputs(BF, torch.int64, 9000, 700, 136, 8, 0.1)
    ids[::2] = 3
    dy, ids = dy.cuda(), ids.cuda()
    first = G.gconv_embed_bwd(dy, ids, 700)
    with torch.cuda.stream(torch.cuda.Stream()):
        G.gconv_embed_bwd(dy, ids, 700)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.gconv_embed_bwd(dy, ids, 700)
    for _ in range(3):
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(G.gconv_embed_bwd(dy, ids, 700), first)
