"""The short causal convolution against its 64-bit definition: forward, gradients, single tokens."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


def rand(gen, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).to(dtype)


def inputs(dtype, lens, dim, taps, bias, states, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    return dict(x=rand(gen, T, dim, dtype=dtype), w=rand(gen, dim, taps, dtype=dtype, std=taps ** -0.5),
                bias=rand(gen, dim, dtype=dtype, std=0.3) if bias else None, dy=rand(gen, T, dim, dtype=dtype),
                init=rand(gen, N, taps - 1, dim, dtype=dtype) if states else None,
                dfinal=rand(gen, N, taps - 1, dim, dtype=dtype) if states else None)


def cuda(t):
    return t.cuda() if t is not None else None


def reference(s, lens, act):
    one = lambda **k: R.shortconv(k["x"], s["w"], s["bias"], act, k["init"], k["dy"], k["dfinal"])  # noqa: E731
    return R.sequences(one, lens, {"x": s["x"], "dy": s["dy"]}, {"init": s["init"], "dfinal": s["dfinal"]}, ("dw", "dbias"))


def compare(s, lens, act, packed, x=None, dy=None):
    want = reference(s, lens, act)
    N, D = len(lens), s["x"].shape[1]
    shape = (sum(lens), D) if packed else (N, lens[0], D)
    x = s["x"].view(shape).cuda() if x is None else x
    dy = s["dy"].view(shape).cuda() if dy is None else dy
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if packed else None
    kw = dict(act=act, cu_seqlens=cu, initial_state=cuda(s["init"]))
    y, final = G.gconv_shortconv_fwd(x, s["w"].cuda(), cuda(s["bias"]), **kw)
    got = G.gconv_shortconv_bwd(dy, x, s["w"].cuda(), cuda(s["bias"]), d_final_state=cuda(s["dfinal"]), **kw)
    assert y.shape == x.shape and got[0].shape == x.shape
    R.check("y", y.reshape(-1, D), *want["y"])
    assert torch.equal(final.cpu().double(), want["final"][0])
    for name, v in zip(("dx", "dw", "dbias", "dinit"), got):
        if v is not None:
            R.check(name, v.reshape(want[name][0].shape), *want[name])
    assert (got[2] is None) == (s["bias"] is None) and (got[3] is None) == (s["init"] is None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("taps", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("act", ["none", "sigmoid", "silu"])
def test_taps_and_activations(dtype, taps, act):
    lens = [37] * 3
    compare(inputs(dtype, lens, 40, taps, True, True, taps), lens, act, False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dim", [1, 3, 8, 13, 64, 129, 520])
@pytest.mark.parametrize("length", [1, 2, 3, 5, 66])
def test_sizes(dtype, dim, length):
    lens = [length] * 2
    compare(inputs(dtype, lens, dim, 4, dim % 2 == 0, length % 2 == 0, dim), lens, "silu", False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [0, 1, 0], [1, 1, 1, 2, 0, 3, 1], [130, 0, 64, 1, 7, 200, 2], [0, 0]])
def test_packed(dtype, lens):
    for states in (False, True):
        compare(inputs(dtype, lens, 24, 4, True, states, len(lens)), lens, "silu", True)


def test_tokens_of_no_sequence_are_not_read():
    gen = torch.Generator().manual_seed(3)
    lens, D, K = [5, 0, 9], 20, 3
    s = inputs(F32, lens, D, K, True, True, 5)
    want = reference(s, lens, "silu")
    T = 3 + sum(lens) + 6
    x, dy = torch.full((T, D), float("nan")), torch.full((T, D), float("inf"))
    x[3:17], dy[3:17] = s["x"], s["dy"]
    cu = (torch.tensor([0] + lens).cumsum(0) + 3).to(torch.int32).cuda()
    kw = dict(act="silu", cu_seqlens=cu, initial_state=s["init"].cuda())
    y, final = G.gconv_shortconv_fwd(x.cuda(), s["w"].cuda(), s["bias"].cuda(), **kw)
    dx, dw, db, di = G.gconv_shortconv_bwd(dy.cuda(), x.cuda(), s["w"].cuda(), s["bias"].cuda(), d_final_state=s["dfinal"].cuda(), **kw)
    R.check("y", y[3:17], *want["y"])
    R.check("dx", dx[3:17], *want["dx"])
    for t in (y, dx):
        assert not t[:3].any() and not t[17:].any()
    R.check("dw", dw, *want["dw"])
    R.check("dbias", db, *want["dbias"])
    R.check("dinit", di, *want["dinit"])
    assert torch.equal(final.cpu().double(), want["final"][0])
    del gen


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Slices of wider tensors at odd places, time-major ones, and a row that repeats."""
    lens, D = [21] * 3, 30
    s = inputs(dtype, lens, D, 4, True, False, 2)
    wide = torch.zeros(3, 21, 2 * D + 7, dtype=dtype, device="cuda")
    wide[..., 5:5 + D] = s["x"].view(3, 21, D).cuda()
    swapped = s["dy"].view(3, 21, D).transpose(0, 1).contiguous().cuda().transpose(0, 1)
    compare(s, lens, "silu", False, x=wide[..., 5:5 + D], dy=swapped)
    s["dy"] = s["dy"][:1].expand(63, D).contiguous()
    compare(s, lens, "silu", False, dy=s["dy"][:1].cuda().expand(3, 21, D))


def test_an_input_reaches_its_taps_alone():
    x = torch.randn(1, 40, 16)
    x[0, 20, 3] = float("inf")
    w = torch.randn(16, 4)
    y, _ = G.gconv_shortconv_fwd(x.cuda(), w.cuda(), act="none")
    off = ~torch.isfinite(y.cpu())
    assert off[0, 20:24, 3].all() and int(off.sum()) == 4


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("taps", [1, 2, 4, 8])
def test_steps_go_on_as_the_whole(dtype, taps):
    """A prompt's state and then tokens one by one give what the whole sequence gives, bit by bit."""
    gen = torch.Generator().manual_seed(taps)
    B, T, D = 5, 12, 70
    x, w, bias = rand(gen, B, T, D, dtype=dtype).cuda(), rand(gen, D, taps, dtype=dtype).cuda(), rand(gen, D, dtype=dtype).cuda()
    whole, last = G.gconv_shortconv_fwd(x, w, bias)
    _, state = G.gconv_shortconv_fwd(x[:, :7], w, bias)
    pool = torch.full((9, taps - 1, D), 7.0, dtype=dtype, device="cuda")
    slots = torch.tensor([8, 2, 0, 5, 4], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(7, T):
        assert torch.equal(G.gconv_shortconv_step(x[:, t], w, pool, bias, slots=slots), whole[:, t])
    assert torch.equal(pool[slots.long()], last)
    assert (pool[[1, 3, 6, 7]] == 7).all()


def test_step_of_idle_rows():
    x, w = torch.randn(4, 33, device="cuda"), torch.randn(33, 3, device="cuda")
    pool = torch.randn(3, 2, 33, device="cuda")
    before = pool.clone()
    y = G.gconv_shortconv_step(x, w, pool, slots=torch.tensor([-1, 1, 3, 1 << 30], dtype=torch.int32, device="cuda"))
    assert not y[[0, 2, 3]].any() and y[1].any()
    assert torch.equal(pool[[0, 2]], before[[0, 2]]) and torch.equal(pool[1, 0], before[1, 1]) and torch.equal(pool[1, 1], x[1])


def test_two_runs_are_equal_and_a_graph_replays():
    s = inputs(BF, [300, 77], 264, 4, True, True, 9)
    cu = torch.tensor([0, 300, 377], dtype=torch.int32, device="cuda")
    args = [s[k].cuda() for k in ("dy", "x", "w", "bias")]
    kw = dict(cu_seqlens=cu, initial_state=s["init"].cuda(), d_final_state=s["dfinal"].cuda())
    first = G.gconv_shortconv_bwd(*args, **kw)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        G.gconv_shortconv_bwd(*args, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = G.gconv_shortconv_bwd(*args, **kw)
    for _ in range(3):
        for t in out:
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, first):
            assert torch.equal(a, b)
        assert torch.equal(G.gconv_shortconv_bwd(*args, **kw)[1], first[1])
