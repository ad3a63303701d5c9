"""The selective state space scan against its 64-bit definition: forward, gradients, single tokens."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
WIDE, NARROW = ("u", "dt", "gate", "dy"), ("b", "c")


def inputs(dtype, lens, dim, states, groups=1, gate=True, skip=True, bias=True, held=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    n = lambda *s, std=1.0, t=F32: (torch.randn(*s, generator=gen) * std).to(t)  # noqa: E731
    s = {k: n(T, dim, t=dtype) for k in WIDE}
    s.update({k: n(T, groups, states, t=dtype) for k in NARROW})
    s["a"] = -torch.exp(n(dim, states, std=0.7)) * torch.arange(1, states + 1)
    s["skip"], s["dt_bias"] = n(dim) if skip else None, n(dim, std=0.5) - 3 if bias else None
    if not gate:
        s["gate"] = None
    s["init"], s["dfinal"] = (n(N, dim, states) if held else None for _ in range(2))
    return s


def cuda(t):
    return t.cuda() if t is not None else None


def reference(s, lens, softplus):
    one = lambda **k: R.scan(k["u"], k["dt"], s["a"], k["b"], k["c"], s["skip"], k["gate"], s["dt_bias"], softplus, k["init"],  # noqa: E731
                             k["dy"], k["dfinal"])
    return R.sequences(one, lens, {k: s[k] for k in WIDE + NARROW}, {"init": s["init"], "dfinal": s["dfinal"]}, ("da", "dskip", "ddt_bias"))


def compare(s, lens, packed, softplus=True, **given):
    want = reference(s, lens, softplus)
    lead = (sum(lens),) if packed else (len(lens), lens[0])
    t = {k: (s[k].unflatten(0, lead) if not packed else s[k]).cuda() if s[k] is not None else None for k in WIDE + NARROW}
    t.update(given)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda() if packed else None
    kw = dict(skip=cuda(s["skip"]), gate=t["gate"], dt_bias=cuda(s["dt_bias"]), softplus=softplus, cu_seqlens=cu, initial_state=cuda(s["init"]))
    args = (t["u"], t["dt"], s["a"].cuda(), t["b"], t["c"])
    y, final = G.gconv_scan_fwd(*args, **kw)
    got = G.gconv_scan_bwd(t["dy"], *args, d_final_state=cuda(s["dfinal"]), **kw)
    flat = lambda v, like: v.reshape(like.shape)  # noqa: E731
    R.check("y", flat(y, want["y"][0]), *want["y"])
    R.check("final", final, *want["final"])
    for name, v in zip(("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit"), got):
        if v is not None:
            R.check(name, flat(v, want[name][0]), *want[name])
    for i, k in ((5, "skip"), (6, "gate"), (7, "dt_bias"), (8, "init")):
        assert (got[i] is None) == (s[k] is None)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("states", [1, 3, 4, 5, 8, 13, 16, 17, 32, 50, 64])
def test_states(dtype, states):
    lens = [35] * 2
    compare(inputs(dtype, lens, 70, states, seed=states), lens, False)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("dim,groups", [(1, 1), (2, 2), (63, 1), (64, 1), (130, 1), (130, 2), (256, 4)])
@pytest.mark.parametrize("length", [1, 7, 16, 65, 150])
def test_sizes(dtype, dim, groups, length):
    lens = [length] * 2
    compare(inputs(dtype, lens, dim, 6, groups, seed=dim + length), lens, False)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("skip,bias,held", [(False, False, False), (True, False, True), (False, True, False)])
@pytest.mark.parametrize("softplus", [False, True])
def test_what_may_be_absent(gate, skip, bias, held, softplus):
    lens = [70]
    s = inputs(F32, lens, 33, 5, gate=gate, skip=skip, bias=bias, held=held, seed=4)
    if not softplus:
        s["dt"] = s["dt"].abs() * 0.2  # steps are positive, or the state grows without end
        s["dt_bias"] = s["dt_bias"].abs() * 0.1 if bias else None
    compare(s, lens, False, softplus)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [0, 3, 0], [1, 1, 2, 0, 1, 15, 1], [130, 0, 64, 1, 7, 33, 2], [16, 16, 48, 8]])
def test_packed(dtype, lens):
    for held in (False, True):
        compare(inputs(dtype, lens, 40, 16, 2, held=held, seed=len(lens)), lens, True)


@pytest.mark.parametrize("lens", [[0], [0, 0, 0]])
def test_sequences_without_tokens(lens):
    s = inputs(F32, lens, 10, 4)
    compare(s, lens, True)
    u = torch.zeros(len(lens), 0, 10, device="cuda")
    b = torch.zeros(len(lens), 0, 1, 4, device="cuda")
    y, final = G.gconv_scan_fwd(u, u, s["a"].cuda(), b, b, initial_state=s["init"].cuda())
    assert y.shape == u.shape and torch.equal(final.cpu(), s["init"])


def test_tokens_of_no_sequence_are_not_read():
    lens, D, S = [20, 0, 45], 70, 16
    s = inputs(F32, lens, D, S, seed=8)
    want = reference(s, lens, True)
    T = 5 + sum(lens) + 130
    t = {}
    for k in WIDE + NARROW:
        t[k] = torch.full((T,) + s[k].shape[1:], float("nan"))
        t[k][5:70] = s[k]
        t[k] = t[k].cuda()
    cu = (torch.tensor([0] + lens).cumsum(0) + 5).to(torch.int32).cuda()
    kw = dict(skip=s["skip"].cuda(), gate=t["gate"], dt_bias=s["dt_bias"].cuda(), cu_seqlens=cu, initial_state=s["init"].cuda())
    args = (t["u"], t["dt"], s["a"].cuda(), t["b"], t["c"])
    y, final = G.gconv_scan_fwd(*args, **kw)
    got = dict(zip(("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit"),
                   G.gconv_scan_bwd(t["dy"], *args, d_final_state=s["dfinal"].cuda(), **kw)))
    R.check("final", final, *want["final"])
    got["y"] = y
    for name, v in got.items():
        if name in ("y", "du", "ddt", "dgate", "db", "dc"):
            assert not v[:5].any() and not v[70:].any(), name
            v = v[5:70]
        R.check(name, v, *want[name])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides(dtype):
    """Slices of one projection at odd places, and time-major gradients."""
    lens, D, S, g = [50] * 3, 66, 7, 2
    s = inputs(dtype, lens, D, S, g, seed=6)
    row = torch.zeros(3, 50, 3 + 2 * D + 2 * g * S + 1, dtype=dtype, device="cuda")
    given, at = {}, 3
    for k in ("u", "gate", "b", "c"):
        size = D if k in WIDE else g * S
        view = row[..., at:at + size]
        view.copy_(s[k].reshape(3, 50, size).cuda())
        given[k] = view if k in WIDE else view.unflatten(-1, (g, S))
        at += size
    given["dy"] = s["dy"].view(3, 50, D).transpose(0, 1).contiguous().cuda().transpose(0, 1)
    compare(s, lens, False, **given)


def test_chunks_agree_with_one_run():
    """A sequence long enough to be cut into chunks, narrow enough that it has to be."""
    lens = [2100]
    compare(inputs(F32, lens, 8, 4, seed=12), lens, False)


def test_strong_and_no_decay():
    """Decays that leave nothing, none at all, and steps past float32's exponentials."""
    lens = [90]
    s = inputs(F32, lens, 20, 4, gate=False, seed=13)
    s["a"][:, 0], s["a"][:, 1], s["a"][:, 2] = 0.0, -1e4, -float("inf")
    s["dt"][:, 3], s["dt"][:, 4], s["dt"][:, 5] = -200.0, -40.0, 30.0
    s["dt_bias"][:] = 0.0
    s["init"], s["dfinal"] = None, None
    want = reference({**s, "a": s["a"].clamp(min=-1e30)}, lens, True)
    kw = dict(skip=s["skip"].cuda(), dt_bias=s["dt_bias"].cuda())
    y, final = G.gconv_scan_fwd(s["u"][None].cuda(), s["dt"][None].cuda(), s["a"].cuda(), s["b"][None].cuda(), s["c"][None].cuda(), **kw)
    # (channel 3's steps are 0 in float32 and 1e-87 in 64 bits, which decays of 1e30 tell apart)
    keep = [i for i in range(20) if i != 3]
    R.check("y", y[0][:, keep], want["y"][0][:, keep], want["y"][1][:, keep])
    R.check("final", final[:, keep], want["final"][0][:, keep], want["final"][1][:, keep])
    got = dict(zip(("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit"),
                   G.gconv_scan_bwd(s["dy"][None].cuda(), s["u"][None].cuda(), s["dt"][None].cuda(), s["a"].cuda(), s["b"][None].cuda(),
                                    s["c"][None].cuda(), **kw)))
    for name in ("du", "ddt"):
        R.check(name, got[name][0][:, keep], want[name][0][:, keep], want[name][1][:, keep])
    R.check("da", got["da"][keep], want["da"][0][keep], want["da"][1][keep])


def test_infinite_decay_in_packed_chunks():
    """Nothing of the state is left by any token, through chunks that end in tokens of no sequence."""
    lens = [100, 0, 190]
    s = inputs(F32, lens, 20, 4, seed=21)
    s["a"][:, 1], s["a"][::3] = -float("inf"), -float("inf")
    T, at = 3 + sum(lens) + 200, slice(3, 293)
    want = reference({**s, "a": s["a"].clamp(min=-1e30)}, lens, True)
    t = {k: torch.zeros((T,) + s[k].shape[1:]) for k in WIDE + NARROW}
    for k in t:
        t[k][at] = s[k]
        t[k] = t[k].cuda()
    cu = (torch.tensor([0] + lens).cumsum(0) + 3).to(torch.int32).cuda()
    kw = dict(skip=s["skip"].cuda(), gate=t["gate"], dt_bias=s["dt_bias"].cuda(), cu_seqlens=cu, initial_state=s["init"].cuda())
    args = (t["u"], t["dt"], s["a"].cuda(), t["b"], t["c"])
    y, final = G.gconv_scan_fwd(*args, **kw)
    R.check("y", y[at], *want["y"])
    R.check("final", final, *want["final"])
    got = dict(zip(("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit"),
                   G.gconv_scan_bwd(t["dy"], *args, d_final_state=s["dfinal"].cuda(), **kw)))
    for name, v in got.items():
        R.check(name, v[at] if name in ("du", "ddt", "db", "dc", "dgate") else v, *want[name])


def test_what_is_not_a_number_stays_in_its_channel_and_time():
    s = inputs(F32, [60], 130, 8, seed=14)
    t = {k: s[k][None].cuda() for k in WIDE + NARROW}
    t["u"][0, 30, 70] = float("nan")
    y, final = G.gconv_scan_fwd(t["u"], t["dt"], s["a"].cuda(), t["b"], t["c"], gate=t["gate"])
    off = ~torch.isfinite(y.cpu())[0]
    assert off[30:, 70].all() and int(off.sum()) == 30
    assert int((~torch.isfinite(final.cpu())).sum()) == 8


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("states,groups", [(1, 1), (6, 2), (16, 1), (40, 4), (64, 1)])
def test_steps(dtype, states, groups):
    """A prompt's state and then tokens one by one, against the definition of the whole."""
    B, T, D = 3, 9, 4 * groups * 7
    s = inputs(dtype, [T] * B, D, states, groups, held=False, seed=states)
    want = reference(s, [T] * B, True)
    t = {k: s[k].unflatten(0, (B, T)).cuda() for k in WIDE + NARROW}
    kw = dict(skip=s["skip"].cuda(), dt_bias=s["dt_bias"].cuda())
    a = s["a"].cuda()
    _, state = G.gconv_scan_fwd(t["u"][:, :4], t["dt"][:, :4], a, t["b"][:, :4], t["c"][:, :4], gate=t["gate"][:, :4], **kw)
    pool = torch.full((7, D, states), 3.0, device="cuda")
    slots = torch.tensor([6, 1, 3], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    y = torch.stack([G.gconv_scan_step(t["u"][:, i], t["dt"][:, i], a, t["b"][:, i], t["c"][:, i], pool, gate=t["gate"][:, i], slots=slots, **kw)
                     for i in range(4, T)], 1)
    pick = lambda v: v.unflatten(0, (B, T))[:, 4:]  # noqa: E731
    R.check("y", y, pick(want["y"][0]), pick(want["y"][1]))
    R.check("state", pool[slots.long()], *want["final"])
    assert (pool[[0, 2, 4, 5]] == 3).all()


def test_step_of_idle_rows_and_many():
    """More sequences than a workgroup takes one after another, some of them idle."""
    B, D, S = 700, 48, 16
    s = inputs(F32, [1] * B, D, S, held=True, seed=1)
    args = [s["u"].cuda(), s["dt"].cuda(), s["a"].cuda(), s["b"].cuda(), s["c"].cuda()]
    pool = s["init"].cuda()
    slots = torch.arange(B, dtype=torch.int32)
    slots[::7] = -1
    before = pool.clone()
    y = G.gconv_scan_step(*args, pool, gate=s["gate"].cuda(), slots=slots.cuda())
    ref, final = G.gconv_scan_fwd(*[v[:, None] if v.shape[0] == B else v for v in args], gate=s["gate"][:, None].cuda(), initial_state=before)
    idle = slots < 0
    assert not y[idle.cuda()].any() and torch.equal(pool[idle.cuda()], before[idle.cuda()])
    live = ~idle.cuda()
    assert (y[live] - ref[live, 0]).abs().max() <= 1e-5 * ref.abs().max()
    assert (pool[live] - final[live]).abs().max() <= 1e-6 * final.abs().max()


def test_two_runs_are_equal_and_a_graph_replays():
    lens = [300, 0, 77]
    s = inputs(BF, lens, 200, 16, seed=9)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    t = {k: cuda(v) for k, v in s.items()}
    kw = dict(skip=t["skip"], gate=t["gate"], dt_bias=t["dt_bias"], cu_seqlens=cu, initial_state=t["init"])
    args = (t["u"], t["dt"], t["a"], t["b"], t["c"])

    def both():
        return G.gconv_scan_fwd(*args, **kw) + G.gconv_scan_bwd(t["dy"], *args, d_final_state=t["dfinal"], **kw)

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
