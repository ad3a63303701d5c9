"""The sequence operators where offsets pass 2^31 elements and 2^32 bytes, and with very many heads:
the answers are those of the same rows in small tensors."""
from __future__ import annotations

import pytest

from seq_ref import F64, orthogonalize

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def normal(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("pitch", [1 << 21, (1 << 21) + 3])  # rows on 16 bytes, and on none
def test_linattn_rows_far_apart(pitch):
    """Tokens 4 MB apart, 9 GB in all."""
    T, H, Hk, dk, dv = 2200, 4, 2, 64, 32
    wide = torch.empty(T, pitch, dtype=torch.bfloat16, device="cuda")
    row = normal(1, T, H * dk + Hk * (dk + dv))
    wide[:, 8:8 + row.shape[1]] = row
    far = wide[:, 8:8 + row.shape[1]]
    do = normal(2, T, H, dv)
    g = torch.tensor([-0.5, -0.1, -0.02, -0.004]).cuda()
    cu = torch.tensor([0, 900, 2200], dtype=torch.int32).cuda()
    state = normal(3, 2, H, dk, dv, dtype=torch.float32)
    print("linattn far", pitch, flush=True)

    def call(p):
        q, k, v = (p[:, a:b].unflatten(-1, (h, d)) for a, b, h, d in (
            (0, H * dk, H, dk), (H * dk, (H + Hk) * dk, Hk, dk), ((H + Hk) * dk, row.shape[1], Hk, dv)))
        kw = dict(cu_seqlens=cu, initial_state=state)
        return G.gconv_linattn_fwd(q, k, v, g, **kw) + G.gconv_linattn_bwd(do, q, k, v, g, **kw)

    assert all(torch.equal(a, b) for a, b in zip(call(far), call(row)))


@pytest.mark.parametrize("heads", [600, 1000])
def test_linattn_many_heads(heads):
    """More heads than workgroups that the plan aims at: a segment is a whole sequence, or several's length."""
    q, k, v, do = (normal(i, 3, 200, 1, 16).repeat(1, 1, heads, 1) for i in range(4))
    g = torch.full((heads,), -0.1).cuda()
    print("linattn heads", heads, flush=True)
    got = G.gconv_linattn_fwd(q, k, v, g) + G.gconv_linattn_bwd(do, q, k, v, g)[:3]
    one = [t[:, :, :1].contiguous() for t in (q, k, v, do)]
    want = G.gconv_linattn_fwd(*one[:3], g[:1]) + G.gconv_linattn_bwd(one[3], *one[:3], g[:1])[:3]
    for a, b in zip(got, want):
        axis = 1 if a.dtype == torch.float32 else 2
        assert torch.equal(a, a.narrow(axis, 0, 1).expand_as(a))
        # other segments: the terms in another order
        off = (a.narrow(axis, 0, 1) - b).double().norm() / b.double().norm()
        assert off <= 3 * 2.0 ** -8, off


@pytest.mark.parametrize("type_", [torch.float32, torch.bfloat16])
def test_step_in_a_large_pool(type_):
    """66000 states of 4 heads of 128 x 128: 17 GB."""
    pool, H, d = 66000, 4, 128
    state = torch.empty(pool, H, d, d, device="cuda")
    slots = torch.tensor([pool - 1, 0, 33001, 65536], dtype=torch.int32).cuda()
    few = normal(4, 4, H, d, d, dtype=torch.float32)
    state[slots.long()] = few
    q, k, v = (normal(5 + i, 4, H, d, dtype=type_) for i in range(3))
    g = torch.full((H,), -0.2).cuda()
    print("step far", type_, flush=True)
    a = G.gconv_linattn_step(q, k, v, g, state, slots=slots)
    b = G.gconv_linattn_step(q, k, v, g, few)
    assert torch.equal(a, b) and torch.equal(state[slots.long()], few)


@pytest.mark.parametrize("gate", ["full", "sequence"])
def test_norm_of_many_rows(gate):
    """2^24 + 256 rows of 128: each row's answers are those of the same row in a short call."""
    block, times, D = 65537, 256, 128  # 2^24 + 256 rows, a block a sequence
    t = {n: normal(i, 1, block, D) for i, n in enumerate(("x", "b", "z", "dy", "dh"))}
    w1, sc, w2 = (normal(9 + i, D) for i in range(3))
    if gate == "sequence":
        t["z"] = t["z"][:, :1].contiguous()
    print("norm far", gate, flush=True)

    def call(t):
        kw = dict(gate=t["z"], w_post=w1, scale=sc, w_pre=w2)
        return G.gconv_normgate_fwd(t["x"], t["b"], **kw) + G.gconv_normgate_bwd(t["dy"], t["dh"], t["x"], t["b"], **kw)[:3]

    small = call(t)
    large = call({n: v.repeat(times, 1, 1) for n, v in t.items()})
    for i, (a, b) in enumerate(zip(large, small)):
        if gate == "sequence" and i == 4:  # the sum over a sequence's tokens: in another order
            off = (a.double() - b.double()).norm(dim=-1) / b.double().norm()
            assert off.max() <= 2.0 ** -7, off.max()
            continue
        assert all(torch.equal(a[j], b[0]) for j in range(times)), i


@pytest.mark.parametrize("groups,m,n", [(65536, 64, 640), (36000, 200, 320)])
def test_ortho_of_many_groups(groups, m, n):
    """Of few rows by several workgroups each, and by the general kernels: over 2^31 elements."""
    base = normal(1, 16, m, n, dtype=torch.float32)
    u = base.repeat(groups // 16, 1, 1).view(groups * m, n)
    print("ortho far", groups, m, n, flush=True)
    got = G.gconv_orthogonalize(u, groups=groups).view(groups // 16, 16, m, n)
    del u
    assert all(torch.equal(got[i], got[0]) for i in range(0, groups // 16, 97)) and torch.equal(got[-1], got[0])
    for j in (0, 15):
        want = orthogonalize(base[j].cpu(), 1, 5, 1e-7)
        assert float((got[-1, j].cpu().to(F64) - want).norm() / want.norm()) <= 5e-3 + 2.0 ** -8
