"""The token operators where offsets pass 2^31 elements: the far end against the same call on its own."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

BF = torch.bfloat16


def close(got, want, dtype):
    assert (got.float() - want.float()).abs().max() <= torch.finfo(dtype).eps * 4 * want.float().abs().max()


def rows(n, d, seed, dtype=BF):
    """n x d values without a 32-bit copy of all of them: 4099 random rows, over and over."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    few = torch.randn(4099, d, generator=gen, device="cuda").to(dtype)
    return few.repeat(-(-n // 4099), 1)[:n]


def test_shortconv():
    T, D, cut = 263000, 8192, 262900
    x, w = rows(T, D, 1), torch.randn(D, 4, device="cuda").to(BF)
    y, final = G.gconv_shortconv_fwd(x[None], w)
    own, last = G.gconv_shortconv_fwd(x[None, cut:], w)
    assert torch.equal(y[0, cut + 3:], own[0, 3:]) and torch.equal(final, last)
    dx, _, _, _ = G.gconv_shortconv_bwd(y, x[None], w)
    part, _, _, _ = G.gconv_shortconv_bwd(y[:, cut:], x[None, cut:], w)
    assert torch.equal(dx[0, cut + 3:], part[0, 3:])


def test_scan():
    T, D, S, cut = 530000, 4096, 2, 529800
    u = rows(T, D, 2)[None]
    b = rows(T, S, 3)[None, :, None]
    a = -torch.ones(D, S, device="cuda") * torch.tensor([1.0, 2.0], device="cuda")
    _, start = G.gconv_scan_fwd(u[:, :cut], u[:, :cut], a, b[:, :cut], b[:, :cut])
    y, final = G.gconv_scan_fwd(u, u, a, b, b)
    own, last = G.gconv_scan_fwd(u[:, cut:], u[:, cut:], a, b[:, cut:], b[:, cut:], initial_state=start)
    close(y[0, cut:], own[0], BF)
    close(final, last, BF)
    du, ddt = G.gconv_scan_bwd(y, u, u, a, b, b)[:2]
    own = G.gconv_scan_bwd(y[:, cut:], u[:, cut:], u[:, cut:], a, b[:, cut:], b[:, cut:], initial_state=start)
    close(du[0, cut:], own[0][0], BF)
    close(ddt[0, cut:], own[1][0], BF)


def test_steps():
    slots, D, S = 40000, 4096, 16
    state = torch.zeros(slots, D, S, device="cuda")
    state[-3:] = torch.randn(3, D, S, device="cuda")
    own = state[-3:].clone()
    u, b = torch.randn(3, D, device="cuda"), torch.randn(3, 1, S, device="cuda")
    a = -torch.rand(D, S, device="cuda")
    y = G.gconv_scan_step(u, u, a, b, b, state, slots=torch.arange(slots - 3, slots, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, G.gconv_scan_step(u, u, a, b, b, own)) and torch.equal(state[-3:], own)
    pool = torch.zeros(180000, 3, D, dtype=BF, device="cuda")
    pool[-2:] = torch.randn(2, 3, D, device="cuda").to(BF)
    own, x, w = pool[-2:].clone(), torch.randn(2, D, device="cuda").to(BF), torch.randn(D, 4, device="cuda").to(BF)
    y = G.gconv_shortconv_step(x, w, pool, slots=torch.tensor([179998, 179999], dtype=torch.int32, device="cuda"))
    assert torch.equal(y, G.gconv_shortconv_step(x, w, own)) and torch.equal(pool[-2:], own)


def test_embed():
    V, D = 1100000, 2048
    table = rows(V, D, 4)
    ids = torch.tensor([V - 1, 5, V - 2, V, V - 1], device="cuda")
    y = G.gconv_embed_fwd(table, ids)
    assert torch.equal(y[[0, 1, 2, 4]], table[ids[[0, 1, 2, 4]]]) and not y[3].any()
    dt = G.gconv_embed_bwd(y, ids, V)
    assert torch.equal(dt[V - 2], y[2]) and torch.equal(dt[V - 1].float(), (y[0].float() * 2).to(BF).float())
    assert int((dt != 0).any(1).sum()) == 3


def test_xent():
    V, D = 1100000, 2048
    w = rows(V, D, 5) * 0.02
    h, t = torch.randn(6, D, device="cuda").to(BF), torch.tensor([V - 1, 0, V - 700, 77, V - 1, -1], device="cuda")
    loss, lse = G.gconv_xent_fwd(h, w, t)
    # rows of w repeat: 4099 of them, the first V % 4099 once more often
    z = h.double() @ w[:4099].double().T
    times = torch.full((4099,), V // 4099, device="cuda", dtype=torch.float64)
    times[:V % 4099] += 1
    want = torch.logsumexp(z + times.log(), 1)
    assert (lse.double() - want).abs().max() <= 1e-4 and not loss[5]
    assert (loss[:5].double() - (want[:5] - z[torch.arange(5), t[:5] % 4099])).abs().max() <= 1e-4
    dl = torch.ones(6, device="cuda")
    dh, dw = G.gconv_xent_bwd(dl, h, w, t, lse)
    p = torch.exp(z - want[:, None])
    p[5] = 0
    dz = p * times
    dz[torch.arange(5), t[:5] % 4099] -= 1
    off = (dh.double() - dz @ w[:4099].double()).norm() / (dz @ w[:4099].double()).norm()
    assert off <= 4e-3
    for v, who in ((V - 1, [0, 4]), (V - 700, [2]), (V - 2, [])):
        own = p[:, v % 4099].clone()
        for i in who:
            own[i] -= 1
        want_row = own @ h.double()
        assert (dw[v].double() - want_row).norm() <= 1e-2 * want_row.norm()
