"""The selective scan with decay rates that leave nothing of a state, next to steps of 0 that leave all of it."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402
import token_ref as R  # noqa: E402
from test_gpu_scan import NARROW, WIDE, inputs, reference  # noqa: E402

NAMES = ("du", "ddt", "da", "db", "dc", "dskip", "dgate", "ddt_bias", "dinit")


def run(s, cu):
    t = {k: v.cuda() if v is not None else None for k, v in s.items()}
    kw = dict(skip=t["skip"], gate=t["gate"], dt_bias=t["dt_bias"], cu_seqlens=cu, initial_state=t["init"])
    args = [t[k] for k in ("u", "dt", "a", "b", "c")]
    y, final = G.gconv_scan_fwd(*args, **kw)
    out = dict(zip(NAMES, G.gconv_scan_bwd(t["dy"], *args, d_final_state=t["dfinal"], **kw)))
    out.update(y=y, final=final)
    return out


def skipped(rate, seed):
    """Packed sequences with some channels' and states' rates at `rate`, and tokens whose step is 0 in float32 (1e-87
    in 64 bits): the state goes through them, and with it its gradient, large ones among them."""
    lens = [70, 0, 45]
    s = inputs(torch.float32, lens, 20, 4, seed=seed)
    s["a"][:, 1], s["a"][::3] = rate, rate
    s["dt_bias"][:] = 0.0
    for at in (0, 3, 4, 40, 69, 70, 90, 114):
        s["dt"][at] = -200.0
    s["init"] *= 50
    s["dfinal"] *= 50
    return s, lens


def against_definition(s, lens):
    # (in 64 bits a rate of -1e30 leaves nothing after a step that float32 holds, and all after one of 1e-87)
    want = reference({**s, "a": s["a"].clamp(min=-1e30)}, lens, True)
    got = run(s, torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda())
    for name, v in got.items():
        R.check(name, v, *want[name])


def test_steps_of_zero_under_an_infinite_decay():
    s, lens = skipped(-float("inf"), 31)
    against_definition(s, lens)


@pytest.mark.parametrize("rate", [-2.4e38, -3e38, torch.finfo(torch.float32).min])
def test_rates_at_the_end_of_float32(rate):
    """Times log2(e) such a rate is past float32: it counts as -infinity."""
    s, lens = skipped(rate, 32)
    against_definition(s, lens)


@pytest.mark.parametrize("rate", [-3e38, torch.finfo(torch.float32).min, -float("inf")])
def test_rates_at_the_end_of_float32_one_token(rate):
    """... and in a step, where a token of step 0 leaves the state as it was and another leaves nothing of it."""
    gen = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    u, b, c, state = n(3, 10), n(3, 1, 4), n(3, 1, 4), n(3, 10, 4)
    dt = torch.tensor([-200.0, 0.5, -200.0], device="cuda")[:, None].expand(3, 10).contiguous()
    before = state.clone()
    G.gconv_scan_step(u, dt, torch.full((10, 4), rate, device="cuda"), b, c, state)
    assert torch.equal(state[[0, 2]], before[[0, 2]])
    step = torch.log1p(torch.exp(torch.tensor(0.5, dtype=torch.float64)))
    want = step * (u[1, :, None] * b[1]).double().cpu()
    R.check("state", state[1], want, 12 * R.U * want.abs())
