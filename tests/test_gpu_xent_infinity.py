"""The cross entropy of logits of +infinity next to large finite ones (bfloat16, whose infinities are kept)."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import grouped_convolution_amd as G  # noqa: E402

INF = float("inf")


@pytest.mark.parametrize("tokens,vocab", [(3, 600), (40, 600), (300, 9000), (5, 40000)])
@pytest.mark.parametrize("size", [0.5, 4.0, 1e30])
def test_an_infinite_logit_makes_lse_infinite(tokens, vocab, size):
    """Whichever column it is in, and however large the others are: 64 x about 0.9 x size."""
    gen = torch.Generator().manual_seed(vocab)
    h = (torch.randn(tokens, 64, generator=gen).abs() + 0.1).to(torch.bfloat16).cuda()
    for at in ([0], [vocab // 2], [vocab - 1], [3, vocab - 2]):
        w = torch.full((vocab, 64), size, dtype=torch.bfloat16, device="cuda")
        w[at] = INF
        targets = torch.full((tokens,), 5, device="cuda")
        loss, lse = G.gconv_xent_fwd(h, w, targets)
        assert (lse == INF).all() and (loss == INF).all(), at
        # the target's own logit infinite: infinity less infinity
        loss, lse = G.gconv_xent_fwd(h, w, torch.full((tokens,), at[0], device="cuda"))
        assert (lse == INF).all() and torch.isnan(loss).all(), at


def test_what_is_not_a_number_outweighs_infinity():
    h = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    for at in (1, 300, 599):
        w = torch.full((600, 64), 4.0, dtype=torch.bfloat16, device="cuda")
        w[299] = INF
        w[at] = float("nan")
        loss, lse = G.gconv_xent_fwd(h, w, torch.zeros(4, dtype=torch.int64, device="cuda"))
        assert torch.isnan(lse).all() and torch.isnan(loss).all(), at


def test_infinite_rows_leave_other_tokens_alone():
    """A token whose logits of those rows are -infinity: they add nothing to its sum."""
    gen = torch.Generator().manual_seed(3)
    h = (torch.randn(20, 64, generator=gen).abs() + 0.1).to(torch.bfloat16)
    h[7] = -h[7]
    w = torch.full((600, 64), 4.0, dtype=torch.bfloat16)
    w[100] = INF
    t = torch.zeros(20, dtype=torch.int64)
    loss, lse = G.gconv_xent_fwd(h.cuda(), w.cuda(), t.cuda())
    others = torch.arange(20) != 7
    assert (lse[others.cuda()] == INF).all()
    want = 4 * h[7].double().sum() + torch.tensor(599.0, dtype=torch.float64).log()
    # 64 terms of one sign summed in float32, and the sum of 599 exponentials
    assert abs(float(lse[7]) - float(want)) <= (64 + 8) * 2.0 ** -24 * abs(float(want)) + (40 + 600 ** 0.5) * 2.0 ** -24
