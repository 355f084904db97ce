"""Tokens drawn where a few hundred elements are kept, and where top-p's cut lies anywhere in a row, against the 64-bit reference."""
import pytest

import sampling_reference as ref
from test_gpu_sampling import KINDS, draw, logits_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("k", [255, 257, 600, 1023, 1024, 1025])
@pytest.mark.parametrize("V", [1024, 1027, 4100, 50257])
def test_some_hundreds(kind, k, V):
    x, u = logits_of(4, V, kind, seed=k + V)
    for settings in (dict(), dict(top_p=0.9), dict(min_p=0.01, top_p=0.5), dict(temperature=9.0, top_p=0.98), dict(temperature=0.02)):
        ref.check(x, u, draw(x, u, top_k=k, **settings), top_k=k, **settings)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("settings", [dict(top_k=300), dict(top_k=900, top_p=0.7), dict(top_p=0.6), dict(top_k=20, top_p=0.9)], ids=str)
def test_equal_values(kind, settings):
    # steps of 1/2 from a spread of 2: hundreds of equal values around every cut; then rows that are mostly masked
    import torch
    x, u = logits_of(6, 20011, kind, spread=2.0, seed=5, lift=False)
    x = (x.float() * 2).round().div(2)
    x[3:, ::3] = float("-inf")
    x[4, 700:] = float("-inf")
    x[5, :] = 1.5
    x = x.to(getattr(torch, kind))
    ref.check(x, u, draw(x, u, **settings), **settings)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("spread", [0.0, 2.0 ** -9, 0.5, 8.0, 100.0])
@pytest.mark.parametrize("V", [1500, 70001])
def test_share_anywhere(kind, spread, V):
    import torch
    x, u = logits_of(5, V, kind, spread=spread, seed=V, lift=False)
    p = torch.tensor([1e-6, 0.25, 0.75, 0.999999, 1 - 2.0 ** -24])
    for settings in (dict(), dict(top_k=V // 2), dict(min_p=0.2), dict(temperature=0.3, top_k=V - 1, min_p=1e-5)):
        ref.check(x, u, draw(x, u, top_p=p, **settings), top_p=p, **settings)


def test_long_slices_of_many_rows():
    # one CTA a row: the longest slices, and the coarsest rough weights
    x, u = logits_of(640, 90001, "bfloat16", spread=1.0, seed=3, lift=False)
    rows = range(0, 640, 61)
    for settings in (dict(top_p=0.9), dict(top_k=1000), dict(top_k=30000, top_p=0.8)):
        ref.check(x, u, draw(x, u, **settings), rows=rows, **settings)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("settings", [dict(top_k=1), dict(top_p=0.0), dict(top_k=700, top_p=1e-9), dict(min_p=1.0), dict(temperature=1e-3)], ids=str)
def test_a_single_token_is_certain(kind, settings):
    # the largest stands alone: its probability is 1, so its logarithm is 0 and nothing near it
    x, u = logits_of(7, 9001, kind, seed=11, lift=False)
    x[:, 4321] = 40.0
    token, logp = draw(x, u, **settings)
    assert token.tolist() == [4321] * 7
    assert logp.tolist() == [0.0] * 7


@pytest.mark.parametrize("settings", [dict(), dict(top_k=5), dict(top_p=1 - 2.0 ** -24)], ids=str)
def test_nearly_certain_tokens(settings):
    # ln of a share near 1 to as many bits as fp32 has: what is left weighs w with w right to 2^-30.5, its quotient and
    # log1p are off by 2^-23 at most, so 2^-22 of the result is allowed (and units of 2^-43 for each of the three others)
    import torch
    B = 6
    x = torch.full((B, 3000), -float("inf"))
    gap = torch.tensor([6.0, 8.0, 10.0, 13.0, 16.0, 20.0])
    x[:, 17], x[:, 1500], x[:, 2999], x[:, 18] = gap, 0.0, -1.0, -0.5
    token, logp = draw(x, torch.full((B,), 2.0 ** -20), **settings)
    assert token.tolist() == [17] * B
    # the others in descending order; top-p keeps one when what comes before it does not reach its share yet
    w = torch.exp(x.double()[:, [1500, 18, 2999]] - gap[:, None].double())
    before = 1 + w.cumsum(1) - w
    kept = before < settings.get("top_p", 2.0) * (1 + w.sum(1, keepdim=True))
    want = -torch.log1p((w * kept).sum(1))
    assert ((logp.cpu().double() - want).abs() <= 2.0 ** -22 * want.abs() + 3 * 2.0 ** -43).all(), (logp, want)


def test_long_rows_of_few_values():
    # so many rows that one CTA might take each, and so many equal values that their weights' sums pass 32 bits
    import torch
    gen = torch.Generator().manual_seed(9)
    x = torch.where(torch.rand((2, 400001), generator=gen) < 0.1, 1.0078125, 1.0).bfloat16()
    x[:, 7] = 3.0
    u = torch.rand(400, generator=gen)
    for settings in (dict(top_p=0.5), dict(top_k=390000, top_p=0.7), dict(temperature=0.37, top_p=0.04)):
        many = x.cuda()[torch.arange(400) % 2]
        got = draw(many, u, **settings)
        rows = [0, 1, 198, 399]
        ref.check(x[[r % 2 for r in rows]], u[rows], [t[rows] for t in got], **settings)


@pytest.mark.parametrize("V", [400001, 720000])
def test_long_rows_of_one_value(V):
    # every weight is the largest: each element holds 1 / V, which V equal whole numbers show without any error
    import torch
    u = torch.rand(300, generator=torch.Generator().manual_seed(2))
    x = torch.full((300, V), -2.5, dtype=torch.float16, device="cuda")
    token, logp = draw(x, u)
    want = (u.double() * V).floor().int()            # (24 bits times V is exact in 64)
    assert torch.equal(token.cpu(), want)
    token, logp = draw(x, u, top_p=0.25)
    assert torch.equal(token.cpu(), (u.double() * -(-V // 4)).floor().int())
