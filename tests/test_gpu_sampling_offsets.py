"""Tokens drawn from logits that lie far from 0, against the 64-bit reference: shares depend on differences only, however
large what the logits have in common is."""
import pytest

import sampling_reference as ref
from test_gpu_sampling import KINDS, draw

pytestmark = pytest.mark.gpu

# temperatures whose log2(e) / T rounds to fp32 with much left over, which a large logit multiplies
TEMPERATURES = [0.71, 1.0, 1.33, 2.79, 5.0, 11.37]


@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("at", [100, 900, 1020, 1100, 1500, 2200, 2900, 3600, 4090, 4200, 20000])
@pytest.mark.parametrize("sign", [1, -1])
def test_far_from_zero(T, at, sign):
    """The largest logit at about +-at in units of T ln 2 (base-2 exponents)."""
    import torch
    gen = torch.Generator().manual_seed(at)
    x = torch.randn((5, 3000), generator=gen) * 2 * T
    x = x - x.amax(1, keepdim=True) + sign * at * T * 0.6931471805599453
    u = torch.rand(5, generator=gen)
    for settings in (dict(), dict(top_k=60), dict(top_k=1200, min_p=1e-4)):
        ref.check(x, u, draw(x, u, temperature=T, **settings), temperature=T, **settings)


@pytest.mark.parametrize("kind", KINDS)
def test_two_tokens(kind):
    """Two logits by themselves: the logarithms of both shares, in types whose steps there are as large as 16."""
    import torch
    x = torch.tensor([[-10000.0, -10001.0], [-10000.0, -10016.0], [6000.0, 6016.0], [2000.0, 2001.0], [-4000.0, -3996.0]]).to(getattr(torch, kind))
    for T in TEMPERATURES:
        for u in (0.0, 1 - 2.0 ** -24):
            us = torch.full((5,), u)
            ref.check(x, us, draw(x, us, temperature=T), temperature=T)


def test_moved_logits_draw_the_same():
    """Differences in whole steps that fp32 holds at either place: the same tokens and, but for roundings, the same logarithms."""
    import torch
    gen = torch.Generator().manual_seed(3)
    x = torch.randint(-4000, 0, (40, 5000), generator=gen).float() / 256
    u = torch.rand(40, generator=gen)
    for T in TEMPERATURES:
        want = draw(x, u, temperature=T)
        for by in (-9000.0, -3000.0, 2000.0, 12000.0):
            got = draw(x + by, u, temperature=T)
            ref.check(x + by, u, got, temperature=T)
            # each is within 2^-24 |logp| + 2^-30 of the same number
            assert ((got[1] - want[1]).abs() <= 2.02 * 2.0 ** -24 * want[1].abs() + 2.0 ** -29)[got[0] == want[0]].all()
