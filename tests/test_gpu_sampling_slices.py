"""Tokens drawn with a small top-k from rows whose largest elements lie together, so that one CTA's slice of the row holds
more of them than it has room to list, against the 64-bit reference."""
import pytest

import sampling_reference as ref
from test_gpu_sampling import KINDS, draw

pytestmark = pytest.mark.gpu


def _row(kind, V, n, where, equal, seed=0):
    """Logits [1, V] below 4 with n lifted to between 5 and 6, each in a piece of 16 bytes of its own."""
    import torch
    vec = 4 if kind == "float32" else 8
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((1, V), generator=gen).clamp(max=4.0)
    if where == "warps":
        # the first 32 pieces of each warp's part of a slice, where 8 CTAs of 8 warps share the row
        part = -(-(-(-((V + 2 * vec - 2) // vec) // 8)) // 8)
        piece = torch.cat([torch.arange(min(part, 32)) + w * part for w in range(8)])[:n]
        at = piece * vec
    else:
        first = {"start": 0, "middle": V // 2 // vec, "end": V // vec - n}[where]
        at = (first + torch.arange(n)) * vec
    n = len(at)
    # steps of 1/512 at 5: all different in 32 bits; in 16 some are equal, and cut by their indices
    high = torch.full((n,), 5.5) if equal else 5 + torch.randperm(n, generator=gen) / 512
    x[0, at] = high
    return x.to(getattr(torch, kind)), n


def _check(x, k, **settings):
    """One row by itself, and in a batch that leaves fewer CTAs to a row: right, and the same bits."""
    import torch
    u = torch.tensor([0.0, 0.17, 0.5, 0.83, 1 - 2.0 ** -24])
    alone = []
    for i in range(len(u)):
        got = draw(x, u[i:i + 1], top_k=k, **settings)
        ref.check(x, u[i:i + 1], got, top_k=k, **settings)
        alone.append(got)
    for B in (60, 300):
        token, logp = draw(x.expand(B, -1).contiguous(), u.repeat(B // 5), top_k=k, **settings)
        for i, (t, p) in enumerate(alone):
            assert bool((token[i::5] == t).all()) and bool((logp[i::5] == p).all()), (B, i)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("where", ["start", "middle", "end", "warps"])
@pytest.mark.parametrize("equal", [True, False], ids=["equal", "distinct"])
@pytest.mark.parametrize("n", [129, 200, 256])
def test_exactly_as_many_as_are_kept(kind, where, equal, n):
    V = 8000 if kind == "float32" else 16000
    x, n = _row(kind, V, n, where, equal, seed=n)
    for k in {n - 1, n, min(n + 1, 256)}:
        _check(x, k)


@pytest.mark.parametrize("kind,V", [("float32", 32000), ("float32", 131072), ("bfloat16", 128256), ("float16", 50257)])
@pytest.mark.parametrize("k", [130, 150, 200, 256])
def test_long_rows(kind, V, k):
    x, n = _row(kind, V, k, "warps", False, seed=k)
    assert n == k
    _check(x, k)


@pytest.mark.parametrize("settings", [dict(top_p=0.6), dict(min_p=0.3), dict(min_p=0.5, top_p=0.9), dict(temperature=0.7, top_p=0.999),
                                      dict(temperature=3.0)], ids=str)
@pytest.mark.parametrize("n", [129, 200])
def test_with_other_filters(settings, n):
    x, n = _row("float32", 8000, n, "start", False, seed=n)
    for k in (n - 1, n, n + 1):
        _check(x, k, **settings)


def test_settings_by_row():
    import torch
    B = 6
    x, n = _row("float32", 8000, 200, "start", True)
    x = x.expand(B, -1).contiguous()
    u = torch.tensor([0.05, 0.3, 0.5, 0.7, 0.9, 0.99])
    s = dict(top_k=torch.tensor([128, 129, 199, 200, 201, 256], dtype=torch.int32), temperature=torch.full((B,), 1.3),
             top_p=torch.tensor([1.0, 0.5, 1.0, 1.0, 0.9, 1.0]))
    ref.check(x, u, draw(x, u, **s), **s)
