"""Tokens drawn from logits against the 64-bit reference (sampling_reference.py)."""
import numpy as np
import pytest

import sampling_reference as ref

pytestmark = pytest.mark.gpu
KINDS = ("float32", "bfloat16", "float16")


def logits_of(B, V, kind="float32", spread=3.0, seed=0, lift=True):
    import torch
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((B, V), generator=gen) * spread
    if lift and V > 8:
        at = torch.randint(0, V, (B, 4), generator=gen)
        x.scatter_(1, at, x.amax(1, keepdim=True) + 2 * torch.rand((B, 4), generator=gen))
    return x.to(getattr(torch, kind)), torch.rand(B, generator=gen)


def draw(x, u, **kw):
    import torch
    from indexer_topk_long_gb300 import sample
    kw = {k: v.cuda() if torch.is_tensor(v) else v for k, v in kw.items()}
    got = sample(x.cuda(), u.cuda(), **kw)
    torch.cuda.synchronize()
    return got


SETTINGS = [dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=0.02), dict(temperature=0.7, top_k=20, top_p=0.95, min_p=0.001),
            dict(top_k=1), dict(top_p=0.0), dict(min_p=1.0), dict(temperature=0.0), dict(temperature=2.5, top_k=1500, top_p=0.99),
            dict(top_k=5000), dict(temperature=1.3, top_p=0.999)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("settings", SETTINGS, ids=str)
@pytest.mark.parametrize("B,V", [(3, 32000), (5, 131071), (40, 2049)])
def test_settings(kind, settings, B, V):
    x, u = logits_of(B, V, kind, seed=V)
    ref.check(x, u, draw(x, u, **settings), **settings)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 31, 32, 33, 511, 512, 513, 2047, 2048, 2049, 4095, 8191, 16385, 65537, 262144, 360000])
def test_vocabularies(kind, V):
    """From one token to the largest, rows that begin at every place of 16 bytes."""
    x, u = logits_of(9 if V < 100000 else 2, V, kind, seed=V)
    for settings in (dict(), dict(top_k=40, top_p=0.9), dict(temperature=1.5, top_p=0.97)):
        ref.check(x, u, draw(x, u, **settings), **settings)


@pytest.mark.parametrize("kind", KINDS)
def test_strided_rows(kind):
    """A slice of a padded buffer: rows apart and off 16 bytes; what lies between them is not read as logits."""
    import torch
    big = torch.full((6, 5003), 100.0, dtype=getattr(torch, kind))
    x, u = logits_of(6, 4999, kind)
    big[:, 3:5002] = x
    big = big.cuda()
    from indexer_topk_long_gb300 import sample
    for settings in (dict(), dict(top_k=30), dict(top_p=0.8)):
        ref.check(x, u, sample(big[:, 3:5002], u.cuda(), **settings), **settings)


def test_settings_by_row():
    import torch
    B = 64
    x, u = logits_of(B, 20011, seed=4)
    rng = np.random.RandomState(5)
    s = dict(temperature=torch.from_numpy(rng.choice([0.0, 0.3, 1.0, 1.7], B).astype(np.float32)),
             top_k=torch.from_numpy(rng.choice([-1, 0, 1, 40, 700, 19999, 20011, 50000], B).astype(np.int32)),
             top_p=torch.from_numpy(rng.choice([0.0, 0.5, 0.99, 1.0, 7.0], B).astype(np.float32)),
             min_p=torch.from_numpy(rng.choice([0.0, 0.01, 0.3], B).astype(np.float32)))
    ref.check(x, u, draw(x, u, **s), **s)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [100, 5000, 70000])
def test_equal_logits(kind, V):
    """All equal: ties go to the lowest index at every cut, and u to its share of indices exactly."""
    import torch
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 1 / 3])
    x = torch.full((6, V), 1.25, dtype=getattr(torch, kind))
    for s in (dict(), dict(top_k=17), dict(top_k=4000), dict(top_p=0.5), dict(top_k=4000, top_p=0.25), dict(top_p=0.0), dict(min_p=1.0)):
        got = draw(x, u, **s)
        assert ref.check(x, u, got, **s) == 0
    n = V // 2
    got = draw(x, u, top_p=0.5)[0].cpu()
    if V % 2 == 0:
        assert got.tolist() == [min(int(float(a) * n), n - 1) for a in u]


@pytest.mark.parametrize("V", [1000, 40000])
def test_few_values(V):
    """Three values only: cuts fall among thousands of equal logits."""
    import torch
    gen = torch.Generator().manual_seed(1)
    x = torch.randint(0, 3, (8, V), generator=gen).float()
    u = torch.rand(8, generator=gen)
    for s in (dict(top_k=V // 2), dict(top_k=V // 2, top_p=0.9), dict(top_p=0.6), dict(top_p=0.95, temperature=3.0), dict(top_k=3), dict(min_p=0.3)):
        ref.check(x, u, draw(x, u, **s), **s)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V", [50, 30000])
def test_masked_logits(kind, V):
    """-inf and the type's lowest value in masked places, all but one masked, and all."""
    import torch
    low = torch.finfo(getattr(torch, kind)).min
    x, u = logits_of(7, V, kind)
    x[0, ::2] = -float("inf")
    x[1, 1:] = -float("inf")
    x[2, :-1] = -float("inf")
    x[3] = -float("inf")
    x[4, ::3] = low
    x[5, :-5] = low
    x[6, 20:] = -float("inf")
    for s in (dict(), dict(top_k=5), dict(top_k=V // 2 + 5), dict(top_p=0.9), dict(top_p=0.9, top_k=V - 10), dict(temperature=0.0), dict(min_p=0.1)):
        got = draw(x, u, **s)
        ref.check(x, u, got, **s)
        assert got[0][3] == -1 and got[1][3] == -float("inf")


@pytest.mark.parametrize("V", [60, 20000])
def test_rows_that_cannot_be_drawn_from(V):
    import torch
    x, u = logits_of(6, V)
    x[1, V - 1] = float("nan")
    x[2, 3] = float("inf")
    x[3] = float("nan")
    x[4, 0] = float("nan")
    x[4, 1:] = -float("inf")
    for s in (dict(), dict(top_k=4), dict(top_p=0.5), dict(temperature=0.0)):
        token, logp = draw(x, u, **s)
        assert token[[1, 2, 3, 4]].tolist() == [-1] * 4 and bool(logp[[1, 2, 3, 4]].isnan().all())
        ref.check(x, u, (token, logp), **s, rows=[0, 5])
    x, u = logits_of(9, V)
    t = torch.tensor([1, -1, float("nan"), float("inf"), 1, 1, 1, 1, 1.0])
    p = torch.tensor([1, 1, 1, 1, -0.1, float("nan"), 1, 1, 1.0])
    m = torch.tensor([0, 0, 0, 0, 0, 0, -0.5, 1.5, 0])
    u[8] = float("nan")
    token, logp = draw(x, u, temperature=t, top_p=p, min_p=m)
    assert token[1:].tolist() == [-1] * 8 and bool(logp[1:].isnan().all())
    ref.check(x, u, (token, logp), rows=[0])


def test_random_numbers_outside_their_range():
    import torch
    x, _ = logits_of(4, 9000)
    got = draw(x, torch.tensor([-0.5, 1.0, 7.0, float("inf")]))[0]
    assert torch.equal(got.cpu(), draw(x, torch.tensor([0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24]))[0].cpu())


@pytest.mark.parametrize("values", ["outlier", "far", "tiny", "steps", "signs", "wide"])
@pytest.mark.parametrize("settings", [dict(top_k=9000), dict(top_p=0.7), dict(top_k=9000, top_p=0.7), dict(top_k=40), dict(), dict(temperature=1e-3, top_p=0.5),
                                      dict(temperature=1e30, top_k=9000, top_p=0.6), dict(temperature=1e-38)], ids=str)
def test_ranges(values, settings):
    """What equal bins over a range split badly: outliers, values at both ends of fp32, subnormal ones, steps
    over all exponents, both signs of zero."""
    import torch
    V = 20000
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((2, V), generator=gen)
    if values == "outlier":
        x[:, 7], x[:, 11] = -1e30, 40.0
    elif values == "far":
        x[:, ::2], x[:, 5] = -3.4e38, 3.4e38
    elif values == "tiny":
        x = torch.randint(0, 3000, (2, V), generator=gen).float() * 2.0 ** -149
    elif values == "steps":
        x = -torch.exp2(torch.randint(-149, 127, (2, V), generator=gen).double()).float()
    elif values == "signs":
        x = torch.where(x > 0, 0.0, -0.0)
    else:
        x *= 1e37
    u = torch.rand(2, generator=gen)
    if values == "signs":
        x0 = torch.zeros_like(x)
        ref.check(x0, u, draw(x, u, **settings), **settings)
    else:
        ref.check(x, u, draw(x, u, **settings), **settings)


def test_the_same_whatever_the_split():
    """One row by itself (8 CTAs), in a small and in a large batch: the same bits."""
    import torch
    x, u = logits_of(1, 50000, seed=8)
    for s in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.95), dict(top_k=3000)):
        one = draw(x, u, **s)
        for B in (5, 30, 200):
            many = draw(x.expand(B, -1).contiguous(), u.expand(B).contiguous(), **s)
            assert bool((many[0] == one[0]).all()) and bool((many[1] == one[1]).all())


def test_shares_of_draws():
    """Evenly spread random numbers: each token comes as often as its probability says, to one draw."""
    import torch
    x, _ = logits_of(1, 300, seed=2)
    n = 4096
    u = (torch.arange(n) + 0.5) / n
    s = dict(temperature=1.2, top_k=30)
    token, logp = draw(x.expand(n, -1).contiguous(), u, **s)
    count = torch.bincount(token.long().cpu(), minlength=300)
    p = torch.zeros(300)
    p[token.long().cpu()] = logp.cpu().exp()
    assert int((count > 0).sum()) <= 30
    assert bool(((count - p * n).abs() <= 1.001).all())


def test_streams_and_graphs():
    import torch
    from indexer_topk_long_gb300 import sample
    x, u = logits_of(33, 70001, "bfloat16")
    x, u = x.cuda(), u.cuda()
    want = sample(x, u, top_k=50, top_p=0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = sample(x, u, top_k=50, top_p=0.9, stream=side)
    torch.cuda.synchronize()
    token, logp = torch.empty_like(want[0]), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):                           # calls that follow each other
            y = x * 1.0
            assert sample(y, u, top_k=50, top_p=0.9, token=token, logp=logp)[0] is token
    for _ in range(3):
        token.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for got in (there, (token, logp)):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    import torch
    from indexer_topk_long_gb300 import LtkError, sample
    x, u = (t.cuda() for t in logits_of(3, 100))
    cases = [(dict(logits=x[0]), "2-D"), (dict(logits=x.double()), "float32"), (dict(logits=x.cpu()), "CUDA"), (dict(logits=x[:, ::2]), "contiguous"),
             (dict(logits=x[:1].expand(3, 100)), "overlap"), (dict(logits=x[:, :0]), "no tokens"), (dict(u=u[:2]), "shape"), (dict(u=u.double()), "float32"),
             (dict(u=u.cpu()), "expected a tensor on"), (dict(temperature=-1.0), "temperature"), (dict(temperature=float("inf")), "temperature"),
             (dict(temperature=float("nan")), "temperature"), (dict(top_p=-0.1), "top_p"), (dict(min_p=1.1), "min_p"), (dict(top_k=2**31), "top_k"),
             (dict(top_k=torch.zeros(3, dtype=torch.int64, device="cuda")), "int32"), (dict(top_p=torch.zeros(4, device="cuda")), "shape"),
             (dict(min_p=torch.zeros(6, device="cuda")[::2]), "contiguous"), (dict(token=torch.zeros(3, device="cuda")), "int32"),
             (dict(logp=torch.zeros(2, device="cuda")), "shape")]
    for kw, msg in cases:
        with pytest.raises(ValueError, match=msg):
            sample(**{**dict(logits=x, u=u), **kw})
    with pytest.raises(LtkError, match="UNSUPPORTED"):
        sample(torch.zeros((1, 360001), device="cuda"), u[:1])
    token, logp = sample(x[:0], u[:0])
    assert token.shape == logp.shape == (0,)
