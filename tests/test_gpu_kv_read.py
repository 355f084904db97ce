"""Tokens read back from the paged cache.  Without rotation a value is one product of fp32 numbers rounded
to 16 bits, so results are compared bit for bit; rotated back, two fp32 products and a sum (three roundings of
2^-24 of |a| + |b|) come before the last one of 2^-8 (bf16) or 2^-11 (f16) of the value."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu
KIND = {"bf16": "bfloat16", "f16": "float16"}


def expected(s, lens, cu, name, cos=None, sin=None, interleaved=False):
    """fp32 (before the last rounding; fp64 with rotation), and |a| + |b| of rotated pairs."""
    rows, size = [], []
    for b, n in enumerate(cu[1:]):
        pos = np.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b])
        pg = s.table[b][pos // s.c.page]
        codes = ref.E4M3[s.c.codes[name][pg, :, pos % s.c.page]].astype(np.float32)
        with np.errstate(all="ignore"):
            x = codes * s.c.scale[name][pg][..., None]
        x = np.where(s.c.scale[name][pg][..., None] == 0, np.float32(0), x)
        y = np.abs(x).astype(np.float64)
        if cos is not None and name == "k":
            x = x.astype(np.float64)
            rot = 2 * cos.shape[1]
            lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            c, z = cos[pos].astype(np.float64)[:, None], sin[pos].astype(np.float64)[:, None]
            a, d = x[..., lo].copy(), x[..., hi].copy()
            x[..., lo], x[..., hi] = a * c + d * z, d * c - a * z
            y[..., lo] = y[..., hi] = np.abs(a) + np.abs(d)
        rows.append(x)
        size.append(y)
    return np.concatenate(rows), np.concatenate(size)


def ints_of(*xs):
    import torch
    return [torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in xs]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hkv,d,page", [(8, 128, 64), (1, 64, 16), (3, 64, 128), (5, 128, 32)])
def test_bit_for_bit(dtype, hkv, d, page):
    """Whole sequences, tails and single tokens, blocks of any scale and of scale 0."""
    import torch
    lens = [1, page, page + 1, 3 * page - 1, 200, 7]
    s = ref.Setup(lens, [1, page, 1, 3 * page - 1, 37, 0], hkv, hkv, d, page, dtype)
    rng = np.random.RandomState(1)
    for name in "kv":
        s.c.scale[name] *= rng.uniform(0.5, 2, s.c.scale[name].shape).astype(np.float32)
        s.c.scale[name][s.table[3, 1], 0] = 0
    cache, ints = s.gpu()
    k, v = cache.read(*ints, s.cu[-1], dtype=getattr(torch, KIND[dtype]))
    torch.cuda.synchronize()
    assert cache.status() == 0
    for got, name in ((k, "k"), (v, "v")):
        want = torch.from_numpy(expected(s, lens, s.cu, name)[0]).to(got.dtype)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype,d,rot,interleaved", [("bf16", 128, 128, False), ("bf16", 128, 48, True), ("f16", 64, 16, False), ("f16", 64, 64, True),
                                                     ("bf16", 64, 32, False), ("f16", 128, 16, True)])
def test_keys_rotated_back(dtype, d, rot, interleaved):
    import torch
    lens = [70, 129, 300]
    s = ref.Setup(lens, [70, 30, 5], 2, 2, d, 32, dtype)
    angle = np.random.RandomState(2).uniform(-4, 4, (301, rot // 2))
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    cache, ints = s.gpu()
    k, v = cache.read(*ints, s.cu[-1], dtype=getattr(torch, KIND[dtype]), cos=torch.from_numpy(cos).cuda(), sin=torch.from_numpy(sin).cuda(),
                      interleaved=interleaved)
    assert cache.status() == 0
    want, size = expected(s, lens, s.cu, "k", cos, sin, interleaved)
    tol = ref.U[dtype] * 1.01 * np.abs(want) + 3 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == "f16" else 0)
    assert np.all(np.abs(k.double().cpu().numpy() - want) <= tol)
    assert torch.equal(v.cpu(), torch.from_numpy(expected(s, lens, s.cu, "v")[0]).to(v.dtype))


def test_what_append_wrote_comes_back():
    """Keys appended with a rotation and read with it: a code's rounding (2^-4 of the block's scale's
    octave at most: half of 2^-3 of a power of two not above twice the value, or of 2^-9 of the scale) is all
    that is lost, besides fp32 and the last rounding.  Read without it and appended elsewhere: the same values."""
    import torch
    from indexer_topk_long_gb300 import PagedKVCache
    gen = torch.Generator(device="cuda").manual_seed(5)
    n, h, d, page = 150, 4, 128, 32
    cache = PagedKVCache(20, h, d, page=page)
    k, v = (torch.randn((n, h, d), device="cuda", generator=gen).bfloat16() for _ in range(2))
    table = torch.randperm(20, device="cuda", generator=gen).to(torch.int32)[:10].view(2, 5).contiguous()
    lens, cu = ints_of([100, 50], [0, 100, 150])
    angle = torch.rand((100, d // 2), device="cuda", generator=gen) * 6
    cache.append(k, v, table, lens, cu, angle.cos(), angle.sin())
    k2, v2 = cache.read(table, lens, cu, n, cos=angle.cos(), sin=angle.sin())
    assert float((v2.float() - v.float()).abs().max()) <= 2.0 ** -4 * 8 and float((k2.float() - k.float()).abs().max()) <= 2.0 ** -3 * 8
    assert float((k2.float() - k.float()).norm() / k.float().norm()) < 2.0 ** -4
    kr, vr = cache.read(table, lens, cu, n)
    other = PagedKVCache(20, h, d, page=page)
    other.append(kr, vr, table, lens, cu)
    for a, b in zip((kr, vr), other.read(table, lens, cu, n)):
        assert torch.equal(a, b)
    assert cache.status() == other.status() == 0


def test_tokens_that_are_not_there():
    """Pages outside the pool, positions before the first, past the table and past the rotation's: NaN and
    reported; rows of no sequence are left as they were."""
    import torch
    s = ref.Setup([40, 20, 33], [10, 20, 33], 2, 2, 64, 16)
    cache, (table, lens, cu) = s.gpu()
    good_k, good_v = cache.read(table, lens, cu, 63)
    assert cache.status() == 0
    t2 = table.clone()
    t2[1, 1] = s.pages
    k, v = cache.read(t2, lens, cu, 63)
    assert cache.status() == 1
    bad = torch.zeros(63, dtype=torch.bool)
    bad[10 + 16:30] = True
    for got, good in ((k, good_k), (v, good_v)):
        assert torch.equal(got.isnan().all(-1).all(-1).cpu(), bad) and torch.equal(got[~bad.cuda()], good[~bad.cuda()])
    l2 = lens.clone()
    l2[1] = 18                                       # two of the 20 lie before its first token
    k, _ = cache.read(table, l2, cu, 63)
    assert cache.status() == 1 and torch.equal(k.isnan().all(-1).all(-1).nonzero().flatten().cpu(), torch.tensor([10, 11]))
    l2[1] = table.shape[1] * 16 + 1                  # one past the table's last column
    k, _ = cache.read(table, l2, cu, 63)
    assert cache.status() == 1 and bool(k[29].isnan().all())
    cos = torch.ones((30, 8), device="cuda")
    k, _ = cache.read(table, lens, cu, 63, cos=cos, sin=torch.zeros_like(cos))
    assert cache.status() == 1
    assert torch.equal(k.isnan().all(-1).all(-1).nonzero().flatten().cpu(), torch.cat([torch.arange(0, 10), torch.arange(60, 63)]))
    k, v = (torch.full((70, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read(table, lens, cu, 70, k_out=k, v_out=v)
    assert cache.status() == 0
    assert torch.equal(k[:63], good_k) and torch.equal(v[:63], good_v)
    assert bool((k[63:] == 9).all()) and bool((v[63:] == 9).all())


def test_many_tokens_and_streams():
    """More tokens than one wave of CTAs holds; another stream; a graph."""
    import torch
    s = ref.Setup([5000, 1, 3000], [5000, 1, 2999], 1, 1, 64, 128)
    cache, ints = s.gpu()
    k, v = cache.read(*ints, 8000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k2, v2 = cache.read(*ints, 8000, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        k3, v3 = cache.read(*ints, 8000)
    graph.replay()
    torch.cuda.synchronize()
    assert cache.status() == 0
    want = [torch.from_numpy(expected(s, s.lens, s.cu, n)[0]).bfloat16().cuda() for n in "kv"]
    for a, b in ((k, v), (k2, v2), (k3, v3)):
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals():
    import torch
    from indexer_topk_long_gb300 import LtkError
    s = ref.Setup([40], [10], 2, 2, 64, 16)
    cache, ints = s.gpu()
    cos = torch.ones((50, 8), device="cuda")
    with pytest.raises(ValueError, match="dtype"):
        cache.read(*ints, 10, dtype=torch.float32)
    with pytest.raises(ValueError, match="both or neither"):
        cache.read(*ints, 10, cos=cos)
    with pytest.raises(ValueError, match="equal shape"):
        cache.read(*ints, 10, cos=cos, sin=cos[:4])
    with pytest.raises(ValueError, match="k_out"):
        cache.read(*ints, 10, k_out=torch.zeros((9, 2, 64), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="v_out"):
        cache.read(*ints, 10, v_out=torch.zeros((10, 2, 64), dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError, match="n: "):
        cache.read(*ints, -1)
    with pytest.raises(ValueError, match="32-bit"):
        cache.read(*ints, 2**31)
    with pytest.raises(LtkError, match="ARG"):
        cache.read(*ints, 10, cos=torch.ones((50, 40), device="cuda"), sin=torch.ones((50, 40), device="cuda"))
    with pytest.raises(LtkError, match="UNSUPPORTED"):
        cache.read(*ints, 10, cos=torch.ones((50, 12), device="cuda"), sin=torch.ones((50, 12), device="cuda"))
    k, v = cache.read(*ints, 0)
    assert k.shape == v.shape == (0, 2, 64) and cache.status() == 0
