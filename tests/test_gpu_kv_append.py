"""Appending to the paged 8-bit cache: codes and scales bit for bit against the
plain implementation (the operation fixes every rounding), queries likewise."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


def _tables(n, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * freq
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def _inputs(N, hq, hkv, d, dtype, seed, gain=1.0):
    import torch
    rng = np.random.RandomState(seed)
    x = torch.from_numpy((rng.randn(N, hq + 2 * hkv, d) * gain).astype(np.float32)).to(
        torch.bfloat16 if dtype == "bf16" else torch.float16)
    return x


def _run(cache, plain, ints, qkv, hq, hkv, cos, sin, interleaved, table, lens, cu):
    import torch
    x = qkv.cuda()
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    ct, st = (torch.from_numpy(t).cuda() for t in (cos, sin))
    got = cache.append(k, v, *ints, ct, st, interleaved=interleaved, q=q)
    f = qkv.float().numpy()
    plain.append(f[:, hq:hq + hkv], f[:, hq + hkv:], table, lens, cu, cos, sin, interleaved)
    assert cache.status() == 0
    return got, f[:, :hq]


def _same(cache, plain):
    np.testing.assert_array_equal(cache.k_scale.cpu().numpy(), plain.scale["k"])
    np.testing.assert_array_equal(cache.v_scale.cpu().numpy(), plain.scale["v"])
    for name, t in (("k", cache.k_codes), ("v", cache.v_codes)):
        np.testing.assert_array_equal(t.cpu().numpy(), plain.codes[name])


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype,rot,inter", [
    ([1], [1], 4, 1, 128, 64, "bf16", 128, False),
    ([17, 64, 65, 5], [1, 1, 1, 1], 8, 2, 128, 64, "bf16", 128, False),
    ([200, 33], [150, 33], 2, 2, 64, 16, "f16", 32, True),
    ([130, 40, 90], [0, 40, 77], 6, 3, 128, 32, "bf16", 96, False),
    ([300], [299], 5, 1, 64, 128, "bf16", 64, False),
    ([129], [129], 40, 1, 128, 128, "f16", 48, True),
    ([70, 70], [13, 0], 1, 1, 128, 16, "bf16", 16, False),
])
def test_append_matches_definition(lens, new, hq, hkv, d, page, dtype, rot, inter):
    s = ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=3)
    for name in "kv":                      # the spare rows are data of nobody here
        s.c.codes[name][s.c.codes[name] == 0x7F] = 0
    cache, ints = s.gpu()
    cos, sin = _tables(max(lens), rot)
    qkv = _inputs(s.cu[-1], hq, hkv, d, dtype, 5)
    got, q = _run(cache, s.c, ints, qkv, hq, hkv, cos, sin, inter, s.table, s.lens, s.cu)
    _same(cache, s.c)
    import torch
    for b in range(len(lens)):
        for i in range(new[b]):
            t, p = s.cu[b] + i, lens[b] - new[b] + i
            want = torch.from_numpy(ref.rotate(q[t], cos[p], sin[p], inter)).to(qkv.dtype)
            assert torch.equal(got[t].cpu(), want)


def test_growing_page_one_token_at_a_time():
    """Each token is larger than the last: the page's exponent grows and its held codes follow."""
    d, page = 128, 16
    s = ref.Setup([20], [1], 1, 2, d, page, seed=1)
    for name in "kv":
        s.c.codes[name][:] = 0
        s.c.scale[name][:] = 0
    cache, ints = s.gpu()
    cos, sin = _tables(20, d)
    import torch
    for p in range(20):
        qkv = _inputs(1, 1, 2, d, "bf16", 100 + p, gain=2.0 ** (p - 10))
        lens = torch.tensor([p + 1], dtype=torch.int32).cuda()
        _run(cache, s.c, [ints[0], lens, ints[2]], qkv, 1, 2, cos, sin, False, s.table, [p + 1], s.cu)
        _same(cache, s.c)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 1e38, 0.0])
@pytest.mark.parametrize("where", ["k", "v"])
def test_values_the_format_cannot_hold(value, where):
    """The token is held as NaN keys and zero values; its neighbours are as without it."""
    s = ref.Setup([40], [40], 1, 2, 64, 32, seed=2)
    for name in "kv":
        s.c.codes[name][:] = 0
    cache, ints = s.gpu()
    cos, sin = _tables(40, 64)
    qkv = _inputs(40, 1, 2, 64, "bf16", 9)
    qkv[7, 1 if where == "k" else 3, 11] = value
    if value == 0.0:
        qkv[:] = 0
    _run(cache, s.c, ints, qkv, 1, 2, cos, sin, False, s.table, s.lens, s.cu)
    _same(cache, s.c)
    if value != 0.0:
        assert (s.c.codes["k"][s.table[0, 0], 0, 7] == 0x7F).all()
        assert (s.c.codes["v"][s.table[0, 0], 0, 7] == 0).all()


def test_without_rotation_or_queries():
    s = ref.Setup([50], [50], 1, 2, 64, 32, seed=4)
    for name in "kv":
        s.c.codes[name][:] = 0
    cache, ints = s.gpu()
    x = _inputs(50, 0, 2, 64, "f16", 6).cuda()
    assert cache.append(x[:, :2], x[:, 2:], *ints) is None
    f = x.float().cpu().numpy()
    none = np.zeros((50, 0), np.float32)
    s.c.append(f[:, :2], f[:, 2:], s.table, s.lens, s.cu, none, none, False)
    _same(cache, s.c)


def test_bad_page_or_position_is_reported_and_written_nowhere():
    import torch
    s = ref.Setup([40, 20], [40, 20], 1, 1, 64, 16, seed=4)
    cache, ints = s.gpu()
    before = cache.k_codes.clone()
    x = _inputs(60, 0, 1, 64, "bf16", 6).cuda()
    ints[0].fill_(s.pages)                # one past the pool
    cache.append(x[:, :1], x[:, 1:], *ints)
    assert cache.status() == 1 and cache.status() == 0
    assert torch.equal(cache.k_codes, before)
    ints[0].fill_(-5)
    cache.append(x[:, :1], x[:, 1:], *ints)
    assert cache.status() == 1
    assert torch.equal(cache.k_codes, before)
    ints[1].fill_(10)                     # shorter than its new tokens: negative positions
    cache.append(x[:, :1], x[:, 1:], *ints)
    assert cache.status() == 1
    assert torch.equal(cache.k_codes, before)


def test_rotation_table_too_short():
    s = ref.Setup([40], [40], 1, 1, 64, 64, seed=4)
    cache, ints = s.gpu()
    import torch
    cos, sin = (torch.from_numpy(t).cuda() for t in _tables(30, 64))
    x = _inputs(40, 1, 1, 64, "bf16", 6).cuda()
    cache.append(x[:, 1:2], x[:, 2:], *ints, cos, sin, q=x[:, :1])
    assert cache.status() == 1
    pg = int(s.table[0, 0])
    assert (cache.k_codes[pg, 0, 30:40] == 0x7F).all() and not (cache.k_codes[pg, 0, :30] == 0x7F).all(-1).any()
