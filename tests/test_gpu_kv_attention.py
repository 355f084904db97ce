"""Attention over the paged 8-bit cache against the plain implementation in 64 bits."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


# (engine, rows the hint speaks of): the kernel for few rows (8 or 16 a unit), then narrow, whole and paired tiles
KERNELS = [(1, 8), (1, 16), (2, 64), (2, 128), (2, 1000)]


def _gpu(s, engine, rows):
    """Pairs of tiles are for long sequences: the page table says so."""
    return s.gpu(engine, 20000 if rows > 256 else 0)


def _hint(s, rows):
    return max(1, rows // (s.q.shape[1] // s.c.heads))


def _dense(s, window=0, sinks=0, max_q=None, scale=None):
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, window, sinks, scale=scale)
    for engine, rows in [(0, None)] + KERNELS:
        cache, ints = _gpu(s, engine, rows or 0)
        out, lse = cache.attention(s.q.cuda(), *ints, window=window, sinks=sinks, scale=scale,
                                   max_q=max_q if rows is None else _hint(s, rows))
        assert cache.status() == 0
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, s.dtype)


def _selected(s, idx):
    import torch
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, idx=idx)
    for engine in (0, 1, 2):
        cache, ints = s.gpu(engine)
        out, lse = cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints)
        assert cache.status() == 0
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, s.dtype)


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype", [
    ([1], [1], 1, 1, 128, 64, "bf16"),
    ([2, 1, 3], [1, 1, 1], 4, 2, 64, 16, "f16"),
    ([127, 128, 129, 1000], [1, 1, 1, 1], 8, 2, 128, 64, "bf16"),
    ([777], [1], 8, 8, 64, 16, "f16"),
    ([300, 31], [3, 2], 10, 2, 128, 32, "bf16"),
    ([513, 40, 16], [0, 1, 4], 7, 1, 64, 128, "bf16"),
    ([200], [1], 16, 1, 128, 16, "f16"),
    ([5000], [1], 4, 1, 128, 64, "bf16"),
])
def test_few_rows(lens, new, hq, hkv, d, page, dtype):
    _dense(ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=11))


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype", [
    ([40], [40], 4, 4, 128, 64, "bf16"),
    ([129], [129], 2, 1, 64, 16, "f16"),
    ([700, 90, 260], [64, 90, 1], 10, 2, 128, 32, "bf16"),
    ([600], [37], 64, 1, 128, 64, "bf16"),
    ([600, 300], [5, 2], 128, 1, 64, 128, "f16"),
    ([513, 512, 511], [100, 0, 33], 7, 1, 128, 16, "f16"),
    ([400], [300], 5, 1, 128, 128, "bf16"),
])
def test_many_rows(lens, new, hq, hkv, d, page, dtype):
    s = ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=12)
    _dense(s)


@pytest.mark.parametrize("max_q", [0, 1, 5, 15, 300])
def test_any_hint_gives_the_same_answer(max_q):
    _dense(ref.Setup([260, 77, 1], [70, 1, 1], 6, 2, 128, 32, "bf16", seed=13), max_q=max_q)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (100, 4), (128, 130), (1000, 7),
                                          (257, 500)])
@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype", [
    ([900, 130, 5], [1, 1, 1], 8, 2, 128, 64, "bf16"),
    ([700, 130, 90], [150, 20, 90], 7, 1, 64, 16, "f16"),
])
def test_window_and_sinks(lens, new, hq, hkv, d, page, dtype, window, sinks):
    _dense(ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=14), window, sinks)


@pytest.mark.parametrize("new", [1, 50])
def test_blocks_of_very_different_scale(new):
    """Scales spread over many binary orders: the weights' folding of the value scale holds."""
    s = ref.Setup([500], [new], 4, 1, 128, 16, "bf16", seed=15, spread=0.0)
    rng = np.random.RandomState(5)
    s.c.scale["v"] *= np.exp2(rng.randint(-14, 15, s.c.scale["v"].shape)).astype(np.float32)
    _dense(s)


@pytest.mark.parametrize("new", [1, 40])
def test_large_scores(new):
    """One key dominates by far, first or last: the running maximum moves by much."""
    for at in (0, 299):
        s = ref.Setup([340], [new], 4, 2, 128, 64, "bf16", seed=16)
        for h in range(2):
            s.c.codes["k"][s.table[0, at // 64], h, at % 64] = 0x68      # a large positive code throughout
        s.q = s.q.abs()
        _dense(s, scale=0.02)


def test_sequence_shorter_than_its_queries_and_empty():
    """Queries before the first token (and of an empty sequence) see nothing: 0 and -inf."""
    import torch
    for engine, rows in KERNELS:
        s = ref.Setup([30, 30], [50, 4], 4, 1, 128, 16, "bf16", seed=17)
        s.lens = [30, 0]
        cache, ints = _gpu(s, engine, rows)
        out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
        assert (out[:20] == 0).all() and torch.isneginf(lse[:20]).all()
        assert (out[50:] == 0).all() and torch.isneginf(lse[50:]).all()
        want = s.c.attend(s.q64()[20:50], s.table[:1], [30], [0, 30])
        ref.check(out[20:50].double().cpu().numpy(), lse[20:50].double().cpu().numpy(), want, "bf16")


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_a_poisoned_token_reaches_only_the_queries_that_see_it(engine, rows):
    s = ref.Setup([100], [40], 4, 1, 128, 16, "bf16", seed=18)
    s.c.codes["k"][s.table[0, 80 // 16], 0, 80 % 16] = 0x7F
    s.c.codes["v"][s.table[0, 80 // 16], 0, 80 % 16] = 0
    cache, ints = _gpu(s, engine, rows)
    out, _ = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
    bad = out.isnan()
    assert not bad[:20].any() and bad[20:].all()
    want = s.c.attend(s.q64()[:20], s.table, [80], [0, 20])
    ref.check(out[:20].double().cpu().numpy(), np.zeros((20, 4)), (want[0], np.zeros((20, 4)), want[2]), "bf16")


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_bad_page_is_reported(engine, rows):
    s = ref.Setup([100, 64], [20, 20], 4, 1, 128, 16, "bf16", seed=19)
    cache, ints = _gpu(s, engine, rows)
    ints[0][0, 2] = s.pages + 7
    out, _ = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
    assert cache.status() == 1 and cache.status() == 0
    assert out[:20].isnan().all() and not out[20:].isnan().any()


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_bad_page_reaches_only_the_queries_that_see_it(engine, rows):
    """The page after the first ten queries' positions is outside the pool."""
    s = ref.Setup([90], [40], 4, 1, 128, 16, "bf16", seed=27)
    cache, ints = _gpu(s, engine, rows)
    ints[0][0, 4] = -3                      # positions 64 .. 79; queries at 50 .. 89
    out, _ = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
    assert cache.status() == 1
    bad = out.isnan()
    assert not bad[:14].any() and bad[14:].all()
    want = s.c.attend(s.q64()[:14], s.table, [64], [0, 14])
    ref.check(out[:14].double().cpu().numpy(), np.zeros((14, 4)), (want[0], np.zeros((14, 4)), want[2]), "bf16")


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype,k", [
    ([1], [1], 4, 1, 128, 64, "bf16", 1),
    ([900], [1], 64, 1, 128, 64, "bf16", 300),
    ([900, 60, 200], [2, 3, 1], 8, 2, 128, 16, "f16", 129),
    ([400], [33], 64, 1, 64, 32, "bf16", 128),
    ([400], [9], 128, 1, 128, 64, "f16", 200),
    ([500, 20], [5, 20], 15, 3, 64, 128, "bf16", 77),
    ([700], [3], 40, 2, 128, 16, "bf16", 513),
])
def test_selected(lens, new, hq, hkv, d, page, dtype, k):
    s = ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=21)
    rng = np.random.RandomState(1)
    idx = np.full((s.cu[-1], k), -1, np.int32)
    for b in range(len(lens)):
        for i in range(new[b]):
            p = lens[b] - new[b] + i
            pick = rng.permutation(p + 1)[:k]
            idx[s.cu[b] + i, :len(pick)] = pick
    _selected(s, idx)


@pytest.mark.parametrize("new,hq,hkv,d,k", [(1500, 64, 1, 64, 130), (700, 40, 1, 64, 300), (160, 128, 1, 64, 260),
                                             (400, 200, 1, 64, 128), (330, 96, 2, 64, 140)])
def test_selected_more_units_than_sms(new, hq, hkv, d, k):
    """Whole units in turn, then a rest that is cut; more than 128 rows a KV head."""
    s = ref.Setup([new + 300], [new], hq, hkv, d, 32, "f16", seed=28)
    rng = np.random.RandomState(3)
    idx = np.stack([rng.permutation(300)[:k] for _ in range(new)]).astype(np.int32)
    import torch
    pick = np.unique(np.concatenate([rng.randint(0, new, 12), [0, new - 1]]))
    for engine in (1, 2):
        cache, ints = s.gpu(engine)
        out, lse = cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints)
        assert cache.status() == 0
        for i, p in zip(pick, 300 + pick):  # each alone, as a sequence's last token
            want = s.c.attend(s.q64()[i:i + 1], s.table, [p + 1], [0, 1], idx=idx[i:i + 1])
            ref.check(out[i:i + 1].double().cpu().numpy(), lse[i:i + 1].double().cpu().numpy(), want, "f16")


def test_many_sequences_and_heads():
    """More row tiles than threads look at in one go, empty sequences among them."""
    rng = np.random.RandomState(4)
    lens = rng.randint(1, 40, 900)
    new = np.minimum(lens, rng.choice([0, 0, 1, 2, 5], 900))
    _dense(ref.Setup(lens, new, 6, 3, 64, 16, "bf16", seed=29))


def test_cu_q_that_does_not_rise():
    """Reported; nothing is read or written out of bounds, and the next call is right."""
    import torch
    s = ref.Setup([60, 50], [40, 30], 4, 1, 128, 16, "bf16", seed=30)
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    for engine, rows in KERNELS:
        cache, ints = _gpu(s, engine, rows)
        for bad in ([0, 50, 30], [0, 40, 1 << 30], [-7, 40, 70]):
            cu = torch.tensor(bad, dtype=torch.int32).cuda()
            cache.attention(s.q.cuda(), ints[0], ints[1], cu, max_q=_hint(s, rows))
            assert cache.status() == (1 if engine == 2 else 0)      # the few-row kernel clamps
        out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "bf16")
    x = s.q.cuda()
    cache.append(x[:, :1], x[:, 1:2], ints[0], ints[1], torch.tensor([0, 50, 30], dtype=torch.int32).cuda())
    torch.cuda.synchronize()


def test_selected_empty_slots_anywhere():
    """Empty slots between the others, whole empty tiles, a row of nothing but empty slots,
    entries past the query's position."""
    for hq, engine in ((4, 1), (4, 2), (64, 1), (64, 2), (100, 2)):
        s = ref.Setup([600], [6], hq, 1, 128, 64, "bf16", seed=22)
        rng = np.random.RandomState(2)
        idx = np.full((6, 400), -1, np.int32)
        for i in range(6):
            idx[i, rng.permutation(400)[:150]] = rng.permutation(590)[:150]
        idx[1, :256] = -1
        idx[2] = -1
        idx[3, :10] = 599                   # not visible to query 3 (position 597)
        idx[3, 10:20] = 1 << 30
        idx[4, 1:] = -1
        cache, ints = s.gpu(engine)
        import torch
        out, lse = cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints)
        want = s.c.attend(s.q64(), s.table, s.lens, s.cu, idx=idx)
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "bf16")
        assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()


def test_same_bits_every_time_and_under_capture():
    """Splits are merged in a fixed order; a replayed graph reads its buffers anew."""
    import torch
    for hq, new, engine in ((8, 1, 1), (8, 100, 2), (64, 3, 1), (64, 3, 2), (100, 1, 2)):
        s = ref.Setup([3000], [new], hq, 1, 128, 64, "bf16", seed=23)
        cache, ints = _gpu(s, engine, new * hq)
        q = s.q.cuda()
        idx = torch.randperm(2900, device="cuda")[:500].to(torch.int32).expand(new, 500).contiguous()
        first = [t.clone() for t in cache.attention(q, *ints) + cache.attention_selected(q, idx, *ints)]
        for _ in range(5):
            again = cache.attention(q, *ints) + cache.attention_selected(q, idx, *ints)
            assert all(torch.equal(a, b) for a, b in zip(first, again))
        outs = [torch.empty_like(t) for t in first]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cache.attention(q, *ints, out=outs[0], lse=outs[1])
            cache.attention_selected(q, idx, *ints, out=outs[2], lse=outs[3])
        for _ in range(2):
            for t in outs:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_another_stream():
    import torch
    s = ref.Setup([1000, 400], [1, 1], 8, 2, 128, 64, "bf16", seed=24)
    cache, ints = s.gpu()
    q = s.q.cuda()
    want, want_lse = cache.attention(q, *ints)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = cache.attention(q, *ints, stream=side)
    del q, s
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_strided_queries():
    import torch
    s = ref.Setup([300, 90], [2, 30], 6, 2, 128, 32, "bf16", seed=25)
    cache, ints = s.gpu()
    wide = torch.randn((32, 10, 128), device="cuda").to(torch.bfloat16)
    wide[:, :6] = s.q.cuda()
    out, lse = cache.attention(wide[:, :6], *ints)
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "bf16")


def test_cache_beyond_32_bit_offsets():
    """Codes past 2^32 bytes: the last pages of a 5 GB pool."""
    import torch
    pages, heads, d, page = 5 * (1 << 30) // (64 * 128 * 8), 8, 128, 64
    s = ref.Setup([300], [1], 8, 8, d, page, "bf16", seed=26)
    from indexer_topk_long_gb300 import PagedKVCache
    cache = PagedKVCache(pages, heads, d, page=page)
    shift = pages - s.pages
    for name, codes, scale in (("k", cache.k_codes, cache.k_scale), ("v", cache.v_codes, cache.v_scale)):
        codes[shift:] = torch.from_numpy(s.c.codes[name]).cuda()
        scale[shift:] = torch.from_numpy(s.c.scale[name]).cuda()
    table = torch.from_numpy(np.where(s.table >= 0, s.table + shift, -1).astype(np.int32)).cuda()
    lens, cu = (torch.tensor(x, dtype=torch.int32).cuda() for x in (s.lens, s.cu))
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    idx = torch.randperm(300, device="cuda")[None].to(torch.int32)
    tiles = PagedKVCache(pages, heads, d, page=page, k_codes=cache.k_codes, v_codes=cache.v_codes,
                         k_scale=cache.k_scale, v_scale=cache.v_scale, engine=2)
    for out, lse in (cache.attention(s.q.cuda(), table, lens, cu),
                     tiles.attention(s.q.cuda(), table, lens, cu, max_q=200),
                     cache.attention_selected(s.q.cuda(), idx, table, lens, cu),
                     tiles.attention_selected(s.q.cuda(), idx, table, lens, cu)):
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "bf16")
