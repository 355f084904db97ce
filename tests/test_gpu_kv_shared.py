"""Attention of sequences that begin with the same pages, against the 64-bit reference, which knows
nothing of what they share.  The bound is that of the attention (kv_reference): joining the two parts
adds the error of their logarithms, fp32 numbers below 2^7 in base 2, so 2^-17 of a weight, and the
bound's 2^-10 for scores holds 2^-14 more than the scores' 120 * 2^-17."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


def shared(groups, common, own, new, hq, hkv, d, page, dtype="bf16", seed=0):
    """A batch in groups of consecutive sequences: groups[g] of them, whose first common[g] pages
    are those of the group's first."""
    of = np.repeat(np.arange(len(groups)), groups)
    s = ref.Setup([common[of[b]] * page + own[b] for b in range(len(own))], new, hq, hkv, d, page, dtype, seed)
    first = np.concatenate([[0], np.cumsum(groups)])
    for b in range(len(own)):
        n = common[of[b]]
        s.table[b, :n] = s.table[first[of[b]], :n]
    s.first = first
    return s


def run(s, engine=0, groups=True, max_q=None, columns=0, **kw):
    import torch
    cache, ints = s.gpu(engine, columns)
    g = torch.tensor(s.first, dtype=torch.int32).cuda() if groups else None
    out, lse = cache.attention_shared(s.q.cuda(), *ints, groups=g, max_q=max_q, **kw)
    torch.cuda.synchronize()
    assert cache.status() == 0
    return out, lse, cache, ints


def check(s, out, lse):
    ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), s.c.attend(s.q64(), s.table, s.lens, s.cu), s.dtype)


@pytest.mark.parametrize("engine", [0, 1, 2])
@pytest.mark.parametrize("hq,hkv,d,page,dtype", [(8, 2, 128, 64, "bf16"), (7, 1, 64, 16, "f16"), (4, 4, 64, 128, "bf16"), (40, 2, 128, 32, "f16")])
def test_one_group(engine, hq, hkv, d, page, dtype):
    own = [1, 5, page, page + 1, 2 * page - 1]
    s = shared([5], [300 // page], own, [1] * 5, hq, hkv, d, page, dtype)
    check(s, *run(s, engine, groups=False)[:2])


@pytest.mark.parametrize("engine", [0, 1, 2])
def test_groups_of_all_sizes(engine):
    """One alone, one of many, one that shares nothing, prefixes of one page to nine."""
    sizes, common = [1, 9, 2, 3], [3, 9, 1, 0]
    own = [40, 1, 2, 16, 17, 31, 60, 8, 100, 33, 5, 7, 300, 20, 1]
    new = [1, 1, 2, 1, 3, 1, 20, 1, 1, 2, 1, 1, 64, 0, 1]
    s = shared(sizes, common, own, new, 6, 2, 64, 16, "f16")
    check(s, *run(s, engine, max_q=64)[:2])


@pytest.mark.parametrize("engine", [1, 2])
@pytest.mark.parametrize("new", [33, 150])
def test_chunks_behind_a_document(engine, new):
    """Causal within each sequence's own tokens; rows of one tile, of pairs and of the narrow form."""
    s = shared([4], [5], [new, new + 7, new + 64, new + 1], [new, new, new - 20, 1], 4, 2, 128, 64)
    check(s, *run(s, engine, groups=False, max_q=new)[:2])


@pytest.mark.parametrize("engine", [0, 1, 2])
def test_long_prefix_over_all_sms(engine):
    """The prefix is cut over the CTAs and joined again before the second step."""
    s = shared([3], [50], [3, 70, 129], [1, 1, 2], 8, 1, 128, 128)
    check(s, *run(s, engine, groups=False, max_q=2)[:2])


@pytest.mark.parametrize("engine", [0, 1, 2])
def test_what_is_not_shared(engine):
    """Tables that part inside the prefix, a first page of its own, a query inside the prefix, a sequence
    without queries and one without tokens: each still gets its own attention."""
    s = shared([8], [6], [5, 6, 7, 8, 9, 10, 1, 4], [1, 1, 1, 1, 0, 1, 1, 1], 4, 2, 64, 16)
    free = [p for p in range(s.pages) if p not in set(s.table.ravel().tolist())]
    s.table[1, 4] = free.pop()                       # parts after four pages
    s.table[2, 0] = free.pop()                       # shares nothing
    s.lens[3] = 3 * 16 + 1                           # its query sees three whole pages
    s.lens[5] = 9                                    # not one whole page
    s.table[4] = -1                                  # no queries: its table is not looked at
    s.lens[4] = 0
    s.lens[6] = 0                                    # a query that sees nothing
    s.table[6] = -1
    out, lse, _, _ = run(s, engine, groups=False)
    check(s, out, lse)
    assert float(out[5].abs().max()) == 0 and bool((lse[5] == -np.inf).all())   # sequence 6's query (4 has none)


@pytest.mark.parametrize("engine", [1, 2])
def test_the_same_page_table_for_all(engine):
    """Copies of one sequence: all but the last page is shared."""
    s = shared([4], [4], [64] * 4, [1] * 4, 4, 1, 128, 64)
    s.table[:] = s.table[0]
    out, lse, _, _ = run(s, engine, groups=False)
    check(s, out, lse)


@pytest.mark.parametrize("engine", [1, 2])
def test_the_bits_do_not_depend_on_what_else_runs(engine):
    """Twice, after other calls, from a graph and on another stream: the same bits."""
    import torch
    s = shared([3, 4], [20, 7], [1, 40, 3, 9, 10, 200, 64], [1, 2, 1, 1, 1, 5, 1], 8, 2, 128, 32)
    out, lse, cache, ints = run(s, engine, max_q=5)
    q, g = s.q.cuda(), torch.tensor(s.first, dtype=torch.int32).cuda()
    cache.attention(q, *ints)
    again = cache.attention_shared(q, *ints, groups=g, max_q=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = cache.attention_shared(q, *ints, groups=g, max_q=5, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = cache.attention_shared(q, *ints, groups=g, max_q=5)
    for _ in range(3):
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for got in (again, there, held):
            assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    assert cache.status() == 0


@pytest.mark.parametrize("engine", [1, 2])
def test_two_graphs(engine):
    """Two captured calls of different batches, replayed in turn: neither lives on what the other leaves."""
    import torch
    a = shared([3], [20], [1, 40, 3], [1, 2, 1], 8, 2, 128, 32)
    cache, ints = a.gpu(engine)
    q = a.q.cuda()
    few = [ints[0][:2].contiguous(), ints[1][:2].contiguous(), ints[2][:3].contiguous()]
    want = [cache.attention_shared(q, *ints, max_q=2), cache.attention_shared(q[:3], *few, max_q=2)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for x, i in ((q, ints), (q[:3], few)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(cache.attention_shared(x, *i, max_q=2))
        graphs.append(g)
    for turn in (0, 1, 1, 0, 1):
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got[turn], want[turn]))


@pytest.mark.parametrize("engine", [0, 1, 2])
def test_scores_far_apart(engine):
    """One part holds all of a row's weight, for some rows the shared one and for some their own."""
    s = shared([4], [6], [17, 18, 40, 33], [1] * 4, 4, 2, 64, 32, "f16")
    for h in range(2):
        s.c.scale["k"][s.table[0, :6], h] *= 2.0 ** 6          # shared keys: scores of some hundreds
    out, lse, _, _ = run(s, engine, groups=False)
    want, want_lse, A = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    # scores are 64 times those of the bound's derivation, and so are their errors
    tol = 2.0 ** -11 * 1.01 * np.abs(want) + (2.0 ** -11 + 64 * 2.0 ** -10 + 2.0 ** -11) * A + 2.0 ** -24
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 64 * 60 * 2.0 ** -17 + 2.0 ** -18 * (1 + np.abs(want_lse)))


@pytest.mark.parametrize("engine", [0, 1, 2])
def test_bad_pages_and_groups(engine):
    """A page outside the pool in the shared part: NaN for all who see it, reported.  Groups that do not
    rise: reported, and every sequence gets its own attention."""
    import torch
    s = shared([3, 2], [4, 4], [5, 6, 7, 8, 9], [1] * 5, 4, 2, 64, 16)
    cache, ints = s.gpu(engine)
    good, g = ints[0].clone(), torch.tensor(s.first, dtype=torch.int32).cuda()
    ints[0][:3, 2] = s.pages + 5
    out, lse = cache.attention_shared(s.q.cuda(), *ints, groups=g)
    assert cache.status() == 1
    assert bool(out[:3].isnan().all()) and not bool(out[3:].isnan().any()) and bool(lse[:3].isnan().all())
    for bad in ([0, 4, 3], [1, 3, 5], [0, 3, 4], [0, 3, 6], [-1, 3, 5], [0, 2**31 - 1, 5]):
        out, lse = cache.attention_shared(s.q.cuda(), good, *ints[1:], groups=torch.tensor(bad, dtype=torch.int32).cuda())
        assert cache.status() == 1
        check(s, out, lse)
    assert cache.status() == 0


def test_queries_past_the_table():
    """A sequence longer than its table: its query sees a page that is not there, the others do not."""
    import torch
    s = shared([3], [4], [16, 16, 16], [1] * 3, 4, 2, 64, 16)
    cache, ints = s.gpu(1)
    ints[1][1] = 5 * 16 + 1
    out, lse = cache.attention_shared(s.q.cuda(), *ints)
    assert cache.status() == 1
    assert bool(out[1].isnan().all())
    s.lens[1] = 80
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    keep = [0, 2]
    ref.check(out[keep].double().cpu().numpy(), lse[keep].double().cpu().numpy(), tuple(x[keep] for x in want), s.dtype)


def test_refusals():
    import torch
    from indexer_topk_long_gb300 import LtkError
    s = shared([2], [2], [3, 4], [1, 1], 4, 2, 64, 16)
    cache, ints = s.gpu()
    q = s.q.cuda()
    for bad, msg in ((torch.zeros(4, dtype=torch.int32, device="cuda"), "groups"), (torch.zeros(1, dtype=torch.int32, device="cuda"), "groups"),
                     (torch.zeros(2, dtype=torch.int64, device="cuda"), "int32"), (torch.zeros((2, 1), dtype=torch.int32, device="cuda"), "groups"),
                     (torch.zeros(2, dtype=torch.int32), "expected a tensor on")):
        with pytest.raises(ValueError, match=msg):
            cache.attention_shared(q, *ints, groups=bad)
    with pytest.raises(ValueError, match="32-bit"):
        cache.attention_shared(q, *ints, max_q=2**31)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(max_q=-1)):
        with pytest.raises(LtkError, match="ARG"):
            cache.attention_shared(q, *ints, **kw)
    with pytest.raises(LtkError, match="ARG"):
        cache.attention_shared(torch.zeros((2, 3, 64), dtype=torch.bfloat16, device="cuda"), *ints)
    # the C call's workspace: too small, or none
    from indexer_topk_long_gb300 import kv
    import ctypes
    b = kv.check_batch(*ints, 2, cache.device)
    out, lse = torch.empty_like(q), torch.empty((2, 4), device="cuda")
    size = ctypes.c_ulonglong(0)
    assert cache.lib.ltk_kv_shared_bytes(cache.h, 2, 2, 4, ctypes.byref(size)) == 0
    space = torch.empty(size.value, dtype=torch.uint8, device="cuda")
    for at, n in ((space.data_ptr(), size.value - 1), (None, size.value), (space.data_ptr() + 4, size.value)):
        assert cache.lib.ltk_kv_attention_shared(cache.h, ctypes.byref(b), None, 0, 0, q.data_ptr(), 256, 4, 1, 0.125, out.data_ptr(),
                                                 lse.data_ptr(), at, n, None) == 1
    empty = cache.attention_shared(q[:0], *ints[:2], torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert empty[0].shape == (0, 4, 64)


@pytest.mark.parametrize("hq,hkv,d,page,new", [(8, 2, 128, 64, 1), (32, 1, 64, 16, 3), (8, 1, 128, 32, 40)])
def test_chosen_by_the_table(hq, hkv, d, page, new):
    """A wide page table is taken for long sequences, which are attended to in two steps: few rows, a
    tile's, pairs'."""
    import torch
    s = shared([6, 2], [9, 4], [new + i for i in range(8)], [new] * 8, hq, hkv, d, page)
    out, lse, cache, ints = run(s, 0, max_q=new, columns=1 << 18)
    check(s, out, lse)
    before = cache.attention(s.q.cuda(), *ints, max_q=new)
    assert not torch.equal(before[1], lse)           # (joined sums differ in the last bits)
