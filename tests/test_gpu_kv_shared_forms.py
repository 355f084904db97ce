"""Attention of sequences that begin with the same pages, in the forms that its costs choose: a wide page table is taken for
long sequences, so that these short ones are attended to in two steps, by every kernel of the first one."""
import pytest

from test_gpu_kv_shared import check, run, shared

pytestmark = pytest.mark.gpu


# rows of a KV head in the first step: few, 17 to 64 (narrow tiles), up to 128, pairs; groups of uneven sizes pass
# these borders within one call
@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 64, 16), (8, 2, 128, 64), (16, 2, 128, 32), (3, 3, 64, 128)])
@pytest.mark.parametrize("sizes", [[3], [5], [15], [17], [33], [4, 6, 1], [13, 17, 20], [2, 70]], ids=str)
def test_rows_of_the_first_step(sizes, hq, hkv, d, page):
    B = sum(sizes)
    common = [max(1, (200 + 150 * g) // page) for g in range(len(sizes))]
    own = [1 + (7 * b) % (page + 9) for b in range(B)]
    new = [1 + (b % 3 == 2 and own[b] > 2) for b in range(B)]
    s = shared(sizes, common, own, new, hq, hkv, d, page, "f16" if B % 2 else "bf16", seed=B)
    out, lse, cache, ints = run(s, 0, max_q=2, columns=1 << 16)
    check(s, out, lse)


def test_graphs_of_two_shapes():
    """Two captured calls of different forms on one cache, replayed in turn, give what each gave by itself."""
    import torch
    a = shared([17], [9], [3 + b for b in range(17)], [1] * 17, 8, 2, 128, 64, seed=1)
    cache, ints = a.gpu(0, 1 << 16)
    q = a.q.cuda()
    part = [x.contiguous() for x in (ints[0][:5], ints[1][:5], ints[2][:6])]
    calls = [lambda: cache.attention_shared(q, *ints, max_q=1), lambda: cache.attention_shared(q[:5], *part, max_q=1)]
    want = [[t.clone() for t in call()] for call in calls]
    graphs, got = [], []
    for call in calls:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(call())
        graphs.append(g)
    for g in (0, 1, 1, 0, 0, 1):
        graphs[g].replay()
        torch.cuda.synchronize()
        for x, y in zip(want[g], got[g]):
            assert torch.equal(x, y)
