"""The example that runs append, the indexer and both attentions together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_attention.py")
    spec = importlib.util.spec_from_file_location("sparse_attention", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("prompt,chunk,q_heads,kv_heads,dim,page", [(700, 256, 8, 2, 128, 64), (333, 100, 4, 4, 64, 16)])
def test_all_keys_give_dense_attention(prompt, chunk, q_heads, kv_heads, dim, page):
    """A window of the whole context gives dense attention's bits, and a selection of 512 keys
    gives its results for every token that sees no more than those."""
    import torch
    ex = _example()
    sizes = dict(prompt=prompt, chunk=chunk, decode=3, q_heads=q_heads, kv_heads=kv_heads, dim=dim, page=page)
    total = prompt + 3
    dense, _ = ex.run(**sizes, topk=512, dense=True)
    wide, _ = ex.run(**sizes, topk=512, window=total + 1)
    assert torch.equal(dense, wide)
    sparse, times = ex.run(**sizes, topk=512)
    assert len(times) == -(-prompt // chunk) + 3
    few = dense[:min(total, 512)].double()
    # the first 512 tokens see at most 512 keys, whichever path they take: the same softmax,
    # rounded once to bf16 (2^-8) from weights in f16 and sums in other orders
    off = (sparse[:len(few)].double() - few).norm() / few.norm()
    assert off < 2.0 ** -7
    assert sparse.isfinite().all()


def test_example_with_window_and_sinks():
    ex = _example()
    out, times = ex.run(prompt=600, chunk=200, decode=2, topk=64, window=50, sinks=4)
    assert out.isfinite().all() and out.shape == (602, 32, 128) and [n for n, _ in times] == [200] * 3 + [1] * 2


@pytest.mark.parametrize("new", [[1] * 6, [40, 1, 7, 0, 90, 3]])
def test_a_step_in_one_graph(new):
    """Append and both attentions captured together: each starts while the one before it ends,
    and a replay gives the bits of the calls made one by one."""
    import torch
    from indexer_topk_long_gb300 import PagedKVCache
    lens = [700, 64, 1000, 130, 90, 300]
    B, hkv, g, d, page = len(lens), 2, 4, 128, 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    width, N = -(-max(lens) // page), sum(new)
    ints = dict(dtype=torch.int32, device="cuda")
    table = torch.randperm(B * width, device="cuda", generator=gen).to(torch.int32).view(B, width)
    cu = torch.tensor([sum(new[:i]) for i in range(B + 1)], **ints)
    held = torch.tensor([n - m for n, m in zip(lens, new)], **ints)
    seq = torch.tensor(lens, **ints)
    first = torch.tensor([sum(lens[i] - new[i] for i in range(j)) for j in range(B + 1)], **ints)

    def rand(n, h):
        return torch.randn((n, h, d), device="cuda", generator=gen).bfloat16()
    k0, v0, k, v, q = rand(int(first[-1]), hkv), rand(int(first[-1]), hkv), rand(N, hkv), rand(N, hkv), rand(N, hkv * g)
    angle = torch.rand((max(lens), d // 2), device="cuda", generator=gen)
    cos, sin = angle.cos(), angle.sin()
    idx = torch.argsort(torch.rand((N, 1000), device="cuda", generator=gen), dim=1)[:, :200].to(torch.int32).contiguous()

    def step(cache):
        q2 = cache.append(k, v, table, seq, cu, cos, sin, q=q)
        out, lse = cache.attention(q2, table, seq, cu, max_q=max(new))
        win, _ = cache.attention(q2, table, seq, cu, max_q=max(new), window=50, sinks=2)
        sel, lse2 = cache.attention_selected(q2, idx, table, seq, cu)
        return q2, out, lse, win, sel, lse2

    def fresh():
        cache = PagedKVCache(B * width, hkv, d, page=page)
        cache.append(k0, v0, table, held, first, cos, sin)
        return cache
    want = []
    cache = fresh()
    for t in step(cache):
        torch.cuda.synchronize()
        want.append(t.clone())
    cache = fresh()
    before = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(cache)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache)
    for _ in range(3):
        for t, b in zip((cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale), before):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert cache.status() == 0
        for a, b in zip(got, want):
            assert torch.equal(a, b)
