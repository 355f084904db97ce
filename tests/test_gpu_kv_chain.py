"""Calls that follow each other without a pause: each kernel starts while the one before it ends."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,engine", [(256, 1), (24, 2)])
def test_attention_sees_scales_and_codes_that_have_just_grown(B, engine):
    """Every append raises the exponent of all partly filled pages (their codes and scales change,
    32 scales to a line and each written by another block), and attention reads them at once.
    In a graph the bits are those of calls with a pause between them."""
    import torch
    from indexer_topk_long_gb300 import PagedKVCache
    hkv, g, d, page, steps, held = 8, 2 if engine == 1 else 8, 128, 32, 6, 40
    gen = torch.Generator(device="cuda").manual_seed(7)
    ints = dict(dtype=torch.int32, device="cuda")
    width = -(-(held + steps) // page)
    table = torch.randperm(B * width, device="cuda", generator=gen).to(torch.int32).view(B, width)
    cu = torch.arange(B + 1, **ints)
    lens = [torch.full((B,), held + i + 1, **ints) for i in range(steps)]

    def rand(n, h, gain=1.0):
        return (torch.randn((n, h, d), device="cuda", generator=gen) * gain).bfloat16()
    k0, v0 = rand(B * held, hkv, 0.25), rand(B * held, hkv, 0.25)
    new = [(rand(B, hkv, 2.0 ** (i - 2)), rand(B, hkv, 2.0 ** (2 * i)), rand(B, hkv * g, 0.5)) for i in range(steps)]
    angle = torch.rand((held + steps, d // 2), device="cuda", generator=gen)
    cos, sin = angle.cos(), angle.sin()
    idx = torch.argsort(torch.rand((B, held + 1), device="cuda", generator=gen), dim=1)[:, :30].to(torch.int32).contiguous()

    def fresh():
        cache = PagedKVCache(B * width, hkv, d, page=page, engine=engine)
        cache.append(k0, v0, table, torch.full((B,), held, **ints), torch.arange(B + 1, **ints) * held, cos, sin)
        return cache

    def run(cache, pause):
        results = []
        for i in range(steps):
            k, v, q = new[i]
            q = cache.append(k, v, table, lens[i], cu, cos, sin, q=q)
            pause()
            results += [q, *cache.attention(q, table, lens[i], cu, max_q=1)]
            pause()
            results += cache.attention_selected(q, idx, table, lens[i], cu)
            pause()
        return results
    cache = fresh()
    want = [t.clone() for t in run(cache, torch.cuda.synchronize)]
    cache = fresh()
    buffers = (cache.k_codes, cache.v_codes, cache.k_scale, cache.v_scale)
    before = [t.clone() for t in buffers]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(cache, lambda: None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(cache, lambda: None)
    for _ in range(10):
        for t, b in zip(buffers, before):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert cache.status() == 0
        assert not any(t.isnan().any() for t in got)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
