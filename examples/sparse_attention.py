"""One layer of sparse attention over a paged 8-bit cache, with random weights and tokens.

A prompt comes in chunks and then token by token.  Every step appends its keys and values
to the cache (rotating keys and queries on the way) and attends: to everything before it
while the context is short, and from then on to the ``--topk`` keys that IndexerTopK finds
for each query.  One layer of every few attends within a window and to the first tokens
instead; the example runs that too.

    python examples/sparse_attention.py --prompt 32768 --chunk 2048 --topk 2048 --decode 32
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from indexer_topk_long_gb300 import IndexerTopK, PagedKVCache  # noqa: E402

INDEX_HEADS, INDEX_DIM = 64, 128


def rotation_tables(positions: int, dim: int, base: float = 10000.0):
    angles = torch.arange(positions, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, dim, 2) / dim)
    return angles.cos().float().cuda(), angles.sin().float().cuda()


class SparseLayer:
    """The cache, the indexer's keys and the rotation tables of one layer and one sequence."""

    def __init__(self, max_len: int, max_new: int, q_heads: int, kv_heads: int, dim: int, page: int, topk: int):
        pages = -(-max_len // page)
        self.topk, self.page_count = topk, pages
        self.cache = PagedKVCache(pages, kv_heads, dim, page=page)
        # one handle for chunks and one for single tokens, each sized for its calls
        self.indexers = [IndexerTopK(max_T=n, max_S=max_len, k=topk, heads=INDEX_HEADS, dim=INDEX_DIM)
                         for n in (max_new, 1)]
        self.index_keys = torch.zeros((max_len, INDEX_DIM), dtype=torch.bfloat16, device="cuda")
        self.table = torch.randperm(pages, device="cuda").to(torch.int32)[None]     # pages in any order
        self.cos, self.sin = rotation_tables(max_len, dim)
        self.length = 0
        self.chosen = None          # keys chosen for the step before

    def step(self, q, k, v, index_q, index_w, index_k, dense: bool = False, window: int = 0, sinks: int = 0):
        """Appends n tokens and returns their attention's output [n, q_heads, dim] and lse."""
        n = q.shape[0]
        first, self.length = self.length, self.length + n
        lens = torch.tensor([self.length], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        q = self.cache.append(k, v, self.table, lens, cu, self.cos, self.sin, q=q)
        self.index_keys[first:self.length] = index_k
        if window or dense or self.length <= self.topk:
            return self.cache.attention(q, self.table, lens, cu, max_q=n, window=window, sinks=sinks)
        at = torch.arange(first, self.length, dtype=torch.int32, device="cuda")
        # each query's threshold starts from the keys that the step before it chose
        indexer = self.indexers[n == 1]
        sample = indexer.make_sample(self.chosen, self.length, min(3 * self.topk, 16384, self.length))
        idx, _ = indexer(index_q, index_w, self.index_keys[:self.length], at, prev_topk=sample)
        self.chosen = idx
        return self.cache.attention_selected(q, idx, self.table, lens, cu)


def tokens(n: int, q_heads: int, kv_heads: int, dim: int, rng):
    """What the layer's projections would give for n tokens."""
    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=rng, device="cuda").to(dtype)
    return dict(q=normal(n, q_heads, dim), k=normal(n, kv_heads, dim), v=normal(n, kv_heads, dim),
                index_q=normal(n, INDEX_HEADS, INDEX_DIM), index_w=normal(n, INDEX_HEADS, dtype=torch.float32).abs(),
                index_k=normal(n, INDEX_DIM))


def run(prompt: int, chunk: int, decode: int, topk: int, q_heads: int = 32, kv_heads: int = 4, dim: int = 128,
        page: int = 64, window: int = 0, sinks: int = 0, dense: bool = False, seed: int = 0):
    """Returns the outputs of all tokens, and (tokens, milliseconds) of each step."""
    rng = torch.Generator(device="cuda").manual_seed(seed)
    layer = SparseLayer(prompt + decode, chunk, q_heads, kv_heads, dim, page, topk)
    outs, times = [], []
    while layer.length < prompt + decode:
        n = min(chunk, prompt - layer.length) if layer.length < prompt else 1
        new = tokens(n, q_heads, kv_heads, dim, rng)
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        out, _ = layer.step(**new, dense=dense, window=window, sinks=sinks)
        t1.record()
        outs.append(out)
        times.append((n, t0, t1))
    torch.cuda.synchronize()
    if layer.cache.status() != 0:
        raise RuntimeError("the cache reports an error")
    return torch.cat(outs), [(n, a.elapsed_time(b)) for n, a, b in times]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("prompt", 32768), ("chunk", 2048), ("decode", 32), ("topk", 2048), ("q-heads", 32),
                        ("kv-heads", 4), ("dim", 128), ("page", 64), ("window", 1024), ("sinks", 4)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    sizes = dict(prompt=a.prompt, chunk=a.chunk, decode=a.decode, topk=a.topk, q_heads=a.q_heads, kv_heads=a.kv_heads,
                 dim=a.dim, page=a.page)
    for name, more in (("sparse", {}), ("window", dict(window=a.window, sinks=a.sinks)), ("dense", dict(dense=True))):
        run(**sizes, **more)                                        # warm up
        out, times = run(**sizes, **more)
        chunks, single = [t for n, t in times if n > 1], sorted(t for n, t in times if n == 1)
        last = "last chunk %8.3f ms" % chunks[-1] if chunks else ""
        print("%-7s %s  %s  finite %s" % (name, last, "one token %7.3f ms" % single[len(single) // 2] if single else "",
                                          bool(out.isfinite().all())))


if __name__ == "__main__":
    main()
