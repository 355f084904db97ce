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
