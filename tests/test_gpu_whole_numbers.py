"""Numbers that have to be whole are not cut without a word."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [2.5, 0.5, -0.25, 1e9 + 0.5])
def test_top_k(k):
    import torch
    from indexer_topk_long_gb300 import sample
    x, u = torch.randn((2, 100), device="cuda"), torch.rand(2, device="cuda")
    with pytest.raises(ValueError, match="top_k: expected a whole number"):
        sample(x, u, top_k=k)
    for whole in (3, 3.0):                           # a whole number of another type is one
        assert torch.equal(sample(x, u, top_k=whole)[0], sample(x, u, top_k=torch.full((2,), 3, dtype=torch.int32, device="cuda"))[0])


@pytest.mark.parametrize("n", [9.5, 0.25])
def test_read(n):
    import kv_reference as ref
    import torch
    s = ref.Setup([40], [10], 2, 2, 64, 16)
    cache, ints = s.gpu()
    with pytest.raises(ValueError, match="n: expected the number of tokens"):
        cache.read(*ints, n)
    want = cache.read(*ints, 10)
    assert all(torch.equal(a, b) for a, b in zip(cache.read(*ints, 10.0), want))
