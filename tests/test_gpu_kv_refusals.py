"""Refusals of the paged cache's calls that need a live handle."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cache():
    from indexer_topk_long_gb300 import PagedKVCache
    return PagedKVCache(8, 2, 128, page=64)


def _ints():
    import torch
    return [torch.zeros((1, 4), dtype=torch.int32, device="cuda"), torch.full((1,), 3, dtype=torch.int32, device="cuda"),
            torch.tensor([0, 3], dtype=torch.int32, device="cuda")]


def _x(heads, n=3, d=128, dtype="bfloat16"):
    import torch
    return torch.zeros((n, heads, d), dtype=getattr(torch, dtype), device="cuda")


def test_binding_refuses(cache):
    import torch
    from indexer_topk_long_gb300 import LtkError, PagedKVCache
    i = _ints()
    cos = torch.zeros((10, 64), device="cuda")
    with pytest.raises(ValueError, match="heads"):
        cache.append(_x(3), _x(3), *i)
    with pytest.raises(ValueError, match="like the others"):
        cache.append(_x(2), _x(2, dtype="float16"), *i)
    with pytest.raises(ValueError, match="both or neither"):
        cache.append(_x(2), _x(2), *i, cos=cos)
    with pytest.raises(ValueError, match="equal shape"):
        cache.append(_x(2), _x(2), *i, cos=cos, sin=cos[:5])
    with pytest.raises(ValueError, match="without q"):
        cache.append(_x(2), _x(2), *i, q_out=_x(4))
    with pytest.raises(LtkError, match="ARG"):       # rotates more than a head holds
        cache.append(_x(2), _x(2), *i, cos=torch.zeros((10, 72), device="cuda"), sin=torch.zeros((10, 72), device="cuda"))
    with pytest.raises(LtkError, match="UNSUPPORTED"):
        cache.append(_x(2), _x(2), *i, cos=torch.zeros((10, 20), device="cuda"), sin=torch.zeros((10, 20), device="cuda"))
    with pytest.raises(LtkError, match="ARG"):       # 3 query heads over 2 KV heads
        cache.attention(_x(3), *i)
    for kw in (dict(window=-1), dict(sinks=-2), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(LtkError, match="ARG"):
            cache.attention(_x(4), *i, **kw)
    with pytest.raises(ValueError, match="out"):
        cache.attention(_x(4), *i, out=_x(2))
    with pytest.raises(ValueError, match="lse"):
        cache.attention(_x(4), *i, lse=torch.zeros(12, device="cuda"))
    with pytest.raises(ValueError, match="idx"):
        cache.attention_selected(_x(4), torch.zeros((2, 5), dtype=torch.int32, device="cuda"), *i)
    with pytest.raises(ValueError, match="int32"):
        cache.attention_selected(_x(4), torch.zeros((3, 5), dtype=torch.int64, device="cuda"), *i)
    with pytest.raises(LtkError, match="ARG"):
        cache.attention_selected(_x(4), torch.zeros((3, 0), dtype=torch.int32, device="cuda"), *i)
    with pytest.raises(ValueError, match="all four"):
        PagedKVCache(8, 2, 128, k_codes=cache.k_codes)
    with pytest.raises(ValueError, match="shape"):
        PagedKVCache(9, 2, 128, k_codes=cache.k_codes, v_codes=cache.v_codes, k_scale=cache.k_scale,
                     v_scale=cache.v_scale)


def test_nothing_to_do(cache):
    import torch
    i = _ints()
    i[2].zero_()
    assert cache.append(_x(2, 0), _x(2, 0), *i, q=_x(4, 0)).shape == (0, 4, 128)
    out, lse = cache.attention(_x(4, 0), *i)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    out, lse = cache.attention_selected(_x(4, 0), torch.zeros((0, 5), dtype=torch.int32, device="cuda"), *i)
    assert out.shape == (0, 4, 128)


def test_closed_cache():
    from indexer_topk_long_gb300 import PagedKVCache
    c = PagedKVCache(2, 1, 64, page=16)
    c.close()
    c.close()
    with pytest.raises(ValueError, match="closed"):
        c.attention(_x(1, d=64), *_ints())


def test_misaligned_pointers(cache):
    from indexer_topk_long_gb300 import ltk
    i = _ints()
    q, out = _x(4), _x(4)
    b = ltk.KvBatch(i[0].data_ptr(), 4, i[1].data_ptr(), i[2].data_ptr(), 1, 3)

    def call(batch=b, q_at=0, stride=512, out_at=0, dtype=0):
        return cache.lib.ltk_kv_attention(cache.h, ctypes.byref(batch), dtype, q.data_ptr() + q_at, stride, 4, 1, 0.1, 0,
                                          0, out.data_ptr() + out_at, None, None)
    assert call() == 0
    assert call(q_at=8) == 1 and call(out_at=2) == 1 and call(stride=516) == 1 and call(stride=8) == 1
    assert call(dtype=1) == 1 and call(dtype=9) == 1
    assert call(batch=ltk.KvBatch(i[0].data_ptr() + 2, 4, i[1].data_ptr(), i[2].data_ptr(), 1, 3)) == 1
    assert call(batch=ltk.KvBatch(i[0].data_ptr(), 4, i[1].data_ptr(), None, 1, 3)) == 1
    assert call(batch=ltk.KvBatch(i[0].data_ptr(), 0, i[1].data_ptr(), i[2].data_ptr(), 1, 3)) == 1
    assert call(batch=ltk.KvBatch(i[0].data_ptr(), 1 << 30, i[1].data_ptr(), i[2].data_ptr(), 1, 3)) == 1
    assert call(batch=ltk.KvBatch(i[0].data_ptr(), 4, i[1].data_ptr(), i[2].data_ptr(), 1, -3)) == 1
