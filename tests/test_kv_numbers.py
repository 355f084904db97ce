"""Whole numbers that 32 bits do not hold are refused, not cut (no GPU: the C entry point is a stand-in)."""
import pytest
import torch

from indexer_topk_long_gb300 import PagedKVCache, kv


def _cache(calls):
    """A binding on the CPU whose attention call is recorded instead of made."""
    c = PagedKVCache.__new__(PagedKVCache)
    c.h, c.heads, c.dim, c.device, c._index = 1, 2, 64, torch.device("cpu"), 0
    c._torch, c._int32, c._float32, c._default_scale = torch, torch.int32, torch.float32, 0.125
    c._raw_stream, c._codes = (lambda i: 0), {torch.bfloat16: 0}
    c._attend = lambda *a: calls.append(a) or 0
    c.close = lambda: None
    return c


def _batch():
    ints = dict(dtype=torch.int32)
    return (torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((1, 2), **ints), torch.full((1,), 3, **ints),
            torch.tensor([0, 3], **ints))


@pytest.mark.parametrize("name", ["window", "sinks", "max_q"])
@pytest.mark.parametrize("value", [2**31, 2**32, 2**32 + 5, 2**40 + 1, -2**31 - 1, -2**32 + 5])
def test_numbers_beyond_32_bits(name, value):
    calls = []
    with pytest.raises(ValueError, match=name + ".*32-bit"):
        _cache(calls).attention(*_batch(), **{name: value})
    assert not calls


@pytest.mark.parametrize("name", ["window", "sinks", "max_q"])
@pytest.mark.parametrize("value", [0, 1, 2**31 - 1, -1, -2**31])
def test_numbers_of_32_bits_reach_the_library(name, value):
    """(which refuses the negative ones)"""
    calls = []
    _cache(calls).attention(*_batch(), **{name: value})
    assert value in calls[0]


@pytest.mark.parametrize("what", [dict(heads=2**32 + 1), dict(dim=2**32 + 64), dict(page=2**32 + 64), dict(engine=2**32)])
def test_configuration_beyond_32_bits(ltk_lib, what):
    with pytest.raises(ValueError, match="32-bit"):
        PagedKVCache(**{**dict(num_pages=4, heads=1, dim=64), **what})


def test_the_check_itself():
    kv._int32s(a=0, b=-2**31, c=2**31 - 1)
    with pytest.raises(ValueError, match="c: "):
        kv._int32s(a=0, c=2**31)
