"""The token sampler without a GPU: the C entry point's refusals, made before any CUDA call, and the reference
that the GPU tests use, on cases worked out by hand."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sampling_reference as ref
from indexer_topk_long_gb300 import ltk, sample


def _call(lib, logits=64, dtype=3, stride=10, B=2, V=10, u=64, token=64, logp=64, settings=(None, None, None, None, 1.0, 0, 1.0, 0.0)):
    s = ltk.Sampling(*settings) if settings is not None else None
    return lib.ltk_sample_tokens(logits, dtype, stride, B, V, None if s is None else ctypes.byref(s), u, token, logp, None)


@pytest.mark.parametrize("kw", [
    dict(dtype=1), dict(dtype=4), dict(dtype=-1), dict(V=0), dict(B=-1), dict(stride=9), dict(settings=None), dict(logits=None), dict(logits=66),
    dict(logits=65, dtype=0), dict(u=None), dict(u=2), dict(token=None), dict(logp=None), dict(logp=65)])
def test_refused_on_the_host(ltk_lib, kw):
    assert _call(ltk_lib, **kw) == 1


@pytest.mark.parametrize("at,value", [(0, 2), (1, 3), (2, 1), (3, 2), (4, -1.0), (4, math.inf), (4, math.nan), (6, -0.5), (6, math.nan), (7, -0.1),
                                      (7, 1.5), (7, math.nan)])
def test_settings_refused_on_the_host(ltk_lib, at, value):
    s = [None, None, None, None, 1.0, 0, 1.0, 0.0]
    s[at] = value
    assert _call(ltk_lib, settings=s) == 1


def test_sizes_on_the_host(ltk_lib):
    assert _call(ltk_lib, V=360001, stride=360001) == 6
    assert _call(ltk_lib, V=720001, stride=720001, dtype=0) == 6
    assert _call(ltk_lib, B=0, logits=None, u=None, token=None, logp=None) == 0


def test_binding_wants_cuda_tensors():
    with pytest.raises(ValueError, match="CUDA"):
        sample(torch.zeros((2, 5)), torch.zeros(2))


def _tokens(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    return ref.sample_row(np.asarray(x, dtype=np.float64), u, temperature, top_k, top_p, min_p)[0]


def test_reference_by_hand():
    x = np.log([1, 2, 4, 1])                         # weights 1, 2, 4, 1
    assert [_tokens(x, u) for u in (0.0, 0.1, 0.13, 0.37, 0.38, 0.87, 0.9)] == [[0], [0], [1], [1], [2], [2], [3]]
    assert _tokens(x, 0.99, top_k=3) == [2] and _tokens(x, 0.0, top_k=3) == [0]        # 2, 1, and of the equal ones the first
    assert _tokens(x, 0.0, top_p=0.7) == [1] and _tokens(x, 0.0, top_p=0.45) == [2]
    assert _tokens(x, 0.0, min_p=0.3) == [1] and _tokens(x, 0.9, min_p=0.3) == [2]
    assert _tokens(x, 0.0, top_k=2, top_p=0.6) == [2]                                   # 4 of 6 reach 0.6
    assert _tokens(x, 0.0, temperature=0.0) == [2]
    assert _tokens([-np.inf] * 3, 0.5) == [-1] and _tokens([0, np.nan], 0.5) == [-1]
    assert _tokens([-np.inf, 1.0], 0.0) == [1]


def test_reference_notices_mistakes():
    """Filters in another order, a draw by rank instead of by index, ties to the higher index: other tokens."""
    x = np.log([1, 2, 4, 1])
    assert _tokens(x, 0.0, top_k=3) != [2]           # by rank the first would be the largest
    assert _tokens(x, 0.99, top_k=3) != [3]          # ties to the higher index would keep 3
    # top-p before min-p: 0.9 of 8 keeps all four weights, then min-p two; after it: 0.9 of 6 keeps both
    assert _tokens(np.log([10, 1, 1, 1, 1, 1, 1, 4]), 0.99, top_p=0.7, min_p=0.3) == [0]
