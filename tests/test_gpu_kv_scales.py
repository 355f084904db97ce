"""Scales and magnitudes at the edge: blocks without a scale, scales that are no powers
of two, scores far from zero, query heads of very different size."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _dense, _gpu, _hint, _selected

pytestmark = pytest.mark.gpu


# --- blocks without a scale hold zeros ---------------------------------------------------------
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (70, 20)])
@pytest.mark.parametrize("new", [1, 40])
def test_zero_scale_is_a_block_of_zeros(new, window, sinks):
    """Value scales of 0 on a seen page, on a page that the window leaves out of a tile that it
    reaches into, and on a page that was never written (both scales and all codes 0)."""
    s = ref.Setup([520, 300], [new, new], 4, 2, 128, 16, "bf16", seed=31)
    for b, pages in ((0, (0, 20, 26, 30)), (1, (3, 12, 18))):
        for pg in pages:
            s.c.scale["v"][s.table[b, pg]] = 0
    s.c.scale["v"][s.table[0, 31], 1] = 0              # of one head only
    for name in "kv":
        s.c.scale[name][s.table[1, 16]] = 0
        s.c.codes[name][s.table[1, 16]] = 0
    _dense(s, window, sinks)


@pytest.mark.parametrize("hq,k", [(4, 130), (40, 77), (64, 300), (100, 200)])
def test_zero_scale_on_listed_keys(hq, k):
    s = ref.Setup([500], [7], hq, 1, 64, 32, "bf16", seed=32)
    for pg in (0, 3, 4, 9):
        s.c.scale["v"][s.table[0, pg]] = 0
    s.c.scale["k"][s.table[0, 5]] = 0
    rng = np.random.RandomState(6)
    idx = np.stack([rng.permutation(490)[:k] for _ in range(7)]).astype(np.int32)
    _selected(s, idx)


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_only_zero_scales(engine, rows):
    """Everything seen is zero: the output is, and lse still counts the keys."""
    import torch
    s = ref.Setup([200], [30], 4, 1, 128, 64, "f16", seed=33)
    s.c.scale["v"][:] = 0
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu)
    cache, ints = _gpu(s, engine, rows)
    idx = torch.arange(200, device="cuda").to(torch.int32).expand(30, 200).contiguous()
    for out, lse in (cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows)),
                     cache.attention_selected(s.q.cuda(), idx, *ints)):
        assert (out == 0).all()
        ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "f16")


@pytest.mark.parametrize("hq", [4, 64, 100])
def test_zero_scale_beside_tiny_scales(hq):
    """A block without a scale does not push the others' weights out of their type's range."""
    s = ref.Setup([300], [3], hq, 1, 128, 16, "bf16", seed=34, spread=0.0)
    s.c.scale["v"] *= np.float32(2.0 ** -24)
    s.c.scale["v"][s.table[0, 2]] = 0
    _dense(s)
    _selected(s, np.stack([np.random.RandomState(i).permutation(290)[:150] for i in range(3)]).astype(np.int32))
