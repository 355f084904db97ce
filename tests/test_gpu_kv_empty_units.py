"""Row tiles whose queries see nothing, between others, many to a CTA."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("engine,rows", KERNELS)
@pytest.mark.parametrize("pattern", ["alternate", "runs"])
def test_empty_sequences_with_queries_between_others(engine, rows, pattern):
    """600 sequences of 128 queries (a pair of row tiles each, eight key tiles' worth to a CTA): empty
    ones, ones whose queries all lie before their first token but one, and ordinary ones."""
    import torch
    B, new = 600, 128
    rng = np.random.RandomState(51)
    if pattern == "alternate":
        lens = [0 if b % 2 else 300 - b % 70 for b in range(B)]
    else:
        lens = list(rng.choice([0, 0, 0, 1, 140, 300], B))
        lens[:12] = [0] * 12
        lens[-9:] = [0] * 9
    s = ref.Setup(lens, [new] * B, 2, 1, 64, 128, "bf16", seed=52)
    cache, ints = _gpu(s, engine, rows)
    q = s.q.cuda()
    out, lse = cache.attention(q, *ints, max_q=_hint(s, rows))
    assert cache.status() == 0
    first = torch.tensor(s.lens).repeat_interleave(new).view(B, new) - new
    sees = (first + torch.arange(new)).view(-1) >= 0
    assert (out[~sees.cuda()] == 0).all() and torch.isneginf(lse[~sees.cuda()]).all()
    assert torch.isfinite(lse[sees.cuda()]).all()
    for b in [i for i in range(B) if lens[i] > 0][::40]:
        got = slice(b * new + max(new - lens[b], 0), (b + 1) * new)
        want = s.c.attend(s.q64()[got], s.table[b:b + 1], [lens[b]], [0, got.stop - got.start])
        ref.check(out[got].double().cpu().numpy(), lse[got].double().cpu().numpy(), want, "bf16")
