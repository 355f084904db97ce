"""Rows whose scores are far from zero are no rows that see nothing."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("engine,rows", KERNELS)
def test_scores_far_from_zero(engine, rows, sign):
    """Scores of 8e34 either way over equal keys of one page.  (One page: a value scale is added
    to the score as its logarithm, so at this size the scores' last bit outweighs what two
    pages' scales differ by.)"""
    import torch
    s = ref.Setup([16], [8], 4, 1, 64, 16, "bf16", seed=36)
    s.c.codes["k"][:] = 0x38                           # 1
    s.c.scale["k"][:] = 1
    s.q[:] = sign * 2.0 ** 113
    cache, ints = _gpu(s, engine, rows)
    idx = torch.arange(16, device="cuda").to(torch.int32).expand(8, 16).contiguous()
    want = s.c.attend(np.zeros((8, 4, 64)), s.table, s.lens, s.cu)      # equal weights
    score = sign * 2.0 ** 113 * 64 / 8                 # beside which ln of the number of keys is nothing
    for out, lse in (cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows)),
                     cache.attention_selected(s.q.cuda(), idx, *ints)):
        ref.check(out.double().cpu().numpy(), np.zeros((8, 4)), (want[0], np.zeros((8, 4)), want[2]), "bf16")
        assert ((lse.double() / score - 1).abs() < 2.0 ** -20).all()
