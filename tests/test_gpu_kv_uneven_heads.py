import numpy as np
import pytest
import kv_reference as ref
pytestmark = pytest.mark.gpu

# --- query heads of very different size ---------------------------------------------------------
@pytest.mark.parametrize("dtype,up", [("bf16", 40), ("bf16", 90), ("f16", 24)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("engine", [1, 2])
def test_a_large_head_leaves_the_others_alone(engine, d, dtype, up):
    """Heads 3 and 40 of 64 on one KV head are 2^up times the others: the others' results are
    as exact as without them."""
    import torch
    s = ref.Setup([300], [4], 64, 1, d, 32, dtype, seed=37)
    if dtype == "f16":                                 # small ones instead: f16 ends at 65504
        q = s.q.double() * 2.0 ** -12
        q[:, [3, 40]] *= 2.0 ** up
        scale = d ** -0.5 * 2.0 ** 12
    else:
        q = s.q.double()
        q[:, [3, 40]] *= 2.0 ** up
        scale = d ** -0.5
    s.q = q.to(s.q.dtype)
    idx = np.stack([np.random.RandomState(i).permutation(296)[:150] for i in range(4)]).astype(np.int32)
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, idx=idx, scale=scale)
    cache, ints = s.gpu(engine)
    out, lse = cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints, scale=scale)
    assert cache.status() == 0
    rest = [h for h in range(64) if h not in (3, 40)]
    ref.check(out[:, rest].double().cpu().numpy(), lse[:, rest].double().cpu().numpy(),
              tuple(t[:, rest] for t in want), dtype)
    assert out.isfinite().all()
