"""Windows and first tokens of any 32-bit size: one that reaches past everything hides nothing."""
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(2**31 - 1, 0), (2**31 - 2, 4), (2**31 - 40, 2**31 - 1), (2**30, 1),
                                          (50, 2**31 - 1), (0, 2**31 - 1)])
@pytest.mark.parametrize("engine,rows", KERNELS)
def test_window_beyond_everything(engine, rows, window, sinks):
    """Sequences shorter than their queries by two and more among them."""
    import torch
    lens, new = [3, 300, 0, 140, 1, 20], [50, 40, 7, 1, 60, 20]
    s = ref.Setup(lens, new, 4, 2, 64, 32, "bf16", seed=55)
    cache, ints = _gpu(s, engine, rows)
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), window=window, sinks=sinks)
    assert cache.status() == 0
    for b, (n, m) in enumerate(zip(lens, new)):
        at, live = s.cu[b], min(n, m)
        none = slice(at, at + m - live)
        assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()
        got = slice(at + m - live, at + m)
        want = s.c.attend(s.q64()[got], s.table[b:b + 1], [n], [0, live])
        ref.check(out[got].double().cpu().numpy(), lse[got].double().cpu().numpy(), want, "bf16")
