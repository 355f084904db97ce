"""Scores so large that fp32 holds them to a few binary orders only: still a softmax."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 25 * 1.3, 2.0 ** 26, 2.0 ** 26 * 1.37, 2.0 ** 26 * 1.9, 2.0 ** 27 * 1.1,
                                 2.0 ** 27 * 1.45, 2.0 ** 27 * 1.85, 2.0 ** 28 * 1.25])
@pytest.mark.parametrize("hq", [4, 64, 100])
@pytest.mark.parametrize("order", ["mixed", "rising"])
def test_large_scores_take_their_largest(hq, order, top):
    """Scores are a product of one element, so exact, and differ by a sixteenth or not at all: each
    query takes the mean of the values of its largest keys."""
    import torch
    s = ref.Setup([400], [5], hq, 1, 64, 16, "bf16", seed=57, spread=0.0)
    rng = np.random.RandomState(8)
    codes = rng.choice(np.concatenate([np.arange(0x40, 0x7F, 2), np.arange(0xC0, 0xFF, 2)]), 400)
    if order == "rising":
        codes = codes[np.argsort(ref.E4M3[codes], kind="stable")]
    s.c.codes["k"][:] = 0
    s.c.scale["k"][:] = s.c.scale["v"][:] = 1
    for j in range(400):
        s.c.codes["k"][s.table[0, j // 16], 0, j % 16, 0] = codes[j]
    s.q[:] = 0
    s.q[:, :, 0] = torch.where(torch.arange(hq) % 3 == 0, -1.0, 1.0).to(s.q.dtype)
    scale = float(np.float32(top * np.log(2.0) / 448))         # the largest exponent (base 2) is `top`
    idx = np.stack([np.sort(rng.permutation(395)[:300]) for _ in range(5)]).astype(np.int32)

    def same(got, want):
        out, lse = (t.double().cpu().numpy() for t in got)
        ref.check(out, np.zeros(lse.shape), (want[0], np.zeros(lse.shape), want[2]), "bf16")
        # (the exponents' product with ln 2 and the scale are rounded to fp32)
        np.testing.assert_allclose(lse, want[1], rtol=2.0 ** -21)
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, scale=scale)
    for engine, rows in KERNELS:
        cache, ints = _gpu(s, engine, rows)
        same(cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), scale=scale), want)
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, idx=idx, scale=scale)
    for engine in (1, 2):
        cache, ints = s.gpu(engine)
        same(cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints, scale=scale), want)
