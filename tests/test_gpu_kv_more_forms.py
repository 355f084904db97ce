"""Forms of the cache's kernels at sizes that the other tests do not reach: the listed kernel's
whole waves at 128 elements a head, append by token with other types and pairings, batches of
chunks and single tokens together."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_append import _inputs, _run, _same, _tables
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,hq,hkv,d,k,dtype", [
    (1100, 64, 1, 128, 130, "bf16"),       # seven waves of units and a rest, units of two tiles
    (500, 64, 1, 128, 700, "bf16"),        # units of six tiles, more than the rings hold
    (320, 40, 2, 128, 128, "f16"),         # one tile a unit, rows that do not fill a half
    (460, 17, 1, 128, 1, "bf16"),          # one key
    (330, 64, 1, 64, 2048, "bf16"),
])
def test_listed_whole_waves(new, hq, hkv, d, k, dtype):
    import torch
    held = max(k, 300)
    s = ref.Setup([new + held], [new], hq, hkv, d, 64, dtype, seed=71)
    rng = np.random.RandomState(4)
    idx = np.stack([rng.permutation(held)[:k] for _ in range(new)]).astype(np.int32)
    idx[::7, k // 3:k // 2] = -1           # empty slots in some
    pick = np.unique(np.concatenate([rng.randint(0, new, 10), [0, 151, 152, new - 1]]))
    cache, ints = s.gpu(2)
    for _ in range(2):
        out, lse = cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints)
        assert cache.status() == 0
        for i in pick:                     # each alone, as a sequence's last token
            want = s.c.attend(s.q64()[i:i + 1], s.table, [held + i + 1], [0, 1], idx=idx[i:i + 1])
            ref.check(out[i:i + 1].double().cpu().numpy(), lse[i:i + 1].double().cpu().numpy(), want, dtype)


@pytest.mark.parametrize("lens,new,hq,hkv,d,page,dtype,rot,inter", [
    ([1], [1], 4, 1, 64, 16, "f16", 64, True),
    ([17, 64, 65, 5, 33, 16], [1, 1, 1, 1, 1, 1], 14, 2, 64, 16, "f16", 32, True),
    ([17, 64, 65, 5], [1, 1, 1, 1], 8, 2, 128, 64, "f16", 128, False),
    ([130, 40, 90], [0, 8, 7], 6, 3, 128, 32, "bf16", 96, True),
    ([18, 50, 128], [6, 8, 8], 5, 1, 64, 16, "bf16", 48, False),
])
def test_append_by_token(lens, new, hq, hkv, d, page, dtype, rot, inter):
    import torch
    assert sum(new) <= 8 * len(lens)
    s = ref.Setup(lens, new, hq, hkv, d, page, dtype, seed=72)
    for name in "kv":
        s.c.codes[name][s.c.codes[name] == 0x7F] = 0
    cache, ints = s.gpu()
    cos, sin = _tables(max(lens), rot)
    got, q = _run(cache, s.c, ints, _inputs(s.cu[-1], hq, hkv, d, dtype, 6, 4.0), hq, hkv, cos, sin, inter, s.table, s.lens, s.cu)
    _same(cache, s.c)
    for b in range(len(lens)):
        for i in range(new[b]):
            t, p = s.cu[b] + i, lens[b] - new[b] + i
            assert torch.equal(got[t].cpu(), torch.from_numpy(ref.rotate(q[t], cos[p], sin[p], inter)).to(got.dtype))


@pytest.mark.parametrize("engine,rows", [(0, 1200)] + KERNELS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 4)])
def test_chunks_and_single_tokens_together(engine, rows, window, sinks):
    s = ref.Setup([700] + [90, 1, 1300, 128, 129, 500, 17] + [260], [300] + [1] * 7 + [45], 4, 1, 64, 32, "bf16", seed=73)
    cache, ints = _gpu(s, engine, rows)
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), window=window, sinks=sinks)
    assert cache.status() == 0
    want = s.c.attend(s.q64(), s.table, s.lens, s.cu, window, sinks)
    ref.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), want, "bf16")
