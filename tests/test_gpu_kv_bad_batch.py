"""Batches that contradict themselves: what is reported, and that nothing else is touched."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [[40, 30], [2, 3]])
@pytest.mark.parametrize("bad", ["falls", "beyond", "negative"])
def test_append_under_a_cu_q_that_does_not_rise(new, bad):
    """Both append forms: pages that the table does not name stay as they are, and so do the
    tokens before the new ones; the next call is right."""
    import torch
    lens = [60, 50]
    s = ref.Setup(lens, new, 1, 2, 64, 16, "bf16", seed=61)
    for name in "kv":
        s.c.codes[name][s.c.codes[name] == 0x7F] = 0
    cache, ints = s.gpu()
    N = s.cu[-1]
    cu = {"falls": [0, N - 1, 1], "beyond": [0, new[0], 1 << 30], "negative": [-7, new[0], N]}[bad]
    x = torch.randn((N, 4, 64), generator=torch.Generator().manual_seed(2)).bfloat16() * 0.01   # (no scale grows)
    held = {n: s.c.codes[n].copy() for n in "kv"}
    cache.append(x[:, :2].cuda(), x[:, 2:].cuda(), ints[0], ints[1], torch.tensor(cu, dtype=torch.int32).cuda())
    cache.status()
    spare = np.setdiff1d(np.arange(s.pages), s.table[s.table >= 0])
    assert len(spare) == 2
    for name, codes in (("k", cache.k_codes), ("v", cache.v_codes)):
        got = codes.cpu().numpy()
        np.testing.assert_array_equal(got[spare], held[name][spare])
        for b in range(2):                              # no sequence has more than N new tokens
            for p in range(max(lens[b] - N, 0)):
                np.testing.assert_array_equal(got[s.table[b, p // 16], :, p % 16], held[name][s.table[b, p // 16], :, p % 16])
    for n, c, sc in (("k", cache.k_codes, cache.k_scale), ("v", cache.v_codes, cache.v_scale)):
        c.copy_(torch.from_numpy(held[n]))
        sc.copy_(torch.from_numpy(s.c.scale[n]))
    cache.append(x[:, :2].cuda(), x[:, 2:].cuda(), *ints)
    assert cache.status() == 0
    none = np.zeros((60, 0), np.float32)
    f = x.float().numpy()
    s.c.append(f[:, :2], f[:, 2:], s.table, lens, s.cu, none, none, False)
    for n, c, sc in (("k", cache.k_codes, cache.k_scale), ("v", cache.v_codes, cache.v_scale)):
        np.testing.assert_array_equal(c.cpu().numpy(), s.c.codes[n])
        np.testing.assert_array_equal(sc.cpu().numpy(), s.c.scale[n])


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_queries_before_the_first_token_are_not_reported(engine, rows):
    import torch
    s = ref.Setup([30, 30], [50, 4], 4, 1, 64, 16, "bf16", seed=62)
    s.lens = [30, 0]
    cache, ints = _gpu(s, engine, rows)
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows))
    assert cache.status() == 0
    assert (out[:20] == 0).all() and torch.isneginf(lse[:20]).all() and (out[50:] == 0).all()
    idx = torch.arange(40, device="cuda").to(torch.int32).expand(54, 40).contiguous()
    out, lse = cache.attention_selected(s.q.cuda(), idx, *ints)
    assert cache.status() == 0
    assert (out[:20] == 0).all() and torch.isneginf(lse[:20]).all() and (out[50:] == 0).all()
    cache.append(s.q[:, :1].cuda(), s.q[:, 1:2].cuda(), *ints)
    assert cache.status() == 1
