"""Appending to pages that others filled under scales that are no powers of two."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [([20, 70], [1, 1]), ([20, 70], [40, 30])])
def test_append_keeps_what_a_page_of_another_scale_holds(lens, new):
    """Both append forms.  The page's scale becomes the power of two above it (or what the new
    tokens need), and its held codes are rounded to that, whatever they were scaled by."""
    import torch
    lens = [n + m - 1 for n, m in zip(lens, new)]
    s = ref.Setup(lens, new, 1, 2, 64, 64, seed=35)
    for name in "kv":
        s.c.codes[name][s.c.codes[name] == 0x7F] = 0
        s.c.scale[name] *= np.float32(1.3)
        s.c.scale[name][s.table[1, 0], 0] = 0.3
        s.c.scale[name][s.table[1, 0], 1] = 48.0
    cache, ints = s.gpu()
    x = torch.randn((s.cu[-1], 4, 64), generator=torch.Generator().manual_seed(1)).bfloat16()
    cache.append(x[:, :2].cuda(), x[:, 2:].cuda(), *ints)
    assert cache.status() == 0
    f = x.float().numpy()
    for b in range(2):
        p0 = lens[b] - new[b]
        pg, off = s.table[b, p0 // 64], p0 % 64
        if off == 0:
            continue
        for name, at, codes, scale in (("k", 0, cache.k_codes, cache.k_scale), ("v", 2, cache.v_codes, cache.v_scale)):
            for h in range(2):
                was = float(s.c.scale[name][pg, h])
                fresh = f[s.cu[b]:s.cu[b] + min(new[b], 64 - off), at + h]
                e = max(ref.exponent(np.abs(fresh).max()), int(np.ceil(np.log2(was))))
                assert float(scale[pg, h]) == 2.0 ** e
                held = ref.E4M3[s.c.codes[name][pg, h, :off]] * was * 2.0 ** -e
                got = codes[pg, h].cpu().numpy()
                np.testing.assert_array_equal(got[:off], ref.encode(held))
                np.testing.assert_array_equal(got[off:off + len(fresh)], ref.encode(fresh.astype(np.float64) * 2.0 ** -e))
