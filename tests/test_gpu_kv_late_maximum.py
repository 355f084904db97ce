"""Maxima that come late in a tile."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _gpu, _hint

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("engine,rows", KERNELS)
def test_late_maxima_do_not_round_weights_again(engine, rows):
    """One tile whose 32-key quarters each bring a maximum 7.25 binary orders above the last.
    All values but the maxima's are equal, so an output is off by what its weights are: one
    rounding to f16 each (2^-11), the output's own (2^-11), and fp32's (below 2^-18)."""
    c = 0.90673828125                                  # exponent (base 2) of a key code of 1; f16 and bf16 hold q
    s = ref.Setup([128], [1], 4, 1, 64, 64, "f16", seed=38)
    for name in "kv":
        s.c.codes[name][:] = 0
    s.c.scale["k"][:], s.c.scale["v"][:] = 1, 2.0 ** 8
    for j in range(128):
        pg = s.table[0, j // 64]
        s.c.codes["v"][pg, 0, j % 64] = 0x7E           # 448
        if j in (32, 64, 96):
            s.c.codes["k"][pg, 0, j % 64, 0] = ref.encode(np.float64(j // 4))
            s.c.codes["v"][pg, 0, j % 64] = 0
    s.q[:] = 0
    s.q[:, :, 0] = c
    scale = float(np.float32(np.log(2.0)))
    want, want_lse, A = s.c.attend(s.q64(), s.table, s.lens, s.cu, scale=scale)
    cache, ints = _gpu(s, engine, rows)
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), scale=scale)
    off = np.abs(out.double().cpu().numpy() / want - 1)
    assert off.max() <= 2.0 ** -10 + 2.0 ** -17, off.max() * 2.0 ** 11
    np.testing.assert_allclose(lse.cpu().numpy(), want_lse, rtol=2.0 ** -18)


@pytest.mark.parametrize("orders", [20, 24, 26, 28, 30])
@pytest.mark.parametrize("engine,rows", KERNELS)
def test_a_late_maximum_far_above_leaves_what_f16_holds(engine, rows, orders):
    """A maximum 2^20 to 2^30 above the keys before it, in the last quarter of a tile, and with a
    value of zero: the others' weights, powers of two from 2^-12 to 2^-22, are exact in f16, so the
    output is off by its own rounding (2^-11) and fp32's (below 2^-17)."""
    s = ref.Setup([128], [1], 4, 1, 64, 64, "f16", seed=39)
    for name in "kv":
        s.c.codes[name][:] = 0
    s.c.scale["k"][:], s.c.scale["v"][:] = 1, 2.0 ** 8
    for j in range(128):
        s.c.codes["v"][s.table[0, j // 64], 0, j % 64] = 0 if j == 100 else 0x7E       # 448
    s.c.codes["k"][s.table[0, 1], 0, 36, 0] = ref.encode(np.float64(orders))
    assert ref.E4M3[ref.encode(np.float64(orders))] == orders
    s.q[:] = 0
    s.q[:, :, 0] = 1
    scale = float(np.float32(np.log(2.0)))
    want, want_lse, A = s.c.attend(s.q64(), s.table, s.lens, s.cu, scale=scale)
    cache, ints = _gpu(s, engine, rows)
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), scale=scale)
    off = np.abs(out.double().cpu().numpy() / want - 1)
    assert off.max() <= 2.0 ** -11 + 2.0 ** -17, off.max() * 2.0 ** 11
    np.testing.assert_allclose(lse.cpu().numpy(), want_lse, rtol=2.0 ** -18)
