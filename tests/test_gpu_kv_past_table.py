"""Sequences that are longer than their page table: reported, nothing written, NaN where seen."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import KERNELS, _hint

pytestmark = pytest.mark.gpu


def _inputs(n, heads, d, seed=1):
    import torch
    return torch.randn((n, heads, d), generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("past", [1, 3, 200])
@pytest.mark.parametrize("new", [1, 6, 60])
def test_append_past_the_page_table(new, past):
    """Tokens whose position has no column in the table are reported and written nowhere, the
    ones before them are stored where they belong."""
    import torch
    page, room = 16, 64
    s = ref.Setup([room, 40], [0, 2], 2, 2, 64, page, seed=41)
    s.c.scale["v"][s.table[0, 3]] *= 0.5
    for name in "kv":
        s.c.codes[name][s.c.codes[name] == 0x7F] = 0
    cache, ints = s.gpu()
    lens, cu = [room + past, 40], [0, new, new + 2]
    ints[1], ints[2] = (torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, cu))
    x = _inputs(new + 2, 6, 64)
    angle = np.arange(room + past)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    q = cache.append(x[:, 2:4].cuda(), x[:, 4:].cuda(), *ints, torch.from_numpy(cos).cuda(), torch.from_numpy(sin).cuda(),
                     q=x[:, :2].cuda())
    assert cache.status() == 1 and cache.status() == 0
    f = x.float().numpy()
    kept = max(new - past, 0)
    keep = list(range(kept)) + [new, new + 1]
    s.c.append(f[keep, 2:4], f[keep, 4:], s.table, [room if kept else 0, 40], [0, kept, kept + 2], cos, sin, False)
    for name, codes, scale in (("k", cache.k_codes, cache.k_scale), ("v", cache.v_codes, cache.v_scale)):
        np.testing.assert_array_equal(codes.cpu().numpy(), s.c.codes[name])
        np.testing.assert_array_equal(scale.cpu().numpy(), s.c.scale[name])
    for t in range(new):                                # queries are rotated by where they are
        p = room + past - new + t
        assert torch.equal(q[t].cpu(), torch.from_numpy(ref.rotate(f[t, :2], cos[p], sin[p], False)).bfloat16())


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (30, 5)])
@pytest.mark.parametrize("past", [1, 5, 300])
@pytest.mark.parametrize("engine,rows", KERNELS)
def test_attention_past_the_page_table(engine, rows, past, window, sinks):
    """Queries whose position has no column in the table are reported and get NaN; the others of
    the sequence, and the other sequences, see what they would see without them."""
    import torch
    room, new = 256, 20
    s = ref.Setup([room, 100], [new, 3], 4, 1, 64, 16, seed=42)
    cache, ints = s.gpu(engine)
    ints[1][0] = room + past
    out, lse = cache.attention(s.q.cuda(), *ints, max_q=_hint(s, rows), window=window, sinks=sinks)
    assert cache.status() == 1 and cache.status() == 0
    kept = max(new - past, 0)
    assert out[kept:new].isnan().all() and lse[kept:new].isnan().all()
    keep = list(range(kept)) + list(range(new, new + 3))
    want = s.c.attend(s.q64()[keep], s.table, [room, 100], [0, kept, kept + 3], window, sinks)
    ref.check(out[keep].double().cpu().numpy(), lse[keep].double().cpu().numpy(), want, "bf16")


@pytest.mark.parametrize("hq", [4, 64, 100])
@pytest.mark.parametrize("engine", [1, 2])
def test_listed_keys_past_the_page_table(engine, hq):
    """A listed key without a column in the table counts as one on a page outside the pool."""
    import torch
    room, new, past = 256, 6, 4
    s = ref.Setup([room], [new], hq, 1, 64, 16, seed=43)
    cache, ints = s.gpu(engine)
    ints[1][0] = room + past                            # queries at 254 .. 259
    rng = np.random.RandomState(3)
    idx = np.stack([rng.permutation(250)[:40] for _ in range(new)]).astype(np.int32)
    call = lambda: cache.attention_selected(s.q.cuda(), torch.from_numpy(idx).cuda(), *ints)  # noqa: E731
    want = [s.c.attend(s.q64()[i:i + 1], s.table, [room], [0, 1], idx=idx[i:i + 1]) for i in range(new)]

    def same(out, lse, rows):
        for i in rows:
            ref.check(out[i:i + 1].double().cpu().numpy(), lse[i:i + 1].double().cpu().numpy(), want[i], "bf16")
    out, lse = call()
    assert cache.status() == 0
    same(out, lse, range(new))
    idx[4, 7] = 257                                     # query 4 is at 258 and sees it
    idx[1, 9] = 257                                     # query 1 is at 255 and does not
    want[1] = s.c.attend(s.q64()[1:2], s.table, [room], [0, 1], idx=idx[1:2])
    out, lse = call()
    assert cache.status() == 1
    assert out[4].isnan().all()
    same(out, lse, [0, 1, 2, 3, 5])
