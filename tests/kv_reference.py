"""Plain implementation of the paged 8-bit cache for the tests: append bit for bit
(fp32 products and sums rounded one by one, as the operation is defined), attention
in 64 bits, both on the CPU with numpy.

Error bound of an attention output, derived from the kernels' arithmetic before
any run.  With p_j the exact softmax weights and A = sum_j p_j |v_j| (per element):
  - the stored output is rounded once: |out| * u, u = 2^-8 (bf16, 8 significant bits) or 2^-11 (f16, 11);
  - each weight meets its value code as an f16 number: at most 2^-11 * A;
  - a score is an fp32 sum of D exact products; its error, at most
    D * 2^-24 * scale * sum |q k| <= 2^-17 * 60 for the inputs here (Cauchy bound
    60 on scale * sum |q k|), moves p_j by that relative amount, in numerator
    and denominator: 2 * 60 * 2^-17 < 2^-10; exp2's and the sums' fp32 errors are below 2^-18.
So |error| <= u |out| + (2^-11 + 2^-10 + 2^-17) A (+ 2^-24 for f16's subnormals),
and lse is within 60 * 2^-17 + 2^-18 * (1 + |lse|).
"""
import numpy as np

E_MIN, E_MAX = -40, 40


def _e4m3_table():
    t = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        t[c] = -v if s else v
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]


def encode(x):
    """fp32/64 array (|x| <= 448) to e4m3 codes, nearest, ties to even."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = a - _POS[lo], _POS[hi] - a
    pick = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(amax):
    e = E_MIN
    if amax > 0:
        m, ex = np.frexp(np.float32(amax))
        e = int(ex) - 9 + (1 if m > 0.875 else 0)
    return min(max(e, E_MIN), E_MAX)


def rotate(x, cos, sin, interleaved):
    """x fp32 [..., d], cos/sin fp32 [rot / 2]."""
    x = x.astype(np.float32).copy()
    rot = 2 * cos.shape[-1]
    if rot == 0:
        return x
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., lo].copy(), x[..., hi].copy()
    with np.errstate(all="ignore"):
        x[..., lo] = a * cos - b * sin
        x[..., hi] = b * cos + a * sin
    return x


class Cache:
    def __init__(self, pages, heads, page, dim):
        self.page, self.heads, self.dim = page, heads, dim
        self.codes = {n: np.zeros((pages, heads, page, dim), np.uint8) for n in "kv"}
        self.scale = {n: np.zeros((pages, heads), np.float32) for n in "kv"}

    def append(self, k, v, table, lens, cu, cos, sin, interleaved):
        """k, v fp32 values of the 16-bit inputs [N, heads, dim]."""
        for b in range(len(lens)):
            n = cu[b + 1] - cu[b]
            p0 = lens[b] - n
            if n == 0:
                continue
            for first in range(p0 - p0 % self.page, lens[b], self.page):
                page = table[b][first // self.page]
                rows = range(max(first, p0), min(first + self.page, lens[b]))
                for h in range(self.heads):
                    kv = {"k": [], "v": []}
                    bad = []
                    for p in rows:
                        t = cu[b] + p - p0
                        kr = rotate(k[t, h], cos[p], sin[p], interleaved)
                        vr = v[t, h].astype(np.float32)
                        lim = np.float32(448 * 2.0 ** E_MAX)
                        bad.append(not (np.all(np.abs(kr) <= lim) and np.all(np.abs(vr) <= lim)))
                        kv["k"].append(kr)
                        kv["v"].append(vr)
                    for name, fill in (("k", 0x7F), ("v", 0)):
                        x = np.stack(kv[name])
                        good = x[~np.array(bad)]
                        e = exponent(np.abs(good).max() if good.size else 0.0)
                        off = rows[0] - first
                        if off > 0:
                            e_old = int(np.frexp(self.scale[name][page, h])[1]) - 1
                            if e > e_old:
                                held = E4M3[self.codes[name][page, h, :off]] * 2.0 ** (e_old - e)
                                nan = np.isnan(held)
                                self.codes[name][page, h, :off] = np.where(nan, 0x7F, encode(np.where(nan, 0, held)))
                            e = max(e, e_old)
                        self.scale[name][page, h] = np.float32(2.0 ** e)
                        for i, p in enumerate(rows):
                            self.codes[name][page, h, p - first] = \
                                fill if bad[i] else encode(x[i].astype(np.float64) * 2.0 ** -e)

    def values(self, name, table_row, h, pos):
        pg = np.asarray(table_row)[np.asarray(pos) // self.page]
        return E4M3[self.codes[name][pg, h, np.asarray(pos) % self.page]] * \
            self.scale[name][pg, h].astype(np.float64)[:, None]

    def attend(self, q, table, lens, cu, window=0, sinks=0, idx=None, scale=None):
        """q fp64 [N, hq, d] -> out, lse, A (see the module's text), all fp64."""
        N, hq, d = q.shape
        G = hq // self.heads
        scale = d ** -0.5 if scale is None else scale
        out, A = np.zeros((N, hq, d)), np.zeros((N, hq, d))
        lse = np.full((N, hq), -np.inf)
        for b in range(len(lens)):
            n = cu[b + 1] - cu[b]
            for i in range(n):
                p, t = lens[b] - n + i, cu[b] + i
                j = np.arange(lens[b]) if idx is None else idx[t][idx[t] >= 0]
                j = j[j <= p]
                if window > 0:
                    j = j[(j > p - window) | (j < sinks)]
                if len(j) == 0:
                    continue
                for h in range(self.heads):
                    K, V = self.values("k", table[b], h, j), self.values("v", table[b], h, j)
                    for g in range(h * G, h * G + G):
                        s = scale * (K @ q[t, g])
                        m = s.max()
                        w = np.exp(s - m)
                        lse[t, g] = m + np.log(w.sum())
                        w /= w.sum()
                        out[t, g], A[t, g] = w @ V, w @ np.abs(V)
        return out, lse, A


U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def check(out, lse, ref, dtype):
    """out, lse fp64 copies of the kernel's results against attend()'s."""
    want, want_lse, A = ref
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(out), nan)
    tol = U[dtype] * 1.01 * np.abs(want) + (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -17) * A + \
        (2.0 ** -24 if dtype == "f16" else 0.0)
    off = np.abs(out - want) - tol
    assert np.all(off[~nan] <= 0), f"worst {np.nanmax(off)}"
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(want_lse))
    fin = np.isfinite(want_lse)
    assert np.all(np.abs(lse[fin] - want_lse[fin]) <= 60 * 2.0 ** -17 + 2.0 ** -18 * (1 + np.abs(want_lse[fin])))


class Setup:
    """A ragged batch over a shuffled pool, a filled cache and queries."""

    def __init__(self, lens, new, hq, hkv, d, page, dtype="bf16", seed=0, spread=1.0):
        rng = np.random.RandomState(seed)
        self.dtype, self.lens, self.new = dtype, list(lens), list(new)
        self.cu = [0] + list(np.cumsum(new))
        held = [-(-n // page) for n in lens]
        self.pages, self.width = max(sum(held), 1) + 2, max(max(held), 1)
        order = rng.permutation(self.pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(held):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.c = Cache(self.pages, hkv, page, d)
        for name in "kv":
            x = rng.randn(self.pages, hkv, page, d) * np.exp2(np.round(rng.randn(self.pages, hkv) * spread))[:, :, None, None] \
                * (0.5 if name == "k" else 1.0)
            for pg in range(self.pages):
                for h in range(hkv):
                    e = exponent(np.abs(x[pg, h]).max())
                    self.c.scale[name][pg, h] = 2.0 ** e
                    self.c.codes[name][pg, h] = encode(x[pg, h] * 2.0 ** -e)
        # rows past a sequence's length hold NaN codes: they must not be read
        for b, n in enumerate(lens):
            if n % page:
                for name in "kv":
                    self.c.codes[name][self.table[b, n // page], :, n % page:] = 0x7F
        import torch
        self.q = torch.from_numpy(rng.randn(self.cu[-1], hq, d).astype(np.float32)).to(
            torch.bfloat16 if dtype == "bf16" else torch.float16)

    def q64(self):
        return self.q.double().numpy()

    def gpu(self, engine=0, columns=0):
        """The framework's cache on the same data, and the batch's tensors; the page table
        padded to ``columns`` (its width is what the choice of kernel knows of lengths)."""
        import torch
        from indexer_topk_long_gb300 import PagedKVCache
        dev = {n: torch.from_numpy(self.c.codes[n]).cuda() for n in "kv"}
        scl = {n: torch.from_numpy(self.c.scale[n]).cuda() for n in "kv"}
        cache = PagedKVCache(self.pages, self.c.heads, self.c.dim, page=self.c.page, k_codes=dev["k"],
                             v_codes=dev["v"], k_scale=scl["k"], v_scale=scl["v"], engine=engine)
        ints = [torch.tensor(np.asarray(x), dtype=torch.int32).cuda() for x in (self.table, self.lens, self.cu)]
        if columns > ints[0].shape[1]:
            ints[0] = torch.nn.functional.pad(ints[0], (0, columns - ints[0].shape[1]), value=-1)
        return cache, ints
