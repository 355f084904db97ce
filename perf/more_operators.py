"""What a server needs to continue one prompt in many ways: cases, plain forms and work.

shared    attention of a decode step (or of short chunks) whose sequences come in groups that begin
          with the same pages of the 8-bit cache: the pages that a group has in common are read once
          for all of its queries, the rest for each sequence.
read      the cache read back: tokens' keys and values in 16 bits, keys rotated back by their
          positions' angles if asked (to fork a sequence inside a page, to move tokens elsewhere).
sample    a token for each row of logits from a given random number: temperature, then min-p, top-k
          and top-p, each on what the one before left.

The module's plain name `own` chooses between the plain forms here (elementary tensor operations)
and the framework's calls.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _shared(name, G, B, q_min, q_max, pre_min, pre_max, own_min, own_max, hq, hkv, d, page, dtype):
    return dict(name=name, op="shared", G=G, B=B, q_min=q_min, q_max=q_max, pre_min=pre_min, pre_max=pre_max,
                own_min=own_min, own_max=own_max, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype)


def _read(name, B, n_min, n_max, ctx_min, ctx_max, hkv, d, page, dtype, rot, interleaved):
    return dict(name=name, op="read", B=B, n_min=n_min, n_max=n_max, ctx_min=ctx_min, ctx_max=ctx_max, hkv=hkv,
                d=d, page=page, dtype=dtype, rot=rot, interleaved=interleaved)


def _sample(name, B, V, dtype, spread, temperature, top_k, top_p, min_p, mixed):
    return dict(name=name, op="sample", B=B, V=V, dtype=dtype, spread=spread, temperature=temperature, top_k=top_k,
                top_p=top_p, min_p=min_p, mixed=mixed)


def listed():
    return [
        # four continuations of a short prompt, one token each: latency
        _shared("shared_few", 1, 4, 1, 1, 1000, 1000, 1, 40, 8, 8, 64, 16, "f16"),
        # many samples of one long prompt
        _shared("shared_decode", 1, 128, 1, 1, 32768, 32768, 16, 512, 32, 8, 128, 64, "bf16"),
        # a few samples of a very long one: the prompt's keys are what is read
        _shared("shared_long", 1, 16, 1, 1, 262144, 262144, 64, 2048, 32, 8, 128, 64, "bf16"),
        # requests on several prompts of different lengths, one or two tokens each, odd group of heads
        _shared("shared_groups", 6, 47, 1, 2, 900, 16000, 1, 700, 14, 2, 64, 32, "f16"),
        # questions' chunks behind one document: matrix work
        _shared("shared_chunks", 1, 16, 200, 256, 8192, 8192, 200, 260, 32, 8, 128, 64, "bf16"),
        # a fork inside a page: the tokens of the last page are read to be appended elsewhere
        _read("read_fork", 1, 37, 37, 4005, 4005, 8, 128, 64, "bf16", 0, False),
        # a whole long sequence
        _read("read_long", 1, 131072, 131072, 131072, 131072, 8, 128, 64, "bf16", 0, False),
        # several sequences to be moved to other positions: keys without their rotation
        _read("read_ragged", 24, 200, 9000, 300, 9000, 2, 64, 16, "f16", 32, True),
        # one user's next token: latency
        _sample("sample_one", 1, 32000, "f32", 3.0, 0.8, 50, 0.9, 0.0, False),
        # a decode batch with the usual filters
        _sample("sample_filtered", 256, 131072, "f32", 3.0, 0.8, 64, 0.95, 0.0, False),
        # the plain distribution over an odd vocabulary
        _sample("sample_plain", 192, 131071, "bf16", 2.0, 1.0, 0, 1.0, 0.0, False),
        # every request its own settings, no top-k among them: nuclei of a few to thousands of tokens
        _sample("sample_mixed", 128, 65537, "f16", 2.5, 1.1, 0, 0.95, 0.001, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "read", "sample", "sample"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "sample":
        V = _log(rng, 300, 262144)
        B = max(1, min(_log(rng, 1, 512), (256 * 131072) // V))
        c = _sample("", B, V, rng.choice(["f32", "f32", "bf16", "f16"]), rng.choice([1.0, 2.0, 3.0, 4.0]),
                    rng.choice([0.6, 0.8, 1.0, 1.0, 1.3]), rng.choice([0, 0, 1, 20, 50, _log(rng, 2, 5000)]),
                    rng.choice([1.0, 0.5, 0.9, 0.95, 0.99]), rng.choice([0.0, 0.0, 0.002, 0.05]), rng.random() < 0.4)
    elif op == "read":
        B = _log(rng, 1, 64)
        ctx = _log(rng, 20, 131072 // B)
        n = _log(rng, 1, ctx)
        c = _read("", B, max(1, n // rng.choice([1, 4, 30])), n, max(1, ctx // rng.choice([1, 3, 20])), ctx,
                  rng.choice([1, 2, 4, 8]), d, page, dtype, rng.choice([0, 0, 16, 32, d]), rng.random() < 0.5)
    else:
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        G = rng.choice([1, 1, 1, 2, 5])
        B = G * _log(rng, 2, 128 // G)
        q = rng.choice([1, 1, 1, 2, 5, _log(rng, 2, max(2, 4096 // B))])
        most = min((1 << 28) // (hkv * d), (1 << 36) // (B * q * hq * d) * G) // G
        pre = max(page, min(_log(rng, 256, 262144), most))
        tail = max(q, _log(rng, 1, max(2, 65536 // B)) if q == 1 else q + rng.choice([0, 3, 60]))
        c = _shared("", G, B, q if rng.random() < 0.5 else 1, q, max(page, pre // rng.choice([1, 2, 10])), pre,
                    max(q, tail // 20), tail, hq, hkv, d, page, dtype)
    del c["name"]
    return c


def _spread(lo, hi, n, turn):
    """n whole numbers between lo and hi, even over their logarithm, in a mixed order."""
    if n == 1 or lo == hi:
        return np.full(n, hi, dtype=np.int64)
    at = (np.arange(n) * turn) % 1.0
    at = np.argsort(np.argsort(at)) / (n - 1)
    return np.round(np.exp(math.log(lo) + at * (math.log(hi) - math.log(lo)))).astype(np.int64)


def _batch(case):
    """Of a shared case: each group's first sequence [G + 1], its common tokens (whole pages),
    and each sequence's tokens behind those and new tokens."""
    G, B, page = case["G"], case["B"], case["page"]
    first = np.linspace(0, B, G + 1).round().astype(np.int64)
    if G > 2:
        first[1:-1] += np.arange(G - 1) % 2          # groups of different sizes
    common = np.maximum(_spread(case["pre_min"], case["pre_max"], G, 0.6180339887) // page, 1) * page
    tail = _spread(case["own_min"], case["own_max"], B, 0.6180339887)
    new = np.minimum(_spread(case["q_min"], case["q_max"], B, 0.7548776662), tail)
    return first, common, tail, new


def _lengths(case):
    """Of a read case: cached tokens of each sequence and how many of its last are read."""
    lens = _spread(case["ctx_min"], case["ctx_max"], case["B"], 0.6180339887)
    n = _spread(case["n_min"], case["n_max"], case["B"], 0.7548776662)
    return lens, np.minimum(n, lens)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _cached(gen, pages, hkv, page, d):
    """A filled cache: codes [pages, hkv, page, d] and power-of-two scales [pages, hkv] of normal
    values with a few large channels, as projected keys and values have them."""
    codes = torch.empty((pages, hkv, page, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, hkv), dtype=torch.float32, device="cuda")
    channel = torch.ones((hkv, 1, d), device="cuda")
    channel[:, :, ::29] = 3.0
    for at in range(0, pages, 4096):
        n = min(4096, pages - at)
        x = torch.randn((n, hkv, page, d), device="cuda", generator=gen) * channel
        unit = torch.exp2(torch.ceil(torch.log2(x.abs().amax((2, 3)) / 448)))
        codes[at:at + n] = (x / unit[:, :, None, None]).to(E4M3).view(torch.uint8)
        scale[at:at + n] = unit
    return codes, scale


def _ints(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).cuda()


def _prepare_sample(case, seed, gen):
    B, V = case["B"], case["V"]
    x = torch.randn((B, V), device="cuda", generator=gen) * case["spread"]
    # a few tokens that the model favours, more strongly in some rows than in others
    favoured = torch.randint(0, V, (B, 8), device="cuda", generator=gen)
    lift = 4.0 * torch.rand((B, 1), device="cuda", generator=gen) * torch.rand((B, 8), device="cuda", generator=gen)
    x.scatter_(1, favoured, x.amax(1, keepdim=True) + lift - 1.0)
    s = dict(op="sample", logits=x.to(TYPES[case["dtype"]]), u=torch.rand(B, device="cuda", generator=gen))
    names = ("temperature", "top_k", "top_p", "min_p")
    if case["mixed"]:
        rng = np.random.RandomState(int(seed) % (1 << 32))
        s["temperature"] = torch.from_numpy((case["temperature"] * rng.uniform(0.5, 1.2, B)).astype(np.float32)).cuda()
        s["top_k"] = _ints(case["top_k"] * rng.randint(0, 3, B))
        s["top_p"] = torch.from_numpy((1 - (1 - case["top_p"]) * rng.uniform(0.0, 3.0, B)).clip(0.1, 1).astype(np.float32)).cuda()
        s["min_p"] = torch.from_numpy((case["min_p"] * rng.randint(0, 3, B)).astype(np.float32)).cuda()
    else:
        s.update({n: case[n] for n in names})
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    if case["op"] == "sample":
        return _prepare_sample(case, seed, gen)
    hkv, d, page, kind = case["hkv"], case["d"], case["page"], TYPES[case["dtype"]]
    if case["op"] == "shared":
        first, common, tail, new = _batch(case)
        group = np.repeat(np.arange(case["G"]), np.diff(first))
        lens = common[group] + tail
    else:
        lens, new = _lengths(case)
        group, common = np.arange(case["B"]), np.zeros(case["B"], dtype=np.int64)
    B = case["B"]
    held, kept = -(-lens // page), common // page
    pages = int((held - kept[group]).sum() + kept.sum())
    width = int(held.max())
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at, start = 0, []
    for n in kept.tolist():
        start.append((at, at + n))
        at += n
    for b in range(B):
        lo, hi = start[group[b]]
        table[b, :hi - lo] = order[lo:hi]
        n = int(held[b]) - (hi - lo)
        table[b, hi - lo:int(held[b])] = order[at:at + n]
        at += n
    s = dict(op=case["op"], page=page, N=int(new.sum()), max_q=int(new.max()), kind=kind, table=table,
             lens=_ints(lens), cu=_ints(np.concatenate([[0], np.cumsum(new)])))
    s["k_codes"], s["k_scale"] = _cached(gen, pages, hkv, page, d)
    s["v_codes"], s["v_scale"] = _cached(gen, pages, hkv, page, d)
    if case["op"] == "shared":
        s["q"] = torch.randn((s["N"], case["hq"], d), device="cuda", generator=gen).to(kind)
        s["groups"] = _ints(first)
        # what the plain form goes by: sizes that a scheduler knows on the host
        s["first"], s["common"], s["tail"], s["new"] = first.tolist(), common.tolist(), tail.tolist(), new.tolist()
    else:
        s["cos"] = s["sin"] = None
        s["interleaved"] = case["interleaved"]
        if case["rot"]:
            rot = case["rot"]
            freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
            angle = torch.arange(int(lens.max()), device="cuda", dtype=torch.float64)[:, None] * freq
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if own:
        from indexer_topk_long_gb300 import PagedKVCache
        s["cache"] = PagedKVCache(pages, hkv, d, page=page, k_codes=s["k_codes"], v_codes=s["v_codes"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _values(codes, scale, table):
    """Cached values of pages table [..., n] in 32 bits: [..., hkv, n * page, d]."""
    t = table.clamp(min=0).long()
    x = codes[t].view(E4M3).float() * scale[t][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_shared(s):
    (N, hq, d), hkv, page = s["q"].shape, s["k_scale"].shape[1], s["page"]
    G, q_most = hq // hkv, s["max_q"]
    new = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=N)
    at = torch.arange(N, device="cuda") - s["cu"][seq]
    out = torch.empty((N, hq, d), device="cuda")
    lse = torch.empty((N, hq), device="cuda")
    row = 0
    for g, pre in enumerate(s["common"]):
        b0, b1 = s["first"][g], s["first"][g + 1]
        rows = slice(row, row + sum(s["new"][b0:b1]))
        row, n = rows.stop, b1 - b0
        last = max(s["tail"][b0:b1])
        # this group's queries by sequence: [n, hkv, G * q_most, d]
        i, j = seq[rows] - b0, at[rows]
        q = torch.zeros((n, q_most, hq, d), device="cuda")
        q[i, j] = s["q"][rows].float() * d ** -0.5
        q = q.view(n, q_most, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, G * q_most, d)
        of_all = q.transpose(0, 1).reshape(hkv, n * G * q_most, d)
        t0 = s["table"][b0, :pre // page]
        score0 = of_all @ _values(s["k_codes"], s["k_scale"], t0).transpose(-1, -2)
        t1 = s["table"][b0:b1, pre // page:pre // page - (-last // page)]
        score1 = q @ _values(s["k_codes"], s["k_scale"], t1).transpose(-1, -2)
        key = torch.arange(score1.shape[-1], device="cuda")
        lens = s["lens"][b0:b1] - pre
        p = (lens - new[b0:b1])[:, None] + torch.arange(q_most, device="cuda")
        seen = (key <= p[..., None])[:, None, None].expand(n, 1, G, q_most, len(key)).reshape(n, 1, G * q_most, -1)
        score1 = torch.where(seen, score1, float("-inf"))
        m0 = score0.amax(-1).reshape(hkv, n, -1).transpose(0, 1)
        m = torch.maximum(m0, score1.amax(-1))[..., None]
        w0 = torch.exp_(score0.sub_(m.transpose(0, 1).reshape(hkv, -1, 1)))
        w1 = torch.exp_(score1.sub_(m))
        v1 = _values(s["v_codes"], s["v_scale"], t1)
        v1 = torch.where((key < lens[:, None])[:, None, :, None], v1, 0)
        o0 = (w0 @ _values(s["v_codes"], s["v_scale"], t0)).reshape(hkv, n, -1, d).transpose(0, 1)
        total = w0.sum(-1).reshape(hkv, n, -1).transpose(0, 1) + w1.sum(-1)
        o = (o0 + w1 @ v1) / total[..., None]
        out[rows] = o.reshape(n, hq, q_most, d)[i, :, j]
        lse[rows] = (torch.log(total) + m[..., 0]).reshape(n, hq, q_most)[i, :, j]
    return out.to(s["q"].dtype), lse


def _plain_read(s):
    n = s["cu"][1:] - s["cu"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["N"])
    pos = (s["lens"] - n)[seq] + torch.arange(s["N"], device="cuda") - s["cu"][seq]
    at, off = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    k = s["k_codes"][at, :, off].view(E4M3).float() * s["k_scale"][at][..., None]
    v = s["v_codes"][at, :, off].view(E4M3).float() * s["v_scale"][at][..., None]
    if s["cos"] is not None:
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        rot = 2 * cos.shape[-1]
        r, rest = k[..., :rot], k[..., rot:]
        if s["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos + b * sin, b * cos - a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos + b * sin, b * cos - a * sin], -1)
        k = torch.cat([r, rest], -1)
    return k.to(s["kind"]), v.to(s["kind"])


def _column(x, kind):
    return x.to(kind)[:, None] if torch.is_tensor(x) else x


def _plain_sample(s):
    f64 = torch.float64
    B, V = s["logits"].shape
    # 64 bits: sums over a whole vocabulary are compared with a random number times their total
    x, at = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    t = _column(s["temperature"], f64)
    if not torch.is_tensor(t):
        t = float(np.float32(t))
    w = torch.exp((x - x[:, :1]) / t)
    rank = torch.arange(V, device="cuda")
    min_p = _column(s["min_p"], f64)
    kept = w >= (min_p if torch.is_tensor(min_p) else float(np.float32(min_p)))
    k = _column(s["top_k"], torch.int64)
    kept &= torch.where(k > 0, rank < k, True) if torch.is_tensor(k) else (rank < k if k > 0 else True)
    w = torch.where(kept, w, 0)
    run = w.cumsum(1)
    p = _column(s["top_p"], f64)
    p = p if torch.is_tensor(p) else torch.full((B, 1), float(np.float32(p)), dtype=f64, device="cuda")
    kept &= (p >= 1) | (run - w < p * run[:, -1:])
    w = torch.where(kept, w, 0)
    by_index = torch.zeros_like(w).scatter_(1, at, w)
    run = by_index.cumsum(1)
    total = run[:, -1:]
    token = (run <= s["u"].double()[:, None] * total).sum(1)
    logp = torch.log(by_index.gather(1, token[:, None]) / total)[:, 0]
    return token.to(torch.int32), logp.float()


def run(state):
    s = state
    if s["op"] == "shared":
        if own:
            return s["cache"].attention_shared(s["q"], s["table"], s["lens"], s["cu"], groups=s["groups"], max_q=s["max_q"])
        return _plain_shared(s)
    if s["op"] == "read":
        if own:
            return s["cache"].read(s["table"], s["lens"], s["cu"], s["N"], dtype=s["kind"], cos=s["cos"], sin=s["sin"],
                                   interleaved=s["interleaved"])
        return _plain_read(s)
    if own:
        from indexer_topk_long_gb300 import sample
        return sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
    return _plain_sample(s)


# ---------------------------------------------------------------------------------------------
# Work and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "f32" else 2
        B, V = case["B"], case["V"]
        return {"bytes": B * V * size + B * (12 + (16 if case["mixed"] else 0)), "flops": 4 * B * V}
    hkv, d, page = case["hkv"], case["d"], case["page"]
    if case["op"] == "read":
        lens, n = _lengths(case)
        N, pages = int(n.sum()), int((-(-lens // page) - (lens - n) // page).sum())
        return {"bytes": N * hkv * d * 6 + pages * (hkv * 8 + 4) + int(n.max()) * case["rot"] * 4,
                "flops": 3 * N * hkv * case["rot"]}
    first, common, tail, new = _batch(case)
    group = np.repeat(np.arange(case["G"]), np.diff(first))
    keys = int(common.sum() + tail.sum())
    pairs = int((new * (common[group] + tail - new) + new * (new + 1) // 2).sum())
    N, hq = int(new.sum()), case["hq"]
    return {"bytes": N * hq * (4 * d + 4) + keys * hkv * 2 * d + keys // page * (4 + 8 * hkv), "flops": 4 * d * hq * pairs}


def _exact_shared(s):
    """Every sequence by itself, with no thought of what it shares."""
    page, cu, lens = s["page"], s["cu"].tolist(), s["lens"].tolist()
    N, hq, d = s["q"].shape
    hkv = s["k_scale"].shape[1]
    out = torch.empty((N, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((N, hq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        rows = slice(cu[b], cu[b + 1])
        at = s["table"][b, :-(-n // page)].long()
        k, v = ((s[x + "_codes"][at].view(E4M3).double() * s[x + "_scale"][at].double()[..., None, None])
                .transpose(0, 1).reshape(hkv, -1, d)[:, :n] for x in "kv")
        hidden = torch.arange(n, device="cuda")[None] > torch.arange(n - (rows.stop - rows.start), n, device="cuda")[:, None]
        for h in range(hq):
            g = h // (hq // hkv)
            t = (s["q"][rows, h].double() @ k[g].T) / math.sqrt(d)
            t = t.masked_fill(hidden, -math.inf)
            lse[rows, h] = torch.logsumexp(t, 1)
            out[rows, h] = torch.exp(t - lse[rows, h, None]) @ v[g]
    return out, lse


def _exact_read(s):
    cu, lens, page = s["cu"].tolist(), s["lens"].tolist(), s["page"]
    both = []
    for name in "kv":
        parts = []
        for b, n in enumerate(lens):
            pos = torch.arange(n - (cu[b + 1] - cu[b]), n, device="cuda")
            at = s["table"][b].long()[pos // page]
            x = s[name + "_codes"][at, :, pos % page].view(E4M3).double() * s[name + "_scale"][at].double()[..., None]
            if name == "k" and s["cos"] is not None:
                turn = torch.complex(s["cos"][pos].double(), -s["sin"][pos].double())[:, None]
                half = turn.shape[-1]
                i = torch.arange(half, device="cuda")
                lo, hi = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
                z = torch.complex(x[..., lo], x[..., hi]) * turn
                x[..., lo], x[..., hi] = z.real, z.imag
            parts.append(x)
        both.append(torch.cat(parts))
    return tuple(both)


def _exact_sample(s):
    """Row by row: what is left is a shrinking list of tokens."""
    x = s["logits"].double().cpu().numpy()
    B = len(x)
    of = {n: (s[n].cpu().numpy() if torch.is_tensor(s[n]) else np.full(B, s[n])) for n in ("temperature", "top_k", "top_p", "min_p")}
    u = s["u"].double().cpu().numpy()
    token, logp = np.empty(B, np.int32), np.empty(B)
    for r in range(B):
        z = (x[r] - x[r].max()) / np.float64(np.float32(of["temperature"][r]))
        left = np.flatnonzero(np.exp(z) >= np.float64(np.float32(of["min_p"][r])))
        k, p = int(of["top_k"][r]), np.float64(np.float32(of["top_p"][r]))
        left = left[np.lexsort((left, -z[left]))]
        if k > 0:
            left = left[:k]
        mass = np.exp(z[left])
        if p < 1:
            run = np.cumsum(mass)
            left = left[:int(np.searchsorted(run, p * run[-1])) + 1]
        left = np.sort(left)
        run = np.cumsum(np.exp(z[left]))
        i = min(int(np.searchsorted(run, u[r] * run[-1], side="right")), len(left) - 1)
        token[r], logp[r] = left[i], z[left[i]] - math.log(run[-1])
    return torch.from_numpy(token).cuda(), torch.from_numpy(logp).cuda()


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"shared": _exact_shared, "read": _exact_read, "sample": _exact_sample}[s["op"]](s)
