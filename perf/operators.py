"""The paged 8-bit key/value cache and the attention that reads it: cases, plain forms and work.

Three operators, as a serving step runs them one after the other:

append     keys and values of new tokens go into a paged cache held in e4m3 codes with one
           power-of-two scale for each page and head; keys (and the step's queries) are rotated
           by their positions on the way.
attention  the step's queries against their sequences' cached tokens, causal, optionally limited
           to a sliding window plus a few first tokens that stay visible.
selected   the same attention over a list of key positions for each query (what the indexer's
           top-k returns; -1 is an empty slot).

The module's plain name `own` chooses between the plain forms here (elementary torch operations in
32 bits) and the framework's calls.
"""
import math

import numpy as np
import torch

own = False

E_MIN, E_MAX = -40, 40          # range of a block's scale exponent
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def _append(name, B, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, page, dtype, rot, interleaved):
    return dict(name=name, op="append", B=B, q_min=q_min, q_max=q_max, ctx_min=ctx_min,
                ctx_max=ctx_max, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, rot=rot,
                interleaved=interleaved)


def _attention(name, B, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, page, dtype, window, sinks):
    return dict(name=name, op="attention", B=B, q_min=q_min, q_max=q_max, ctx_min=ctx_min,
                ctx_max=ctx_max, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, window=window,
                sinks=sinks)


def _selected(name, B, q_min, q_max, ctx_min, ctx_max, hq, hkv, d, page, dtype, k):
    return dict(name=name, op="selected", B=B, q_min=q_min, q_max=q_max, ctx_min=ctx_min,
                ctx_max=ctx_max, hq=hq, hkv=hkv, d=d, page=page, dtype=dtype, k=k)


def listed():
    return [
        # one sequence decoding: a single new token, where only latency counts
        _append("append_one", 1, 1, 1, 4001, 4001, 32, 8, 128, 64, "bf16", 128, False),
        # a decode batch: one new token for each of many sequences
        _append("append_decode_batch", 256, 1, 1, 64, 2048, 32, 8, 128, 64, "bf16", 128, False),
        # a prefill chunk that starts in the middle of a page
        _append("append_chunk", 1, 8192, 8192, 8229, 8229, 32, 8, 128, 64, "bf16", 128, False),
        # ragged chunks of several requests: f16, rotation of half of each head in adjacent pairs
        _append("append_ragged", 13, 1, 700, 900, 5000, 14, 2, 64, 16, "f16", 32, True),
        # one short sequence, one head for each query head: latency
        _attention("decode_short", 1, 1, 1, 777, 777, 8, 8, 64, 16, "f16", 0, 0),
        # one sequence at 256K context: the cache is streamed once, bandwidth
        _attention("decode_256k", 1, 1, 1, 262144, 262144, 32, 8, 128, 64, "bf16", 0, 0),
        # a decode batch of very different lengths
        _attention("decode_ragged", 64, 1, 1, 128, 32768, 32, 8, 128, 64, "bf16", 0, 0),
        # a prefill chunk at the end of a 32K context: matrix work
        _attention("chunk_32k", 1, 2048, 2048, 32768, 32768, 32, 8, 128, 64, "bf16", 0, 0),
        # several requests' chunks with a sliding window and four first tokens, odd group of heads
        _attention("window_ragged", 24, 1, 300, 500, 9000, 14, 2, 64, 32, "f16", 1024, 4),
        # the decode step behind the indexer: 2048 keys chosen out of 1M, one shared head
        _selected("selected_decode_1m", 1, 1, 1, 1 << 20, 1 << 20, 64, 1, 128, 64, "bf16", 2048),
        # two tokens each for several sequences, some shorter than the list
        _selected("selected_ragged", 16, 2, 2, 300, 131072, 32, 8, 128, 16, "f16", 1000),
        # the indexer's prefill chunk at 1M context
        _selected("selected_chunk_1m", 1, 8192, 8192, 1 << 20, 1 << 20, 64, 1, 128, 64, "bf16", 2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "selected"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "selected":
        hkv = rng.choice([1, 1, 2, 8])
        hq = hkv * rng.choice([1, 4, 5, 8]) if hkv > 1 else rng.choice([16, 32, 64, 64, 128])
        B = _log(rng, 1, 32)
        q = _log(rng, 1, 4096 if B == 1 else 8)
        k = _log(rng, 17, 2048)
        ctx = _log(rng, 256, (1 << 20) if B * hkv <= 2 else 65536)
        q = max(1, min(q, ctx, (1 << 36) // (k * hq * d) // B, (1 << 31) // (k * hkv * d) // B))
        c = _selected("", B, 1, q, max(q, ctx // 50), ctx, hq, hkv, d, page, dtype, k)
    else:
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 5, 7, 8])
        B = _log(rng, 1, 128)
        kind = rng.choice(["decode", "chunk", "mixed"])
        if op == "append":
            q = 1 if kind == "decode" else _log(rng, 2, max(2, 8192 // B))
            ctx = max(q, _log(rng, 16, 8192 if B > 8 else 32768))
            rot = d if rng.random() < 0.6 else rng.choice([16, 32, 48])
            c = _append("", B, q if kind == "chunk" else 1, q, min(ctx, max(q, 16)), ctx, hq, hkv, d,
                        page, dtype, rot, rng.random() < 0.4)
        else:
            q = 1 if kind == "decode" else _log(rng, 2, max(2, 2048 // B))
            most = (1 << 28) // (B * hkv * d) if kind == "decode" else (1 << 38) // (B * q * hq * d)
            ctx = max(q, min(_log(rng, 16, 262144), max(64, min(most, (1 << 19) // B))))
            window = rng.choice([0, 0, 128, 1000, 4096])
            c = _attention("", B, q if kind == "chunk" else 1, q, min(ctx, max(q, ctx // 40, 1)), ctx,
                           hq, hkv, d, page, dtype, window, rng.choice([0, 1, 4, 64]) if window else 0)
    del c["name"]
    return c


def _spread(lo, hi, B, turn):
    """B whole numbers between lo and hi, even over their logarithm, in a mixed order."""
    if B == 1 or lo == hi:
        return np.full(B, hi, dtype=np.int64)
    at = (np.arange(B) * turn) % 1.0
    at = np.argsort(np.argsort(at)) / (B - 1)
    return np.round(np.exp(math.log(lo) + at * (math.log(hi) - math.log(lo)))).astype(np.int64)


def _lengths(case):
    """Cached tokens of each sequence (new ones among them) and new tokens of each."""
    lens = _spread(case["ctx_min"], case["ctx_max"], case["B"], 0.6180339887)
    new = _spread(case["q_min"], case["q_max"], case["B"], 0.7548776662)
    return lens, np.minimum(new, lens)


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _scale_exponent(amax):
    """Smallest e in the allowed range with amax <= 448 * 2^e (int32)."""
    mant, ex = torch.frexp(amax)
    e = ex - 9 + (mant > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _cached(gen, pages, hkv, page, d):
    """A filled cache: codes [pages, hkv, page, d] and scales [pages, hkv] of normal values with a
    few large channels, as projected keys and values have them."""
    codes = torch.empty((pages, hkv, page, d), dtype=torch.uint8, device="cuda")
    scale = torch.empty((pages, hkv), dtype=torch.float32, device="cuda")
    channel = torch.ones((hkv, 1, d), device="cuda")
    channel[:, :, ::29] = 3.0
    for at in range(0, pages, 4096):
        n = min(4096, pages - at)
        x = torch.randn((n, hkv, page, d), device="cuda", generator=gen) * channel
        e = _scale_exponent(x.abs().amax((2, 3)))
        codes[at:at + n] = (x * _pow2(-e)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[at:at + n] = _pow2(e)
    return codes, scale


def _selection(gen, case, lens, new):
    """Key positions chosen by each query: k of a pool of 3k that 64 neighbouring queries share."""
    k, rows = case["k"], []
    for b in range(case["B"]):
        for q0 in range(0, int(new[b]), 64):
            n = min(64, int(new[b]) - q0)
            seen = int(lens[b] - new[b]) + q0 + 1
            m = min(3 * k, seen)
            edge = torch.arange(m + 1, device="cuda", dtype=torch.float64).mul_(seen / m).floor_()
            u = torch.rand(m, device="cuda", generator=gen, dtype=torch.float64)
            pool = (edge[:-1] + (u * (edge[1:] - edge[:-1])).floor()).clamp_(max=seen - 1).to(torch.int32)
            pick = torch.rand((n, m), device="cuda", generator=gen).argsort(1)[:, :k]
            row = torch.full((n, k), -1, dtype=torch.int32, device="cuda")
            row[:, :pick.shape[1]] = pool[pick]
            rows.append(row)
    return torch.cat(rows)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, new = _lengths(case)
    B, hkv, hq, d, page = case["B"], case["hkv"], case["hq"], case["d"], case["page"]
    kind = TYPES[case["dtype"]]
    held = -(-lens // page)
    width, pages, N = int(held.max()), int(held.sum()), int(new.sum())
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    first = np.concatenate([[0], np.cumsum(held)])
    for b in range(B):
        table[b, :int(held[b])] = order[int(first[b]):int(first[b + 1])]
    s = dict(op=case["op"], page=page, N=N, max_q=int(new.max()), max_len=int(lens.max()), width=width,
             table=table, lens=torch.from_numpy(lens).to(torch.int32).cuda(),
             cu_q=torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(torch.int32).cuda())
    s["k_codes"], s["k_scale"] = _cached(gen, pages, hkv, page, d)
    s["v_codes"], s["v_scale"] = _cached(gen, pages, hkv, page, d)
    s["q"] = torch.randn((N, hq, d), device="cuda", generator=gen).to(kind)
    if case["op"] == "append":
        # k and v are slices of the projection's output, as a layer has them
        qkv = torch.randn((N, hq + 2 * hkv, d), device="cuda", generator=gen).to(kind)
        qkv[:, hq:hq + hkv, ::29] *= 3
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        rot, s["interleaved"] = case["rot"], case["interleaved"]
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(s["max_len"], device="cuda", dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    elif case["op"] == "selected":
        s["idx"] = _selection(gen, case, lens, new)
    else:
        s["window"], s["sinks"] = case["window"], case["sinks"]
    if own:
        from indexer_topk_long_gb300 import PagedKVCache
        s["cache"] = PagedKVCache(pages, hkv, d, page=page, k_codes=s["k_codes"], v_codes=s["v_codes"],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------
def _tokens(s):
    """Sequence and position of each new token."""
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=s["N"])
    at = torch.arange(s["N"], device="cuda") - s["cu_q"][seq]
    return new, seq, (s["lens"] - new)[seq] + at, at


def _rotate(x, cos, sin, interleaved):
    x = x.float()
    rot = 2 * cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _store(x, bad, fill, codes, scale, s, new, seq, pos):
    """x [N, hkv, d] into codes and scale; tokens marked bad are held as the code `fill`.
    Every sequence has one new token at least."""
    page = s["page"]
    at = s["table"][seq, pos // page].long()
    amax = torch.where(bad, 0, x.abs().amax(-1))
    most = torch.zeros_like(scale).index_reduce_(0, at, amax, "amax")
    e = _scale_exponent(most)
    # a page that held tokens before keeps the larger exponent, and its codes follow
    first = s["lens"] - new
    part = s["table"][torch.arange(len(new), device="cuda"), first // page].long()
    kept = first % page
    e_old = torch.frexp(scale[part])[1] - 1
    e_new = torch.where((kept > 0)[:, None], torch.maximum(e_old, e[part]), e[part])
    held = codes[part]
    grown = held.view(torch.float8_e4m3fn).float() * _pow2(e_old - e_new)[:, :, None, None]
    old = torch.arange(page, device="cuda")[None, :] < kept[:, None]
    codes[part] = torch.where(old[:, None, :, None], grown.to(torch.float8_e4m3fn).view(torch.uint8), held)
    e[part] = e_new
    touched = torch.zeros(len(scale), dtype=torch.bool, device="cuda")
    touched[at] = True
    scale.copy_(torch.where(touched[:, None], _pow2(e), scale))
    new_codes = (x * _pow2(-e[at])[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at, :, pos % page] = torch.where(bad[:, :, None], fill, new_codes)


def _plain_append(s):
    new, seq, pos, _ = _tokens(s)
    cos, sin = s["cos"][pos], s["sin"][pos]
    k, v = _rotate(s["k"], cos, sin, s["interleaved"]), s["v"].float()
    limit = 448.0 * 2.0 ** E_MAX
    bad = ~((k.abs() <= limit).all(-1) & (v.abs() <= limit).all(-1))
    _store(k, bad, 0x7F, s["k_codes"], s["k_scale"], s, new, seq, pos)
    _store(v, bad, 0, s["v_codes"], s["v_scale"], s, new, seq, pos)
    q = _rotate(s["q"], cos, sin, s["interleaved"]).to(s["q"].dtype)
    return q


def _values(codes, scale, table):
    """Cached values of whole sequences in 32 bits: [B, hkv, width * page, d]."""
    t = table.clamp(min=0).long()
    x = codes[t].view(torch.float8_e4m3fn).float() * scale[t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _softmax_product(score, seen, v):
    """out and lse of masked scores [..., q, s] over values [..., s, d]; 0 and -inf where nothing is seen."""
    score = torch.where(seen, score, float("-inf"))
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0, m)
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total == 0, 1, total)
    return out, (torch.log(total) + m).squeeze(-1)


def _plain_attention(s):
    new, seq, pos, at = _tokens(s)
    B, (N, hq, d), hkv = len(new), s["q"].shape, s["k_scale"].shape[1]
    k, v = _values(s["k_codes"], s["k_scale"], s["table"]), _values(s["v_codes"], s["v_scale"], s["table"])
    q = torch.zeros((B, s["max_q"], hq, d), device="cuda")
    q[seq, at] = s["q"].float()
    q = q.view(B, s["max_q"], hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    score = (q @ k.transpose(-1, -2)) * d ** -0.5
    p = (s["lens"] - new)[:, None] + torch.arange(s["max_q"], device="cuda")
    j = torch.arange(k.shape[2], device="cuda")
    seen = j <= p[..., None]
    if s["window"]:
        seen &= (j > p[..., None] - s["window"]) | (j < s["sinks"])
    seen = seen[:, None, None].expand(B, 1, hq // hkv, s["max_q"], len(j)).flatten(2, 3)
    v = torch.where(torch.arange(v.shape[2], device="cuda")[:, None] < s["lens"][:, None, None, None], v, 0)
    out, lse = _softmax_product(score, seen, v)
    out = out.view(B, hq, s["max_q"], d)[seq, :, at]
    lse = lse.view(B, hq, s["max_q"])[seq, :, at]
    return out.to(s["q"].dtype), lse


def _plain_selected(s):
    new, seq, pos, _ = _tokens(s)
    (N, hq, d), hkv = s["q"].shape, s["k_scale"].shape[1]
    seen = (s["idx"] >= 0) & (s["idx"] <= pos[:, None])
    j = torch.where(seen, s["idx"], 0).long()
    at, off = s["table"][seq[:, None], j // s["page"]].long(), j % s["page"]
    k = s["k_codes"][at, :, off].view(torch.float8_e4m3fn).float() * s["k_scale"][at][..., None]
    v = s["v_codes"][at, :, off].view(torch.float8_e4m3fn).float() * s["v_scale"][at][..., None]
    v = torch.where(seen[:, :, None, None], v, 0)
    q = s["q"].float().view(N, hkv, hq // hkv, d)
    score = (q @ k.permute(0, 2, 3, 1)) * d ** -0.5
    out, lse = _softmax_product(score, seen[:, None, None], v.transpose(1, 2))
    return out.reshape(N, hq, d).to(s["q"].dtype), lse.reshape(N, hq)


def run(state):
    s = state
    if s["op"] == "append":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["table"], s["lens"], s["cu_q"], s["cos"], s["sin"],
                                  interleaved=s["interleaved"], q=s["q"])
        else:
            q = _plain_append(s)
        e4m3 = torch.float8_e4m3fn
        return dict(q=q, k=s["k_codes"].view(e4m3), v=s["v_codes"].view(e4m3), k_scale=s["k_scale"],
                    v_scale=s["v_scale"])
    if s["op"] == "attention":
        if own:
            return s["cache"].attention(s["q"], s["table"], s["lens"], s["cu_q"], max_q=s["max_q"],
                                        window=s["window"], sinks=s["sinks"])
        return _plain_attention(s)
    if own:
        return s["cache"].attention_selected(s["q"], s["idx"], s["table"], s["lens"], s["cu_q"])
    return _plain_selected(s)


# ---------------------------------------------------------------------------------------------
# Work and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    lens, new = _lengths(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    N = int(new.sum())
    if case["op"] == "append":
        pages = int((-(-lens // page) - (lens - new) // page).sum())
        return {"bytes": N * (hq * d * 4 + hkv * d * 6 + case["rot"] * 4) + pages * hkv * 8,
                "flops": 3 * N * case["rot"] * (hq + hkv)}
    io = N * hq * (4 * d + 4)
    pairs = keys = 0
    for n, q in zip(lens.tolist(), new.tolist()):
        p = np.arange(n - q, n)
        if case["op"] == "selected":
            starts = p[::64]
            got = np.minimum(case["k"], np.repeat(starts, 64)[:q] + 1)
            pairs += int(got.sum())
            keys += min(n, int(np.minimum(3 * case["k"], starts + 1).sum()), int(got.sum()))
        elif case["window"]:
            lo = np.maximum(0, p - case["window"] + 1)
            pairs += int((p - lo + 1 + np.minimum(case["sinks"], lo)).sum())
            keys += int(n - lo[0] + min(case["sinks"], lo[0]))
        else:
            pairs += int((p + 1).sum())
            keys += n
    if case["op"] == "selected":
        io += N * case["k"] * 4
    return {"bytes": io + keys * hkv * 2 * d, "flops": 4 * d * hq * pairs}


def _e4m3(x):
    """x (64 bits) rounded to the nearest e4m3 value, ties to even."""
    ex = torch.frexp(x)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(x), ex - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    dev = "cuda"
    lens, cu, page = s["lens"].tolist(), s["cu_q"].tolist(), s["page"]
    N, hkv, d = s["k"].shape
    rot = 2 * s["cos"].shape[1]

    def turned(x, pos):
        x = x.double().clone()
        c, z = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = x[..., lo].clone(), x[..., hi].clone()
        x[..., lo], x[..., hi] = a * c - b * z, b * c + a * z
        return x

    kept = {n: s[n + "_codes"].view(torch.float8_e4m3fn).double() for n in "kv"}
    scale = {n: s[n + "_scale"].double() for n in "kv"}
    q = torch.empty(s["q"].shape, dtype=torch.float64, device=dev)
    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        p0 = lens[b] - n
        pos = torch.arange(p0, lens[b], device=dev)
        rows = slice(cu[b], cu[b + 1])
        q[rows] = turned(s["q"][rows], pos)
        at = s["table"][b].long()[p0 // page:(lens[b] - 1) // page + 1]
        span, off = len(at) * page, p0 % page
        for name, x in (("k", turned(s["k"][rows], pos)), ("v", s["v"][rows].double())):
            x = torch.cat([torch.zeros((off, hkv, d), dtype=torch.float64, device=dev), x,
                           torch.zeros((span - off - n, hkv, d), dtype=torch.float64, device=dev)])
            x = x.view(len(at), page, hkv, d).transpose(1, 2)
            amax = x.abs().amax((2, 3))
            unit = torch.exp2(torch.ceil(torch.log2(amax.clamp(min=2.0 ** -60) / 448)).clamp(E_MIN, E_MAX))
            if off:
                unit[0] = torch.maximum(unit[0], scale[name][at[0]])
            held = kept[name][at]
            ratio = (scale[name][at] / unit)[..., None, None]
            row = torch.arange(span, device=dev).view(len(at), 1, page, 1)
            held = torch.where(row < off, _e4m3(held * ratio), held)
            kept[name][at] = torch.where((row >= off) & (row < off + n), _e4m3(x / unit[..., None, None]), held)
            scale[name][at] = unit
    return dict(q=q, k=kept["k"], v=kept["v"], k_scale=scale["k"], v_scale=scale["v"])


def _exact_rows(q, k, v, seen):
    """q [r, d], k and v [s, d], seen [r, s], all in 64 bits."""
    t = (q @ k.T) / math.sqrt(q.shape[1])
    t = t.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(t, 1)
    w = torch.exp(t - lse[:, None]).masked_fill(~seen, 0.0)
    return w @ v, lse


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if s["op"] == "append":
        return _exact_append(s)
    page, cu, lens = s["page"], s["cu_q"].tolist(), s["lens"].tolist()
    N, hq, d = s["q"].shape
    hkv = s["k_scale"].shape[1]
    G = hq // hkv
    out = torch.zeros((N, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((N, hq), -math.inf, dtype=torch.float64, device="cuda")

    def rows_of(name, b, h, j):
        at = s["table"][b].long()[j // page]
        return s[name + "_codes"][at, h, j % page].view(torch.float8_e4m3fn).double() * s[name + "_scale"][at, h].double()[:, None]

    for b in range(len(lens)):
        n = cu[b + 1] - cu[b]
        p = torch.arange(lens[b] - n, lens[b], device="cuda")
        if s["op"] == "selected":
            for i in range(cu[b], cu[b + 1]):
                j = s["idx"][i].long()
                j = j[(j >= 0) & (j <= p[i - cu[b]])]
                if not len(j):
                    continue
                all_seen = torch.ones((G, len(j)), dtype=torch.bool, device="cuda")
                for h in range(hkv):
                    g = slice(h * G, h * G + G)
                    out[i, g], lse[i, g] = _exact_rows(s["q"][i, g].double(), rows_of("k", b, h, j), rows_of("v", b, h, j), all_seen)
            continue
        j = torch.arange(lens[b], device="cuda")
        seen = j[None] <= p[:, None]
        if s["window"]:
            seen &= (p[:, None] - j[None] < s["window"]) | (j[None] < s["sinks"])
        for h in range(hkv):
            k, v = rows_of("k", b, h, j), rows_of("v", b, h, j)
            for g in range(h * G, h * G + G):
                out[cu[b]:cu[b + 1], g], lse[cu[b]:cu[b + 1], g] = _exact_rows(s["q"][cu[b]:cu[b + 1], g].double(), k, v, seen)
    return out, lse
