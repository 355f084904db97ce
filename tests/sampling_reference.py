"""Plain 64-bit implementation of the token sampler, row by row, for the tests.

The kernels' weights are right to 2^-32 of themselves and 2^-44 of the largest, so a sum of n of them is right to
2^-31 of itself for the inputs here (n below 2^19, a largest of 1 among them: n 2^-44 <= 2^-25 only where all the others
are next to nothing, and then their share of the total is too).  Where a border lies nearer to its target than
`SLACK` of the total, the row says so and either side of it is accepted; borders that are whole numbers of equal
weights are exact on both sides."""
import numpy as np

SLACK = 2.0 ** -30


def sample_row(x, u, temperature, top_k, top_p, min_p):
    """(accepted tokens, logp of each, how many are kept) for x fp64 [V]."""
    f = lambda v: np.float64(np.float32(v))
    x = np.asarray(x, dtype=np.float64)
    if np.isnan(x).any() or (x == np.inf).any():
        return [-1], [np.nan], 0
    m = x.max()
    if m == -np.inf:
        return [-1], [-np.inf], 0
    if temperature == 0:
        return [int(np.argmax(x))], [0.0], 1
    with np.errstate(over="ignore"):
        z = (x - m) / f(temperature)
    w = np.exp(z)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    order = order[w[order] >= f(min_p)]
    if top_k > 0:
        order = order[:top_k]
    cuts = [len(order)]
    if f(top_p) < 1:
        run = np.cumsum(w[order])
        goal = f(top_p) * run[-1]
        cuts = sorted({int(np.searchsorted(run, g)) + 1 for g in (goal, goal - SLACK * run[-1], goal + SLACK * run[-1])
                       if g == goal or not _exact(w[order])})
    tokens, logps = [], []
    for n in cuts:
        kept = np.sort(order[:max(min(n, len(order)), 1)])
        run = np.cumsum(w[kept])
        goal = f(u) * run[-1]
        for g in (goal,) if _exact(w[kept]) else (goal, goal - SLACK * run[-1], goal + SLACK * run[-1]):
            i = min(int(np.searchsorted(run, g, side="right")), len(kept) - 1)
            while i > 0 and w[kept[i]] == 0:
                i -= 1
            if kept[i] not in tokens:
                tokens.append(int(kept[i]))
                logps.append(z[kept[i]] - np.log(run[-1]))
    return tokens, logps, cuts[0]


def _exact(w):
    return bool((w == w[0]).all())


def check(logits, u, got, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None):
    """got = (token, logp) of the framework for logits [B, V] (any type), settings numbers or [B]."""
    x = logits.double().cpu().numpy()
    token, logp = got[0].cpu().numpy(), got[1].double().cpu().numpy()
    u = u.double().cpu().numpy()
    of = lambda s, r: s[r].item() if hasattr(s, "shape") else s
    doubtful = 0
    for r in range(len(x)) if rows is None else rows:
        tokens, logps, _ = sample_row(x[r], u[r], of(temperature, r), of(top_k, r), of(top_p, r), of(min_p, r))
        doubtful += len(tokens) > 1
        assert token[r] in tokens, (r, int(token[r]), tokens, u[r])
        want = logps[tokens.index(token[r])]
        # (x - m) log2(e) / T and the logarithm in double, rounded to fp32; the total to 2^-31
        assert np.isnan(logp[r]) == np.isnan(want)
        assert np.isnan(want) or logp[r] == want or abs(logp[r] - want) <= 2.0 ** -24 * 1.01 * abs(want) + 2.0 ** -30, (r, logp[r], want)
    return doubtful
