"""Plain definitions of the row operators in 64 bits or more, for the tests:
one row, token or request at a time, no code shared with the kernels."""
import numpy as np

LD = np.longdouble


def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob) of one row of logits (any float array)."""
    x = np.asarray(x, dtype=np.float64)
    live = [i for i in range(x.size) if x[i] > -np.inf]
    if not live:
        return -1, -np.inf
    live = np.array(live)
    ranked = live[np.argsort(-x[live], kind="stable")]
    if not temperature > 0:
        return int(ranked[0]), 0.0
    best = x[ranked[0]]
    xr = x[ranked]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.exp((xr.astype(LD) - LD(best)) / LD(temperature))
    # scores at the largest weigh 1 (also +inf); below +inf nothing else weighs
    w = np.where(xr == best, LD(1), np.where(np.isnan(w), LD(0), w))
    w = np.where(w < LD(2.0) ** -44, LD(0), w)
    if 0 < top_k < w.size:
        w = w[:top_k]
    if top_p < 1:
        run = np.cumsum(w)
        n = 1 + int(np.count_nonzero(run[:-1] < LD(top_p) * run[-1]))
        w = w[:n]
    if min_p > 0:
        w = w[w >= min(1.0, float(min_p))]
    kept = ranked[:w.size]
    place = np.argsort(kept)
    run = np.cumsum(w[place])
    if not u > 0:
        u = 0.0
    u = min(float(u), 1.0 - 2.0 ** -24)
    at = int(np.searchsorted(run, LD(u) * run[-1], side="right"))
    return int(kept[place[at]]), float(np.log(w[place[at]] / run[-1]))


def _score(x, scoring):
    """64-bit scores of one token's logits; masked experts weigh nothing."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            s = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))),
                         np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
            return np.where(x > -np.inf, s, 0.0)
        live = x > -np.inf
        if not live.any():
            return np.zeros_like(x)
        top = x[live].max()
        e = np.where(live, np.where(x == top, 1.0, np.exp(x - top)), 0.0)
        return e / e.sum()


def route_token(x, top_k, scoring, bias=None, groups=1, topk_groups=1, group_score="max",
                renormalize=True, scale=1.0):
    """(indices, weights) of one token."""
    x = np.asarray(x, dtype=np.float64)
    E = x.size
    s = _score(x, scoring)
    c = s + np.asarray(bias, dtype=np.float64) if bias is not None else x.copy()
    c = np.where((x > -np.inf) & (c > -np.inf), c, -np.inf)
    if groups > 1:
        size = E // groups
        score = []
        for g in range(groups):
            own = sorted((e for e in range(g * size, (g + 1) * size) if c[e] > -np.inf),
                         key=lambda e: (-c[e], e))
            if not own:
                score.append(-np.inf)
            elif group_score == "max":
                score.append(c[own[0]])
            else:
                by = c if bias is not None else s
                score.append(sum(by[e] for e in own[:2]))
        best = sorted(range(groups), key=lambda g: (-score[g], g))[:topk_groups]
        for g in range(groups):
            if g not in best:
                c[g * size:(g + 1) * size] = -np.inf
    order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:top_k]
    w = np.array([s[e] for e in order])
    if renormalize:
        if scoring == "softmax" and len(order):
            w = _score(x[order], "softmax")   # the whole's sum cancels
        total = w.sum()
        w = w / total if total > 0 else np.zeros_like(w)
    idx = np.full(top_k, -1, dtype=np.int32)
    out = np.zeros(top_k)
    idx[:len(order)] = order
    out[:len(order)] = w * scale
    return idx, out


def weights_of(x, idx, scoring, renormalize, scale):
    """The weights as a function of one token's logits at given experts."""
    ok = [(j, e) for j, e in enumerate(idx) if 0 <= e < len(x) and x[e] > -np.inf]
    out = np.zeros(len(idx))
    if not ok:
        return out
    s = _score(x, scoring)
    w = np.array([s[e] for _, e in ok])
    if renormalize:
        if scoring == "softmax":
            z = np.array([x[e] for _, e in ok], dtype=np.float64)
            w = np.exp(z - z.max())
        w = w / w.sum() if w.sum() > 0 else w * 0
    for (j, _), v in zip(ok, w):
        out[j] = v * scale
    return out


def route_grad_token(x, idx, g, scoring, renormalize, scale):
    """(gradient, magnitude of its terms) of one token's weights, by the formula."""
    x = np.asarray(x, dtype=np.float64)
    E = x.size
    ok = [(j, int(e)) for j, e in enumerate(idx) if 0 <= e < E and x[e] > -np.inf]
    out, size = np.zeros(E), np.zeros(E)
    if not ok:
        return out, size
    s = _score(x, scoring)
    if scoring == "softmax" and renormalize:
        top = max(x[e] for _, e in ok)
        s = np.where(x > -np.inf, np.exp(np.minimum(x - top, 0)), 0.0)
    total = sum(s[e] for _, e in ok)
    if renormalize and not total > 0:
        return out, size
    dot = sum(g[j] * s[e] for j, e in ok)
    ds = np.zeros(E)
    mag = np.zeros(E)
    for j, e in ok:
        if renormalize:
            ds[e] += (g[j] - dot / total) / total
            mag[e] += (abs(g[j]) + abs(dot / total)) / total
        else:
            ds[e] += g[j]
            mag[e] += abs(g[j])
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            other = _score(-x, "sigmoid")
        out, size = ds * s * other, mag * s * other
    elif renormalize:
        out, size = ds * s, mag * s
    else:
        out, size = s * (ds - dot), s * (mag + abs(dot))
    return out * scale, size * abs(scale)


def extend_tables(tables, kv_lens, new_tokens, free, start, bs, max_tokens, wide=False):
    tables = np.array(tables, dtype=np.int64)
    R, width = tables.shape
    start = max(int(start), 0)
    taken = 0
    starts, req, pos, slots = [0], [], [], []
    for r in range(R):
        kv = max(int(kv_lens[r]), 0)
        new = min(max(int(new_tokens[r]), 0), kv)
        old = kv - new
        held, need = min(-(-old // bs), width), min(-(-kv // bs), width)
        for b in range(held, need):
            at = start + taken
            tables[r, b] = free[at] if at < len(free) else -1
            taken += 1
        for p in range(old, kv):
            b = p // bs
            block = tables[r, b] if b < width else -1
            slot = block * bs + p % bs if block >= 0 else -1
            if not wide and slot > 2 ** 31 - 1:
                slot = -1
            req.append(r), pos.append(p), slots.append(slot)
        starts.append(len(req))
    def pad(v):
        return np.array((v + [-1] * max_tokens)[:max_tokens], dtype=np.int64)
    return tables, np.array(starts), pad(req), pad(pos), pad(slots), start + taken


def slots_of(indices, tables, bs, owner, wide=False):
    indices = np.asarray(indices, dtype=np.int64)
    out = np.full(indices.shape, -1, dtype=np.int64)
    R, width = tables.shape
    for r in range(indices.shape[0]):
        q = int(owner[r])
        if not 0 <= q < R:
            continue
        for j, i in enumerate(indices[r]):
            if i >= 0 and i // bs < width and tables[q, i // bs] >= 0:
                s = int(tables[q, i // bs]) * bs + int(i) % bs
                out[r, j] = s if wide or s <= 2 ** 31 - 1 else -1
    return out
