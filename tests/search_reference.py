"""Plain definitions of a beam search's operators in 64 bits, for the tests: one
request, row or token at a time, no code shared with the kernels."""
import numpy as np

LD = np.longdouble


def beams(x, scores, k, ended=None, end_token=0, lengths=None, penalty=0.0):
    """(totals, parents, tokens) of one request: x [beams][vocab], scores [beams]."""
    found = []
    for b in range(x.shape[0]):
        s = float(scores[b])
        if not np.isfinite(s):
            continue
        done = ended is not None and bool(ended[b])
        norm = 1.0
        if lengths is not None:
            norm = float(max(int(lengths[b]) + (0 if done else 1), 1)) ** float(penalty)
        if done:
            found.append((s / norm, b, end_token, s))
            continue
        row = x[b].astype(np.float64)
        live = np.flatnonzero(row > -np.inf)
        if live.size == 0:
            continue
        top = row[live].max()
        if top == np.inf:
            live = np.flatnonzero(row == np.inf)
            lse, base = float(np.log(LD(live.size))), np.zeros(row.size)
        else:
            # (against the largest: its own size would swallow the sum's logarithm)
            lse, base = float(np.log(np.exp((row[live] - top).astype(LD)).sum())), row - top
        for i in live[np.argsort(-base[live], kind="stable")[:k]]:
            total = s + (base[i] - lse)
            found.append((total / norm, b, int(i), total))
    found.sort(key=lambda c: (-c[0], c[1], c[2]))
    found = (found + [(0.0, -1, -1, -np.inf)] * k)[:k]
    return [c[3] for c in found], [c[1] for c in found], [c[2] for c in found]


def block_tables(tables, lens, parents, block_size, tail=None):
    """(new tables, [(child row, source block, target block, tokens)])."""
    R, k = parents.shape
    W = tables.shape[0] // R
    out = np.full((R * k, tables.shape[1]), -1, dtype=np.int32)
    copies = []
    for r in range(R):
        n = max(int(lens[r]), 0)
        full, part = n // block_size, n % block_size
        for j in range(k):
            if W == k:
                out[r * k + j] = tables[r * W + j]
            p = int(parents[r, j])
            if not 0 <= p < W:
                continue
            out[r * k + j, :full] = tables[r * W + p, :full]
            if part and full < tables.shape[1]:
                mine = int(tail[r * k + j]) if tail is not None else int(tables[r * W + j, full])
                out[r * k + j, full] = mine
                copies.append((r * k + j, int(tables[r * W + p, full]), mine, part))
    return out, copies


def positions(table, n, block_size, num_blocks):
    """(block, offset) of the first n positions, those in the cache alone, and which they are."""
    p = np.arange(max(0, min(int(n), table.size * block_size)))
    b = table[p // block_size]
    ok = (b >= 0) & (b < num_blocks)
    return b[ok], (p % block_size)[ok], p[ok]


def attention(q, k, v, entries, scale):
    """One token: q [heads][dim]; entries: [(blocks, offsets)] of what it sees;
    k, v [blocks][block_size][kv_heads][dim].  (out, lse, bound of out, of lse,
    weights): the bounds without the types' rounding, see `bounds`."""
    heads, dim = q.shape
    kv = k.shape[2]
    per = heads // kv
    ks = np.concatenate([k[b, o] for b, o in entries]) if entries else np.zeros((0, kv, dim))
    vs = np.concatenate([v[b, o] for b, o in entries]) if entries else np.zeros((0, kv, dim))
    n = ks.shape[0]
    out, lse = np.zeros((heads, dim)), np.full(heads, -np.inf)
    spread, size, delta = np.zeros((heads, dim)), np.zeros((heads, dim)), np.zeros(heads)
    weights = np.zeros((heads, n))
    for h in range(heads):
        if n == 0:
            continue
        a = ks[:, h // per] @ q[h] * scale
        top = a.max()
        w = np.exp(a - top)
        z = w.sum()
        weights[h] = w / z
        out[h] = weights[h] @ vs[:, h // per]
        lse[h] = top + np.log(z)
        spread[h] = weights[h] @ np.abs(vs[:, h // per])
        size[h] = np.abs(vs[:, h // per]).sum(0)
        # a score: dim products added up in 32 bits, then scaled and taken from
        # the largest (each to 2^-24 of the values), and the exponential
        delta[h] = (dim + 8) * 2.0 ** -24 * scale * (np.abs(ks[:, h // per]) @ np.abs(q[h])).max() + 2.0 ** -21
    return out, lse, spread, size, delta, weights


def bounds(out, lse, spread, size, delta, n, half_step, smallest):
    """What out and lse may be off by: weights rounded to the type (half_step of
    themselves; in float16 those below its normal numbers by 2^-25, beside a
    largest of 1 at least), their errors from the scores' (twice: in the weight
    and in the sum), n additions in 32 bits, and out's own rounding."""
    fp32 = 2 * delta + (n + 64) * 2.0 ** -24
    off = (half_step + fp32)[:, None] * 1.01 * spread + smallest * size + half_step[:, None] * np.abs(out) + smallest
    return off, fp32 + 2.0 ** -22 * np.abs(np.where(np.isinf(lse), 0.0, lse))


def keep(mass, n, budget, sinks, recent):
    """The kept positions of one row, rising."""
    n = max(0, min(int(n), mass.size))
    if n <= budget:
        return np.arange(n)
    fixed = np.r_[np.arange(sinks), np.arange(n - recent, n)]
    rest = np.arange(sinks, n - recent)
    m = mass[rest].astype(np.float64)
    # NaN below -inf, equal ones by position
    order = np.lexsort((rest, -np.where(np.isnan(m), -np.inf, m), np.isnan(m)))
    return np.sort(np.r_[fixed, rest[order[:budget - sinks - recent]]]).astype(np.int64)
