"""What is measured of the operators of a beam search over a paged cache: choosing the beams,
reordering what they hold, attention with a prefix that sequences share, the attention mass of
cached positions, and eviction by it.

Each case is one pass of one operator.  With ``own`` false, ``run`` computes it with elementary
torch operations; with ``own`` true it makes the framework's calls.  The beams' choice is made in
64 bits in the plain form: a sum over a hundred thousand weights, and two totals next to each other
at a border, need them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def _beams(requests, beams, k, vocab, dtype, ended, penalty, pad=0, spread=2.0):
    return {"op": "beams", "requests": requests, "beams": beams, "k": k, "vocab": vocab,
            "dtype": dtype, "ended": ended, "penalty": penalty, "pad": pad, "spread": spread}


def _reorder(requests, beams, history, state, longest, block_size, caches, heads, dim):
    return {"op": "reorder", "requests": requests, "beams": beams, "history": history, "state": state,
            "longest": longest, "block_size": block_size, "caches": caches, "heads": heads, "dim": dim}


def _attend(op, groups, members, ragged, prefix, suffix, heads, kv_heads, dim, dtype, block_size, next_n=1):
    return {"op": op, "groups": groups, "members": members, "ragged": ragged, "prefix": prefix,
            "suffix": suffix, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "block_size": block_size, "next_n": next_n}


def _evict(requests, mass_heads, heads, dim, longest, budget, sinks, recent, block_size):
    return {"op": "evict", "requests": requests, "mass_heads": mass_heads, "heads": heads, "dim": dim,
            "longest": longest, "budget": budget, "sinks": sinks, "recent": recent,
            "block_size": block_size}


def listed():
    return [
        # one request of four beams: the call's latency is what counts
        {"name": "beams_one_request", **_beams(1, 4, 8, 32768, "bf16", 0.0, 0.0)},
        # the largest: a batch of searches, some beams at their end, scores weighed by length
        {"name": "beams_batch", **_beams(32, 8, 16, 131072, "fp32", 0.1, 0.8)},
        # five beams over an odd vocabulary in half precision, padded rows
        {"name": "beams_odd", **_beams(48, 5, 10, 50001, "fp16", 0.0, 0.0, pad=7)},
        # a small search's step: token histories, a small state, the open blocks of one layer
        {"name": "reorder_small", **_reorder(2, 4, 200, 1000, 300, 16, 2, 8, 64)},
        # a batch's step: histories, recurrent states, the open blocks of two layers
        {"name": "reorder_batch", **_reorder(32, 8, 1024, 65536, 8192, 64, 4, 8, 128)},
        # four beams over a short prompt: latency
        {"name": "attend_small", **_attend("attend", 1, 4, False, 1000, 100, 32, 8, 128, "bf16", 64)},
        # two long prompts with 32 continuations each
        {"name": "attend_shared", **_attend("attend", 2, 32, False, 32768, 512, 64, 8, 128, "bf16", 64)},
        # groups of different sizes, two new tokens a sequence, narrow heads, odd lengths
        {"name": "attend_ragged", **_attend("attend", 7, 5, True, 5001, 777, 16, 4, 64, "fp16", 16, next_n=2)},
        # the mass of a batch of beam searches' positions
        {"name": "mass_beams", **_attend("mass", 8, 8, False, 8192, 256, 32, 8, 128, "bf16", 64)},
        # groups of different sizes, one key head for all
        {"name": "mass_ragged", **_attend("mass", 3, 4, True, 2999, 301, 8, 1, 64, "fp16", 16)},
        # prompts cut down to an eighth, each head by itself
        {"name": "evict_prompt", **_evict(16, 8, 8, 128, 8192, 1024, 4, 128, 64)},
        # one request at its limit, all heads alike, odd sizes
        {"name": "evict_odd", **_evict(1, 1, 4, 64, 5003, 777, 1, 33, 16)},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["beams", "beams", "reorder", "attend", "attend", "mass", "evict"])
    if op == "beams":
        vocab = _log_int(rng, 1000, 200000)
        beams = _log_int(rng, 1, 16)
        requests = _log_int(rng, 1, max(1, min(64, 256 * 131072 // (vocab * beams))))
        return _beams(requests, beams, rng.randint(beams, 2 * beams), vocab, rng.choice(["fp32", "bf16", "fp16"]),
                      rng.choice([0.0, 0.0, 0.2]), rng.choice([0.0, 0.0, 0.6, 1.0]),
                      pad=rng.choice([0, 0, 1, 8, 33]), spread=round(rng.uniform(1.0, 3.0), 2))
    if op == "reorder":
        beams = _log_int(rng, 1, 16)
        return _reorder(_log_int(rng, 1, 256 // beams), beams, _log_int(rng, 1, 1024), _log_int(rng, 1, 65536),
                        _log_int(rng, 20, 8192), rng.choice([1, 16, 48, 64]), rng.randint(1, 4),
                        rng.choice([1, 2, 8]), rng.choice([64, 80, 128]))
    if op in ("attend", "mass"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 7, 8])
        groups, members = _log_int(rng, 1, 16), _log_int(rng, 1, 32)
        limit = (2 * 32768 * 8) // (groups * kv_heads)
        prefix = _log_int(rng, 1, max(1, min(32768, limit)))
        suffix = _log_int(rng, 4, max(4, min(1024, 64 * 512 * 8 // (groups * members * kv_heads))))
        next_n = rng.choice([1, 1, 2, 3])
        while next_n > 1 and groups * members * next_n * heads > 4096:
            next_n -= 1
        members = max(1, min(members, 4096 // (groups * heads)))
        return _attend(op, groups, members, rng.random() < 0.4, prefix, suffix, heads, kv_heads,
                       rng.choice([64, 128]), rng.choice(["bf16", "fp16"]), rng.choice([16, 32, 64, 128]),
                       next_n=next_n)
    heads = rng.choice([1, 2, 4, 8])
    requests = _log_int(rng, 1, 32)
    longest = _log_int(rng, 64, 16 * 8192 // requests if requests > 8 else 16384)
    budget = _log_int(rng, 16, max(16, min(longest, 1024)))
    recent = rng.randint(0, budget // 2)
    return _evict(requests, rng.choice([1, heads]), heads, rng.choice([64, 128]), longest, budget,
                  rng.randint(0, min(4, budget - recent)), recent, rng.choice([16, 48, 64]))


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _prepare_beams(case, seed):
    R, W, vocab, dev = case["requests"], case["beams"], case["vocab"], "cuda"
    g = _gen(seed, 53)
    # a bulk of unlikely tokens and some dozens that the context makes likely
    x = torch.randn(R * W, vocab + case["pad"], device=dev, generator=g) * case["spread"]
    likely = torch.randint(0, vocab, (R * W, 48), device=dev, generator=g)
    x.scatter_add_(1, likely, torch.randn(R * W, 48, device=dev, generator=g) * 2 + 6)
    banned = torch.randint(0, vocab, (R * W, 16), device=dev, generator=g)
    x.scatter_(1, banned, float("-inf"))
    x = x.to(DTYPES[case["dtype"]])[:, :vocab]
    st = {"case": case, "logits": x, "ended": None, "lengths": None,
          "scores": -20 - 5 * torch.rand(R, W, device=dev, generator=g)}
    if case["ended"]:
        st["ended"] = torch.rand(R, W, device=dev, generator=g) < case["ended"]
    if case["penalty"]:
        st["lengths"] = torch.randint(20, 40, (R, W), device=dev, generator=g, dtype=torch.int32)
    return st


def _prepare_reorder(case, seed):
    R, W, bs, dev = case["requests"], case["beams"], case["block_size"], "cuda"
    g = _gen(seed, 59)
    rows, width = R * W, (case["longest"] + bs - 1) // bs
    # every row holds an open block and is given one for the step; full blocks come from a shared pool
    own_blocks = torch.randperm(2 * rows, device=dev, generator=g).to(torch.int32)
    lens = torch.randint(1, case["longest"] + 1, (R,), device=dev, generator=g).to(torch.int32)
    tables = torch.randint(2 * rows, 2 * rows + 64, (R, 1, width), device=dev, generator=g).to(torch.int32)
    tables = tables.expand(R, W, width).reshape(rows, width).contiguous()
    full = (lens // bs).long().repeat_interleave(W)
    col = torch.arange(width, device=dev)[None, :]
    tables = torch.where(col == full[:, None], own_blocks[:rows, None], tables)
    tables = torch.where(col > full[:, None], -1, tables).to(torch.int32)
    caches = [torch.randn(2 * rows + 64, bs, case["heads"], case["dim"], device=dev, generator=g).bfloat16()
              for _ in range(case["caches"])]
    return {"case": case, "lens": lens, "tables": tables, "tail": own_blocks[rows:].clone(), "caches": caches,
            # most children come from the better beams
            "parents": (torch.rand(R, W, device=dev, generator=g) ** 2 * W).to(torch.int32),
            "history": torch.randint(0, 131072, (rows, case["history"]), device=dev, generator=g, dtype=torch.int32),
            "state": torch.randn(rows, case["state"], device=dev, generator=g)}


def _prepare_attend(case, seed):
    G, bs, dev, dt = case["groups"], case["block_size"], "cuda", DTYPES[case["dtype"]]
    g = _gen(seed, 61)
    S = G * case["members"]
    starts = torch.arange(G + 1, device=dev, dtype=torch.int32) * case["members"]
    if case["ragged"]:
        cuts = torch.randint(0, S + 1, (G - 1,), device=dev, generator=g).sort()[0]
        starts[1:G] = cuts.to(torch.int32)
    T, P, L = case["next_n"], case["prefix"], case["suffix"]
    plens = torch.randint((P + 1) // 2, P + 1, (G,), device=dev, generator=g).to(torch.int32)
    lens = torch.randint(min(T, L), L + 1, (S,), device=dev, generator=g).to(torch.int32)
    pw, sw = (P + bs - 1) // bs, (L + bs - 1) // bs
    ids = torch.randperm(G * pw + S * sw, device=dev, generator=g).to(torch.int32)
    shape = (ids.numel(), bs, case["kv_heads"], case["dim"])
    st = {"case": case, "starts": starts, "plens": plens, "lens": lens,
          "ptables": ids[:G * pw].view(G, pw).clone(), "tables": ids[G * pw:].view(S, sw).clone(),
          "k": torch.randn(shape, device=dev, generator=g).to(dt),
          "v": torch.randn(shape, device=dev, generator=g).to(dt),
          # sharper than unrelated vectors: a query attends to some of its keys
          "q": (torch.randn(S * T, case["heads"], case["dim"], device=dev, generator=g) * 1.5).to(dt)}
    if case["op"] == "mass":
        st["lse"] = _plain_attend(case, st)[1]
        st["pmass"] = torch.rand(G, case["kv_heads"], pw * bs, device=dev, generator=g)
        st["mass"] = torch.rand(S, case["kv_heads"], sw * bs, device=dev, generator=g)
    return st


def _prepare_evict(case, seed):
    R, H, L, B, bs, dev = (case["requests"], case["mass_heads"], case["longest"], case["budget"],
                           case["block_size"], "cuda")
    g = _gen(seed, 67)
    width, kept = (L + bs - 1) // bs, (B + bs - 1) // bs
    mass = torch.exp(2.5 * torch.randn(R, H, width * bs, device=dev, generator=g))
    # positions that nothing has attended to
    mass = torch.where(torch.rand(mass.shape, device=dev, generator=g) < 0.3, 0.0, mass)
    ids = torch.randperm(R * (width + kept), device=dev, generator=g).to(torch.int32)
    shape = (R * (width + kept), bs, case["heads"], case["dim"])
    return {"case": case, "mass": mass,
            "lens": torch.randint((L + 1) // 2, L + 1, (R,), device=dev, generator=g).to(torch.int32),
            "tables": ids[:R * width].view(R, width).clone(), "to": ids[R * width:].view(R, kept).clone(),
            "caches": [torch.randn(shape, device=dev, generator=g).bfloat16() for _ in range(2)]}


_PREPARE = {"beams": _prepare_beams, "reorder": _prepare_reorder, "attend": _prepare_attend,
            "mass": _prepare_attend, "evict": _prepare_evict}


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](case, state)
    return _PLAIN[case["op"]](case, state)


def _own_beams(case, st):
    import exact_row_top_amd as ert
    return ert.select_beams(st["logits"], st["scores"], case["k"], ended=st["ended"], end_token=2,
                            lengths=st["lengths"], length_penalty=case["penalty"])


def _own_reorder(case, st):
    import exact_row_top_amd as ert
    history, state = ert.reorder_beams([st["history"], st["state"]], st["parents"])
    tables = ert.reorder_block_tables(st["tables"], st["lens"], st["parents"], case["block_size"],
                                      caches=st["caches"], tail_blocks=st["tail"])
    return history, state, tables, st["caches"]


def _own_attend(case, st):
    import exact_row_top_amd as ert
    return ert.prefix_attention(st["q"], st["k"], st["v"], st["ptables"], st["plens"], st["tables"],
                                st["lens"], group_starts=st["starts"], next_n=case["next_n"],
                                return_lse=True)


def _own_mass(case, st):
    import exact_row_top_amd as ert
    return ert.attention_mass(st["q"], st["k"], st["lse"], st["ptables"], st["plens"], st["tables"],
                              st["lens"], group_starts=st["starts"], next_n=case["next_n"],
                              prefix_mass=st["pmass"], mass=st["mass"], decay=0.99)


def _own_evict(case, st):
    import exact_row_top_amd as ert
    kept, mass, lens = ert.evict_cache(st["mass"], st["lens"], case["budget"], sinks=case["sinks"],
                                       recent=case["recent"], block_tables=st["tables"],
                                       caches=st["caches"], out_tables=st["to"])
    return kept, mass, lens, st["caches"]


_OWN = {"beams": _own_beams, "reorder": _own_reorder, "attend": _own_attend, "mass": _own_mass,
        "evict": _own_evict}


def _plain_beams(case, st):
    R, W, V = case["requests"], case["beams"], case["vocab"]
    x = st["logits"].double()
    x = torch.where(torch.isnan(x), float("-inf"), x)
    best = x.amax(1, keepdim=True)
    x = x - (best + torch.log(torch.exp(x - best).sum(1, keepdim=True)))
    total = st["scores"].double()[:, :, None] + x.view(R, W, V)
    if st["ended"] is not None:
        ended = st["ended"][:, :, None]
        only = torch.where(torch.arange(V, device=x.device) == 2, st["scores"].double()[:, :, None], float("-inf"))
        total = torch.where(ended, only, total)
    rank = total
    if st["lengths"] is not None:
        n = st["lengths"].double() + (1.0 if st["ended"] is None else torch.where(st["ended"], 0.0, 1.0))
        rank = total / torch.pow(n, case["penalty"])[:, :, None]
    order = torch.sort(rank.view(R, W * V), dim=1, descending=True, stable=True)[1][:, :case["k"]]
    score = total.view(R, W * V).gather(1, order)
    dead = score == float("-inf")
    return (score.float(), torch.where(dead, -1, order // V).int(), torch.where(dead, -1, order % V).int())


def _plain_reorder(case, st):
    R, W, bs = case["requests"], case["beams"], case["block_size"]
    dev = st["parents"].device
    source = (st["parents"].long() + torch.arange(R, device=dev)[:, None] * W).view(-1)
    lens = st["lens"].long().repeat_interleave(W)
    full, part = lens // bs, lens % bs
    col = torch.arange(st["tables"].shape[1], device=dev)[None, :]
    held = st["tables"][source]
    mine = (col == full[:, None]) & (part > 0)[:, None]
    tables = torch.where(mine, st["tail"][:, None], torch.where(col < full[:, None], held, st["tables"]))
    # the parents' open blocks into the children's own
    at = full.clamp(max=col.shape[1] - 1)[:, None]
    src, dst = held.gather(1, at)[:, 0].long().clamp(min=0), st["tail"].long()
    live = (torch.arange(bs, device=dev)[None, :] < part[:, None])[:, :, None, None]
    for cache in st["caches"]:
        cache[dst] = torch.where(live, cache[src], cache[dst])
    return st["history"][source], st["state"][source], tables, st["caches"]


def _pages(cache, tables):
    # [entries, kv heads, positions, dim] in 32 bits
    return cache[tables.long()].flatten(1, 2).float().transpose(1, 2)


def _attend_parts(case, st):
    """Scores of the shared and of the own positions, -inf where masked, and where the queries of a
    group stand in its padded rows."""
    G, S, T, H, D = st["plens"].numel(), st["lens"].numel(), case["next_n"], case["kv_heads"], case["dim"]
    dev, per = st["q"].device, case["heads"] // case["kv_heads"]
    q = st["q"].float().view(S, T, H, per, D) * D ** -0.5
    group = torch.searchsorted(st["starts"][1:].long(), torch.arange(S, device=dev), right=True)
    place = torch.arange(S, device=dev) - st["starts"].long()[group]
    room = S if case["ragged"] else case["members"]
    padded = torch.zeros(G, room, T, H, per, D, device=dev)
    padded[group, place] = q
    shared = torch.matmul(padded.permute(0, 3, 1, 2, 4, 5).reshape(G, H, room * T * per, D),
                          _pages(st["k"], st["ptables"]).transpose(2, 3))
    at = torch.arange(shared.shape[3], device=dev)
    shared = torch.where(at < st["plens"][:, None, None, None], shared, float("-inf"))
    mine = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(S, H, T * per, D),
                        _pages(st["k"], st["tables"]).transpose(2, 3)).view(S, H, T, per, -1)
    at = torch.arange(mine.shape[4], device=dev)
    sees = st["lens"][:, None] - T + 1 + torch.arange(T, device=dev)
    mine = torch.where(at < sees[:, None, :, None, None], mine, float("-inf"))
    return shared.view(G, H, room, T, per, -1), mine, group, place


def _rows_of(x, group, place):
    # [G, H, room, T, per, n] -> [S, H, T, per, n]
    return x[group, :, place]


def _plain_attend(case, st):
    shared, mine, group, place = _attend_parts(case, st)
    S, H, T, per, _ = mine.shape
    D = case["dim"]
    top = shared.amax(5, keepdim=True)
    best = torch.maximum(_rows_of(top, group, place), mine.amax(4, keepdim=True))
    ground = torch.where(top == float("-inf"), 0.0, top)
    weights = torch.exp(shared - ground)
    G, room = shared.shape[0], shared.shape[2]
    value = torch.matmul(weights.view(G, H, room * T * per, -1), _pages(st["v"], st["ptables"]))
    floor = torch.where(best == float("-inf"), 0.0, best)
    scale = torch.exp(_rows_of(ground, group, place) - floor)
    scale = torch.where(_rows_of(top, group, place) == float("-inf"), 0.0, scale)
    total = _rows_of(weights.sum(5, keepdim=True), group, place) * scale
    value = _rows_of(value.view(G, H, room, T, per, D), group, place) * scale
    weights = torch.exp(mine - floor)
    value = value + torch.matmul(weights.view(S, H, T * per, -1), _pages(st["v"], st["tables"])).view(S, H, T, per, D)
    total = total + weights.sum(4, keepdim=True)
    out = torch.where(total > 0, value / total, 0.0).permute(0, 2, 1, 3, 4).reshape(S * T, H * per, D)
    lse = (best + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(S * T, H * per)
    return out.to(st["q"].dtype), lse


def _plain_mass(case, st):
    shared, mine, group, place = _attend_parts(case, st)
    S, H, T, per, _ = mine.shape
    lse = st["lse"].view(S, T, H, per).permute(0, 2, 1, 3)
    whole = torch.full(shared.shape[:5], float("inf"), device=lse.device)
    whole[group, :, place] = lse
    shared = torch.exp(shared - whole[..., None]).sum((2, 3, 4))
    mine = torch.exp(mine - lse[..., None]).sum((2, 3))
    return st["pmass"] * 0.99 + shared, st["mass"] * 0.99 + mine


def _plain_evict(case, st):
    R, H, B, bs = case["requests"], case["mass_heads"], case["budget"], case["block_size"]
    mass, n = st["mass"], st["lens"].long()[:, None, None]
    dev = mass.device
    at = torch.arange(mass.shape[2], device=dev)
    key = torch.where((at < case["sinks"]) | (at >= n - case["recent"]), float("inf"), mass)
    key = torch.where(at < n, key, float("-inf"))
    kept = torch.sort(key, dim=2, descending=True, stable=True)[1][:, :, :B]
    kept = torch.where(kept < n, kept, mass.shape[2]).sort(dim=2)[0]
    kept = torch.nn.functional.pad(kept, (0, B - kept.shape[2]), value=mass.shape[2])
    live = kept < mass.shape[2]
    place = torch.where(live, kept, 0)
    kept_mass = torch.where(live, mass.gather(2, place), 0.0)
    # every kept position's row from its old slot to its new one
    r = torch.arange(R, device=dev)[:, None, None]
    j = torch.arange(B, device=dev)[None, None, :]
    src, dst = st["tables"].long()[r, place // bs], st["to"].long()[r, j // bs]
    per = case["heads"] // H
    h = torch.arange(H, device=dev)[None, :, None]
    for cache in st["caches"]:
        rows = cache.view(cache.shape[0], bs, H, per * case["dim"])
        moved = rows[src, place % bs, h]
        there = rows[dst, (j % bs).expand_as(place), h.expand_as(place)]
        rows[dst, (j % bs).expand_as(place), h.expand_as(place)] = torch.where(live[..., None], moved, there)
    return (torch.where(live, kept, -1).int(), kept_mass, torch.clamp(st["lens"], max=B), st["caches"])


_PLAIN = {"beams": _plain_beams, "reorder": _plain_reorder, "attend": _plain_attend, "mass": _plain_mass,
          "evict": _plain_evict}


# --------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "beams":
        rows, size = case["requests"] * case["beams"], 4 if case["dtype"] == "fp32" else 2
        live = 1.0 - case["ended"]
        return {"bytes": rows * (live * case["vocab"] * size + 9) + case["requests"] * case["k"] * 12,
                "flops": 4 * live * rows * case["vocab"]}
    if op == "reorder":
        rows, bs = case["requests"] * case["beams"], case["block_size"]
        width = (case["longest"] + bs - 1) // bs
        # the parents' rows are read once however many children they have; about 0.6 of the beams are parents
        open_block = (bs - 1) / 2 * case["heads"] * case["dim"] * 2 * case["caches"]
        row = case["history"] * 4 + case["state"] * 4 + width * 4 + open_block
        return {"bytes": 1.6 * rows * row, "flops": 0}
    if op in ("attend", "mass"):
        S, T = case["groups"] * case["members"], case["next_n"]
        P, L = 0.75 * case["prefix"], 0.5 * (case["suffix"] + T)
        cached = (case["groups"] * P + S * L) * case["kv_heads"]
        rows = S * T * case["heads"]
        if op == "attend":
            return {"bytes": cached * case["dim"] * 4 + rows * (case["dim"] * 4 + 4),
                    "flops": 4 * rows * case["dim"] * (P + L)}
        return {"bytes": cached * (case["dim"] * 2 + 8) + rows * (case["dim"] * 2 + 4),
                "flops": 2 * rows * case["dim"] * (P + L)}
    R, H, L, B = case["requests"], case["mass_heads"], 0.75 * case["longest"], case["budget"]
    B = min(B, L)
    moved = 2 * 2 * B * case["heads"] * case["dim"] * 2
    return {"bytes": R * (H * (L * 4 + B * 8) + moved), "flops": R * H * L}


# --------------------------------------------------------------------------------------------
# the definitions in 64 bits on the host
# --------------------------------------------------------------------------------------------

def exact(case, seed):
    if not torch.cuda.is_available():
        return None
    st = prepare(case, seed)
    if case["op"] == "beams":
        return _exact_beams(case, st)
    if case["op"] in ("attend", "mass"):
        return _exact_attend(case, st)
    return None   # values are moved and chosen: nothing is computed


def _host(t):
    if t is None:
        return None
    return (t.float() if t.is_floating_point() else t).cpu().numpy()


def _exact_beams(case, st):
    if st["logits"].numel() > 40_000_000:
        return None
    R, W, k = case["requests"], case["beams"], case["k"]
    x, scores, ended, lengths = (_host(st[n]) for n in ("logits", "scores", "ended", "lengths"))
    outs = [[], [], []]
    for r in range(R):
        found = []
        for b in range(W):
            s, n = float(scores[r, b]), 1.0
            done = ended is not None and bool(ended[r, b])
            if lengths is not None:
                n = float(int(lengths[r, b]) + (0 if done else 1)) ** case["penalty"]
            if done:
                found.append((s / n, b, 2, s))
                continue
            row = x[r * W + b].astype(np.float64)
            live = np.flatnonzero(row > -np.inf)
            top = row[live].max()
            lse = top + math.log(np.exp(row[live] - top).sum(dtype=np.longdouble))
            # a beam's own best k are all that can be chosen
            for i in live[np.argsort(-row[live], kind="stable")[:k]]:
                found.append(((s + (row[i] - lse)) / n, b, int(i), s + (row[i] - lse)))
        found.sort(key=lambda c: (-c[0], c[1], c[2]))
        found = (found + [(0.0, -1, -1, -math.inf)] * k)[:k]
        outs[0].append([c[3] for c in found])
        outs[1].append([c[1] for c in found])
        outs[2].append([c[2] for c in found])
    return np.array(outs[0]), np.array(outs[1], dtype=np.int32), np.array(outs[2], dtype=np.int32)


def _exact_attend(case, st):
    T, H, D, bs = case["next_n"], case["kv_heads"], case["dim"], case["block_size"]
    per = case["heads"] // H
    q, plens, lens, starts, pt, tab = (_host(st[n]) for n in ("q", "plens", "lens", "starts", "ptables", "tables"))
    # (64-bit operations on the device: the host would take minutes over the long prompts)
    keys, values, qd = st["k"].double(), st["v"].double(), st["q"].double()
    S = lens.size
    mass = case["op"] == "mass"
    out, lse = np.zeros((S * T, H * per, D)), np.full((S * T, H * per), -np.inf)
    if mass:
        pm, own_mass = st["pmass"].double() * 0.99, st["mass"].double() * 0.99
        given = st["lse"].double()
    for g in range(plens.size):
        n = int(plens[g])
        pages = torch.from_numpy(pt[g].astype(np.int64)).to(keys.device)
        pk, pv = keys[pages].reshape(-1, H, D)[:n], values[pages].reshape(-1, H, D)[:n]
        for s in range(int(starts[g]), int(starts[g + 1])):
            m = int(lens[s])
            pages = torch.from_numpy(tab[s].astype(np.int64)).to(keys.device)
            sk, sv = keys[pages].reshape(-1, H, D)[:m], values[pages].reshape(-1, H, D)[:m]
            ks = torch.cat([pk, sk]).transpose(0, 1)                    # [H, n + m, D]
            vs = torch.cat([pv, sv]).transpose(0, 1)
            for t in range(T):
                sees = n + max(0, m - T + t + 1)
                a = torch.bmm(qd[s * T + t].view(H, per, D), ks[:, :sees].transpose(1, 2).contiguous()) / math.sqrt(D)
                if mass:
                    p = torch.exp(a - given[s * T + t].view(H, per, 1)).sum(1)
                    pm[g, :, :n] += p[:, :n]
                    own_mass[s, :, :sees - n] += p[:, n:]
                elif sees:
                    z = torch.logsumexp(a, 2, keepdim=True)
                    out[s * T + t] = torch.bmm(torch.exp(a - z), vs[:, :sees]).reshape(H * per, D).cpu().numpy()
                    lse[s * T + t] = z.view(-1).cpu().numpy()
    return (pm, own_mass) if mass else (out, lse)
