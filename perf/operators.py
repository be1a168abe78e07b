"""What is measured of the row operators beside the top-K: sampling a token, routing to experts
and its gradient, block tables with slot maps, and the slots of selected positions.

Each case is one call of one operator.  With ``own`` false, ``run`` computes it with elementary
torch operations; with ``own`` true it makes the framework's call.  Whole-number choices (tokens,
experts, slots) are made in 64 bits in the plain form: a sum over a hundred thousand weights, and
two scores next to each other at a border, need them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def _sample(rows, vocab, dtype, filters, pad=0, spread=2.0):
    return {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "filters": filters,
            "pad": pad, "spread": spread}


def _route(op, tokens, experts, top_k, dtype, scoring, bias, groups, topk_groups, renorm):
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "dtype": dtype,
            "scoring": scoring, "bias": bias, "groups": groups, "topk_groups": topk_groups,
            "renorm": renorm}


def _tables(requests, new_tokens, longest, block_size):
    return {"op": "tables", "requests": requests, "new": new_tokens, "longest": longest,
            "block_size": block_size}


def _slots(rows, k, longest, block_size, next_n):
    return {"op": "slots", "rows": rows, "k": k, "longest": longest, "block_size": block_size,
            "next_n": next_n}


def listed():
    return [
        # one conversation: a single bf16 row, every filter on; the call's latency is what counts
        {"name": "sample_one_row", **_sample(1, 32768, "bf16", "all")},
        # a decode batch as wide as the varlen workload, each request with its own settings
        {"name": "sample_mixed_batch", **_sample(64, 131072, "fp32", "mixed")},
        # the largest: rollouts at a temperature, the whole vocabulary kept
        {"name": "sample_temperature", **_sample(256, 131072, "fp32", "none")},
        # an odd vocabulary in half precision with padded rows, cut by probability alone
        {"name": "sample_nucleus_odd", **_sample(128, 50001, "fp16", "nucleus", pad=7)},
        # a decode step's router: few tokens, softmax scores, no groups
        {"name": "route_decode", **_route("route", 64, 128, 8, "bf16", "softmax", False, 1, 1, True)},
        # a prompt's router: sigmoid scores, balance bias, 4 groups of 8
        {"name": "route_prompt", **_route("route", 16384, 256, 8, "fp32", "sigmoid", True, 8, 4, True)},
        # its gradient in training
        {"name": "route_grad", **_route("route_grad", 16384, 256, 8, "fp32", "sigmoid", True, 8, 4, True)},
        # the gradient through the whole softmax (weights left as they are), odd token count
        {"name": "route_grad_softmax", **_route("route_grad", 4097, 64, 6, "bf16", "softmax", False, 1, 1, False)},
        # a decode step: one new token for each of 64 requests in mid-flight
        {"name": "tables_decode", **_tables(64, 1, 131072, 64)},
        # a prefill step: 61 whole prompts of different lengths, a million tokens at most
        {"name": "tables_prompt", **_tables(61, 0, 16384, 16)},
        # slots of the decode selection: 64 rows of 2048 positions
        {"name": "slots_decode", **_slots(64, 2048, 131072, 64, 1)},
        # slots of the prefill tile's selection: 4 requests x 1024 rows, 1024 positions each
        {"name": "slots_prompt", **_slots(4096, 1024, 16384, 64, 1024)},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "route", "route_grad", "tables", "slots"])
    dtype = rng.choice(["fp32", "bf16", "fp16"])
    if op == "sample":
        vocab = _log_int(rng, 1000, 200000)
        rows = _log_int(rng, 1, min(512, 256 * 131072 // vocab))
        return _sample(rows, vocab, dtype, rng.choice(["none", "all", "mixed", "nucleus"]),
                       pad=rng.choice([0, 0, 1, 8, 33]), spread=round(rng.uniform(1.0, 3.0), 2))
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        per = _log_int(rng, 4, 512 // groups)
        experts = groups * per
        topk_groups = rng.randint((groups + 1) // 2, groups)
        top_k = rng.randint(1, min(16, topk_groups * per))
        tokens = _log_int(rng, 1, 16384 * 256 // max(experts, 64))
        return _route(op, tokens, experts, top_k, dtype, rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, topk_groups, rng.random() < 0.7)
    if op == "tables":
        requests = _log_int(rng, 1, 1000)
        longest = _log_int(rng, 64, min(131072, (1 << 20) // requests + 64))
        return _tables(requests, rng.choice([0, 1, 2, 3, 4]), longest, rng.choice([1, 16, 32, 48, 64, 128]))
    next_n = rng.choice([1, 1, 2, 3, 4])
    rows = _log_int(rng, 1, 2048)
    return _slots(rows, rng.choice([512, 1024, 2048]), _log_int(rng, 4096, 131072),
                  rng.choice([1, 16, 48, 64, 128]), next_n)


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def prepare(case, seed):
    return _PREPARE[case["op"]](case, seed)


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _prepare_sample(case, seed):
    rows, vocab, dev = case["rows"], case["vocab"], "cuda"
    g = _gen(seed, 11)
    # a bulk of unlikely tokens and some dozens that the context makes likely
    x = torch.randn(rows, vocab + case["pad"], device=dev, generator=g) * case["spread"]
    likely = torch.randint(0, vocab, (rows, 48), device=dev, generator=g)
    x.scatter_add_(1, likely, torch.randn(rows, 48, device=dev, generator=g) * 2 + 6)
    banned = torch.randint(0, vocab, (rows, 16), device=dev, generator=g)
    x.scatter_(1, banned, float("-inf"))
    x = x.to(DTYPES[case["dtype"]])[:, :vocab]
    st = {"case": case, "logits": x, "uniforms": torch.rand(rows, device=dev, generator=g),
          "temperature": torch.rand(rows, device=dev, generator=g) * 0.8 + 0.5,
          "top_k": None, "top_p": None, "min_p": None}
    pick = torch.rand(4, rows, device=dev, generator=g)
    if case["filters"] == "all":
        st["top_k"] = torch.randint(20, 100, (rows,), device=dev, generator=g, dtype=torch.int32)
        st["top_p"] = torch.rand(rows, device=dev, generator=g) * 0.2 + 0.79
        st["min_p"] = torch.rand(rows, device=dev, generator=g) * 0.05
    elif case["filters"] == "nucleus":
        st["top_p"] = torch.rand(rows, device=dev, generator=g) * 0.2 + 0.79
    elif case["filters"] == "mixed":
        # each request its own: greedy, cut by count, by probability, by a share of the best, or not
        st["temperature"] = torch.where(pick[0] < 0.15, 0.0, st["temperature"])
        k = torch.randint(1, 400, (rows,), device=dev, generator=g, dtype=torch.int32)
        st["top_k"] = torch.where(pick[1] < 0.4, k, 0).to(torch.int32)
        st["top_p"] = torch.where(pick[2] < 0.5, torch.rand(rows, device=dev, generator=g) * 0.3 + 0.69, 1.0)
        st["min_p"] = torch.where(pick[3] < 0.3, torch.rand(rows, device=dev, generator=g) * 0.1, 0.0)
    return st


def _prepare_route(case, seed):
    T, E, dev = case["tokens"], case["experts"], "cuda"
    g = _gen(seed, 23)
    x = (torch.randn(T, E, device=dev, generator=g) * 1.5).to(DTYPES[case["dtype"]])
    bias = torch.randn(E, device=dev, generator=g) * 0.05 if case["bias"] else None
    st = {"case": case, "logits": x, "bias": bias}
    if case["op"] == "route_grad":
        st["indices"] = _route_plain(case, x, bias)[0]
        st["grad"] = torch.randn(T, case["top_k"], device=dev, generator=g)
    return st


def _prepare_tables(case, seed):
    R, L, bs, dev = case["requests"], case["longest"], case["block_size"], "cuda"
    g = _gen(seed, 37)
    kv = torch.randint(max(1, L // 16), L + 1, (R,), device=dev, generator=g).to(torch.int32)
    # new = 0 stands for whole prompts: every token of the request is new
    new = kv.clone() if case["new"] == 0 else torch.clamp(kv, max=case["new"]).to(torch.int32)
    width = (L + bs - 1) // bs
    ids = torch.randperm(2 * R * width, device=dev, generator=g).to(torch.int32)
    held = (kv - new + bs - 1) // bs
    tables = ids[:R * width].view(R, width).clone()
    tables[torch.arange(width, device=dev)[None, :] >= held[:, None]] = -1
    # the step's padded capacity: what its buffers were made for
    most = R * (L if case["new"] == 0 else case["new"])
    return {"case": case, "tables": tables, "kv_lens": kv, "new_tokens": new,
            "free_blocks": ids[R * width:].clone(), "max_tokens": most,
            "free_start": torch.randint(0, R + 1, (1,), device=dev, generator=g).to(torch.int32)}


def _prepare_slots(case, seed):
    rows, k, L, bs, dev = case["rows"], case["k"], case["longest"], case["block_size"], "cuda"
    g = _gen(seed, 41)
    R = (rows + case["next_n"] - 1) // case["next_n"]
    width = (L + bs - 1) // bs
    tables = torch.randperm(R * width, device=dev, generator=g).to(torch.int32).view(R, width)
    lens = torch.randint(1, L + 1, (rows, 1), device=dev, generator=g)
    idx = (torch.rand(rows, k, device=dev, generator=g) * lens).to(torch.int32)
    # a row shorter than k holds its positions in order, then -1
    col = torch.arange(k, device=dev, dtype=torch.int32)[None, :]
    idx = torch.where(lens <= k, torch.where(col < lens, col, -1), idx).to(torch.int32)
    return {"case": case, "indices": idx, "tables": tables}


_PREPARE = {"sample": _prepare_sample, "route": _prepare_route, "route_grad": _prepare_route,
            "tables": _prepare_tables, "slots": _prepare_slots}


# --------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _OWN[case["op"]](case, state)
    return _PLAIN[case["op"]](case, state)


def _own_sample(case, st):
    import exact_row_top_amd as ert
    return ert.sample_tokens(st["logits"], st["uniforms"], temperature=st["temperature"],
                             top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"],
                             return_logprobs=True)


def _route_args(case):
    return {"scoring": case["scoring"], "renormalize": case["renorm"], "scale": 2.5}


def _own_route(case, st):
    import exact_row_top_amd as ert
    return ert.route_experts(st["logits"], case["top_k"], bias=st["bias"],
                             num_groups=case["groups"], topk_groups=case["topk_groups"],
                             group_score="top2" if case["bias"] else "max", **_route_args(case))


def _own_route_grad(case, st):
    import exact_row_top_amd as ert
    return ert.route_experts_backward(st["grad"], st["logits"], st["indices"], **_route_args(case))


def _own_tables(case, st):
    import exact_row_top_amd as ert
    starts, requests, positions, slots, free_next = ert.extend_block_tables(
        st["tables"], st["kv_lens"], st["new_tokens"], st["free_blocks"], st["free_start"],
        case["block_size"], st["max_tokens"])
    return st["tables"], starts, requests, positions, slots, free_next


def _own_slots(case, st):
    import exact_row_top_amd as ert
    return ert.topk_slots(st["indices"], st["tables"], case["block_size"], next_n=case["next_n"])


_OWN = {"sample": _own_sample, "route": _own_route, "route_grad": _own_route_grad,
        "tables": _own_tables, "slots": _own_slots}


def _plain_sample(case, st):
    x, u = st["logits"].float(), st["uniforms"].double()[:, None]
    rows, vocab = x.shape
    t = st["temperature"].double()[:, None]
    x = torch.where(torch.isnan(x), float("-inf"), x)
    xs, order = torch.sort(x, dim=1, descending=True, stable=True)
    best = xs[:, :1].double()
    w = torch.exp((xs.double() - best) / torch.where(t > 0, t, 1.0))
    w = torch.where(xs == xs[:, :1], 1.0, w) * (xs > float("-inf"))
    rank = torch.arange(vocab, device=x.device)[None, :]
    keep = torch.ones_like(w, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep &= (rank < k) | (k <= 0)
    if st["top_p"] is not None:
        mass = torch.cumsum(w * keep, 1)
        keep &= (mass - w * keep < st["top_p"].double()[:, None] * mass[:, -1:]) | (rank == 0)
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None].clamp(max=1.0)
    kept = torch.zeros_like(w).scatter_(1, order, w * keep)
    mass = torch.cumsum(kept, 1)
    total = mass[:, -1:]
    token = (mass <= u * total).sum(1, keepdim=True).clamp(max=vocab - 1)
    greedy, empty = ~(t > 0), total == 0
    token = torch.where(greedy, order[:, :1], token)
    logprob = torch.log(kept.gather(1, token) / total)
    logprob = torch.where(empty, float("-inf"), torch.where(greedy, 0.0, logprob))
    return torch.where(empty, -1, token)[:, 0].int(), logprob[:, 0].float()


def _route_scores(case, x):
    x = x.double()
    return torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)


def _route_plain(case, logits, bias):
    s = _route_scores(case, logits)
    c = s + bias.double()[None, :] if bias is not None else logits.double()
    G, T, E = case["groups"], s.shape[0], s.shape[1]
    if G > 1:
        by = c.view(T, G, E // G)
        score = by.sort(dim=2, descending=True)[0][:, :, :2].sum(2) if bias is not None else by.amax(2)
        best = score.sort(dim=1, descending=True, stable=True)[1][:, :case["topk_groups"]]
        on = torch.zeros_like(score).scatter_(1, best, 1.0) > 0
        c = torch.where(on[:, :, None], by, float("-inf")).view(T, E)
    idx = c.sort(dim=1, descending=True, stable=True)[1][:, :case["top_k"]]
    w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.int(), (w * 2.5).float()


def _plain_route(case, st):
    return _route_plain(case, st["logits"], st["bias"])


def _plain_route_grad(case, st):
    x, idx, g = st["logits"].float(), st["indices"].long(), st["grad"] * 2.5
    s = torch.sigmoid(x) if case["scoring"] == "sigmoid" else torch.softmax(x, 1)
    chosen = s.gather(1, idx)
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, idx, g)
    if case["scoring"] == "sigmoid":
        dx = ds * s * (1 - s)
    else:
        dx = s * (ds - (g * chosen).sum(1, keepdim=True))
    return dx.to(st["logits"].dtype)


def _plain_tables(case, st):
    bs, most, tables = case["block_size"], st["max_tokens"], st["tables"]
    kv, new = st["kv_lens"].long(), st["new_tokens"].long()
    old = kv - new
    held, need = (old + bs - 1) // bs, (kv + bs - 1) // bs
    fresh = torch.cumsum(need - held, 0) - (need - held)
    col = torch.arange(tables.shape[1], device=kv.device)[None, :]
    at = st["free_start"].long() + fresh[:, None] + col - held[:, None]
    taken = st["free_blocks"][at.clamp(0, st["free_blocks"].numel() - 1)]
    tables = torch.where((col >= held[:, None]) & (col < need[:, None]), taken, tables)
    starts = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    n = torch.arange(most, device=kv.device)
    req = torch.searchsorted(starts[1:], n, right=True)
    live = req < kv.numel()
    r = req.clamp(max=kv.numel() - 1)
    pos = old[r] + n - starts[r]
    block = tables[r, (pos // bs).clamp(max=tables.shape[1] - 1)]
    slots = torch.where(live, block * bs + pos % bs, -1)
    return (tables, starts.int(), torch.where(live, req, -1).int(), torch.where(live, pos, -1).int(),
            slots.int(), (st["free_start"] + (need - held).sum()).int())


def _plain_slots(case, st):
    idx, bs = st["indices"].long(), case["block_size"]
    req = torch.arange(idx.shape[0], device=idx.device) // case["next_n"]
    block = st["tables"][req[:, None], idx.clamp(min=0) // bs]
    return torch.where(idx >= 0, block * bs + idx % bs, -1).int()


_PLAIN = {"sample": _plain_sample, "route": _plain_route, "route_grad": _plain_route_grad,
          "tables": _plain_tables, "slots": _plain_slots}


# --------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = 4 if case.get("dtype") == "fp32" else 2
    if op == "sample":
        rows, vocab = case["rows"], case["vocab"]
        settings = {"none": 8, "nucleus": 12, "all": 20, "mixed": 20}[case["filters"]]
        return {"bytes": rows * (vocab * size + settings + 8), "flops": 4 * rows * vocab}
    if op in ("route", "route_grad"):
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        if op == "route":
            return {"bytes": T * (E * size + k * 8) + (4 * E if case["bias"] else 0),
                    "flops": 6 * T * E}
        # the gradient through sigmoid or renormalised weights needs the chosen logits alone
        whole = case["scoring"] == "softmax" and not case["renorm"]
        return {"bytes": T * ((E if whole else k) * size + k * 8 + E * size),
                "flops": T * (6 * E if whole else 10 * k)}
    if op == "tables":
        R, L, bs = case["requests"], case["longest"], case["block_size"]
        most = R * (L if case["new"] == 0 else case["new"])
        tokens = R * (L // 16 + L) // 2 if case["new"] == 0 else R * case["new"]
        blocks = max(1, tokens // bs)
        return {"bytes": R * 12 + most * 12 + blocks * 8 + 12, "flops": 4 * tokens}
    # each position read and its slot written once; of the tables what a row's request can hold
    rows, k = case["rows"], case["k"]
    requests = (rows + case["next_n"] - 1) // case["next_n"]
    entries = min(requests * (case["longest"] // case["block_size"]), rows * k)
    return {"bytes": rows * k * 8 + entries * 4, "flops": 3 * rows * k}


# --------------------------------------------------------------------------------------------
# the definitions, row by row in 64 bits or more on the host
# --------------------------------------------------------------------------------------------

def exact(case, seed):
    if not torch.cuda.is_available():
        return None
    st = prepare(case, seed)
    host = {k: (v.float() if v.is_floating_point() else v).cpu().numpy()
            for k, v in st.items() if isinstance(v, torch.Tensor)}
    if case["op"] == "sample":
        return _exact_sample(st, host)
    if case["op"] == "route":
        return _exact_route(case, host)
    if case["op"] == "route_grad":
        return _exact_route_grad(case, host)
    return None   # whole numbers only: nothing is rounded


def _exact_sample(st, h):
    if st["logits"].numel() > 40_000_000:
        return None
    tokens, logprobs = [], []
    for r in range(h["logits"].shape[0]):
        x = h["logits"][r].astype(np.float64)
        live = np.flatnonzero(~np.isnan(x) & (x > -np.inf))
        if live.size == 0:
            tokens.append(-1), logprobs.append(-np.inf)
            continue
        temp = float(h["temperature"][r])
        if not temp > 0:
            tokens.append(int(np.argmax(np.where(np.isnan(x), -np.inf, x)))), logprobs.append(0.0)
            continue
        # weights by falling logit; nothing behind the kept prefix is looked at again
        ranked = live[np.argsort(-x[live], kind="stable")]
        w = np.exp((x[ranked].astype(np.longdouble) - x[ranked[0]]) / np.longdouble(temp))
        k = int(h["top_k"][r]) if "top_k" in h else 0
        if 0 < k < w.size:
            w = w[:k]
        if "top_p" in h:
            csum = np.cumsum(w)
            w = w[:1 + int(np.count_nonzero(csum[:-1] < np.longdouble(h["top_p"][r]) * csum[-1]))]
        if "min_p" in h:
            w = w[w >= min(1.0, float(h["min_p"][r]))]
        kept = ranked[:w.size]
        place = np.argsort(kept)
        csum = np.cumsum(w[place])
        at = int(np.searchsorted(csum, np.longdouble(h["uniforms"][r]) * csum[-1], side="right"))
        at = min(at, w.size - 1)
        tokens.append(int(kept[place[at]]))
        logprobs.append(float(np.log(w[place[at]] / csum[-1])))
    return (np.array(tokens, dtype=np.int32), np.array(logprobs))


def _exact_scores(case, x):
    x = x.astype(np.float64)
    if case["scoring"] == "sigmoid":
        return 1.0 / (1.0 + np.exp(-x))
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def _exact_route(case, h):
    s = _exact_scores(case, h["logits"])
    rank_by = s + h["bias"].astype(np.float64) if "bias" in h else h["logits"].astype(np.float64)
    T, E = s.shape
    G = case["groups"]
    if G > 1:
        top = -np.sort(-rank_by.reshape(T, G, E // G), axis=2)
        score = top[:, :, :2].sum(2) if "bias" in h else top[:, :, 0]
        place = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1)
        rank_by = np.where(np.repeat(place < case["topk_groups"], E // G, axis=1), rank_by, -np.inf)
    idx = np.argsort(-rank_by, axis=1, kind="stable")[:, :case["top_k"]]
    w = np.take_along_axis(s, idx, 1)
    if case["renorm"]:
        w = w / w.sum(1, keepdims=True)
    return idx.astype(np.int32), 2.5 * w


def _exact_route_grad(case, h):
    # d weights_j / d logits_e, summed against the given gradient, from the quotient's own derivative
    s, idx, g = _exact_scores(case, h["logits"]), h["indices"], h["grad"].astype(np.float64)
    rows = np.arange(s.shape[0])[:, None]
    c = s[rows, idx]
    up = 2.5 * g
    if case["renorm"]:
        z = c.sum(1, keepdims=True)
        up = up / z - (2.5 * g * c / z ** 2).sum(1, keepdims=True)
    out = np.zeros_like(s)
    if case["scoring"] == "sigmoid":
        out[rows, idx] = up * c * (1 - c)
        return out
    # softmax: s_e (delta_ej - s_j)
    out = -s * (up * c).sum(1, keepdims=True)
    out[rows, idx] += up * c
    return out
