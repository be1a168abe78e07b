"""A beam search's operators where their other tests do not reach: group starts
that fall in part, bounds of zero, bounds that cut, scores of any size, small
weights in float16, more rows than a tile holds, long rows, refusals that leave
everything as it was, and the documented loop over several steps."""
import numpy as np
import pytest

from gpu_helpers import log
from test_search_ops_gpu import (HALF, NINF, Case, _check_attend, _check_beams, _check_evict, _check_mass, _cuda, _dt,
                                 ert)  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# group starts that fall in part: groups that overlap
# ---------------------------------------------------------------------------

FALLS = [([2, 2, 2], [0, 6, 2, 6]), ([2, 2, 2], [0, 4, 1, 6]), ([40, 30, 40], [0, 110, 2, 110]),
         ([1, 0, 2, 1], [0, 3, 2, 2, 4])]


@pytest.mark.parametrize("members,starts", FALLS)
@pytest.mark.parametrize("room", [0, 1 << 21])
def test_attention_leaves_out_prefixes_of_overlapping_groups(ert, members, starts, room):
    c = Case("bf16", 64, 16, members, 200, 50, 8, 2, plens=[200, 150, 100, 50][:len(members)])
    c.starts = np.array(starts, dtype=np.int32)
    c.group = lambda s: None
    _check_attend(ert, c, f"starts {starts} room {room}", room=room)


@pytest.mark.parametrize("members,starts", FALLS)
def test_mass_leaves_out_prefixes_of_overlapping_groups(ert, members, starts):
    c = Case("bf16", 64, 16, members, 200, 50, 8, 2, plens=[200, 150, 100, 50][:len(members)])
    c.starts = np.array(starts, dtype=np.int32)
    c.group = lambda s: None
    _check_mass(ert, c, f"starts {starts}")


def test_mass_of_more_groups_than_a_wave_with_starts_that_fall_late(ert):
    members = [1] * 150
    c = Case("fp16", 64, 16, members, 40, 20, 4, 2)
    _check_mass(ert, c, "150 groups")
    c.starts[140:] = 130
    c.group = lambda s: None
    _check_mass(ert, c, "150 groups, falling at the 140th")


@pytest.mark.parametrize("groups", [1, 2, 3, 5, 63, 64, 65, 66, 200, 768, 769, 2300])
def test_mass_finds_a_fall_wherever_it_is(ert, groups):
    import torch
    g = torch.Generator(device="cuda").manual_seed(groups)
    q = torch.randn(groups, 2, 64, device="cuda", generator=g).half()
    k = torch.randn(groups + 1, 16, 1, 64, device="cuda", generator=g).half()
    pt = torch.arange(groups, device="cuda", dtype=torch.int32).view(-1, 1)
    pl = torch.full((groups,), 16, dtype=torch.int32, device="cuda")
    tab, lens = torch.full((groups, 1), groups, dtype=torch.int32, device="cuda"), torch.zeros(groups, dtype=torch.int32, device="cuda")
    lse, mass = torch.full((groups, 2), 3.0, device="cuda"), torch.rand(groups, 1, 700, device="cuda", generator=g)

    def run(starts):
        return ert.attention_mass(q, k, lse, pt, pl, tab, lens, group_starts=_cuda(starts), prefix_mass=mass, decay=0.5)[0]

    log(f"[mass] {groups} groups, a fall at each of some places")
    rising = np.arange(groups + 1, dtype=np.int32)
    seen = run(rising)
    assert torch.equal(seen[:, :, 16:], mass[:, :, 16:] * 0.5) and bool((seen[:, :, :16] > mass[:, :, :16] * 0.5).all())
    for at in {0, 1, 14, 15, 30, 31, 61, 62, 63, 64, 125, 126, 250, 251, 252, 253, 254, 190, 191, 192, 193, 766, 767, 768, groups // 2, groups - 5, groups - 4, groups - 3, groups - 2, groups - 1}:
        if 0 <= at < groups:
            starts = rising.copy()
            starts[at], starts[at + 1] = starts[at + 1], starts[at]
            assert torch.equal(run(starts), mass * 0.5), at


# ---------------------------------------------------------------------------
# bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("limit,own", [(0, None), (None, 0), (0, 0), (0, 31), (100, 0), (1, 1)])
def test_attention_bounds_of_zero(ert, limit, own):
    c = Case("bf16", 64, 16, [3, 2], 333, 77, 8, 2, next_n=2)
    _check_attend(ert, c, f"limits {limit} {own}", limit=limit, own=own)


@pytest.mark.parametrize("limit,own", [(None, None), (100, None), (None, 31), (100, 31), (0, 31), (100, 0), (0, 0), (5000, 5000)])
def test_mass_within_the_bounds_of_its_attention(ert, limit, own):
    import torch
    c = Case("fp16", 64, 16, [3, 2], 333, 77, 8, 2, next_n=2, plens=[333, 90], lens=[77, 20, 33, 0, 60])
    pt, pl, tab, lens = c.dev()
    starts = _cuda(c.starts)
    log(f"[mass] bounds {limit} {own}")
    kw = dict(next_n=2, group_starts=starts)
    bounds = dict(max_prefix_len=limit, max_len=own)
    out, lse = ert.prefix_attention(c.q, c.k, c.v, pt, pl, tab, lens, return_lse=True, **kw, **bounds)
    got = ert.attention_mass(c.q, c.k, lse, pt, pl, tab, lens, **kw, **bounds)
    cut = [x if b is None else x.clamp(max=b) for x, b in ((pl, limit), (lens, own))]
    want = ert.attention_mass(c.q, c.k, lse, pt, cut[0], tab, cut[1], **kw)
    assert all(a.shape == b.shape and torch.equal(a, b) for a, b in zip(got, want))
    # a token's weights sum to one: 64 bits over what the call wrote, heads of a key head together
    rows = (lse > NINF).sum().item()
    # (each weight to 2^-11 by its log-sum and score, sums in 32 bits)
    assert abs(sum(float(m.double().sum()) for m in got) - rows) <= 2.0 ** -10 * max(rows, 1)


# ---------------------------------------------------------------------------
# scores of any size, small weights
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,scale", [("fp16", 1.0), ("fp16", 64.0), ("bf16", 1.0), ("bf16", 2.0 ** 10)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("room", [0, 1 << 21])
def test_attention_to_one_of_far_scores(ert, dtype, scale, sign, room):
    """Scores whose last bits weigh more than their gaps' exponents: products are
    exact, gaps are far, so all weight is the largest score's."""
    import torch
    rng = np.random.default_rng([3, sign + 1, room])
    D, bs, G, W, H = 64, 16, 2, 140 if room else 5, 2
    P, L = 320, 64
    N = G * P // bs + G * W * L // bs
    k, q = torch.zeros(N, bs, H, D, device="cuda"), torch.zeros(G * W, H, D, device="cuda")
    # whole numbers of eight bits times a power of two: exact in both types, all of a row's distinct
    v = torch.randn(N, bs, H, D, device="cuda").to(_dt(dtype))
    pt = np.arange(G * P // bs, dtype=np.int32).reshape(G, -1)
    tab = (np.arange(G * W * L // bs, dtype=np.int32) + G * P // bs).reshape(G * W, -1)
    q[:, :, 0] = 1.375 * 2.0 ** 14
    q[:, 1, 0] = 1.625 * 2.0 ** 14
    kn = np.zeros((N, bs))
    for g in range(G):
        kn[pt[g]] = sign * rng.integers(1, 200, (P // bs, bs))
    for s in range(G * W):
        kn[tab[s]] = sign * rng.integers(1, 200, (L // bs, bs))
    # one key of each sequence, or of its prefix, beyond all others
    best = 250.0 if sign > 0 else 0.25
    want = torch.zeros(G * W, H, D, dtype=torch.float64, device="cuda")
    for s in range(G * W):
        g = s // W
        if g == 0:      # in the prefix, the same for the group
            b, o = pt[0, 7], 5
        else:
            b, o = tab[s, s % (L // bs)], (3 * s) % bs
        kn[b, o] = sign * best
        want[s] = v[b, o].double()
    k[:, :, :, 0] = torch.from_numpy(kn).cuda().float()[:, :, None] * 128.0
    k, q = k.to(_dt(dtype)), q.to(_dt(dtype))
    log(f"[attend] far scores {dtype} scale={scale} sign={sign} room={room}")
    tables = torch.nn.functional.pad(_cuda(pt), (0, room // bs), value=-1)
    out, lse = ert.prefix_attention(q, k, v, tables, _cuda(np.full(G, P, np.int32)), _cuda(tab),
                                    _cuda(np.full(G * W, L, np.int32)), scale=scale, return_lse=True)
    # one weight: the value times a power of two and back, rounded once
    assert bool(((out.double() - want).abs() <= HALF[dtype] * want.abs()).all())
    z = scale * q[:, :, 0].double() * sign * best * 128.0
    assert bool(((lse.double() - z).abs() <= 2.0 ** -22 * z.abs()).all())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attention_to_scores_a_step_of_their_type_apart(ert, dtype):
    """Scores of 1.5 * 2^27, whose neighbours lie 16 apart: a later tile's weigh
    2^16 times the first ones', just beyond what float16 holds."""
    import torch
    D, bs, n, S = 64, 32, 320, 2048   # (so many that a wave takes all of a row)
    k, v = torch.zeros(n // bs, bs, 1, D, device="cuda"), torch.zeros(n // bs, bs, 1, D, device="cuda")
    q = torch.zeros(S, 1, D, device="cuda")
    q[:, 0, 0], q[:, 0, 1] = 1.5 * 2.0 ** 12, 4.0
    k[..., 0] = 2.0 ** 15
    k[4, :, 0, 1], v[4] = 4.0, 1.0
    tab = torch.arange(n // bs, dtype=torch.int32, device="cuda").expand(S, n // bs).contiguous()
    lens = _cuda(np.array([n, 160] * (S // 2), np.int32))
    q, k, v = (x.to(_dt(dtype)) for x in (q, k, v))
    log(f"[attend] scores 16 apart {dtype}")
    out, lse = ert.prefix_attention(q, k, v, None, None, tab, lens, scale=float(np.log(2)), return_lse=True)
    top = 2.0 ** 16 * 32
    for s, others in ((0, n - 32), (1, 128)):
        # weights and out rounded to the type
        assert float((out[s].double() - top / (top + others)).abs().max()) <= 2 * HALF[dtype]
        z = np.log(2) * (1.5 * 2.0 ** 27 + 16) + np.log(32 + others / 2.0 ** 16)
        assert abs(float(lse[s, 0]) - z) <= 2.0 ** -22 * z


def test_attention_float16_keeps_the_weights_of_a_long_tail(ert):
    """One key of weight 1 and 2^17 - 1 of 2^-25.5, which together are a 362nd of
    the row, one wave over all of them."""
    import torch
    S, H, D, bs, n = 1024, 2, 64, 64, 1 << 17
    blocks = n // bs
    k = torch.zeros(blocks, bs, H, D, dtype=torch.float16, device="cuda")
    v = torch.ones_like(k)
    k[0, 0, :, 0], v[0, 0] = 17.6875, 0.0
    q = torch.zeros(S, H, D, dtype=torch.float16, device="cuda")
    q[:, :, 0] = 1.0
    tab = torch.arange(blocks, dtype=torch.int32, device="cuda").expand(S, blocks).contiguous()
    lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
    log("[attend] a tail of small weights")
    out = ert.prefix_attention(q, k, v, None, None, tab, lens, scale=1.0).double()
    tail = (n - 1) * np.exp(-17.6875)
    want = tail / (1 + tail)
    # each weight to half a step of float16's smallest, 2^-25, where the largest weighs 2^7 at least; the
    # additions in 32 bits; out's own rounding
    off = n * 2.0 ** -32 + want * (n * 2.0 ** -24 + 2.0 ** -11 + 2.0 ** -20)
    assert float((out - want).abs().max()) <= off < want / 4


# ---------------------------------------------------------------------------
# more query rows of a key head than a tile, long rows, crowded rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim,bs", [("bf16", 64, 16), ("fp16", 64, 7), ("bf16", 128, 7), ("fp16", 128, 64)])
def test_more_own_query_rows_than_a_tile(ert, dtype, dim, bs):
    for n, (members, prefix, suffix, heads, kv, next_n) in enumerate([
            ([2], 100, 90, 8, 1, 5), ([1, 2], 70, 130, 4, 2, 33), ([1], 40, 300, 2, 1, 65), ([], 0, 80, 6, 2, 32)]):
        c = Case(dtype, dim, bs, members, prefix, suffix, heads, kv, next_n, seed=n, outside=0 if members else 1)
        what = f"{dtype} dim={dim} bs={bs} members={members} heads={heads}/{kv} next_n={next_n}"
        _check_attend(ert, c, what)
        _check_mass(ert, c, what, seed=n)


@pytest.mark.parametrize("positions", [8192, 8193, 32768, 32769, 70001])
def test_evict_rows_held_in_registers_and_longer(ert, positions):
    rng = np.random.default_rng(positions)
    R, H = 4, 2
    lens = np.array([positions, positions - 1, 33000, positions + 9], dtype=np.int32)
    special = rng.choice([np.nan, np.inf, -np.inf, -0.0, 1e-42], (R, H, positions))
    kinds = {"normal": rng.normal(0, 1, (R, H, positions)), "zeros": np.zeros((R, H, positions)),
             "few": rng.integers(0, 3, (R, H, positions)).astype(float),
             "half": np.where(rng.random((R, H, positions)) < 0.5, 0.0, np.exp(rng.normal(0, 9, (R, H, positions)))),
             "masked": np.where(rng.random((R, H, positions)) < 0.3, special, rng.normal(0, 1, (R, H, positions))),
             "nan": np.full((R, H, positions), np.nan)}
    for name, m in kinds.items():
        mass = _cuda(m.astype(np.float32))
        for budget, sinks, recent in ((1, 0, 0), (1000, 4, 64), (1000, 400, 600), (positions // 2, 0, 7), (positions - 1, 3, 0)):
            _check_evict(ert, mass, lens, budget, sinks, recent,
                         f"{name} positions={positions} budget={budget} sinks={sinks} recent={recent}")


@pytest.mark.parametrize("vocab", [131073, 262145, 1 << 20])
def test_beams_of_crowded_rows_with_several_pieces_a_thread(ert, vocab):
    rng = np.random.default_rng(vocab)
    rows = [np.zeros(vocab), np.where(rng.random(vocab) < 0.5, 1.0, -1.0), np.where(rng.random(vocab) < 0.999, NINF, 2.0),
            rng.integers(-3, 3, vocab).astype(float), np.sort(rng.normal(0, 1, vocab)),
            np.where(np.arange(vocab) < vocab - 70, 0.5, 0.5 + (np.arange(vocab) % 3) * 0.25)]
    x = _cuda(np.array(rows, dtype=np.float32))
    for k in (1, 7, 64):
        for r in range(len(rows)):
            _check_beams(ert, x[r:r + 1], np.array([[-1.5]]), k, f"vocab={vocab} row {r} alone k={k}")
        _check_beams(ert, x, rng.uniform(-9, -1, (2, 3)), k, f"vocab={vocab} together k={k}")


# ---------------------------------------------------------------------------
# refusals, and the loop
# ---------------------------------------------------------------------------

def test_evict_refuses_caches_before_anything_is_written(ert):
    import torch
    def half(*shape):
        return torch.zeros(*shape, dtype=torch.float16, device="cuda")
    mass, lens = torch.rand(2, 1, 64, device="cuda"), torch.tensor([64, 20], dtype=torch.int32, device="cuda")
    tab = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    c, n = half(12, 16, 2, 8), 12 * 16 * 2 * 8
    odd, wide = half(n + 4)[4:].view(12, 16, 2, 8), half(n + 64)
    calls = {"the same cache twice": dict(caches=[c, c]), "a cache not at 16 bytes": dict(caches=[c, odd]),
             "caches that overlap": dict(caches=[wide[:n].view(12, 16, 2, 8), wide[64:].view(12, 16, 2, 8)]),
             "more caches than a call takes": dict(caches=[half(1, 16, 2, 8) for _ in range(65)]),
             "blocks too long": dict(caches=[half(1, (1 << 20) + 1, 1, 8)]),
             "tables of two strides at one place": dict(caches=[c], out_tables=tab.as_strided((2, 2), (2, 1)))}
    for what, kw in calls.items():
        log(f"[evict] refuses {what}")
        out = torch.full((2, 1, 8), 9.0, device="cuda")
        with pytest.raises((ValueError, RuntimeError)):
            ert.evict_cache(mass, lens, 8, block_tables=tab, mass_out=out, **kw)
        assert bool((out == 9).all()), what


def test_documented_loop_over_several_steps(ert):
    """The step that the documentation shows, as often as a search takes it:
    mass, ends and tables follow the beams, the prompt's cache and its mass are
    cut together.  Against a search without paging that masks what was evicted."""
    import torch
    R, W, bs, H, per, D, V, steps, sinks, recent, eos = 2, 3, 4, 2, 2, 64, 301, 9, 2, 3, 5
    g = torch.Generator(device="cuda").manual_seed(21)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    wq, wk, wv = rnd(V, H * per, D).bfloat16(), rnd(V, H, D).bfloat16(), rnd(V, H, D).bfloat16()
    proj = rnd(H * per * D, V) * 0.5
    prompt = torch.randint(0, V, (R, 23), device="cuda", generator=g)
    N = R * 6 + R * W * 4
    k_cache, v_cache = (torch.zeros(N, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    prompt_tables = torch.arange(R * 6, device="cuda", dtype=torch.int32).view(R, 6)
    for r in range(R):
        at = prompt_tables[r].long().repeat_interleave(bs)[:23], (torch.arange(23, device="cuda") % bs)
        k_cache[at], v_cache[at] = wk[prompt[r]], wv[prompt[r]]
    prompt_lens = torch.tensor([23, 17], dtype=torch.int32, device="cuda")
    tables = torch.full((R * W, 4), -1, dtype=torch.int32, device="cuda")
    free, taken = torch.arange(R * 6, N, device="cuda", dtype=torch.int32), torch.zeros(1, dtype=torch.int32, device="cuda")
    scores = torch.tensor([[0.0] + [NINF] * (W - 1)] * R, device="cuda")
    ended = torch.zeros(R, W, dtype=torch.bool, device="cuda")
    tokens = torch.zeros(R, W, dtype=torch.int32, device="cuda")
    history = torch.zeros(R * W, steps, dtype=torch.int32, device="cuda")
    prompt_mass = mass = None
    # the same search kept apart: which prompt positions are left for each head, and the masses by position
    left = [[np.arange(int(n)) for _ in range(H)] for n in prompt_lens.tolist()]
    p_mass, o_mass = np.zeros((R, H, 23)), np.zeros((R * W, H, steps))
    k64, v64, q64 = (x.double().cpu().numpy() for x in (wk, wv, wq))
    host_prompt = prompt.cpu().numpy()
    for step in range(steps):
        lens = torch.full((R * W,), step + 1, dtype=torch.int32, device="cuda")
        _, _, _, slots, taken = ert.extend_block_tables(tables, lens, torch.ones_like(lens), free, taken, bs, R * W)
        history[:, step] = tokens.view(-1)
        last = tokens.view(-1).long()
        k_cache.view(-1, H, D)[slots.long()], v_cache.view(-1, H, D)[slots.long()] = wk[last], wv[last]
        q = wq[last]
        out, lse = ert.prefix_attention(q, k_cache, v_cache, prompt_tables, prompt_lens, tables, lens, return_lse=True)
        prompt_mass, mass = ert.attention_mass(q, k_cache, lse, prompt_tables, prompt_lens, tables, lens,
                                               prefix_mass=prompt_mass, mass=mass, decay=0.99)
        # what it has to be
        hist = history.cpu().numpy()
        p_mass, o_mass = p_mass * np.float32(0.99), o_mass * np.float32(0.99)
        for s in range(R * W):
            r = s // W
            for h in range(H):
                seen, own = host_prompt[r][left[r][h]], hist[s, :step + 1]
                ks = np.concatenate([k64[seen, h], k64[own, h]])
                vs = np.concatenate([v64[seen, h], v64[own, h]])
                for i in range(per):
                    a = ks @ q64[hist[s, step], h * per + i] * D ** -0.5
                    w = np.exp(a - a.max())
                    w /= w.sum()
                    p_mass[r, h, left[r][h]] += w[:seen.size]
                    o_mass[s, h, :step + 1] += w[seen.size:]
                    want, spread = w @ vs, w @ np.abs(vs)
                    # weights and result rounded to bfloat16 (2^-8 each), the rest in 32 bits
                    assert (np.abs(out[s, h * per + i].double().cpu().numpy() - want) <= 2.0 ** -7 * 1.05 * spread + 1e-5).all()
        # (32-bit scores: 72 roundings of sums of products of about 8, 2^-14.8, in the weight and in its log-sum)
        for r in range(R):
            for h in range(H):
                m = prompt_mass[r, h, :left[r][h].size].double().cpu().numpy()
                assert (np.abs(m - p_mass[r, h, left[r][h]]) <= 2.0 ** -13 * p_mass[r, h, left[r][h]] + 1e-9).all(), (step, r, h)
        m = mass[:, :, :step + 1].double().cpu().numpy()
        assert (np.abs(m - o_mass[:, :, :step + 1]) <= 2.0 ** -13 * o_mass[:, :, :step + 1] + 1e-9).all(), step
        logits = out.float().view(R * W, -1) @ proj
        scores, parents, tokens = ert.select_beams(logits, scores, W, ended=ended, end_token=eos)
        ended = ended.gather(1, parents.long().clamp(min=0)) | (tokens == eos)
        history, mass = ert.reorder_beams([history, mass], parents)
        tables = ert.reorder_block_tables(tables, lens.view(R, W)[:, 0].contiguous(), parents, bs,
                                          caches=[k_cache, v_cache], out=tables)
        src = (parents.cpu().numpy() + np.arange(R)[:, None] * W).reshape(-1)
        assert (parents >= 0).all()
        o_mass = o_mass[src]
        n, budget = prompt_lens.tolist(), 14 - 3 * (step // 3)
        kept, prompt_mass, prompt_lens = ert.evict_cache(prompt_mass, prompt_lens, budget, sinks=sinks, recent=recent,
                                                         block_tables=prompt_tables, caches=[k_cache, v_cache])
        for r in range(R):
            for h in range(H):
                # (masses next to each other at the border may come in either order: what the call kept stands,
                # and is what its own mass says)
                stay = kept[r, h].cpu().numpy()
                stay = stay[stay >= 0]
                assert stay.size == min(n[r], budget) and set(range(min(sinks, n[r]))) <= set(stay.tolist())
                left[r][h] = left[r][h][stay]
