"""A beam search's operators on the GPU against their definitions in 64 bits:
the beams' choice, reordering of states and block tables, attention with a
shared prefix, attention mass and eviction; alone, on other streams, in
captured graphs, and together as a search uses them."""
import itertools

import numpy as np
import pytest

import search_reference as ref
from gpu_helpers import log

pytestmark = pytest.mark.gpu

NINF, INF, NAN = float("-inf"), float("inf"), float("nan")
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SMALL = {"bf16": 0.0, "fp16": 2.0 ** -25}


@pytest.fixture(scope="module")
def ert():
    import torch
    import exact_row_top_amd as m
    assert torch.cuda.is_available()
    m.load_library()
    return m


def _dt(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _cuda(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


# ---------------------------------------------------------------------------
# the beams' choice
# ---------------------------------------------------------------------------

def _check_beams(ert, x, scores, k, what, ended=None, lengths=None, penalty=0.0, end_token=0):
    """Beams and tokens equal the definition's, totals to one fp32 rounding
    beside the sum's own 1e-11."""
    import torch
    log(f"[beams] {what}")
    R, W = scores.shape
    host = x.float().cpu().numpy()
    got = ert.select_beams(x, _cuda(scores.astype(np.float32)), k,
                           ended=None if ended is None else _cuda(ended), end_token=end_token,
                           lengths=None if lengths is None else _cuda(lengths.astype(np.int32)),
                           length_penalty=penalty)
    torch.cuda.synchronize()
    total, parent, token = [t.cpu().numpy() for t in got]
    assert total.shape == parent.shape == token.shape == (R, k)
    for r in range(R):
        want = ref.beams(host[r * W:(r + 1) * W], scores[r].astype(np.float32), k,
                         None if ended is None else ended[r], end_token,
                         None if lengths is None else lengths[r], np.float32(penalty))
        assert list(zip(parent[r], token[r])) == list(zip(want[1], want[2])), (what, r)
        for a, b in zip(total[r], want[0]):
            assert a == b or abs(float(a) - b) <= 2.0 ** -24 * abs(b) * 1.001 + 1e-11, (what, r, a, b)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 64, 1000, 2047, 2048, 2049, 6150, 40001])
def test_beam_sizes(ert, dtype, vocab):
    rng = np.random.default_rng([vocab, 3])
    for R, W, k in ((1, 1, 1), (3, 4, 8), (2, 5, 10), (2, 3, 64)):
        x = _cuda(rng.normal(0, 2.5, (R * W, vocab)).astype(np.float32), _dt(dtype))
        _check_beams(ert, x, rng.uniform(-9, -1, (R, W)), k, f"{dtype} vocab={vocab} {R}x{W} k={k}")


@pytest.mark.parametrize("vocab,R,W,k", [(131072, 2, 8, 16), (200003, 1, 3, 64), (1 << 20, 1, 2, 64),
                                         (5000, 3, 32, 64), (5000, 70, 2, 3)])
def test_beam_ranges(ert, vocab, R, W, k):
    rng = np.random.default_rng([vocab, R])
    for spread in (0.1, 3.0):
        x = _cuda(rng.normal(0, spread, (R * W, vocab)).astype(np.float32))
        _check_beams(ert, x, rng.uniform(-9, -1, (R, W)), k, f"vocab={vocab} {R}x{W} k={k} spread={spread}")


def test_beam_ended_lengths_and_dead_beams(ert):
    rng = np.random.default_rng(5)
    R, W, V = 6, 5, 3001
    x = _cuda(rng.normal(0, 3, (R * W, V)).astype(np.float32))
    ended = rng.random((R, W)) < 0.4
    ended[0] = True
    lengths = rng.integers(-3, 50, (R, W))
    scores = rng.uniform(-40, -1, (R, W))
    scores[1, 2:] = NINF
    scores[2] = NINF
    scores[3, 0], scores[3, 1] = INF, NAN
    for penalty in (0.0, 0.7, 1.0, -0.5):
        for e, n in ((None, None), (ended, None), (None, lengths), (ended, lengths)):
            for k in (1, 5, 10):
                _check_beams(ert, x, scores, k, f"penalty={penalty} ended={e is not None} k={k}", ended=e,
                             lengths=n, penalty=penalty, end_token=7)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_beam_scores_far_from_zero(ert, dtype):
    rng = np.random.default_rng(8)
    R, W, V = 2, 4, 5003
    for at in (300.0, 6e4, 2.0 ** 20 - 3, 2.0 ** 20 + 3, 3e7, 1e12, 1e17, 1e30, 3e38):
        if dtype == "fp16" and at > 6e4:
            continue
        for sign in (1.0, -1.0):
            row = sign * at + rng.normal(0, 2, (R * W, V))
            row[:, ::7] -= rng.exponential(1.0, (R * W, (V + 6) // 7)) * at * 0.1
            row[:, 5], row[:, 6] = NINF, NAN
            x = _cuda(np.clip(row, -3.38e38, 3.38e38).astype(np.float32), _dt(dtype))
            _check_beams(ert, x, rng.uniform(-9, -1, (R, W)), 6, f"{dtype} around {sign * at}")


def test_beam_first_step(ert):
    # all beams hold the same row; only the first has a score
    rng = np.random.default_rng(6)
    row = rng.normal(0, 2, (1, 5001)).astype(np.float32)
    x = _cuda(np.repeat(row, 4, 0))
    _check_beams(ert, x, np.array([[0.0, NINF, NINF, NINF]]), 4, "first step")


@pytest.mark.parametrize("dtype,offset,stride", [("fp32", 1, 5003), ("bf16", 3, 5007), ("fp16", 7, 5001)])
def test_beam_equal_rows_tie_whatever_their_alignment(ert, dtype, offset, stride):
    import torch
    rng = np.random.default_rng([offset, stride])
    W, V = 5, 5001
    buf = torch.full((W * stride + 64,), INF, device="cuda", dtype=_dt(dtype))
    buf[::3] = NAN
    x = buf.as_strided((W, V), (stride, 1), offset)
    x.copy_(_cuda(np.repeat(rng.normal(0, 2, (1, V)).astype(np.float32), W, 0), _dt(dtype)))
    got = ert.select_beams(x, _cuda(np.full((1, W), -3.25, np.float32)), 10)
    parent, token = got[1].cpu().numpy()[0], got[2].cpu().numpy()[0]
    # the best token from every beam in turn, then the second best
    host = x[0].float().cpu().numpy()
    order = np.argsort(-host, kind="stable")
    if host[order[0]] > host[order[1]]:
        assert list(parent[:5]) == [0, 1, 2, 3, 4] and set(token[:5]) == {order[0]}
    x.copy_(_cuda(rng.normal(0, 2, (W, V)).astype(np.float32), _dt(dtype)))
    _check_beams(ert, x, rng.uniform(-9, -1, (1, W)), 10, f"{dtype} poisoned neighbours")


@pytest.mark.parametrize("dtype", ["fp32", "fp16"])
def test_beam_ties_and_masked_scores(ert, dtype):
    rng = np.random.default_rng(8)
    V = 9000
    rows = [np.zeros(V), np.full(V, -3.5), np.where(rng.random(V) < 0.5, 1.0, -1.0),
            rng.integers(-3, 3, V).astype(float), np.sort(rng.normal(0, 1, V)), -np.sort(rng.normal(0, 1, V)),
            np.where(rng.random(V) < 0.99, NINF, rng.normal(0, 1, V)), np.full(V, NINF), np.full(V, NAN),
            np.where(rng.random(V) < 0.3, NAN, rng.normal(0, 1, V)),
            np.where(rng.random(V) < 0.01, INF, rng.normal(0, 1, V)), np.full(V, INF),
            np.where(np.arange(V) == V - 1, 60000.0, -60000.0)]
    x = _cuda(np.array(rows, dtype=np.float32), _dt(dtype))
    for k in (1, 7, 64):
        for r in range(len(rows)):
            _check_beams(ert, x[r:r + 1], np.array([[-1.5]]), k, f"{dtype} row {r} alone k={k}")
        # rows whose sums are far apart together
        _check_beams(ert, x[[0, 3, 4, 7, 8, 10]].contiguous(), rng.uniform(-9, -1, (1, 6)), k,
                     f"{dtype} together k={k}")


def test_beam_rows_beyond_32_bit_offsets(ert):
    import torch
    stride = (1 << 27) + 5
    buf = torch.zeros(19 * stride, dtype=torch.float16, device="cuda")
    x = buf.as_strided((18, 4001), (stride, 1))
    rng = np.random.default_rng(9)
    x.copy_(_cuda(rng.normal(0, 2, (18, 4001)).astype(np.float32), torch.float16))
    _check_beams(ert, x, rng.uniform(-9, -1, (9, 2)), 4, "far rows")


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------

def _parents(rng, R, k, W, lost=0.0):
    p = rng.integers(0, W, (R, k)).astype(np.int32)
    p[rng.random((R, k)) < lost] = -1
    return p


@pytest.mark.parametrize("R,W", [(1, 1), (3, 4), (2, 8), (2, 9), (1, 32)])
def test_reorder_rows(ert, R, W):
    import torch
    rng = np.random.default_rng([R, W])
    shapes = [(1,), (3,), (5, 7), (16,), (1000,), (4097,), (2, 3, 1031)]
    types = [torch.int32, torch.float16, torch.uint8, torch.int64, torch.float32, torch.bool, torch.bfloat16]
    states = [torch.randint(0, 2, (R * W, *s), device="cuda").to(t) if t == torch.bool else
              torch.randint(0, 120, (R * W, *s), device="cuda").to(t) for s, t in itertools.product(shapes, types)]
    p = _parents(rng, R, W, W, 0.2)
    src = (np.arange(R)[:, None] * W + p).reshape(-1)
    lost = _cuda(p.reshape(-1) < 0)
    idx = _cuda(np.where(p.reshape(-1) < 0, 0, src))
    log(f"[reorder] {R}x{W}: {len(states)} states")
    got = ert.reorder_beams(states, _cuda(p))
    for s, g in zip(states, got):
        keep = lost.view(-1, *[1] * (s.dim() - 1))
        assert torch.equal(g, torch.where(keep, torch.zeros_like(s), s[idx]))
    want = [torch.where(lost.view(-1, *[1] * (s.dim() - 1)), s, s[idx]) for s in states]
    back = ert.reorder_beams(states, _cuda(p), out=states)
    assert all(torch.equal(a, b) for a, b in zip(states, want)) and back[0] is states[0]


def test_reorder_rows_strided_other_width_and_single(ert):
    import torch
    rng = np.random.default_rng(3)
    R, W, k = 4, 3, 7
    buf = torch.randn(R * W, 301, device="cuda")
    x = buf[:, 5:298]
    p = _parents(rng, R, k, W)
    idx = _cuda((np.arange(R)[:, None] * W + p).reshape(-1))
    assert torch.equal(ert.reorder_beams(x, _cuda(p), beams=W), x[idx])
    to = torch.full((R * k, 400), 7.0, device="cuda")
    ert.reorder_beams(x, _cuda(p), beams=W, out=to[:, 11:304])
    assert torch.equal(to[:, 11:304], x[idx]) and bool((to[:, :11] == 7).all()) and bool((to[:, 304:] == 7).all())
    # in place, with neighbours left alone
    p = _parents(rng, R, W, W)
    idx = _cuda((np.arange(R)[:, None] * W + p).reshape(-1))
    want = buf.clone()
    want[:, 5:298] = x[idx]
    ert.reorder_beams(x, _cuda(p), out=x)
    assert torch.equal(buf, want)
    assert ert.reorder_beams([], _cuda(p)) == []
    assert ert.reorder_beams(torch.empty(0, 5, device="cuda"), torch.empty(0, 3, dtype=torch.int32, device="cuda")).shape == (0, 5)


def test_reorder_rows_side_by_side_and_crossed(ert):
    import torch
    rng = np.random.default_rng(4)
    R, W = 3, 5
    p = _parents(rng, R, W, W)
    idx = _cuda((np.arange(R)[:, None] * W + p).reshape(-1))
    wide = torch.randn(R * W, 53, device="cuda")
    want = wide.clone()
    want[:, :48] = wide[idx][:, :48]
    parts = [wide[:, :20], wide[:, 20:41], wide[:, 41:48]]
    ert.reorder_beams(parts, _cuda(p), out=parts)
    assert torch.equal(wide, want)
    a, b = torch.randn(R * W, 9, device="cuda"), torch.randn(R * W, 9, device="cuda")
    for states, out in (([a, b], [b, a]), ([a, a], [a, a]), ([a, b], [a, a]), ([wide[:, :20], wide[:, 19:30]],) * 2):
        with pytest.raises((ValueError, RuntimeError)):
            ert.reorder_beams(states, _cuda(p), out=out)


def test_same_cache_twice_is_refused(ert):
    import torch
    c = torch.zeros(12, 4, 2, 8, device="cuda")
    tab, lens = torch.arange(12, device="cuda", dtype=torch.int32).view(6, 2), torch.full((2,), 5, dtype=torch.int32, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    with pytest.raises((ValueError, RuntimeError)):
        ert.reorder_block_tables(tab, lens, p, 4, caches=[c, c])
    with pytest.raises((ValueError, RuntimeError)):
        ert.evict_cache(torch.zeros(2, 1, 8, device="cuda"), lens, 3, block_tables=tab[:2], caches=[c, c])


def test_reorder_rows_beyond_32_bit_offsets(ert):
    import torch
    x = torch.zeros(6, 1 << 30, dtype=torch.uint8, device="cuda")
    x[:, ::1 << 20] = torch.arange(1, 7, device="cuda", dtype=torch.uint8)[:, None]
    p = torch.tensor([[5, 0, 0, 2, 4, 1]], dtype=torch.int32, device="cuda")
    ert.reorder_beams(x, p, out=x)
    assert x[:, 1 << 29].tolist() == [6, 1, 1, 3, 5, 2] and x[:, 0].tolist() == [6, 1, 1, 3, 5, 2]


@pytest.mark.parametrize("block_size", [1, 3, 16, 48, 64])
@pytest.mark.parametrize("R,W,k", [(1, 1, 1), (5, 4, 4), (3, 9, 9), (4, 2, 5), (2, 6, 3), (1, 32, 32)])
def test_reorder_block_tables(ert, block_size, R, W, k):
    import torch
    rng = np.random.default_rng([block_size, R, W, k])
    width = 7
    N = 2 * R * (W + k) + 40
    lens = rng.integers(0, width * block_size + 3, R).astype(np.int32)
    if R > 2:
        lens[0], lens[1], lens[2] = 0, block_size * 2, -5
    ids = rng.permutation(N - 40).astype(np.int32)
    tables = rng.integers(N - 40, N, (R * W, width)).astype(np.int32)
    full = np.maximum(np.repeat(lens, W), 0) // block_size
    for i in range(R * W):
        if full[i] < width:
            tables[i, full[i]] = ids[i]
    tail = ids[R * W:R * W + R * k]
    if R > 2:
        tail[-1] = -1          # a block that is not there
        tables[-1] = N + 5
    for shape, dtype in (((2, 24), torch.bfloat16), ((5,), torch.uint8)):
        caches = [torch.randint(0, 200, (N, block_size, *shape), device="cuda").to(dtype) for _ in range(3)]
        for own in ([False, True] if W == k else [True]):
            p = _parents(rng, R, k, W, 0.15)
            t = tail if own else None
            want, copies = ref.block_tables(tables, lens, p, block_size, t)
            expect = [c.clone() for c in caches]
            for _, a, b, n in copies:
                if 0 <= a < N and 0 <= b < N:
                    for e, c in zip(expect, caches):
                        e[b, :n] = c[a, :n]
            for in_place in ([False, True] if W == k else [False]):
                log(f"[tables] bs={block_size} {R}x{W}->{k} own={own} in_place={in_place} {dtype}")
                mine, tab = [c.clone() for c in caches], _cuda(tables)
                got = ert.reorder_block_tables(tab, _cuda(lens), _cuda(p), block_size, caches=mine,
                                               tail_blocks=None if t is None else _cuda(t),
                                               out=tab if in_place else None)
                assert np.array_equal(got.cpu().numpy(), want)
                assert all(torch.equal(a, b) for a, b in zip(mine, expect))
                if not in_place:
                    assert np.array_equal(tab.cpu().numpy(), tables)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Case:
    """A cache, tables and queries; everything unused holds NaN and infinities."""

    def __init__(self, dtype, dim, bs, members, prefix, suffix, heads, kv, next_n=1, seed=0, spread=1.0,
                 outside=0, lens=None, plens=None, layout="plain", bad=False):
        import torch
        rng = np.random.default_rng([dim, bs, len(members), heads, kv, next_n, seed])
        self.dtype, self.bs, self.next_n, self.heads, self.kv, self.dim = dtype, bs, next_n, heads, kv, dim
        G, S = len(members), sum(members) + 2 * outside
        self.starts = (outside + np.r_[0, np.cumsum(members)]).astype(np.int32)
        self.plens = np.array(plens if plens is not None else rng.integers(0, prefix + 1, G), dtype=np.int32)
        self.lens = np.array(lens if lens is not None else rng.integers(0, suffix + 1, S), dtype=np.int32)
        pw, sw = -(-prefix // bs) if G else 0, -(-suffix // bs)
        ids = rng.permutation(G * pw + S * sw + 3).astype(np.int32)
        self.ptab, self.tab = ids[:G * pw].reshape(G, pw).copy(), ids[G * pw:G * pw + S * sw].reshape(S, sw).copy()
        self.N = N = ids.size
        k = rng.normal(0, spread, (N, bs, kv, dim)).astype(np.float32)
        v = rng.normal(0, 1, (N, bs, kv, dim)).astype(np.float32)
        used = np.zeros((N, bs), dtype=bool)
        for t, n in itertools.chain(zip(self.ptab, self.plens), zip(self.tab, self.lens)):
            b, o, _ = ref.positions(t, n, bs, N)
            used[b, o] = True
        poison = np.array([NAN, INF, NINF, 1e30], dtype=np.float32)
        k[~used] = poison[rng.integers(0, 4, (int((~used).sum()), kv, dim))]
        v[~used] = poison[rng.integers(0, 4, (int((~used).sum()), kv, dim))]
        if bad:   # tables that name blocks that are not there
            for t in (self.ptab, self.tab):
                if t.size > 4:
                    t.reshape(-1)[rng.integers(0, t.size, 3)] = [-1, N, 2 ** 31 - 1]
        q = rng.normal(0, 1, (S * next_n, heads, dim)).astype(np.float32)
        if layout == "plain":
            self.k, self.v, self.q = (_cuda(a, _dt(dtype)) for a in (k, v, q))
        else:   # keys and values of a block together, heads before slots; queries inside a wider row
            both = torch.empty(N, 2, kv, bs, dim, dtype=_dt(dtype), device="cuda")
            self.k, self.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
            self.k.copy_(_cuda(k)), self.v.copy_(_cuda(v))
            wide = torch.full((S * next_n, heads + 5, dim + 8), NAN, dtype=_dt(dtype), device="cuda")
            self.q = wide[:, 2:heads + 2, 8:]
            self.q.copy_(_cuda(q))
        self.G, self.S = G, S

    def dev(self):
        return (_cuda(self.ptab) if self.G else None, _cuda(self.plens) if self.G else None, _cuda(self.tab),
                _cuda(self.lens))

    def group(self, s):
        for g in range(self.G):
            if self.starts[g] <= s < self.starts[g + 1]:
                return g
        return None

    def sees(self, s, t, limit=None, own=None):
        """[(blocks, offsets)], [(kind, entry, positions)] of token t of sequence s."""
        parts, where = [], []
        g = self.group(s)
        if g is not None:
            b, o, p = ref.positions(self.ptab[g], self.plens[g] if limit is None else min(self.plens[g], limit), self.bs, self.N)
            parts.append((b, o)), where.append((0, g, p))
        n = min(int(self.lens[s]), self.tab.shape[1] * self.bs)
        n = n if own is None else min(n, own)
        b, o, p = ref.positions(self.tab[s], n - self.next_n + t + 1, self.bs, self.N)
        parts.append((b, o)), where.append((1, s, p))
        return parts, where

    def expect(self, scale=None, limit=None, own=None):
        q, k, v = (x.double().cpu().numpy() for x in (self.q, self.k, self.v))
        scale = self.dim ** -0.5 if scale is None else scale
        return [(ref.attention(q[s * self.next_n + t], k, v, self.sees(s, t, limit, own)[0], scale),
                 self.sees(s, t, limit, own)[1]) for s in range(self.S) for t in range(self.next_n)]


def _check_attend(ert, c, what, scale=None, limit=None, own=None, equal=False, room=0):
    import torch
    log(f"[attend] {what}")
    pt, pl, tab, lens = c.dev()
    if room:   # prefix tables for as many positions as `room`
        pt = torch.nn.functional.pad(pt, (0, (room + c.bs - 1) // c.bs - pt.shape[1]), value=-1)
    out, lse = ert.prefix_attention(c.q, c.k, c.v, pt, pl, tab, lens, next_n=c.next_n, scale=scale,
                                    group_starts=_cuda(c.starts) if c.G and not equal else None,
                                    max_prefix_len=limit, max_len=own, return_lse=True)
    torch.cuda.synchronize()
    got, sums = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert got.shape == tuple(c.q.shape) and out.dtype == c.q.dtype
    for i, ((o, z, spread, size, delta, w), _) in enumerate(c.expect(scale, limit, own)):
        off, loff = ref.bounds(o, z, spread, size, delta, w.shape[1], np.full(c.heads, HALF[c.dtype]), SMALL[c.dtype])
        bad = np.abs(got[i] - o) > off
        assert not bad.any() and not np.isnan(got[i]).any(), (what, i, np.abs(got[i] - o).max(), off.max())
        empty = np.isinf(z)
        assert np.array_equal(np.isneginf(sums[i]), empty), (what, i)
        assert (np.abs(sums[i] - z)[~empty] <= loff[~empty]).all(), (what, i, sums[i], z)
    return lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bs", [1, 7, 16, 48, 64])
def test_attention_sizes(ert, dtype, dim, bs):
    for n, (members, prefix, suffix, heads, kv, next_n) in enumerate([
            ([1], 1, 1, 1, 1, 1), ([2], 70, 33, 4, 2, 1), ([3, 0, 5, 1], 257, 40, 6, 2, 2),
            ([9], 600, 150, 8, 1, 1), ([4, 4], 130, 65, 14, 2, 3), ([40], 300, 20, 2, 2, 1)]):
        c = Case(dtype, dim, bs, members, prefix, suffix, heads, kv, next_n, seed=n)
        _check_attend(ert, c, f"{dtype} dim={dim} bs={bs} members={members} prefix={prefix} suffix={suffix} "
                              f"heads={heads}/{kv} next_n={next_n}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bs", [1, 7, 16, 64])
def test_attention_where_queries_share_a_read(ert, dtype, dim, bs):
    # room for 2^21 positions: waves of 32 queries share the prefix, 2, 4 and 8 of them
    for n, (members, prefix, suffix, heads, kv, next_n) in enumerate([
            ([20, 13], 130, 33, 4, 2, 1), ([9, 0, 30, 1], 333, 40, 6, 2, 2), ([33], 700, 50, 8, 2, 1),
            ([40, 3, 90], 100, 10, 4, 1, 1), ([60], 257, 20, 8, 1, 1), ([70, 129], 65, 5, 6, 2, 1)]):
        c = Case(dtype, dim, bs, members, prefix, suffix, heads, kv, next_n, seed=n)
        _check_attend(ert, c, f"{dtype} dim={dim} bs={bs} members={members} prefix={prefix} suffix={suffix} "
                              f"heads={heads}/{kv} next_n={next_n}", room=1 << 21)


@pytest.mark.parametrize("dtype,dim,bs,next_n", [("bf16", 64, 16, 1), ("fp16", 128, 7, 1), ("bf16", 128, 64, 2), ("fp16", 64, 1, 2)])
def test_attention_of_many_short_sequences(ert, dtype, dim, bs, next_n):
    for members, prefix in (([300, 0, 220], 40), ([], 0)):   # a wave a sequence and key head
        c = Case(dtype, dim, bs, members, prefix, 70, 8, 4, next_n, outside=2 if members else 256)
        _check_attend(ert, c, f"{dtype} dim={dim} bs={bs} many {members}")


def test_attention_long_prefixes_of_many_queries(ert):
    for dtype, dim, members, prefix, heads, kv in (("bf16", 64, [33], 17000, 2, 2), ("fp16", 128, [20, 5], 9001, 8, 2),
                                                   ("bf16", 128, [2, 40, 30], 5000, 8, 1)):
        c = Case(dtype, dim, 64, members, prefix, 20, heads, kv, plens=[prefix - 7 * g for g in range(len(members))])
        _check_attend(ert, c, f"{dtype} {dim} {members} {prefix}", room=1 << 23)
        c = Case(dtype, dim, 64, members, prefix // 2, 20, heads, kv, spread=8.0)
        _check_attend(ert, c, f"{dtype} {dim} {members} spread 8", room=1 << 23)


@pytest.mark.parametrize("members,room", [([3, 2], 0), ([70, 40], 1 << 21)])
def test_attention_leaves_out_prefixes_of_falling_starts(ert, members, room):
    c = Case("bf16", 64, 16, members, 200, 50, 8, 2)
    c.starts = c.starts[::-1].copy()
    c.group = lambda s: None
    _check_attend(ert, c, f"falling starts {members}", room=room)


def test_attention_long_rows_and_many_splits(ert):
    for dtype, members, prefix, suffix, heads, kv in (("bf16", [2], 20000, 3000, 4, 2), ("fp16", [3, 1], 9001, 4097, 4, 1)):
        c = Case(dtype, 128, 64, members, prefix, suffix, heads, kv, plens=[prefix] * len(members),
                 lens=[suffix] * sum(members))
        _check_attend(ert, c, f"{dtype} long {members}")
        for spread in (8.0,):   # scores hundreds apart: one key takes nearly all
            c = Case(dtype, 128, 64, members, 3001, 500, heads, kv, spread=spread)
            _check_attend(ert, c, f"{dtype} spread={spread}")


def test_attention_without_prefix_or_own_positions(ert):
    c = Case("bf16", 64, 16, [], 0, 300, 8, 2, outside=3)
    _check_attend(ert, c, "no prefixes")
    c = Case("bf16", 64, 16, [3, 2], 200, 50, 8, 2, outside=2)
    _check_attend(ert, c, "sequences outside every group")
    c = Case("fp16", 64, 16, [3, 2], 200, 50, 8, 2, lens=[0] * 5)
    _check_attend(ert, c, "prefix alone")
    c = Case("fp16", 128, 16, [3, 2], 200, 50, 8, 2, lens=[0] * 5, plens=[0, 5])
    _check_attend(ert, c, "rows that see nothing")
    c = Case("bf16", 128, 16, [2, 2], 200, 50, 8, 2, next_n=4, lens=[1, 2, 3, 60], plens=[0, -7])
    _check_attend(ert, c, "tokens before the first position, lengths outside the tables")
    c = Case("bf16", 128, 16, [4, 4], 200, 50, 8, 2)
    _check_attend(ert, c, "equal groups", equal=True)


def test_attention_strides_scale_limits_and_bad_blocks(ert):
    for dtype in ("bf16", "fp16"):
        c = Case(dtype, 128, 16, [3, 2], 333, 77, 8, 2, layout="wide")
        _check_attend(ert, c, f"{dtype} strided")
        c = Case(dtype, 64, 24, [3, 2], 333, 77, 8, 4, next_n=2)
        for scale in (0.0, 1.0):
            _check_attend(ert, c, f"{dtype} scale={scale}", scale=scale)
        _check_attend(ert, c, f"{dtype} limits", limit=100, own=31)
        c = Case(dtype, 64, 16, [3, 2], 333, 77, 8, 4, bad=True)
        _check_attend(ert, c, f"{dtype} blocks that are not there")


def test_attention_cache_beyond_32_bit_offsets(ert):
    import torch
    N, bs, H, D = 40000, 64, 8, 128
    k = torch.zeros(N, bs, H, D, dtype=torch.bfloat16, device="cuda")   # 2.6e9 elements
    c = Case("bf16", D, bs, [2], 200, 100, 16, H)
    at = torch.tensor([N - 1 - 3 * i for i in range(c.N)], device="cuda")
    v = torch.zeros_like(k)
    k[at], v[at] = c.k, c.v
    move = at.cpu().numpy().astype(np.int32)
    pt, tab = move[c.ptab], move[c.tab]
    pl, lens = _cuda(c.plens), _cuda(c.lens)
    got = ert.prefix_attention(c.q, k, v, _cuda(pt), pl, _cuda(tab), lens)
    want = ert.prefix_attention(c.q, c.k, c.v, _cuda(c.ptab), pl, _cuda(c.tab), lens)
    assert torch.equal(got, want)
    _check_attend(ert, c, "the same near")


# ---------------------------------------------------------------------------
# attention mass
# ---------------------------------------------------------------------------

def _check_mass(ert, c, what, decay=0.9, given=True, extra=0, seed=0):
    import torch
    log(f"[mass] {what}")
    rng = np.random.default_rng(seed)
    pt, pl, tab, lens = c.dev()
    starts = _cuda(c.starts) if c.G else None
    _, lse = ert.prefix_attention(c.q, c.k, c.v, pt, pl, tab, lens, next_n=c.next_n, group_starts=starts, return_lse=True)
    P, L = (c.ptab.shape[1] * c.bs + extra if c.G else 0), c.tab.shape[1] * c.bs + extra
    m0, m1 = rng.random((c.G, c.kv, P)).astype(np.float32), rng.random((c.S, c.kv, L)).astype(np.float32)
    arg = dict(prefix_mass=_cuda(m0) if c.G else None, mass=_cuda(m1)) if given else {}
    got = ert.attention_mass(c.q, c.k, lse, pt, pl, tab, lens, next_n=c.next_n, group_starts=starts, decay=decay, **arg)
    torch.cuda.synchronize()
    base = [m0.astype(np.float64) * np.float32(decay), m1.astype(np.float64) * np.float32(decay)]
    if not given:
        base = [np.zeros((c.G, c.kv, c.ptab.shape[1] * c.bs)), np.zeros((c.S, c.kv, c.tab.shape[1] * c.bs))]
    off = [np.abs(b) * 2.0 ** -22 for b in base]
    per = c.heads // c.kv
    sums = lse.double().cpu().numpy()
    for i, ((_, z, _, _, delta, w), where) in enumerate(c.expect()):
        at = 0
        for kind, entry, p in where:
            for h in range(c.heads):
                if np.isinf(z[h]):
                    continue
                # the weights against the sum that the call is given
                x = w[h, at:at + p.size] * np.exp(z[h] - sums[i, h])
                base[kind][entry, h // per, p] += x
                off[kind][entry, h // per, p] += x * (2 * delta[h] + 2.0 ** -21 * (1 + abs(z[h])) + c.S * c.next_n * per * 2.0 ** -24)
            at += p.size
    for kind in (0, 1):
        if kind == 0 and not c.G:
            assert got[0] is None
            continue
        g = got[kind].double().cpu().numpy()
        assert g.shape == base[kind].shape and (np.abs(g - base[kind]) <= off[kind] * 1.01 + 1e-37).all(), \
            (what, kind, np.abs(g - base[kind]).max())
    return lse, got


@pytest.mark.parametrize("dtype,dim", [("bf16", 64), ("bf16", 128), ("fp16", 64), ("fp16", 128)])
@pytest.mark.parametrize("bs", [1, 7, 16, 64])
def test_attention_mass(ert, dtype, dim, bs):
    for n, (members, prefix, suffix, heads, kv, next_n) in enumerate([
            ([1], 1, 1, 1, 1, 1), ([3, 0, 5, 1], 257, 40, 6, 2, 2), ([9], 600, 150, 8, 1, 1), ([], 0, 70, 4, 4, 1)]):
        c = Case(dtype, dim, bs, members, prefix, suffix, heads, kv, next_n, seed=n, outside=n % 2 if members else 2)
        _check_mass(ert, c, f"{dtype} dim={dim} bs={bs} members={members}", extra=n * 5, given=n != 2)


def test_attention_mass_layouts_bad_blocks_and_in_place(ert):
    import torch
    c = Case("bf16", 128, 16, [3, 2], 333, 77, 8, 2, layout="wide")
    _check_mass(ert, c, "strided")
    c = Case("fp16", 64, 16, [3, 2], 333, 77, 8, 4, bad=True, plens=[0, 300], lens=[0, 0, 3, 77, 90])
    lse, want = _check_mass(ert, c, "blocks that are not there, rows that see nothing", given=False)
    pt, pl, tab, lens = c.dev()
    a, b = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    for _ in range(2):
        ert.attention_mass(c.q, c.k, lse, pt, pl, tab, lens, group_starts=_cuda(c.starts), decay=0.5, prefix_mass=a,
                           mass=b, prefix_out=a, out=b)
    assert torch.allclose(a, want[0] * 1.5, rtol=1e-6) and torch.allclose(b, want[1] * 1.5, rtol=1e-6)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------

def _check_evict(ert, mass, lens, budget, sinks, recent, what):
    import torch
    log(f"[evict] {what}")
    kept, m, n = ert.evict_cache(mass, _cuda(lens), budget, sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    host = mass.cpu().numpy()
    kept, m, n = kept.cpu().numpy(), m.cpu().numpy(), n.cpu().numpy()
    for r in range(host.shape[0]):
        for h in range(host.shape[1]):
            want = ref.keep(host[r, h], lens[r], budget, sinks, recent)
            assert n[r] == want.size
            assert np.array_equal(kept[r, h], np.r_[want, np.full(budget - want.size, -1)]), (what, r, h)
            assert np.array_equal(m[r, h], np.r_[host[r, h][want], np.zeros(budget - want.size, np.float32)],
                                  equal_nan=True), (what, r, h)


@pytest.mark.parametrize("positions", [1, 2, 63, 65, 1000, 1024, 1025, 16384, 20011])
def test_evict_sizes(ert, positions):
    rng = np.random.default_rng(positions)
    R, H = 4, 3
    lens = np.array([positions, max(1, positions // 2), 0, positions + 9], dtype=np.int32)
    kinds = {"normal": rng.normal(0, 1, (R, H, positions)), "zeros": np.zeros((R, H, positions)),
             "few": rng.integers(0, 3, (R, H, positions)).astype(float),
             "half": np.where(rng.random((R, H, positions)) < 0.5, 0.0, np.exp(rng.normal(0, 9, (R, H, positions)))),
             "masked": np.where(rng.random((R, H, positions)) < 0.3, rng.choice([NAN, INF, NINF, -0.0, 1e-42], (R, H, positions)),
                                rng.normal(0, 1, (R, H, positions)))}
    for name, m in kinds.items():
        mass = _cuda(m.astype(np.float32))
        for budget in sorted({1, 2, max(1, positions // 3), max(1, positions - 1), positions, positions + 5}):
            for sinks, recent in {(0, 0), (min(1, budget), 0), (0, min(7, budget)), (min(4, budget // 2), budget - min(4, budget // 2))}:
                _check_evict(ert, mass, lens, budget, sinks, recent,
                             f"{name} positions={positions} budget={budget} sinks={sinks} recent={recent}")


def test_evict_strided_mass_and_wider_output(ert):
    import torch
    rng = np.random.default_rng(2)
    wide = _cuda(rng.random((5, 4, 700)).astype(np.float32))
    mass = wide[1:4, ::2, 13:513]
    lens = np.array([500, 100, 333], dtype=np.int32)
    _check_evict(ert, mass, lens, 120, 3, 10, "strided")
    out = torch.full((3, 2, 200), 9.0, device="cuda")
    kept, m, _ = ert.evict_cache(mass, _cuda(lens), 120, mass_out=out)
    assert m is out and bool((out[:, :, 120:] == 0).all())
    assert torch.equal(out[0, 0, :120], mass[0, 0][kept[0, 0].long()])


@pytest.mark.parametrize("block_size,heads,cache_heads,dim", [(16, 2, 2, 64), (1, 1, 4, 8), (7, 3, 6, 128), (64, 4, 8, 40)])
def test_evict_moves_rows(ert, block_size, heads, cache_heads, dim):
    import torch
    rng = np.random.default_rng([block_size, heads])
    R, L, budget = 5, 900, 333
    width, to_width = -(-L // block_size), -(-budget // block_size)
    N = R * (width + to_width) + 3
    ids = rng.permutation(N).astype(np.int32)
    tables, to = ids[:R * width].reshape(R, width).copy(), ids[R * width:R * (width + to_width)].reshape(R, to_width).copy()
    tables[4, 1], to[4, 0] = -1, N          # blocks that are not there
    lens = np.array([L, 100, 0, 334, 700], dtype=np.int32)
    mass = rng.random((R, heads, L)).astype(np.float32)
    caches = [torch.randint(0, 100, (N, block_size, cache_heads, dim), device="cuda").to(torch.float16) for _ in range(2)]
    for in_place in (False, True):
        log(f"[evict move] bs={block_size} heads={heads}/{cache_heads} in_place={in_place}")
        mine = [c.clone() for c in caches]
        target = tables if in_place else to
        kept, _, n = ert.evict_cache(_cuda(mass), _cuda(lens), budget, sinks=2, recent=20, block_tables=_cuda(tables),
                                     caches=mine, out_tables=None if in_place else _cuda(to))
        kept, per = kept.cpu().numpy(), cache_heads // heads
        for c, m in zip(caches, mine):
            want = c.cpu().numpy().copy()
            host = c.cpu().numpy()
            for r in range(R):
                for h in range(heads):
                    for j, p in enumerate(kept[r, h]):
                        if p < 0 or j // block_size >= target.shape[1]:
                            continue
                        a, b = tables[r, p // block_size], target[r, j // block_size]
                        if 0 <= a < N and 0 <= b < N:
                            want[b, j % block_size, h * per:(h + 1) * per] = host[a, p % block_size, h * per:(h + 1) * per]
            assert np.array_equal(m.cpu().numpy(), want), (in_place,)


def test_evict_moves_rows_beyond_32_bit_offsets(ert):
    import torch
    N, bs = 600, 1024
    cache = torch.zeros(N, bs, 4, 1024, dtype=torch.bfloat16, device="cuda")   # 5 GB
    cache[590, :, 0, 0] = torch.arange(bs, device="cuda").to(torch.bfloat16)
    mass = torch.zeros(1, 1, bs, device="cuda")
    mass[0, 0, 100:110] = 1.0
    kept, _, n = ert.evict_cache(mass, _cuda(np.array([bs], np.int32)), 10, block_tables=_cuda(np.array([[590]], np.int32)),
                                 caches=cache, out_tables=_cuda(np.array([[599]], np.int32)))
    assert cache[599, :10, 0, 0].tolist() == list(range(100, 110)) and float(cache[599, 10:].abs().sum()) == 0


# ---------------------------------------------------------------------------
# streams, graphs, devices, and a search that uses all of them
# ---------------------------------------------------------------------------

def _step(ert, st):
    """One step of a search: attention and mass, the choice, and what it moves."""
    out, lse = ert.prefix_attention(st["q"], st["k"], st["v"], st["ptab"], st["plens"], st["tab"], st["slens"],
                                    group_starts=st["starts"], return_lse=True)
    mass = ert.attention_mass(st["q"], st["k"], lse, st["ptab"], st["plens"], st["tab"], st["slens"],
                              group_starts=st["starts"], prefix_mass=st["pmass"], decay=0.5)
    found = ert.select_beams(st["logits"], st["scores"], st["scores"].shape[1])
    history = ert.reorder_beams(st["history"], found[1])
    tables = ert.reorder_block_tables(st["tab"], st["lens"], found[1], st["k"].shape[1], caches=[st["k"], st["v"]],
                                      tail_blocks=st["tail"])
    kept = ert.evict_cache(mass[0], st["plens"], 40, sinks=2, recent=8)
    return [out, lse, *mass, *found, history, tables, *kept, st["k"].clone(), st["v"].clone()]


def _search(seed):
    import torch
    R, W, bs = 3, 4, 16
    c = Case("bf16", 64, bs, [W] * R, 200, 60, 8, 2, seed=seed, plens=[200, 150, 30], lens=[37] * 4 + [60] * 4 + [16] * 4)
    g = torch.Generator(device="cuda").manual_seed(seed)
    fresh = torch.zeros(R * W, bs, 2, 64, dtype=torch.bfloat16, device="cuda")
    pt, pl, tab, lens = c.dev()
    return {"q": c.q, "k": torch.cat([c.k, fresh]), "v": torch.cat([c.v, fresh]), "ptab": pt, "plens": pl, "tab": tab,
            "slens": lens, "lens": lens.view(R, W)[:, 0].contiguous(), "starts": _cuda(c.starts),
            "pmass": torch.rand(R, 2, pt.shape[1] * bs, device="cuda", generator=g),
            "logits": torch.randn(R * W, 4001, device="cuda", generator=g),
            "scores": -torch.rand(R, W, device="cuda", generator=g),
            "history": torch.randint(0, 99, (R * W, 30), device="cuda", generator=g),
            "tail": (torch.arange(R * W, device="cuda") + c.N).to(torch.int32)}


def _same(a, b):
    import torch
    return all(torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float())) for x, y in zip(a, b))


def test_ranks_stay_numbers_at_any_penalty(ert):
    import torch
    logits, scores = torch.zeros(6, 1, device="cuda"), torch.zeros(2, 3, device="cuda")
    lengths = torch.tensor([[9, 1, 2 ** 31 - 1]] * 2, dtype=torch.int32, device="cuda")
    for penalty in (-3e38, -400.0, 400.0, 3e38):   # totals of zero over powers of 0 and infinity
        s, b, t = ert.select_beams(logits, scores, 4, lengths=lengths, length_penalty=penalty)
        assert s.tolist() == [[0.0] * 3 + [NINF]] * 2 and t.tolist() == [[0] * 3 + [-1]] * 2
        assert b.tolist() == [[0, 1, 2, -1]] * 2


def test_step_on_another_stream_and_repeated(ert):
    import torch
    st = _search(1)
    want = _step(ert, st)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = [_step(ert, st) for _ in range(3)]
    side.synchronize()
    assert all(_same(a, want) for a in again)
    log("[step] stream argument")
    found = ert.select_beams(st["logits"], st["scores"], 4, stream=side)
    side.synchronize()
    assert _same(found, want[4:7])


def test_step_in_a_graph(ert):
    import torch
    st = _search(2)
    eager = [_step(ert, _search(s)) for s in (2, 3, 4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(ert, st)
    for s, want in zip((2, 3, 4, 2), eager + eager[:1]):
        new = _search(s)
        for name in st:
            st[name].copy_(new[name])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert _same(captured, want), s
        _step(ert, _search(s))   # eager work between the replays


def test_two_graphs_and_an_eager_call_side_by_side(ert):
    import torch
    states = [_search(5), _search(6)]
    want = [_step(ert, s) for s in states]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for s in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_step(ert, s))
        graphs.append(g)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    eager = _search(7)
    ahead = _step(ert, eager)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, sides):
            with torch.cuda.stream(s):
                g.replay()
        between = _step(ert, eager)
        torch.cuda.synchronize()
        assert _same(between, ahead) and all(_same(o, w) for o, w in zip(outs, want))


def test_search_over_a_shared_cache_equals_a_private_one(ert):
    """Some steps of a search with shared prompt, blocks moved by parent, and the
    framework's block tables, against attention over each beam's whole history
    kept apart."""
    import torch
    R, W, bs, H, D, V, steps = 2, 3, 4, 2, 64, 501, 11
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    embed, proj = rnd(V, 3, H, D).bfloat16(), rnd(H * D, V) * 0.5
    prompt = torch.randint(0, V, (R, 10), device="cuda", generator=g)
    N = R * 3 + R * W * 4
    k, v = (torch.zeros(N, bs, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ptab = torch.arange(R * 3, device="cuda", dtype=torch.int32).view(R, 3)
    for r in range(R):
        for i in range(10):
            k[ptab[r, i // bs], i % bs], v[ptab[r, i // bs], i % bs] = embed[prompt[r, i], 1], embed[prompt[r, i], 2]
    plens = torch.full((R,), 10, dtype=torch.int32, device="cuda")
    tab = torch.full((R * W, 4), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(R * 3, N, device="cuda", dtype=torch.int32)
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    scores = torch.tensor([[0.0] + [NINF] * (W - 1)] * R, device="cuda")
    tokens = torch.zeros(R, W, dtype=torch.int32, device="cuda")
    history = torch.zeros(R * W, steps, dtype=torch.int32, device="cuda")
    for step in range(steps):
        lens = torch.full((R * W,), step + 1, dtype=torch.int32, device="cuda")
        _, _, _, slots, taken = ert.extend_block_tables(tab, lens, torch.ones_like(lens), free, taken, bs, R * W)
        history[:, step] = tokens.view(-1)
        x = embed[tokens.view(-1).long()]
        k.view(-1, H, D)[slots.long()], v.view(-1, H, D)[slots.long()] = x[:, 1], x[:, 2]
        out = ert.prefix_attention(x[:, 0], k, v, ptab, plens, tab, lens)
        # each beam's own history, no paging
        whole = torch.cat([prompt.repeat_interleave(W, 0), history[:, :step + 1].long()], 1)
        e = embed[whole].float()
        a = torch.softmax((e[:, :, 1] * x[:, None, 0].float()).sum(3) * D ** -0.5, 1)
        want = (a[..., None] * e[:, :, 2]).sum(1)
        # weights and result rounded to bfloat16 (2^-8 each), the rest in 32 bits
        assert bool(((out.float() - want).abs() <= 2.0 ** -7 * 1.05 * (a[..., None] * e[:, :, 2].abs()).sum(1) + 1e-5).all()), step
        logits = out.float().view(R * W, -1) @ proj
        scores, parents, tokens = ert.select_beams(logits, scores, W)
        ert.reorder_beams(history, parents, out=history)
        ert.reorder_block_tables(tab, lens.view(R, W)[:, 0].contiguous(), parents, bs, caches=[k, v], out=tab)
        for r in range(R * W):
            for i in range(step + 1):
                assert torch.equal(k[tab[r, i // bs], i % bs], embed[history[r, i].long(), 1]), (step, r, i)
