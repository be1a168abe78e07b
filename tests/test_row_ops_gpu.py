"""The row operators on the GPU against their definitions in 64 bits: sampling,
expert routing and its gradient, block tables and slot maps, slots of
selected positions; alone, on other streams, in captured graphs, and together
with the selection as a serving step uses them."""
import itertools

import numpy as np
import pytest

import row_reference as ref
from gpu_helpers import log

pytestmark = pytest.mark.gpu

NINF = float("-inf")


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
# sampling
# ---------------------------------------------------------------------------

def _check_sample(ert, x, u, what, lp_abs=1e-11, **setting):
    """Tokens equal the definition's, log-probabilities to one fp32 rounding
    (2^-24 of the value) beside the weights' own 2^-45 a term (1e-11)."""
    import torch
    host = x.float().cpu().numpy()
    rows = host.shape[0]
    u = np.asarray(u, dtype=np.float32)
    dev = {k: _cuda(np.asarray(v, dtype=np.int32 if k == "top_k" else np.float32))
           for k, v in setting.items()}
    want = [ref.sample_row(host[r], u[r], **{k: (int(v[r]) if k == "top_k" else np.float32(v[r]))
                                             for k, v in setting.items()}) for r in range(rows)]
    ud = _cuda(u)
    for whole in (False, True):
        log(f"[sample] {what} whole_row={whole}")
        tok, lp = ert.sample_tokens(x, ud, return_logprobs=True, whole_row=whole, **dev)
        torch.cuda.synchronize()
        got = tok.cpu().numpy()
        bad = [(r, int(got[r]), want[r][0]) for r in range(rows) if got[r] != want[r][0]]
        assert not bad, (what, whole, bad[:5])
        lp = lp.cpu().numpy().astype(np.float64)
        for r in range(rows):
            w = want[r][1]
            if np.isinf(w):
                assert lp[r] == w
            else:
                assert abs(lp[r] - w) <= 2.0 ** -24 * abs(w) * 1.001 + lp_abs, (what, whole, r, lp[r], w)


def _settings(rng, rows, kind):
    s = {"temperature": rng.uniform(0.4, 1.4, rows)}
    if kind in ("k", "all", "mixed"):
        s["top_k"] = rng.integers(1, 300, rows)
    if kind in ("p", "all", "mixed"):
        s["top_p"] = rng.uniform(0.05, 0.999, rows)
    if kind in ("m", "all", "mixed"):
        s["min_p"] = rng.uniform(0.0, 0.3, rows)
    if kind == "mixed":
        s["temperature"][rng.random(rows) < 0.2] = 0.0
        s["top_k"][rng.random(rows) < 0.5] = 0
        s["top_p"][rng.random(rows) < 0.4] = 1.0
        s["min_p"][rng.random(rows) < 0.5] = 0.0
    return s


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 63, 65, 1000, 2047, 2048, 2049, 6150, 40001])
def test_sample_sizes(ert, dtype, vocab):
    rng = np.random.default_rng([vocab, 1])
    for kind in ("none", "k", "p", "m", "all", "mixed"):
        rows = 5
        x = _cuda(rng.normal(0, 2.5, (rows, vocab)).astype(np.float32), _dt(dtype))
        _check_sample(ert, x, rng.random(rows), f"{dtype} vocab={vocab} {kind}",
                      **_settings(rng, rows, kind))


@pytest.mark.parametrize("vocab,rows", [(131072, 3), (200003, 2), (1 << 20, 1)])
def test_sample_long_rows(ert, vocab, rows):
    rng = np.random.default_rng([vocab, 2])
    for kind, spread in (("none", 2.0), ("p", 0.1), ("p", 2.5), ("all", 3.0), ("mixed", 1.0)):
        x = _cuda(rng.normal(0, spread, (rows, vocab)).astype(np.float32))
        _check_sample(ert, x, rng.random(rows), f"vocab={vocab} {kind} spread={spread}",
                      **_settings(rng, rows, kind))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("offset,stride", [(0, 5007), (1, 5009), (3, 5006), (5, 5021), (7, 5008)])
def test_sample_unaligned_rows_and_poisoned_neighbours(ert, dtype, offset, stride):
    import torch
    rng = np.random.default_rng([offset, stride])
    rows, vocab = 4, 5001
    buf = torch.full((rows * stride + 64,), float("inf"), device="cuda", dtype=_dt(dtype))
    buf[::3] = float("nan")
    x = buf.as_strided((rows, vocab), (stride, 1), offset)
    x.copy_(_cuda(rng.normal(0, 2, (rows, vocab)).astype(np.float32), _dt(dtype)))
    for kind in ("none", "all", "p"):
        _check_sample(ert, x, rng.random(rows), f"{dtype} offset={offset} stride={stride} {kind}",
                      **_settings(rng, rows, kind))


def test_sample_masked_infinite_and_equal_rows(ert):
    rng = np.random.default_rng(3)
    vocab = 4500
    rows = []
    rows.append(np.full(vocab, NINF))                                # nothing left
    rows.append(np.full(vocab, np.nan))                              # nothing left
    one = np.full(vocab, NINF); one[4321] = -3.0e38; rows.append(one)  # one left
    mix = rng.normal(0, 2, vocab); mix[::2] = np.nan; mix[1::4] = NINF; rows.append(mix)
    inf = rng.normal(0, 2, vocab); inf[[77, 2050, 4400]] = np.inf; rows.append(inf)
    rows.append(np.full(vocab, np.inf))                              # all +inf
    rows.append(np.full(vocab, 1.25))                                # all equal
    rows.append(np.full(vocab, np.finfo(np.float32).min))            # the type's lowest value
    two = np.zeros(vocab); two[1000:4000] = 1.0; rows.append(two)    # two classes
    low = rng.normal(0, 1, vocab); low[:4000] = np.finfo(np.float32).min; rows.append(low)
    wide = np.concatenate([[3e38, -3e38], rng.normal(0, 1, vocab - 2)]); rows.append(wide)
    zero = np.where(np.arange(vocab) % 2 == 0, 0.0, -0.0); rows.append(zero)
    x = _cuda(np.array(rows, dtype=np.float32))
    n = len(rows)
    u = np.linspace(0.013, 0.987, n)
    full = np.full(n, 1.0)
    _check_sample(ert, x, u, "special rows, no cut")
    for k in (1, 2, 3, 700, 4499, 4500, 9000):
        _check_sample(ert, x, u, f"special rows top_k={k}", top_k=[k] * n)
    for p in (0.0, 1e-9, 0.37, 0.999):
        _check_sample(ert, x, u, f"special rows top_p={p}", top_p=[p] * n)
    for m in (1e-20, 0.2, 1.0, 7.0):
        _check_sample(ert, x, u, f"special rows min_p={m}", min_p=[m] * n)
    _check_sample(ert, x, u, "special rows, all cuts", top_k=[1500] * n, top_p=[0.61] * n,
                  min_p=[0.05] * n, temperature=0.7 * full)
    for t in (0.0, -1.0, np.nan, np.inf, 1e-30, 1e30):
        _check_sample(ert, x, u, f"special rows T={t}", temperature=[t] * n)
        _check_sample(ert, x, u, f"special rows T={t} top_k", temperature=[t] * n, top_k=[1234] * n)


def test_sample_uniform_ends_and_settings_that_cut_nothing(ert):
    rng = np.random.default_rng(4)
    u = np.array([0.0, 1e-30, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, np.nan, np.inf], dtype=np.float32)
    n = u.size
    x = _cuda(rng.normal(0, 2, (n, 3001)).astype(np.float32))
    _check_sample(ert, x, u, "uniform ends")
    _check_sample(ert, x, u, "uniform ends, cut", top_k=[40] * n, top_p=[0.9] * n)
    _check_sample(ert, x, u, "nothing cut", top_k=[0, -5, 3001, 10 ** 9, 3002] * 2,
                  top_p=[1.0, 1.5, np.nan, np.inf, 1.0] * 2, min_p=[0.0, -1.0, np.nan, 0.0, -0.0] * 2)


def test_sample_crowded_candidates(ert):
    # more equal scores than a segment or the row hands on, ties at the cut,
    # the likely tokens side by side, and a flat row that needs most of it
    rng = np.random.default_rng(5)
    vocab, rows = 50000, 6
    x = np.zeros((rows, vocab))
    x[0] = np.round(rng.normal(0, 1, vocab))
    x[1] = rng.integers(0, 3, vocab)
    x[2] = rng.normal(0, 0.05, vocab)
    x[3] = rng.normal(0, 1, vocab); x[3, 30000:31000] += 8
    x[4] = -np.abs(np.arange(vocab) - 25000) / 3000.0
    x[5] = rng.normal(0, 1, vocab); x[5, ::17] = 4.0
    xd = _cuda(x.astype(np.float32))
    u = rng.random(rows)
    for k in (5, 64, 500, 3333, 20000):
        _check_sample(ert, xd, u, f"crowded top_k={k}", top_k=[k] * rows)
    for p in (0.1, 0.5, 0.95, 0.9999):
        _check_sample(ert, xd, u, f"crowded top_p={p}", top_p=[p] * rows, top_k=[0, 9000] * 3)
    _check_sample(ert, xd, u, "crowded min_p", min_p=[0.5, 1.0, 0.9, 0.1, 0.01, 0.9])


def test_sample_candidate_counts(ert):
    # rows of 1, 2, ... live scores, ties among them: one candidate more or less
    # than the waves, and the workgroup, rank at once
    rng = np.random.default_rng(23)
    counts = [1, 2, 8, 9, 63, 64, 65, 127, 128, 129, 192, 193, 255, 256, 257, 300]
    vocab, rows = 6 * 2048, len(counts)
    x = np.full((rows, vocab), NINF)
    for r, n in enumerate(counts):
        x[r, rng.permutation(vocab)[:n]] = np.round(rng.normal(0, 2, n) * 8) / 8
    xd = _cuda(x.astype(np.float32), _dt("bf16"))
    u = rng.random(rows)
    one = np.ones(rows)
    for k in (1, 2, 64, 65, 200, 256, 257):
        _check_sample(ert, xd, u, f"counts k={k}", top_k=[k] * rows)
        _check_sample(ert, xd, u, f"counts k={k} and more", top_k=[k] * rows, top_p=0.8 * one, min_p=0.02 * one)
    _check_sample(ert, xd, u, "counts top-p", top_p=0.7 * one)
    _check_sample(ert, xd, u, "counts min-p", min_p=0.1 * one)
    _check_sample(ert, xd, u, "counts cut to one", top_k=[300] * rows, top_p=0 * one)
    _check_sample(ert, xd, 0 * u, "counts first", top_k=[300] * rows)
    _check_sample(ert, xd, 0 * u + 0.99999994, "counts last", top_k=[300] * rows)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_sample_low_cuts(ert, dtype):
    # cuts far below the likeliest tokens: each alone, min-p beside them, both
    # at once, ties across the cut, rows with +inf scores
    rng = np.random.default_rng(15)
    vocab, rows = 30011, 6
    x = rng.normal(0, 0.3, (rows, vocab))
    x[1] = rng.normal(0, 1.5, vocab)
    x[2] = np.round(rng.normal(0, 1, vocab) * 8) / 8
    x[3, ::2] = NINF
    x[4, [5, 20000]] = 30.0
    x[5, [7, 8, 29000]] = np.inf
    xd = _cuda(x.astype(np.float32), _dt(dtype))
    u = rng.random(rows)
    one = np.ones(rows)
    _check_sample(ert, xd, u, f"{dtype} low top-p", top_p=0.9 * one, temperature=one)
    _check_sample(ert, xd, u, f"{dtype} low top-p and min-p", top_p=0.9 * one, min_p=0.2 * one)
    _check_sample(ert, xd, u, f"{dtype} low top-k", top_k=[12345] * rows)
    _check_sample(ert, xd, u, f"{dtype} low top-k and min-p", top_k=[12345] * rows, min_p=0.3 * one)
    _check_sample(ert, xd, u, f"{dtype} low min-p", min_p=0.05 * one)
    _check_sample(ert, xd, u, f"{dtype} low top-k and top-p", top_k=[12345] * rows, top_p=0.7 * one)
    _check_sample(ert, xd, u, f"{dtype} hot", temperature=40 * one, top_p=0.5 * one)
    _check_sample(ert, xd, u, f"{dtype} no temperature at all", temperature=np.inf * one, top_p=0.5 * one)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_sample_both_cuts_low(ert, dtype):
    # top-p's share is of what top-k leaves: from small to nearly all of it, k
    # on either side of what the candidates hold, past the row's end, min-p and
    # temperatures beside them, ties on both cuts, few scores that count at all
    rng = np.random.default_rng(16)
    vocab, rows = 24007, 8
    x = rng.normal(0, 0.5, (rows, vocab))
    x[1] = rng.normal(0, 3, vocab)
    x[2] = np.round(rng.normal(0, 1, vocab) * 4) / 4
    x[3, 100:] = NINF
    x[4] = 0.25
    x[5] = rng.normal(0, 1, vocab) + 40 * (rng.random(vocab) < 0.2)
    x[6] = -np.abs(rng.normal(0, 200, vocab))
    x[7, 11] = 9.0
    xd = _cuda(x.astype(np.float32), _dt(dtype))
    u = rng.random(rows)
    one = np.ones(rows)
    for k in (40, 700, 2500, 11000, 24006, 30000):
        for p in (0.05, 0.6, 0.999):
            _check_sample(ert, xd, u, f"{dtype} k={k} p={p}", top_k=[k] * rows, top_p=p * one)
    _check_sample(ert, xd, u, f"{dtype} with min-p", top_k=[9000] * rows, top_p=0.8 * one, min_p=0.4 * one)
    _check_sample(ert, xd, u, f"{dtype} hot", top_k=[9000] * rows, top_p=0.8 * one, temperature=30 * one)
    _check_sample(ert, xd, u, f"{dtype} flat", top_k=[9000] * rows, top_p=0.8 * one, temperature=np.inf * one)
    _check_sample(ert, xd, u, f"{dtype} each row its own", top_k=[9000, 0, 1, 50, 12000, 24007, 300, 5000],
                  top_p=np.array([0.9, 0.5, 0.3, 1.0, 0.01, 0.7, -1.0, 0.95]),
                  temperature=np.array([1, 0.2, 3, 1, 1, 8, 0, 1.0]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_sample_crowds_of_equal_scores(ert, dtype):
    # more scores of the cut's own value than are listed: constant rows, two
    # values, a crowd below a few others, masks between, crowds in some segments
    # only, several crowded values
    rng = np.random.default_rng(29)
    vocab, rows = 20011, 9
    x = np.zeros((rows, vocab))
    x[1, :] = -3.5
    x[1, rng.permutation(vocab)[:300]] = rng.normal(0, 0.5, 300)
    x[2, ::3] = NINF
    x[3] = np.where(rng.random(vocab) < 0.5, 1.0, 0.5)
    x[4, :9000] = -30
    x[5] = rng.normal(-8, 1, vocab)
    x[5, 3000:9000] = -2.25
    x[6] = rng.integers(0, 4, vocab) * 0.25
    x[7, 1] = 2.0
    x[8] = np.round(rng.normal(-20, 2, vocab))
    xd = _cuda(x.astype(np.float32), _dt(dtype))
    u = rng.random(rows)
    one = np.ones(rows)
    for p in (0.01, 0.5, 0.97):
        _check_sample(ert, xd, u, f"{dtype} crowds p={p}", top_p=p * one)
        _check_sample(ert, xd, u, f"{dtype} crowds p={p} and k", top_p=p * one, top_k=[6000] * rows)
    for k in (250, 301, 2500, 8000, 20010):
        _check_sample(ert, xd, u, f"{dtype} crowds k={k}", top_k=[k] * rows)
    _check_sample(ert, xd, u, f"{dtype} crowds min-p", top_k=[8000] * rows, min_p=0.1 * one)
    _check_sample(ert, xd, u, f"{dtype} crowds and min-p", top_p=0.9 * one, min_p=0.5 * one)
    _check_sample(ert, xd, 0 * u, f"{dtype} crowds first", top_p=0.9 * one)
    _check_sample(ert, xd, 0 * u + 0.99999994, f"{dtype} crowds last", top_p=0.9 * one)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_sample_infinities_that_are_candidates(ert, dtype):
    # so many +inf scores in a segment that its floor is +inf, and all of them
    # candidates: the cuts are of those scores alone
    rng = np.random.default_rng(41)
    vocab, counts = 4500, [1, 14, 15, 16, 40, 64, 100, 128]
    x = rng.normal(0, 2, (len(counts) + 2, vocab))
    for r, n in enumerate(counts):
        x[r, np.arange(n) * 16 + r] = np.inf             # one a lane while there are lanes
    x[-2, :4 * 40:4] = np.inf
    x[-2, 2100:2100 + 3 * 60:3] = np.inf                 # in two segments
    x[-1, :300] = np.inf                                 # more than a segment hands on
    xd = _cuda(x.astype(np.float32), _dt(dtype))
    short = _cuda(np.full((x.shape[0], 128), np.inf, dtype=np.float32), _dt(dtype))
    u = rng.random(x.shape[0])
    one = np.ones(x.shape[0])
    for t, name in ((xd, "some"), (short, "all")):
        for p in (0.0, 0.1, 0.5, 0.9):
            _check_sample(ert, t, u, f"{dtype} {name} +inf p={p}", top_p=p * one)
            _check_sample(ert, t, u, f"{dtype} {name} +inf p={p} and min-p", top_p=p * one, min_p=0.3 * one)
            _check_sample(ert, t, u, f"{dtype} {name} +inf p={p} and k", top_p=p * one, top_k=[25] * len(u))
        _check_sample(ert, t, u, f"{dtype} {name} +inf k", top_k=[12] * len(u))
        _check_sample(ert, t, u, f"{dtype} {name} +inf min-p", min_p=0.3 * one)


def _check_sample_near(ert, x, u, what, temperature=None, top_k=None, min_p=None):
    """Scores so far down that their weights are a few units of 2^-43, each off
    by up to half a unit, 2^-44: u Z may then lie in any token whose interval
    of the weights' running sum is within vocab * 2^-44 of it, but only in one
    that has a weight of 2^-44 or more, and u = 0 in the first of those alone."""
    host = x.cpu().numpy().astype(np.longdouble)
    rows, vocab = host.shape
    off = np.longdouble(vocab) * np.longdouble(2) ** -44
    kw = {k: _cuda(np.full(rows, v, np.int32 if k == "top_k" else np.float32))
          for k, v in (("temperature", temperature), ("top_k", top_k), ("min_p", min_p)) if v is not None}
    u = np.float32(u)
    for whole in (False, True):
        log(f"[sample] {what} whole_row={whole}")
        tok, lp = ert.sample_tokens(x, _cuda(np.full(rows, u)), return_logprobs=True, whole_row=whole, **kw)
        tok, lp = tok.cpu().numpy(), lp.cpu().numpy()
        for r in range(rows):
            w = np.exp((host[r] - host[r].max()) / np.longdouble(np.float32(temperature or 1.0)))
            w = np.where(w < np.longdouble(2) ** -44, 0, w)
            if top_k is not None:
                w[np.argsort(-host[r], kind="stable")[top_k:]] = 0
            run, t = np.cumsum(w), tok[r]
            y = np.longdouble(u) * run[-1]
            assert w[t] > 0 and run[t] - w[t] - off <= y <= run[t] + off, (what, whole, r, t)
            assert u > 0 or t == np.flatnonzero(w)[0], (what, whole, r, t)
            want = np.log(w[t] / run[-1])
            assert abs(lp[r] - want) <= 2.0 ** -24 * abs(want) * 1.001 + off / run[-1], (what, whole, r, lp[r], want)


@pytest.mark.parametrize("gap", [29.0, 30.0, 31.0, 37.5, 44.0, 60.0])
def test_sample_segments_far_below_the_best(ert, gap):
    # weights of 2^-44 and less are zero, whatever the other scores of their
    # segment: small uniforms draw the first token that has a weight
    vocab = 3 * 2048 + 777
    x = np.zeros((6, vocab))
    x[0, :2048] = -gap                        # a segment of them in front
    x[1, :4096] = -gap                        # two
    x[2, :-1] = -gap                          # all but the last token
    x[3, :5000] = -gap                        # and a segment of both
    x[3, 100] = -3.0
    x[4, :2048] = -gap                        # one of them a little higher
    x[4, 700] = 0.5 - gap
    x[5, 2048:] = -gap                        # behind
    xd = _cuda(x.astype(np.float32))
    for u in (0.0, 2.0 ** -40, 2.0 ** -24, 0.5, 1 - 2.0 ** -24):
        _check_sample_near(ert, xd, u, f"gap={gap} u={u}, no cut")
        _check_sample_near(ert, xd, u, f"gap={gap} u={u}, cold", temperature=0.05)
        _check_sample_near(ert, xd / 16, u, f"gap={gap} u={u}, colder scores", temperature=1 / 16)
        _check_sample_near(ert, xd, u, f"gap={gap} u={u}, min-p that cuts nothing", min_p=1e-30)
        _check_sample_near(ert, xd, u, f"gap={gap} u={u}, top-k of all but one", top_k=vocab - 1)


def test_sample_top_p_beside_a_tail_without_weight(ert):
    # 129024 scores of 2^-45 together weigh 3.7e-9 of the best, as much as one
    # of the 64 tokens among which 1 - top_p = 2^-24 falls; they count nothing
    vocab = 64 * 2048
    x = np.full((2, vocab), -31.2)
    x[:, 1:2048] = NINF
    x[:, 0] = 0.0
    x[:, 1:65] = -19.5
    x[1] = x[1, ::-1]
    p = np.full(2, 1 - 2.0 ** -24)
    for u in (0.0, 0.5, 1 - 2.0 ** -23, 1 - 2.0 ** -24):
        _check_sample(ert, _cuda(x.astype(np.float32)), np.full(2, u), f"tail u={u}", top_p=p)
        _check_sample(ert, _cuda(x.astype(np.float32)), np.full(2, u), f"tail u={u}, no cut")


def test_sample_low_cuts_side_by_side(ert):
    # rows that several workgroups share, in two graphs and eagerly on two
    # streams at once, again and again
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(24, 60001, device="cuda", generator=g)
    u = torch.rand(24, device="cuda", generator=g)
    p = torch.full((24,), 0.9, device="cuda")
    k = torch.randint(1, 30000, (24,), device="cuda", generator=g, dtype=torch.int32)
    want_p, want_k = ert.sample_tokens(x, u, top_p=p).clone(), ert.sample_tokens(x, u, top_k=k).clone()
    torch.cuda.synchronize()
    graphs = []
    for kw in (dict(top_p=p), dict(top_k=k)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ert.sample_tokens(x, u, **kw)
        graphs.append((graph, out))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(a):
            graphs[0][0].replay()
            one = ert.sample_tokens(x, u, top_p=p)
        with torch.cuda.stream(b):
            graphs[1][0].replay()
            two = ert.sample_tokens(x, u, top_k=k)
        three = ert.sample_tokens(x, u, top_p=p)
        torch.cuda.synchronize()
        for got, want in ((one, want_p), (three, want_p), (graphs[0][1], want_p), (two, want_k),
                          (graphs[1][1], want_k)):
            assert torch.equal(got, want)


def test_sample_both_low_cuts_and_crowds_side_by_side(ert):
    # the same with both cuts, and rows in which one value is crowded
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    x = (torch.randn(20, 50003, device="cuda", generator=g) * 2 - 25).bfloat16()
    x[3] = 0.5
    x[4, ::2] = 1.0
    u = torch.rand(20, device="cuda", generator=g)
    p = torch.full((20,), 0.9, device="cuda")
    k = torch.randint(3, 30000, (20,), device="cuda", generator=g, dtype=torch.int32)
    calls = [dict(top_p=p), dict(top_k=k), dict(top_k=k, top_p=p)]
    want = [ert.sample_tokens(x, u, whole_row=True, **kw).clone() for kw in calls]
    torch.cuda.synchronize()
    graphs = []
    for kw in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = ert.sample_tokens(x, u, **kw)
        graphs.append((graph, out))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(4):
        eager = []
        for stream, kw, (graph, _) in zip(streams, calls, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
                eager.append(ert.sample_tokens(x, u, **kw))
        torch.cuda.synchronize()
        for got, (_, out), right in zip(eager, graphs, want):
            assert torch.equal(got, right) and torch.equal(out, right)


def test_sample_outputs_given_and_empty_batch(ert):
    import torch
    x = torch.randn(4, 999, device="cuda")
    u = torch.rand(4, device="cuda")
    tok = torch.full((4,), -9, dtype=torch.int32, device="cuda")
    lp = torch.full((4,), -9.0, device="cuda")
    got = ert.sample_tokens(x, u, tokens=tok, logprobs=lp)
    assert got[0] is tok and got[1] is lp
    assert torch.equal(tok, ert.sample_tokens(x, u))
    empty = ert.sample_tokens(x[:0], u[:0], return_logprobs=True)
    assert empty[0].shape == (0,) and empty[1].shape == (0,)


def test_sample_follows_the_distribution(ert):
    # a grid of uniforms draws each token as often as its weight says, to one
    # grid step
    import torch
    p = np.array([0.4, 0.1, 0.25, 0.05, 0.2])
    n = 4000
    x = _cuda(np.tile(np.log(p), (n, 1)).astype(np.float32))
    u = (torch.arange(n, device="cuda") + 0.5) / n
    tok = ert.sample_tokens(x, u).cpu().numpy()
    assert np.all(np.abs(np.bincount(tok, minlength=5) - n * p) <= 1.0 + 1e-3)
    assert np.all(np.diff(tok) >= 0)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def _check_route(ert, x, top_k, what, bias=None, **kw):
    """Experts equal the definition's; weights to one fp32 rounding (2^-24)
    beside 64-bit arithmetic (1e-12)."""
    import torch
    log(f"[route] {what}")
    host = x.float().cpu().numpy()
    names = {"num_groups": "groups"}
    want = [ref.route_token(host[t], top_k, bias=bias,
                            **{names.get(k, k): v for k, v in kw.items()})
            for t in range(host.shape[0])]
    b = _cuda(np.asarray(bias, dtype=np.float32)) if bias is not None else None
    idx, w = ert.route_experts(x, top_k, bias=b, **kw)
    torch.cuda.synchronize()
    idx, w = idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    for t, (wi, ww) in enumerate(want):
        assert np.array_equal(idx[t], wi), (what, t, idx[t], wi)
        assert np.all(np.abs(w[t] - ww) <= np.abs(ww) * (2.0 ** -24 + 1e-12) + 2.0 ** -149), (what, t, w[t], ww)


ROUTE_SHAPES = [(1, 1, 1, 1), (2, 2, 1, 1), (8, 2, 1, 1), (8, 3, 4, 2), (60, 6, 1, 1), (64, 8, 8, 3),
                (63, 5, 3, 2), (128, 8, 1, 1), (160, 6, 8, 3), (255, 16, 5, 5), (256, 8, 8, 4),
                (257, 4, 1, 1), (384, 8, 1, 1), (472, 13, 8, 7), (512, 10, 16, 2), (1024, 64, 2, 1)]


@pytest.mark.parametrize("experts,top_k,groups,topk_groups", ROUTE_SHAPES)
def test_route_shapes(ert, experts, top_k, groups, topk_groups):
    rng = np.random.default_rng([experts, top_k])
    for scoring, with_bias, renorm, dtype in itertools.product(
            ("softmax", "sigmoid"), (False, True), (False, True), ("fp32", "bf16")):
        tokens = int(rng.integers(1, 23))
        x = _cuda(rng.normal(0, 1.5, (tokens, experts)).astype(np.float32), _dt(dtype))
        bias = rng.normal(0, 0.1, experts).astype(np.float32) if with_bias else None
        for gs in (("max", "top2") if groups > 1 else ("max",)):
            _check_route(ert, x, top_k, f"E={experts} k={top_k} {scoring} bias={with_bias} "
                         f"renorm={renorm} {dtype} {gs}", bias=bias, scoring=scoring,
                         num_groups=groups, topk_groups=topk_groups, group_score=gs,
                         renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_ties_masks_and_extremes(ert, scoring):
    rng = np.random.default_rng(6)
    E = 64
    rows = [np.zeros(E), rng.integers(-2, 3, E).astype(float), np.full(E, NINF), np.full(E, np.nan)]
    few = np.full(E, NINF); few[[3, 40, 41]] = [0.5, 2.0, 2.0]; rows.append(few)
    half = rng.normal(0, 1, E); half[::2] = NINF; half[1] = np.nan; rows.append(half)
    rows.append(np.full(E, -200.0)); rows.append(np.full(E, 90.0))
    rows.append(np.linspace(-87, 88, E)); rows.append(np.full(E, np.finfo(np.float32).min))
    inf = rng.normal(0, 1, E); inf[[5, 6]] = np.inf; rows.append(inf)
    near = 1.0 + np.arange(E) * 2.0 ** -23; rows.append(near)
    rows.append(near[::-1].copy())
    x = _cuda(np.array(rows, dtype=np.float32))
    equal = np.full(E, 0.25, dtype=np.float32)
    masked = rng.normal(0, 0.1, E).astype(np.float32); masked[[0, 9]] = NINF; masked[11] = np.nan
    for bias, (groups, tg), renorm in itertools.product((None, equal, masked),
                                                        ((1, 1), (8, 2)), (False, True)):
        for gs in (("max", "top2") if groups > 1 else ("max",)):
            _check_route(ert, x, 8, f"special {scoring} bias={bias is not None} groups={groups} {gs} "
                         f"renorm={renorm}", bias=bias, scoring=scoring, num_groups=groups,
                         topk_groups=tg, group_score=gs, renormalize=renorm)


def test_route_bias_keeps_the_largest_out(ert):
    # the chosen lie so far below the token's largest logit that their shares
    # of the whole softmax are zero in 64 bits; divided by their sum they are not
    rng = np.random.default_rng(31)
    x = rng.normal(0, 1, (40, 64)).astype(np.float32)
    x[:, 5] = np.linspace(600, 3000, 40)
    bias = np.zeros(64, dtype=np.float32)
    bias[5] = -4.0
    for renormalize in (True, False):
        for top_k in (1, 6, 40):
            idx, w = ert.route_experts(_cuda(x), top_k, bias=_cuda(bias), renormalize=renormalize)
            for t in range(40):
                want, ww = ref.route_token(x[t], top_k, "softmax", bias, renormalize=renormalize)
                assert np.array_equal(idx[t].cpu().numpy(), want)
                got = w[t].cpu().numpy()
                # one rounding to float32 (of 64-bit shares good to 2^-44), half the least number below its normal range
                assert np.all(np.abs(got - ww) <= 2.0 ** -24 * (1 + 1e-5) * np.abs(ww) + 2.0 ** -150)
                assert not renormalize or abs(got.sum(dtype=np.float64) - 1) < 1e-5


def test_route_many_tokens_strided_and_tied(ert):
    import torch
    rng = np.random.default_rng(7)
    for dtype, experts, pad in (("bf16", 256, 3), ("fp32", 128, 1), ("fp16", 320, 0)):
        buf = torch.full((1111, experts + pad), float("inf"), device="cuda", dtype=_dt(dtype))
        x = buf[:, :experts]
        x.copy_(_cuda(rng.normal(0, 1, (1111, experts)).astype(np.float32), _dt(dtype)))
        _check_route(ert, x, 8, f"many {dtype} zero bias", bias=np.zeros(experts, np.float32),
                     scoring="sigmoid", num_groups=8, topk_groups=4, group_score="top2")
        _check_route(ert, x, 6, f"many {dtype} no bias", scoring="softmax", renormalize=False)


def test_route_fewer_experts_than_asked_for(ert):
    # the groups that stay hold fewer experts than top_k
    rng = np.random.default_rng(17)
    x = _cuda(rng.normal(0, 1, (9, 64)).astype(np.float32))
    bias = rng.normal(0, 0.1, 64).astype(np.float32)
    for b in (None, bias):
        _check_route(ert, x, 16, "two groups of four for sixteen", bias=b, scoring="sigmoid",
                     num_groups=16, topk_groups=2, group_score="top2")
        _check_route(ert, x, 64, "all of them", bias=b, scoring="softmax")


def test_route_near_ties(ert):
    # scores a few 2^-24 apart, and sigmoids that 32 bits cannot tell apart
    rng = np.random.default_rng(18)
    E = 256
    base = rng.normal(0, 1, (40, E)).astype(np.float32)
    base[:, 100:160] = (np.float32(2.0) + np.arange(60, dtype=np.float32) * 2.0 ** -22)[rng.permutation(60)]
    base[20:, 30:60] = 17.0 + rng.random((20, 30)).astype(np.float32) * 12
    for scoring, b in itertools.product(("sigmoid", "softmax"),
                                        (np.zeros(E, np.float32), np.full(E, -3.0, np.float32))):
        _check_route(ert, _cuda(base), 12, f"near ties {scoring}", bias=b, scoring=scoring,
                     num_groups=8, topk_groups=5, group_score="top2")
        _check_route(ert, _cuda(base), 12, f"near ties {scoring}, one group", bias=b, scoring=scoring)


@pytest.mark.parametrize("experts,groups,topk_groups", [(256, 8, 4), (64, 4, 2), (60, 6, 3), (512, 16, 7), (48, 16, 5)])
def test_route_near_group_borders(ert, experts, groups, topk_groups):
    # group scores that are equal, a few 2^-24 apart, or clear; of two, several
    # and all groups; groups with one live expert and with none
    rng = np.random.default_rng([experts, groups])
    size = experts // groups
    T = 96
    x = rng.normal(-2, 0.5, (T, experts)).astype(np.float32)
    for t in range(T):
        near = rng.permutation(groups)[:2 + t % groups] if t % 3 else np.arange(groups)
        for g in range(groups):
            lead = 1.5 if g in near else rng.choice([0.5, 1.0, 2.0, 2.5])
            a, b = rng.permutation(size)[:2]
            step = 2.0 ** -22 * rng.integers(0, 3, 2)
            x[t, g * size + a] = np.float32(lead + step[0])
            x[t, g * size + b] = np.float32(lead - 0.25 * (t % 2) + step[1])
        if t % 5 == 0:
            g = rng.integers(groups)
            x[t, g * size:(g + 1) * size - 1] = NINF
        if t % 7 == 0:
            x[t, :size] = NINF
    bias = (rng.integers(0, 2, experts) * 2.0 ** -23).astype(np.float32)
    for scoring, how in itertools.product(("sigmoid", "softmax"), ("max", "top2")):
        for b in (bias, np.zeros(experts, np.float32)):
            _check_route(ert, _cuda(x), min(8, topk_groups * size), f"group borders {scoring} {how}", bias=b,
                         scoring=scoring, num_groups=groups, topk_groups=topk_groups, group_score=how)
    _check_route(ert, _cuda(x, _dt("bf16")), 4, "group borders bf16", bias=bias, scoring="sigmoid",
                 num_groups=groups, topk_groups=topk_groups, group_score="top2")


def _check_grad(ert, x, idx, g, what, **kw):
    """One fp32 rounding of each of at most three terms (3 * 2^-24 of their
    size), then one rounding to the output type (half a step, or half the
    smallest subnormal)."""
    import torch
    log(f"[route grad] {what}")
    host = x.float().cpu().numpy()
    got = ert.route_experts_backward(_cuda(g.astype(np.float32)), x, _cuda(idx.astype(np.int32)), **kw)
    torch.cuda.synchronize()
    fi = torch.finfo(x.dtype)
    got = got.double().cpu().numpy()
    assert got.shape == host.shape
    for t in range(host.shape[0]):
        want, size = ref.route_grad_token(host[t], idx[t], g[t].astype(np.float32).astype(np.float64), **kw)
        tol = size * (3 * 2.0 ** -24 + 1e-12) * (1 + fi.eps) + np.abs(want) * fi.eps / 2 \
            + fi.smallest_normal * fi.eps / 2 + 2.0 ** -149
        bad = np.flatnonzero(~(np.abs(got[t] - want) <= tol))
        assert bad.size == 0, (what, t, bad[:4], got[t][bad[:4]], want[bad[:4]])


@pytest.mark.parametrize("experts,top_k,groups,topk_groups", ROUTE_SHAPES)
def test_route_gradient(ert, experts, top_k, groups, topk_groups):
    rng = np.random.default_rng([experts, top_k, 1])
    for scoring, renorm, dtype in itertools.product(("softmax", "sigmoid"), (False, True),
                                                    ("fp32", "bf16", "fp16")):
        tokens = int(rng.integers(1, 23))
        x = _cuda(rng.normal(0, 1.5, (tokens, experts)).astype(np.float32), _dt(dtype))
        idx = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)])
        _check_grad(ert, x, idx, rng.normal(0, 1, (tokens, top_k)), f"E={experts} k={top_k} "
                    f"{scoring} renorm={renorm} {dtype}", scoring=scoring, renormalize=renorm, scale=1.5)


def test_route_gradient_masks_repeats_and_extremes(ert):
    rng = np.random.default_rng(8)
    E, K = 48, 4
    x = rng.normal(0, 1, (8, E)).astype(np.float32)
    x[0] = NINF
    x[1] = np.nan
    x[2, 5:] = NINF
    x[3] = -300.0
    x[4] = 95.0
    x[5] = np.linspace(-90, 90, E)
    idx = np.array([[-1] * 4, [-1] * 4, [0, 3, -1, -1], [1, 2, 3, 4], [7, 6, 5, 4], [0, 47, 24, 10],
                    [9, 9, 9, 2], [3, E, -7, 3]])
    g = rng.normal(0, 1, (8, K))
    for scoring, renorm, dtype in itertools.product(("softmax", "sigmoid"), (False, True), ("fp32", "bf16")):
        _check_grad(ert, _cuda(x, _dt(dtype)), idx, g, f"special {scoring} {renorm} {dtype}",
                    scoring=scoring, renormalize=renorm, scale=0.7)


def _sure_gradient(x, idx, g, scoring, renormalize, scale):
    """One token's gradient in extended precision, the size of the terms that
    cancel in it, and the size of what is left of them."""
    LD = np.longdouble
    x, g = x.astype(LD), g.astype(LD)
    live = x > -np.inf
    if scoring == "sigmoid":
        s, other = np.where(live, 1 / (1 + np.exp(-x)), 0), 1 / (1 + np.exp(x))
    else:
        s = np.where(live, np.exp(x - x[live].max()), 0)
        s = s / s.sum()
    ok = [(j, e) for j, e in enumerate(idx) if e >= 0 and live[e]]
    total = sum(s[e] for _, e in ok) if renormalize else LD(1)
    out, terms, rest = (np.zeros(x.size, LD) for _ in range(3))
    if scoring == "sigmoid" and not renormalize:
        for j, e in ok:
            out[e] += g[j] * s[e] * other[e]
        return out * scale, abs(out) * 0, abs(out) * scale
    share = {j: s[e] / total for j, e in ok}
    mean = sum(g[j] * share[j] for j, _ in ok)
    size = sum(abs(g[j]) * share[j] for j, _ in ok)
    for j, e in ok:
        out[e] += share[j] * (g[j] - mean * renormalize)
        terms[e] += share[j] * (abs(g[j]) + size)
        rest[e] += share[j] * (abs(g[j]) * (1 - share[j]) + size - share[j] * abs(g[j]))
    if not renormalize:
        out -= s * mean
        chosen = np.isin(np.arange(x.size), [e for _, e in ok])
        terms += np.where(chosen, 0, s * size)
        rest += np.where(chosen, 0, s * size)
    if scoring == "sigmoid":
        out, terms, rest = (v * other for v in (out, terms, rest))
    return out * scale, terms * scale, rest * scale


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_route_gradient_of_a_sure_choice(ert, dtype):
    # s_e (g_e - sum_j g_j s_j) where the two nearly cancel: a chosen expert
    # with nearly all of the mass, alone and beside others, with equal
    # gradients, named twice.  Sums, products and quotients of 64 bits: at most
    # 32 roundings of 2^-53 of the terms; exponentials good to 2^-45, four of
    # them in what the terms leave; then a rounding to float32 and one to the
    # output's type.
    import torch
    rng = np.random.default_rng(43)
    E, rows = 40, 24
    x = rng.normal(0, 1, (rows, E))
    x[:, 7] += np.linspace(4, 30, rows)
    x[0] = NINF
    x[0, :5] = [20, 0, 0, 0, -1]
    idx = np.tile(np.array([7, 3, 30, 12]), (rows, 1))
    idx[0] = [0, 1, 2, 3]
    idx[5:9, 1:] = -1                                      # the sure one alone
    idx[9:12, 1] = 7                                       # named twice
    g = rng.normal(0, 1, (rows, 4)).astype(np.float32)
    g[12:15] = 1.2345
    g[9:12, 1] = -g[9:12, 0] * np.float32(1 + 2.0 ** -20)
    xd = _cuda(x.astype(np.float32), _dt(dtype))
    host = xd.double().cpu().numpy()
    fi = torch.finfo(xd.dtype)
    for scoring, renorm in itertools.product(("softmax", "sigmoid"), (False, True)):
        kw = dict(scoring=scoring, renormalize=renorm, scale=1.75)
        log(f"[route grad] sure choice {dtype} {kw}")
        got = ert.route_experts_backward(_cuda(g), xd, _cuda(idx.astype(np.int32)), **kw).double().cpu().numpy()
        for t in range(rows):
            want, terms, rest = _sure_gradient(host[t], idx[t], g[t], **kw)
            tol = np.abs(want) * (2.0 ** -24 + fi.eps / 2 * (1 + 2.0 ** -23)) + terms * 2.0 ** -48 \
                + rest * 2.0 ** -43 + fi.smallest_normal * fi.eps / 2 + 2.0 ** -149
            bad = np.flatnonzero(~(np.abs(got[t] - want) <= tol))
            assert bad.size == 0, (dtype, kw, t, bad[:4], got[t][bad[:4]], want[bad[:4]])


@pytest.mark.parametrize("scoring,renorm", itertools.product(("softmax", "sigmoid"), (False, True)))
def test_route_gradient_against_differences(ert, scoring, renorm):
    # central differences of the 64-bit definition: their own error is about
    # h^2 = 1e-10 and 1e-16 / h = 1e-11
    import torch
    rng = np.random.default_rng(9)
    x = rng.normal(0, 1, (3, 24)).astype(np.float32)
    g = rng.normal(0, 1, (3, 5)).astype(np.float32)
    xd = _cuda(x).requires_grad_()
    idx, w = ert.route_experts(xd, 5, scoring=scoring, renormalize=renorm, scale=1.25)
    assert w.requires_grad and not idx.requires_grad
    w.backward(_cuda(g))
    got = xd.grad.double().cpu().numpy()
    idx = idx.cpu().numpy()
    h = 1e-5
    for t in range(3):
        for e in range(24):
            hi, lo = x[t].astype(np.float64), x[t].astype(np.float64)
            hi[e] += h
            lo[e] -= h
            d = (ref.weights_of(hi, idx[t], scoring, renorm, 1.25) -
                 ref.weights_of(lo, idx[t], scoring, renorm, 1.25)) / (2 * h)
            assert abs((d * g[t]).sum() - got[t, e]) <= 1e-6


def test_route_sigmoids_at_the_end_of_64_bits(ert):
    # scores on both sides of 2^-1022 (logits of -708.4), below which they
    # count as zero: weights are shares of what is left, never inf or NaN
    LD = np.longdouble
    rng = np.random.default_rng(47)
    E, K = 16, 4
    at = [-700.0, -707.5, -708.0, -709.0, -709.8, -712.0, -730.0, -744.0, -746.0, -800.0]
    x = np.array([a + rng.uniform(-0.2, 0.2, E) for a in at] +
                 [np.linspace(-712, -704, E), np.linspace(-745, -708.6, E)]).astype(np.float32)
    g = rng.normal(0, 1, (len(x), K)).astype(np.float32)
    # an exponential of 64 bits is good to 2^-45, its argument to 2^-43 of 1022
    rel = 2.0 ** -24 + 2.0 ** -32
    for bias in (None, np.full(E, 0.5, np.float32)):
        xd = _cuda(x).requires_grad_()
        idx, w = ert.route_experts(xd, K, scoring="sigmoid", bias=None if bias is None else _cuda(bias))
        w.backward(_cuda(g))
        idx, w, dx = idx.cpu().numpy(), w.detach().cpu().numpy(), xd.grad.cpu().numpy()
        assert np.isfinite(w).all() and np.isfinite(dx).all()
        for t in range(len(x)):
            s = np.exp(x[t].astype(LD))
            s = np.where(s < LD(2.0) ** -1022, LD(0), s)
            if bias is None:
                assert np.array_equal(idx[t], np.argsort(-x[t], kind="stable")[:K])
            own = s[idx[t]]
            total = own.sum()
            share = own / total if total > 0 else own
            assert np.all(np.abs(w[t] - share) <= rel * share + 2.0 ** -149), (t, w[t], share)
            want = np.zeros(E, LD)
            mean = (g[t].astype(LD) * share).sum()
            want[idx[t]] = share * (g[t] - mean)
            size = np.zeros(E, LD)
            size[idx[t]] = share * (np.abs(g[t]) + abs(mean))
            assert np.all(np.abs(dx[t] - want) <= rel * np.abs(want) + 2.0 ** -32 * size + 2.0 ** -149), (t, dx[t], want)


def test_route_autograd_broadcast_gradient_and_refusals(ert):
    import torch
    x = torch.randn(33, 40, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    idx, w = ert.route_experts(x, 3, scoring="sigmoid", scale=2.0, renormalize=False)
    w.sum().backward()                       # the gradient comes as a broadcast one
    want = ert.route_experts_backward(torch.ones(33, 3, device="cuda"), x.detach(), idx,
                                      scoring="sigmoid", scale=2.0, renormalize=False)
    assert torch.equal(x.grad, want)
    with torch.no_grad():
        assert not ert.route_experts(x, 3)[1].requires_grad
    with pytest.raises(ValueError):
        ert.route_experts(x, 3, stream=torch.cuda.current_stream())
    _, w = ert.route_experts(x, 3)
    gx, = torch.autograd.grad(w.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.float().sum().backward()          # no second derivative


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_beyond_32_bit_offsets(ert, dtype):
    # rows whose elements lie more than 2^31 apart from the first
    import torch
    rng = np.random.default_rng(53)
    stride, rows = (1 << 30) + 24, 4
    buf = torch.empty((rows - 1) * stride + 8192, dtype=_dt(dtype), device="cuda")
    u = rng.random(rows)
    x = buf.as_strided((rows, 5003), (stride, 1))
    x.copy_(_cuda(rng.normal(0, 2, (rows, 5003)).astype(np.float32)))
    one = np.ones(rows)
    _check_sample(ert, x, u, f"{dtype} far rows")
    _check_sample(ert, x, u, f"{dtype} far rows, cuts", top_k=[50, 0, 3000, 7], top_p=0.9 * one)
    y = buf.as_strided((rows, 96), (stride, 1), 3)
    bias = rng.normal(0, 0.1, 96).astype(np.float32)
    near = y.contiguous()
    assert all(torch.equal(a, b) for a, b in zip(
        ert.route_experts(y, 6, scoring="sigmoid", bias=_cuda(bias), num_groups=4, topk_groups=2),
        ert.route_experts(near, 6, scoring="sigmoid", bias=_cuda(bias), num_groups=4, topk_groups=2)))
    idx = _cuda(np.stack([rng.permutation(96)[:6] for _ in range(rows)]).astype(np.int32))
    g = _cuda(rng.normal(0, 1, (rows, 6)).astype(np.float32))
    for renorm in (False, True):
        assert torch.equal(ert.route_experts_backward(g, y, idx, renormalize=renorm),
                           ert.route_experts_backward(g, near, idx, renormalize=renorm))


# ---------------------------------------------------------------------------
# block tables and slots
# ---------------------------------------------------------------------------

def _check_tables(ert, kv, new, bs, what, width=None, num_free=None, start=0, max_tokens=None,
                  wide=False, pad=0, block_base=0, seed=0):
    import torch
    log(f"[tables] {what}")
    rng = np.random.default_rng([seed, len(kv), bs])
    kv, new = np.asarray(kv, np.int32), np.asarray(new, np.int32)
    R = kv.size
    c = np.maximum(kv, 0).astype(np.int64)
    a = np.minimum(np.maximum(new, 0), c)
    need = -(-c // bs)
    width = int(need.max(initial=0)) + 2 if width is None else width
    total_new = int((need - (-(-(c - a) // bs))).sum())
    num_free = total_new + start + 3 if num_free is None else num_free
    ids = (rng.permutation(R * width + num_free) + block_base).astype(np.int32)
    tables = np.full((R, width + pad), -77, np.int32)
    tables[:, :width] = ids[:R * width].reshape(R, width)
    free = ids[R * width:]
    max_tokens = int(a.sum()) + 5 if max_tokens is None else max_tokens
    td = _cuda(tables)
    view = td[:, :width]
    got = ert.extend_block_tables(view, _cuda(kv), _cuda(new), _cuda(free),
                                  torch.tensor([start], dtype=torch.int32, device="cuda"), bs,
                                  max_tokens, slot_dtype=torch.int64 if wide else None)
    torch.cuda.synchronize()
    want = ref.extend_tables(tables[:, :width], kv, new, free, start, bs, max_tokens, wide)
    names = ("token_starts", "token_requests", "positions", "slots")
    assert np.array_equal(view.cpu().numpy(), want[0]), what
    if pad:
        assert (td[:, width:] == -77).all(), "columns behind the table were written"
    for name, g, w in zip(names, got[:4], want[1:5]):
        assert np.array_equal(g.cpu().numpy(), w), (what, name)
    assert int(got[4]) == want[5], what


@pytest.mark.parametrize("bs", [1, 3, 16, 48, 64])
def test_tables_lengths(ert, bs):
    rng = np.random.default_rng(bs)
    kv = [0, 1, bs, bs + 1, 2 * bs - 1, 2 * bs, 500, 513, 64, 0, 7]
    _check_tables(ert, kv, kv, bs, f"whole prompts bs={bs}")
    _check_tables(ert, kv, [1] * len(kv), bs, f"one new each bs={bs}", pad=3)
    _check_tables(ert, kv, [0] * len(kv), bs, f"nothing new bs={bs}")
    _check_tables(ert, kv, rng.integers(0, 9, len(kv)), bs, f"some new bs={bs}", start=4, wide=True)
    _check_tables(ert, [-5, 10, 3], [4, 99, -2], bs, f"lengths out of range bs={bs}")


@pytest.mark.parametrize("requests", [0, 1, 2, 255, 256, 257, 1000, 4096])
def test_tables_request_counts(ert, requests):
    rng = np.random.default_rng(requests)
    kv = rng.integers(0, 90, requests)
    _check_tables(ert, kv, np.minimum(kv, rng.integers(0, 60, requests)), 16,
                  f"{requests} requests", start=11)


def test_tables_long_short_lists_and_narrow_tables(ert):
    _check_tables(ert, [70000, 3, 40001], [70000, 3, 20000], 16, "long prompts")
    _check_tables(ert, [300001, 0, 5, 70002], [300001, 0, 5, 70002], 48, "four tokens a thread")
    _check_tables(ert, [300001, 7, 5, 70002], [300001, 7, 0, 70002], 64, "four tokens a thread, wide",
                  wide=True, max_tokens=370003)
    _check_tables(ert, [100, 200, 300], [100, 50, 300], 16, "free list too short", num_free=9)
    _check_tables(ert, [100, 200, 300], [100, 50, 300], 16, "free list used up", num_free=9, start=20)
    _check_tables(ert, [100, 200, 300], [100, 50, 300], 16, "no free list", num_free=0)
    _check_tables(ert, [100, 200, 300], [100, 50, 300], 16, "table too narrow", width=5)
    _check_tables(ert, [100, 200, 300], [100, 50, 300], 16, "more tokens than places", max_tokens=77)
    _check_tables(ert, [100, 200], [100, 200], 16, "no places", max_tokens=0)
    _check_tables(ert, [100, 200], [100, 200], 16, "padding behind", max_tokens=9000)
    # slots on both sides of 2^31
    for wide in (False, True):
        _check_tables(ert, [300, 5000], [300, 4000], 64, f"far blocks wide={wide}",
                      block_base=(1 << 25) - 60, wide=wide)


@pytest.mark.parametrize("k,bs,next_n,wide", [(512, 64, 1, False), (1024, 16, 3, False), (2048, 48, 2, True),
                                              (1, 1, 1, False), (7, 5, 4, True), (1000, 64, 1, False)])
def test_slots(ert, k, bs, next_n, wide):
    import torch
    rng = np.random.default_rng([k, bs])
    rows = 10
    R, width = (rows + next_n - 1) // next_n, 40
    tables = rng.permutation(R * width).reshape(R, width).astype(np.int32)
    tables[0, 3] = -1
    idx = rng.integers(-1, width * bs, (rows, k)).astype(np.int32)
    idx[1, :] = -1
    idx[2, 0] = width * bs            # past the table
    idx[3, 0] = 2 ** 31 - 1
    owner = np.arange(rows) // next_n
    dt = torch.int64 if wide else torch.int32
    got = ert.topk_slots(_cuda(idx), _cuda(tables), bs, next_n=next_n, slot_dtype=dt)
    assert got.dtype == dt
    assert np.array_equal(got.cpu().numpy(), ref.slots_of(idx, tables, bs, owner, wide))
    owner = rng.integers(-1, R + 1, rows).astype(np.int32)   # requests outside the tables too
    own = _cuda(idx)
    got = ert.topk_slots(own, _cuda(tables), bs, row_requests=_cuda(owner), slot_dtype=dt,
                         slots=None if wide else own)
    assert np.array_equal(got.cpu().numpy(), ref.slots_of(idx, tables, bs, owner, wide))
    if not wide:
        assert got is own


@pytest.mark.parametrize("bs", [1, 2, 3, 5, 7, 48, 100, 641, 65537, 1 << 20, (1 << 30) - 1, 1 << 30])
def test_slots_block_sizes(ert, bs):
    # quotients over the whole range of positions, in and out of the table
    import torch
    rng = np.random.default_rng(bs)
    width = 37
    edge = np.array([q * bs + o for q in range(width + 1) for o in (-1, 0, 1)], dtype=np.int64)
    far = np.concatenate([edge, rng.integers(0, 2 ** 31, 500), [2 ** 31 - 1, 0]])
    idx = far[(far >= 0) & (far < 2 ** 31)].astype(np.int32)[None, :]
    tables = rng.permutation(width).astype(np.int32)[None, :]
    got = ert.topk_slots(_cuda(idx), _cuda(tables), bs, slot_dtype=torch.int64)
    assert np.array_equal(got.cpu().numpy(), ref.slots_of(idx, tables, bs, [0], True))


def test_slots_many_rows(ert):
    # enough rows for the staged tables, rows over several workgroups
    rng = np.random.default_rng(19)
    for rows, k, width in ((1200, 512, 300), (700, 2048, 64), (1030, 1001, 900), (600, 1024, 512),
                           (1030, 1001, 500), (512, 513, 256), (300, 5000, 77)):
        tables = rng.permutation(20 * width).reshape(20, width).astype(np.int32)
        idx = rng.integers(-1, width * 16 + 5, (rows, k)).astype(np.int32)
        owner = rng.integers(0, 20, rows).astype(np.int32)
        got = ert.topk_slots(_cuda(idx), _cuda(tables), 16, row_requests=_cuda(owner)).cpu().numpy()
        at = idx.astype(np.int64)
        ok = (at >= 0) & (at < width * 16)
        want = np.where(ok, tables[owner[:, None], np.where(ok, at // 16, 0)].astype(np.int64) * 16 + at % 16, -1)
        assert np.array_equal(got, want)


def test_slots_of_the_longest_rows(ert):
    # a row of nearly 2^31 positions, written over its indices
    import torch
    n = 2 ** 31 - 701
    idx = torch.arange(n, dtype=torch.int32, device="cuda")
    idx[5] = -1
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    tables = torch.randperm(2048, device="cuda", generator=g).to(torch.int32)[None, :]
    got = ert.topk_slots(idx[None, :], tables, 1 << 20, slots=idx[None, :])[0]
    off = torch.arange(1 << 20, dtype=torch.int32, device="cuda")
    assert int(got[5]) == -1
    got[5] = (int(tables[0, 0]) << 20) + 5
    for b in range(2048):
        own = got[b << 20:(b + 1) << 20]
        assert torch.equal(own, off[:own.numel()] + (int(tables[0, b]) << 20)), b


def test_slots_strided_tables_far_blocks_and_empty(ert):
    import torch
    tables = np.array([[1 << 25, (1 << 25) - 1, 5], [0, 2 ** 31 - 1, 7]], np.int32)
    big = torch.full((2, 9), 3, dtype=torch.int32, device="cuda")
    big[:, :3] = _cuda(tables)
    idx = np.array([[0, 63, 64, 127, 128, -1], [1, 64, 70, 191, 192, 0]], np.int32)
    for wide in (False, True):
        got = ert.topk_slots(_cuda(idx), big[:, :3], 64, slot_dtype=torch.int64 if wide else torch.int32)
        assert np.array_equal(got.cpu().numpy(), ref.slots_of(idx, tables, 64, [0, 1], wide))
    none = ert.topk_slots(_cuda(idx)[:0], big, 64)
    assert none.shape == (0, 6)


def test_binding_names_what_is_missing(ert):
    import torch
    def z(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")
    given = [z(3, 4), z(3), z(3), z(5), z(1)]
    for at, wrong in itertools.product(range(5), (None, [1, 2, 3], 7)):
        args = list(given)
        args[at] = wrong
        with pytest.raises(TypeError):
            ert.extend_block_tables(*args, 16, 4)
    for wrong in (z(3, 4)[:, :1], z(2, 2), torch.zeros((), dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            ert.extend_block_tables(*given[:3], wrong, given[4], 16, 4)
    with pytest.raises(TypeError):
        ert.extend_block_tables(*given[:3], z(5).float(), given[4], 16, 4)
    with pytest.raises(ValueError):
        ert.extend_block_tables(*given[:3], z(5).cpu(), given[4], 16, 4)


# ---------------------------------------------------------------------------
# streams, graphs, and the operators together
# ---------------------------------------------------------------------------

def _step(ert, s):
    """A decode step's choices: slots for the new tokens, the selection, its
    slots, the experts, the next token."""
    starts, owner, pos, slots, nxt = ert.extend_block_tables(
        s["tables"], s["kv"], s["new"], s["free"], s["start"], 64, s["kv"].shape[0] * s["next_n"])
    sel = ert.topk_decode_varlen(s["scores"], s["kv"], 512, next_n=s["next_n"], workspace=s["ws"],
                                 sorted=True, deterministic=True)
    where = ert.topk_slots(sel, s["tables"], 64, next_n=s["next_n"])
    experts, weights = ert.route_experts(s["router"], 4, scoring="sigmoid", bias=s["bias"],
                                         num_groups=4, topk_groups=2, group_score="top2")
    token, lp = ert.sample_tokens(s["logits"], s["u"], temperature=s["t"], top_k=s["k"],
                                  top_p=s["p"], min_p=s["m"], return_logprobs=True)
    return [starts, owner, pos, slots, nxt, sel, where, experts, weights, token, lp, s["tables"]]


def _step_state(ert, seed, requests=6, next_n=2):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rows = requests * next_n
    def rand(*shape):
        return torch.rand(*shape, device="cuda", generator=g)
    kv = torch.tensor([3, 64, 640, 2047, 4000, 1000][:requests], dtype=torch.int32, device="cuda") + seed
    ids = torch.randperm(requests * 70 + 64, device="cuda", generator=g).to(torch.int32)
    tables = ids[:requests * 70].view(requests, 70).clone()
    return {"kv": kv, "new": torch.full((requests,), next_n, dtype=torch.int32, device="cuda"),
            "tables": tables, "free": ids[requests * 70:].clone(), "next_n": next_n,
            "start": torch.tensor([seed % 5], dtype=torch.int32, device="cuda"),
            "scores": torch.randn(rows, 4096, device="cuda", generator=g),
            "ws": ert.new_workspace(rows, 4096, 512),
            "router": torch.randn(rows, 64, device="cuda", generator=g).bfloat16(),
            "bias": torch.randn(64, device="cuda", generator=g) * 0.05,
            "logits": (torch.randn(rows, 9001, device="cuda", generator=g) * 2).half(),
            "u": rand(rows), "t": rand(rows) + 0.3,
            "k": torch.randint(0, 90, (rows,), device="cuda", generator=g, dtype=torch.int32),
            "p": rand(rows) * 0.3 + 0.7, "m": rand(rows) * 0.05}


def _check_step(s, out):
    host = {k: v.float().cpu().numpy() if v.is_floating_point() else v.cpu().numpy()
            for k, v in s.items() if hasattr(v, "cpu")}
    o = [t.cpu().numpy() for t in out]
    rows, n = host["scores"].shape[0], s["next_n"]
    for r in range(rows):
        kv = int(host["kv"][r // n])
        nv = min(kv - n + r % n + 1, 4096) if kv >= n else 0
        x = host["scores"][r, :nv]
        want = np.argsort(-x, kind="stable")[:512] if nv > 512 else np.arange(nv)
        assert np.array_equal(o[5][r, :want.size], want) and (o[5][r, want.size:] == -1).all()
        assert np.array_equal(o[7][r], ref.route_token(host["router"][r], 4, "sigmoid", host["bias"],
                                                       4, 2, "top2")[0])
        assert o[9][r] == ref.sample_row(host["logits"][r], host["u"][r], host["t"][r],
                                         int(host["k"][r]), host["p"][r], host["m"][r])[0]
    assert np.array_equal(o[6], ref.slots_of(o[5], o[11], 64, np.arange(rows) // n))


def test_a_decode_step_together(ert):
    import torch
    for seed in range(3):
        s = _step_state(ert, seed)
        before = s["tables"].cpu().numpy()
        out = _step(ert, s)
        torch.cuda.synchronize()
        want = ref.extend_tables(before, s["kv"].cpu().numpy(), s["new"].cpu().numpy(),
                                 s["free"].cpu().numpy(), int(s["start"]), 64, 12)
        for got, w in zip([out[11], *out[:4]], want[:5]):
            assert np.array_equal(got.cpu().numpy(), w)
        assert int(out[4]) == want[5]
        _check_step(s, out)


def test_a_captured_step_replays(ert):
    # captured once, replayed with new inputs copied in and eager work between
    import torch
    s = _step_state(ert, 0)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(ert, s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _step(ert, s)
    for seed in (1, 2, 3, 4):
        n = _step_state(ert, seed)
        for k, v in n.items():
            if k not in ("next_n", "ws"):
                s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        eager = _step(ert, n)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b), seed
        _check_step(n, eager)


def test_two_captured_graphs_and_eager_calls_share_nothing(ert):
    import torch
    a, b = _step_state(ert, 5), _step_state(ert, 6)
    want_a = [t.clone() for t in _step(ert, a)]
    want_b = [t.clone() for t in _step(ert, b)]
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _step(ert, s)
        graphs.append((g, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for st, (g, _) in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        eager = ert.sample_tokens(a["logits"], a["u"], temperature=a["t"], top_k=a["k"], top_p=a["p"],
                                  min_p=a["m"])
        torch.cuda.synchronize()
        assert torch.equal(eager, want_a[9])
        for (_, out), want in zip(graphs, (want_a, want_b)):
            for x, y in zip(out, want):
                assert torch.equal(x, y)


def test_other_streams(ert):
    import torch
    st = torch.cuda.Stream()
    x = torch.randn(8, 30000, device="cuda") * 2
    u = torch.rand(8, device="cuda")
    p = torch.full((8,), 0.9, device="cuda")
    r = torch.randn(100, 64, device="cuda")
    want = ert.sample_tokens(x, u, top_p=p), *ert.route_experts(r, 4)
    torch.cuda.synchronize()
    for _ in range(4):
        got = ert.sample_tokens(x, u, top_p=p, stream=st), *ert.route_experts(r, 4, stream=st)
        other = ert.sample_tokens(x, u, top_p=p), *ert.route_experts(r, 4)
        torch.cuda.synchronize()
        for g, o, w in zip(got, other, want):
            assert torch.equal(g, w) and torch.equal(o, w)


def test_training_step_captured_beside_eager(ert):
    # forward and backward captured on tensors of their own, with eager work on
    # other leaves between the replays
    import torch
    x = torch.randn(50, 96, device="cuda", requires_grad=True)
    g = torch.randn(50, 6, device="cuda")
    def step(t):
        _, w = ert.route_experts(t, 6, scoring="softmax", renormalize=True, scale=1.5)
        return torch.autograd.grad(w, t, g)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x)
    for seed in range(3):
        torch.manual_seed(seed)
        new = torch.randn(50, 96, device="cuda")
        with torch.no_grad():
            x.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(new.requires_grad_()))
