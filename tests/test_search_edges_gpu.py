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


