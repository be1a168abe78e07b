"""A beam search's step over a paged cache: the choice of the beams, what it does
to their states and block tables, attention with a prefix that sequences
share, the attention mass of cached positions, and eviction by it.

Thin bindings of the C calls declared in ``include/exact_row_top.h``, whose
comments hold the definitions.

    out, lse = prefix_attention(q, k_cache, v_cache, prefix_tables, prefix_lens, tables, lens,
                                return_lse=True)
    prefix_mass, mass = attention_mass(q, k_cache, lse, prefix_tables, prefix_lens, tables, lens,
                                       prefix_mass=prefix_mass, mass=mass)
    scores, parents, tokens = select_beams(logits, scores, k)
    reorder_beams([history, state, mass], parents, out=[history, state, mass])
    reorder_block_tables(tables, kv_lens, parents, block_size, caches=[k_cache, v_cache], out=tables)
    kept, prefix_mass, prefix_lens = evict_cache(prefix_mass, prefix_lens, budget, sinks=4, recent=64,
                                                 block_tables=prefix_tables, caches=[k_cache, v_cache])

Tensors must share one device, which need not be the current one.  The work
runs on the current stream of that device, or on ``stream``, whose pool then
also holds the returned tensors.
"""
from __future__ import annotations

import ctypes

import torch

from .row_ops import (TOPK_DT, _check, _elsewhere, _int32, _lib, _matrix, _raw_stream, _scores,
                      _tables_layout, _tensor, _vector)


def _flat(t, name, dtype, shape, device):
    """Pointer of a contiguous tensor of one shape, or None."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == device.index):
            return t.data_ptr()
    except AttributeError:
        pass
    _tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t.data_ptr()


def _given(t, name, length, device):
    """Pointer of an int32 vector that must be given."""
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    return _vector(t, name, torch.int32, length, device)


def _tables(t, name, rows, device):
    """(pointer, row stride, width) of block tables; any number of rows for None."""
    try:
        (n, width), (stride, inner) = t.shape, t.stride()
        if (t.dtype is torch.int32 and inner == 1 and stride >= width and n == rows and n < 1 << 31
                and width < 1 << 31 and t.get_device() == device.index):
            return t.data_ptr(), stride if n > 1 else width, width
    except (AttributeError, TypeError, ValueError):
        pass
    n, width, stride = _tables_layout(t)
    if rows is not None and n != rows:
        raise ValueError(f"{name} must hold {rows} rows")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t.data_ptr(), stride, width


def select_beams(logits, scores, k, *, ended=None, end_token=0, lengths=None, length_penalty=0.0,
                 stream=None):
    """The k best continuations of each request's beams.

    logits [requests * beams, vocab] (float32, bfloat16 or float16), scores
    float32 [requests, beams]: each beam's sum of log-probabilities so far (one
    that is not finite offers nothing: start with 0 and -inf behind it).  ended:
    bool [requests, beams]; an ended beam offers end_token alone, its score as
    it is.  lengths: int32 [requests, beams], the tokens of each beam; with it
    totals are ranked by total / length ** length_penalty, the new token counted.

    Returns (scores, parents, tokens), float32 / int32 / int32 [requests, k],
    best first: the new total (not divided), the beam and its token; equal
    ranks go to the lower beam, then the lower token.  Places without a
    candidate hold -inf, -1, -1.  beams at most 32, k at most 64."""
    guard = _elsewhere(logits, "logits", stream)
    if guard is not None:
        with guard:
            return select_beams(logits, scores, k, ended=ended, end_token=end_token, lengths=lengths,
                                length_penalty=length_penalty)
    lib = _lib()
    rows, vocab, stride, code = _scores(logits, "logits")
    dev = logits.device
    k, end_token = _int32(k, "k"), _int32(end_token, "end_token")
    if _tensor(scores, "scores").dim() != 2:
        raise ValueError("scores must be 2-D")
    requests, beams = scores.shape
    if requests * beams != rows:
        raise ValueError(f"logits must hold {requests * beams} rows")
    s = _flat(scores, "scores", torch.float32, (requests, beams), dev)
    e = _flat(ended, "ended", torch.bool, (requests, beams), dev)
    n = _flat(lengths, "lengths", torch.int32, (requests, beams), dev)
    if k < 1:
        raise ValueError("k must be at least 1")
    # (sizes one by one, and not in a tuple: a third of a microsecond less each)
    found = torch.empty(requests, k, dtype=torch.float32, device=dev)
    parents = torch.empty(requests, k, dtype=torch.int32, device=dev)
    tokens = torch.empty(requests, k, dtype=torch.int32, device=dev)
    nbytes = lib.topk_beams_workspace_bytes(requests, beams, k, vocab)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.topk_beams(logits.data_ptr(), code, stride, vocab, requests, beams, k, s, e, end_token, n,
                          float(length_penalty), found.data_ptr(), parents.data_ptr(), tokens.data_ptr(),
                          ws.data_ptr(), nbytes, _raw_stream(dev)))
    return found, parents, tokens


def _parents(parents, device):
    try:
        shape = parents.shape
        if (parents.dtype is torch.int32 and len(shape) == 2 and parents.is_contiguous()
                and parents.get_device() == device.index):
            return shape
    except AttributeError:
        pass
    _tensor(parents, "parents")
    if parents.dtype != torch.int32:
        raise TypeError(f"parents must be torch.int32, got {parents.dtype}")
    if parents.dim() != 2 or not parents.is_contiguous():
        raise ValueError("parents must be a contiguous int32 [requests, k] tensor")
    if parents.device != device:
        raise ValueError(f"parents must be on {device}")
    return parents.shape


def _rows_layout(t, name, rows, device):
    """(row stride, row size) in bytes of a tensor of contiguous rows."""
    try:
        if t.is_contiguous() and t.shape[0] == rows and rows and t.get_device() == device.index:
            n = t.nbytes // rows
            return n, n
    except (AttributeError, IndexError):
        pass
    _tensor(t, name)
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dim() < 1 or t.shape[0] != rows:
        raise ValueError(f"{name} must hold {rows} rows")
    size = t.element_size()
    if t.is_contiguous():
        n = t.numel() // rows * size if rows else 0
        return n, n
    if not t[0].is_contiguous():
        raise ValueError(f"{name} must have contiguous rows")
    n = t[0].numel() * size
    stride = t.stride(0) * size if rows > 1 else n
    if stride < n:
        raise ValueError(f"{name} rows overlap")
    return stride, n


def reorder_beams(states, parents, *, beams=None, out=None, stream=None):
    """Rows by parent: row r * k + j of each result is row r * beams +
    parents[r, j] of the state.

    states: a tensor or a list of tensors [requests * beams, ...] of any type
    whose rows are contiguous; parents: int32 [requests, k] as select_beams
    gives them (beams: k, unless told).  out: where the results go, a tensor or
    list like states with requests * k rows; a state may be its own out (then
    beams must be k): rows then move in place.  Rows without a parent (-1) are
    zero in new results and left as they are in given ones.  All arrays move
    in one launch.  beams and k at most 32.  Returns the results, in states'
    form."""
    single = isinstance(states, torch.Tensor)
    states = [states] if single else list(states)
    if out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if len(out) != len(states):
            raise ValueError("out must hold one tensor for each state")
    guard = _elsewhere(parents, "parents", stream)
    if guard is not None:
        with guard:
            got = reorder_beams(states, parents, beams=beams, out=out)
        return got[0] if single else got
    dev = parents.device
    requests, k = _parents(parents, dev)
    beams = k if beams is None else _int32(beams, "beams")
    clear = out is None
    sources = [_rows_layout(t, "states", requests * beams, dev) for t in states]
    if clear:
        out = [torch.empty(requests * k, *t.shape[1:], dtype=t.dtype, device=dev) for t in states]
        targets = [(n, n) for _, n in sources]
    else:
        targets = [_rows_layout(t, "out", requests * k, dev) for t in out]
        for a, b in zip(states, out):
            if a.dtype != b.dtype or a.shape[1:] != b.shape[1:]:
                raise ValueError("out must have its state's type and row shape")
    # one array: sources, targets, their strides, row sizes
    n = len(states)
    each = (ctypes.c_int64 * (5 * n))(*[t.data_ptr() for t in states], *[t.data_ptr() for t in out],
                                      *[s for s, _ in sources], *[s for s, _ in targets],
                                      *[b for _, b in sources])
    at = ctypes.addressof(each)
    _check(_lib().topk_reorder_rows(n, at, at + 8 * n, at + 16 * n, at + 24 * n, at + 32 * n,
                                    parents.data_ptr(), requests, beams, k, 1 if clear else 0,
                                    _raw_stream(dev)))
    return out[0] if single else out


def _caches(caches, block_size, device):
    """(pointer array, caches, blocks, bytes of a slot) of caches of one shape."""
    caches = [caches] if isinstance(caches, torch.Tensor) else caches
    if not caches:
        return None, 0, 0, 0
    try:
        first = caches[0]
        shape, dtype, nbytes = first.shape, first.dtype, first.nbytes
        good = len(shape) >= 2 and shape[1] == block_size
        for c in caches:
            good = (good and c.is_contiguous() and c.shape == shape and c.dtype is dtype
                    and c.get_device() == device.index)
    except (AttributeError, TypeError):
        good = False
    if not good:
        for c in caches:
            _tensor(c, "caches")
            if c.device != device:
                raise ValueError(f"caches must be on {device}")
            if c.dim() < 2 or not c.is_contiguous() or c.shape != shape or c.dtype != dtype:
                raise ValueError("caches must be contiguous [blocks, block_size, ...] tensors of one shape and type")
        raise ValueError(f"caches must hold blocks of {block_size}")
    slots = shape[0] * shape[1]
    slot_bytes = nbytes // slots if slots else 0
    if shape[0] >> 31 or slot_bytes >> 31:
        raise ValueError("caches are too large: their sizes must fit 32 bits")
    return ((ctypes.c_void_p * len(caches))(*[c.data_ptr() for c in caches]), len(caches), shape[0],
            slot_bytes)


def reorder_block_tables(block_tables, kv_lens, parents, block_size, *, caches=(), tail_blocks=None,
                         out=None, stream=None):
    """Block tables by parent, sharing full blocks.

    block_tables: int32 [requests * beams, max_blocks]; kv_lens: int32
    [requests], the tokens that every beam of a request holds; parents: int32
    [requests, k].  Child j of request r gets its parent's entries of full
    blocks.  The block that is open (kv_lens % block_size > 0) becomes the
    child's own, tail_blocks[r * k + j] (int32 [requests * k]) or, without
    tail_blocks, the one that row r * k + j itself holds there; its tokens are
    copied from the parent's in each of the caches ([blocks, block_size, ...],
    contiguous, of one shape).  Entries behind stay the row's own (-1 where k
    is not beams).  A child without a parent keeps its row.

    out: int32 [requests * k, max_blocks], may be block_tables itself.  Open
    blocks of a request are distinct and no other request's.  beams and k at
    most 32.  Returns the new tables."""
    guard = _elsewhere(block_tables, "block_tables", stream)
    if guard is not None:
        with guard:
            return reorder_block_tables(block_tables, kv_lens, parents, block_size, caches=caches,
                                        tail_blocks=tail_blocks, out=out)
    dev = block_tables.device
    requests, k = _parents(parents, dev)
    rows = len(block_tables)
    tables, stride, width = _tables(block_tables, "block_tables", rows, dev)
    beams = rows // requests if requests else k
    if requests * beams != rows:
        raise ValueError(f"block_tables must hold the rows of {requests} requests")
    block_size = _int32(block_size, "block_size")
    lens = _given(kv_lens, "kv_lens", requests, dev)
    tail = _vector(tail_blocks, "tail_blocks", torch.int32, requests * k, dev)
    if tail is None and beams != k:
        raise ValueError("tail_blocks is needed where k differs from the beams of a request")
    pointers, count, blocks, slot_bytes = _caches(caches, block_size, dev)
    if out is None:
        out = torch.empty(requests * k, width, dtype=torch.int32, device=dev)
    to, out_stride, out_width = _tables(out, "out", requests * k, dev)
    if out_width != width:
        raise ValueError(f"out must be an int32 [{requests * k}, {width}] tensor")
    _check(_lib().topk_reorder_blocks(
        tables, stride, width, lens, parents.data_ptr(), requests, beams, k, block_size, tail, to, out_stride,
        count, pointers, blocks, slot_bytes, _raw_stream(dev)))
    return out


def _attend_arguments(q, k_cache, prefix_tables, prefix_lens, block_tables, kv_lens, group_starts,
                      next_n, scale):
    """The arguments that attention and mass share: (device, query arguments,
    key cache layout, blocks and their size, tables and scale, sizes)."""
    dtype, dev = q.dtype, q.device
    code = TOPK_DT.get(dtype)
    if code != 1 and code != 2:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    if q.dim() != 3:
        raise ValueError("q must be 3-D [tokens, heads, dim] with unit inner stride")
    (tokens, heads, dim), (token_stride, head_stride, inner) = q.shape, q.stride()
    if inner != 1 and q.numel():
        raise ValueError("q must be 3-D [tokens, heads, dim] with unit inner stride")
    next_n = _int32(next_n, "next_n")
    if next_n < 1 or tokens % next_n:
        raise ValueError("q must hold next_n tokens for each sequence")
    seqs = tokens // next_n
    keys = _cache_layout(k_cache, "k_cache", dtype, dim, dev)
    blocks, block_size, kv_heads, _ = k_cache.shape
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError("q's heads must be a multiple of the cache's")
    if tokens >> 31 or blocks >> 31 or block_size >> 31:
        raise ValueError("sizes must fit 32 bits")
    own = (*_tables(block_tables, "block_tables", seqs, dev), _given(kv_lens, "kv_lens", seqs, dev))
    if prefix_tables is None:
        if prefix_lens is not None or group_starts is not None:
            raise ValueError("prefix_lens and group_starts need prefix_tables")
        groups, shared, starts = 0, (None, 0, 0, None), None
    else:
        groups = len(prefix_tables)
        shared = (*_tables(prefix_tables, "prefix_tables", groups, dev),
                  _given(prefix_lens, "prefix_lens", groups, dev))
        starts = _vector(group_starts, "group_starts", torch.int32, groups + 1, dev)
        if starts is None and groups and seqs % groups:
            raise ValueError("without group_starts the sequences must form equal groups")
    scale = float(dim) ** -0.5 if scale is None else float(scale)
    query = (q.data_ptr(), code, token_stride if tokens > 1 else 0, head_stride if heads > 1 else 0, seqs,
             next_n, heads, kv_heads, dim)
    return (dev, query, keys, (blocks, block_size), (*shared, starts, groups, *own, scale),
            (tokens, heads, kv_heads, dim, seqs, groups, next_n))


def _bounds(tables, block_size, max_prefix_len, max_len):
    """(tables, bounds, positions that the rows hold within them): the C calls
    take a bound of 0 for none, so a bound of zero takes the table's width."""
    tables = list(tables)
    bounds, room = [], []
    for at, name, bound in ((2, "max_prefix_len", max_prefix_len), (8, "max_len", max_len)):
        if bound is not None:
            bound = _int32(bound, name)
            if bound < 0:
                raise ValueError(f"{name} must not be negative")
            if bound == 0:
                tables[at] = 0
        bounds.append(bound or 0)
        room.append(min(tables[at] * block_size, bound or tables[at] * block_size))
    return tables, bounds, room


def _cache_layout(cache, name, dtype, dim, device):
    """(pointer, block, slot and head strides) of a cache."""
    try:
        (blocks, size, heads, d), (b, s, h, inner) = cache.shape, cache.stride()
        if cache.dtype is dtype and d == dim and inner == 1 and cache.get_device() == device.index:
            return cache.data_ptr(), b if blocks > 1 else 0, s if size > 1 else 0, h if heads > 1 else 0
    except (AttributeError, TypeError, ValueError):
        pass
    _tensor(cache, name)
    if cache.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {cache.dtype}")
    if cache.device != device:
        raise ValueError(f"{name} must be on {device}")
    raise ValueError(f"{name} must be [blocks, block_size, heads, {dim}] with unit inner stride")


def prefix_attention(q, k_cache, v_cache, prefix_tables, prefix_lens, block_tables, kv_lens, *,
                     group_starts=None, next_n=1, scale=None, max_prefix_len=None, max_len=None,
                     out=None, return_lse=False, stream=None):
    """Decode attention over a paged cache for sequences that share prefixes.

    q: [sequences * next_n, heads, dim] (bfloat16 or float16, dim 64 or 128);
    k_cache, v_cache: [blocks, block_size, kv_heads, dim] with any strides that
    are multiples of 8 and a unit inner one.  Group g, the sequences
    group_starts[g] .. group_starts[g + 1] - 1 (int32 [groups + 1]; None: equal
    groups), sees the first prefix_lens[g] positions of prefix_tables[g] (int32
    [groups, max_blocks]; None: no prefixes); token t of sequence s then sees
    the first kv_lens[s] - next_n + t + 1 positions of block_tables[s], its
    own.  scale: dim ** -0.5 unless given, never negative.  max_prefix_len and
    max_len (0 and up) bound the lengths (which are cut to them) where the tables
    have room for far more: the work is planned for the longest rows there can be.

    Returns out, [sequences * next_n, heads, dim] in q's type, or (out, lse)
    with the float32 log-sums [sequences * next_n, heads], which attention_mass
    takes.  Tokens that see nothing give 0 and -inf.  Not differentiable."""
    guard = _elsewhere(q, "q", stream)
    if guard is not None:
        with guard:
            return prefix_attention(q, k_cache, v_cache, prefix_tables, prefix_lens, block_tables,
                                    kv_lens, group_starts=group_starts, next_n=next_n, scale=scale,
                                    max_prefix_len=max_prefix_len, max_len=max_len, out=out,
                                    return_lse=return_lse)
    dev, query, keys, paging, tables, sizes = _attend_arguments(
        q, k_cache, prefix_tables, prefix_lens, block_tables, kv_lens, group_starts, next_n, scale)
    tokens, heads, kv_heads, dim, seqs, groups, next_n = sizes
    values = _cache_layout(v_cache, "v_cache", q.dtype, dim, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must have k_cache's shape")
    bounds, room = (0, 0), (tables[2] * paging[1], tables[8] * paging[1])
    if max_prefix_len is not None or max_len is not None:
        tables, bounds, room = _bounds(tables, paging[1], max_prefix_len, max_len)
    if out is None:
        out = torch.empty(tokens, heads, dim, dtype=q.dtype, device=dev)
    else:
        out = _matrix(out, "out", q.dtype, (tokens, heads, dim), dev)
    lse = torch.empty(tokens, heads, dtype=torch.float32, device=dev) if return_lse else None
    lib = _lib()
    nbytes = lib.topk_attend_workspace_bytes(groups, seqs, tables[4] is not None, next_n, heads, kv_heads,
                                             dim, *room)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.topk_attend(*query, *keys, *values, *paging, *tables, *bounds, out.data_ptr(),
                           lse.data_ptr() if lse is not None else None, ws.data_ptr(), nbytes,
                           _raw_stream(dev)))
    return (out, lse) if return_lse else out


def _mass(mass, out, name, entries, kv_heads, positions, device):
    """(positions, given mass' pointer, result) of one kind of mass rows."""
    for t in (mass, out):
        if t is not None:
            what = name if t is mass else f"{name}'s out"
            if _tensor(t, what).dim() != 3:
                raise ValueError(f"{what} must be 3-D")
            positions = t.shape[2]
    if positions >> 31:
        raise ValueError(f"{name} is too large: its sizes must fit 32 bits")
    shape = (entries, kv_heads, positions)
    given = _flat(mass, name, torch.float32, shape, device)
    if out is None:
        out = torch.empty(entries, kv_heads, positions, dtype=torch.float32, device=device)
    else:
        out = _matrix(out, f"{name}'s out", torch.float32, shape, device)
    return positions, given, out


def attention_mass(q, k_cache, lse, prefix_tables, prefix_lens, block_tables, kv_lens, *,
                   group_starts=None, next_n=1, scale=None, prefix_mass=None, mass=None, decay=1.0,
                   prefix_out=None, out=None, max_prefix_len=None, max_len=None, stream=None):
    """Accumulated attention mass of cached positions: decay times the mass
    given, plus the weights that the step's tokens gave each position, added up
    over the tokens and the query heads of a key head.

    q to scale, max_prefix_len and max_len as in the prefix_attention call that
    gave lse: positions behind the bounds have no part in it.  prefix_mass:
    float32 [groups, kv_heads, positions], mass: float32 [sequences, kv_heads,
    positions] (None: zeros, as many positions as the tables hold).  prefix_out
    and out: where the results go, may be prefix_mass and mass.  Returns
    (prefix mass, mass); the first is None without prefix_tables."""
    guard = _elsewhere(q, "q", stream)
    if guard is not None:
        with guard:
            return attention_mass(q, k_cache, lse, prefix_tables, prefix_lens, block_tables, kv_lens,
                                  group_starts=group_starts, next_n=next_n, scale=scale,
                                  prefix_mass=prefix_mass, mass=mass, decay=decay,
                                  prefix_out=prefix_out, out=out, max_prefix_len=max_prefix_len,
                                  max_len=max_len)
    dev, query, keys, paging, tables, sizes = _attend_arguments(
        q, k_cache, prefix_tables, prefix_lens, block_tables, kv_lens, group_starts, next_n, scale)
    tokens, heads, kv_heads, dim, seqs, groups, next_n = sizes
    if lse is None:
        raise TypeError("lse must be a torch.Tensor")
    weights = _flat(lse, "lse", torch.float32, (tokens, heads), dev)
    if prefix_tables is None:
        if prefix_mass is not None or prefix_out is not None:
            raise ValueError("prefix_mass needs prefix_tables")
        shared, given_shared, prefix_out = 0, None, None
    else:
        shared, given_shared, prefix_out = _mass(prefix_mass, prefix_out, "prefix_mass", groups, kv_heads,
                                                 tables[2] * paging[1], dev)
    own, given_own, out = _mass(mass, out, "mass", seqs, kv_heads, tables[8] * paging[1], dev)
    bounds = (0, 0)
    if max_prefix_len is not None or max_len is not None:
        tables, bounds, _ = _bounds(tables, paging[1], max_prefix_len, max_len)
    _check(_lib().topk_attend_mass_bounded(*query, *keys, *paging, *tables, *bounds, weights, float(decay),
                                           given_shared, prefix_out.data_ptr() if prefix_out is not None else None,
                                           shared, given_own, out.data_ptr(), own, _raw_stream(dev)))
    return prefix_out, out


def evict_cache(mass, kv_lens, budget, *, sinks=0, recent=0, block_tables=None, caches=(),
                out_tables=None, mass_out=None, stream=None):
    """Keeps the budget positions of each (request, head) that matter most.

    mass: float32 [requests, heads, positions] with a unit inner stride;
    kv_lens: int32 [requests].  Where a request holds more than budget
    positions, the first `sinks`, the last `recent` and those with the largest
    mass stay (equal masses: the lower position; NaN below all); else all.

    Returns (kept, kept mass, new lengths): int32 [requests, heads, budget], the
    kept positions in rising order, then -1; float32, their mass, then 0
    (mass_out: where it goes, float32 [requests, heads, >= budget]); int32
    [requests].

    With caches (contiguous [blocks, block_size, kv_heads, ...] tensors of one
    shape, rows of block_tables, int32 [requests, max_blocks]) the kept
    positions' rows move to the front: position j of head h comes from position
    kept[r, h, j], and from then on has kept mass[r, h, j]: the mass given no
    longer fits the cache.  heads divides kv_heads; with one, all heads keep the
    same positions.  out_tables: the rows' new blocks, none of them in block_tables;
    None: in place."""
    guard = _elsewhere(mass, "mass", stream)
    if guard is not None:
        with guard:
            return evict_cache(mass, kv_lens, budget, sinks=sinks, recent=recent, block_tables=block_tables,
                               caches=caches, out_tables=out_tables, mass_out=mass_out)
    if mass.dtype != torch.float32:
        raise TypeError(f"mass must be torch.float32, got {mass.dtype}")
    if mass.dim() != 3:
        raise ValueError("mass must be 3-D [requests, heads, positions] with unit inner stride")
    dev = mass.device
    (requests, heads, positions), (stride0, stride1, inner) = mass.shape, mass.stride()
    if inner != 1 and positions > 1 and mass.numel():
        raise ValueError("mass must be 3-D [requests, heads, positions] with unit inner stride")
    if requests >> 31 or heads >> 31 or positions >> 31:
        raise ValueError("mass is too large: its sizes must fit 32 bits")
    lens = _given(kv_lens, "kv_lens", requests, dev)
    budget, sinks, recent = _int32(budget, "budget"), _int32(sinks, "sinks"), _int32(recent, "recent")
    if budget < 1 or sinks < 0 or recent < 0 or sinks + recent > budget:
        raise ValueError("budget must be at least 1, and sinks and recent within it")
    caches = [caches] if isinstance(caches, torch.Tensor) else caches
    if caches:
        if block_tables is None:
            raise ValueError("caches need block_tables")
        shape = _tensor(caches[0], "caches").shape
        if len(shape) < 3:
            raise ValueError("caches must be [blocks, block_size, kv_heads, ...] tensors")
        pointers, count, blocks, slot_bytes = _caches(caches, shape[1], dev)
        # (all that the move could refuse, before the choice writes anything)
        if count > 64 or shape[1] > 1 << 20:
            raise ValueError("at most 64 caches with blocks of at most 2 ** 20 positions")
        size, free = blocks * shape[1] * slot_bytes, 0
        for p in sorted(pointers) if size else ():
            if p & 15 or p < free:
                raise ValueError("caches must be aligned to 16 bytes and must not overlap")
            free = p + size
        if heads < 1 or shape[2] % heads:
            raise ValueError("mass' heads must divide the caches' heads")
        if (slot_bytes // heads) % 16:
            raise ValueError("a head's share of a cache slot must be a multiple of 16 bytes")
        tables = _tables(block_tables, "block_tables", requests, dev)
        to = tables if out_tables is None else _tables(out_tables, "out_tables", requests, dev)
        if to[0] == tables[0] and to[1] != tables[1] and requests > 1:
            raise ValueError("out_tables must be block_tables or lie apart from them")
    kept = torch.empty(requests, heads, budget, dtype=torch.int32, device=dev)
    new_lens = torch.empty(requests, dtype=torch.int32, device=dev)
    width = budget
    if mass_out is None:
        mass_out = torch.empty(requests, heads, budget, dtype=torch.float32, device=dev)
        out = mass_out.data_ptr()
    else:
        if _tensor(mass_out, "mass_out").dim() != 3 or mass_out.shape[2] < budget:
            raise ValueError("mass_out must be [requests, heads, budget or more]")
        width = mass_out.shape[2]
        out = _flat(mass_out, "mass_out", torch.float32, (requests, heads, width), dev)
    lib, raw = _lib(), _raw_stream(dev)
    _check(lib.topk_evict_keep(mass.data_ptr(), stride0 if requests > 1 else 0, stride1 if heads > 1 else 0,
                               positions, requests, heads, lens, budget, sinks, recent, kept.data_ptr(), out,
                               width, new_lens.data_ptr(), raw))
    if caches:
        _check(lib.topk_evict_move(kept.data_ptr(), requests, heads, budget, *tables, *to, shape[1], count,
                                   pointers, blocks, slot_bytes, raw))
    return kept, mass_out, new_lens
