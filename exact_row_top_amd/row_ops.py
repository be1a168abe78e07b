"""Row operators beside the top-K selection: sampling a token per row of logits,
routing tokens to experts (with its gradient), block tables and slot maps of a
paged cache, and the slots of selected positions.

Thin bindings of the C calls declared in ``include/exact_row_top.h``, whose
comments hold the definitions.  Equal scores go to the lower index everywhere.

    token = sample_tokens(logits, uniforms, temperature=t, top_k=k, top_p=p, min_p=m)
    experts, weights = route_experts(logits, 8, scoring="sigmoid", bias=b, num_groups=8,
                                     topk_groups=4, group_score="top2")
    starts, requests, positions, slots, free_next = extend_block_tables(
        tables, kv_lens, new_tokens, free_blocks, free_start, block_size, max_tokens)
    slots = topk_slots(indices, tables, block_size)

Tensors must share one device, which need not be the current one.  The work
runs on the current stream of that device, or on ``stream``, whose pool then
also holds the returned tensors.
"""
from __future__ import annotations

import operator

import torch

TOPK_DT = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
TOPK_SAMPLE_WHOLE_ROW = 1
TOPK_ROUTE_SIGMOID, TOPK_ROUTE_TOP2, TOPK_ROUTE_RENORMALIZE = 1, 2, 4

_calls = None


def _lib():
    global _calls
    if _calls is None:
        from . import load_library
        _calls = load_library()
    return _calls


def _check(status):
    if status != 0:
        from . import TOPK_EINVAL, TopKError, strerror
        raise TopKError(status, "a size, count or setting outside the call's range"
                        if status == TOPK_EINVAL else strerror(status))


def _tensor(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t


def _fits(name, rows, width):
    if rows >> 31 or width >> 31:
        raise ValueError(f"{name} is too large: its sizes must fit 32 bits")


def _scores(t, name):
    """(rows, width, row stride, dtype code) of a score matrix."""
    code = TOPK_DT.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, width = t.shape
    _fits(name, rows, width)
    if t.is_contiguous():
        return rows, width, width, code
    stride = t.stride(0) if rows > 1 else width
    if rows and width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit inner stride")
    if stride < width:
        raise ValueError(f"{name} rows overlap")
    return rows, width, stride, code


def _vector(t, name, dtype, length, device):
    """Pointer of a contiguous 1-D tensor of `length` values, or None."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.dim() == 1 and t.numel() == length and t.is_contiguous()
                and t.get_device() == device.index):
            return t.data_ptr()
    except AttributeError:
        pass
    _tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 1 or t.shape[0] != length or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{length}] tensor")
    raise ValueError(f"{name} must be on {device}")


def _matrix(t, name, dtype, shape, device):
    """A contiguous matrix the caller gave, checked; a new one for None."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _tensor(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t


def _int32(v, name):
    v = operator.index(v)
    if not -(1 << 31) <= v < (1 << 31):
        raise ValueError(f"{name} must fit 32 bits")
    return v


class _On:
    """Makes a tensor's device (and a given stream) current around a call."""

    def __init__(self, device, stream):
        if stream is not None:
            if stream.device != device:
                raise ValueError(f"stream must be on {device}")
            self.guard = torch.cuda.stream(stream)
        else:
            self.guard = torch.cuda.device(device)

    def __enter__(self):
        return self.guard.__enter__()

    def __exit__(self, *a):
        return self.guard.__exit__(*a)


def _elsewhere(t, name, stream):
    """A guard if the call has to leave the current device or stream."""
    _tensor(t, name)
    if stream is not None or t.device.index != torch._C._cuda_getDevice():
        return _On(t.device, stream)
    return None


def _raw_stream(device):
    return torch._C._cuda_getCurrentRawStream(device.index)


def sample_tokens(logits, uniforms, *, temperature=None, top_k=None, top_p=None, min_p=None,
                  tokens=None, logprobs=None, return_logprobs=False, whole_row=False, stream=None):
    """One token per row of logits [rows, vocab] (float32, bfloat16 or float16).

    uniforms: float32 [rows], one number in [0, 1) for each row's draw.
    temperature, top_p, min_p: float32 [rows], top_k: int32 [rows]; None leaves
    the setting out.  top_k <= 0, top_p >= 1 and min_p <= 0 cut nothing; a
    temperature that is not > 0 takes the row's best token.  The cuts apply in
    the order top-k, top-p (over what top-k kept), min-p; the draw runs over
    the kept tokens in index order.  NaN and -inf logits are never drawn; a row
    of nothing else gives -1.

    Returns the tokens, int32 [rows], or (tokens, logprobs) with the float32
    log-probability of each token among the kept ones.  Weights of 2^-44 of a
    row's largest and less count as zero; sums of weights, and with them the
    borders between tokens, are good to vocab * 2^-44 of it beside 2^-44 of
    themselves.  whole_row reads
    every row a second time instead of using the candidates and sums of the
    first reading (for tests; the same results within that bound)."""
    guard = _elsewhere(logits, "logits", stream)
    if guard is not None:
        with guard:
            return sample_tokens(logits, uniforms, temperature=temperature, top_k=top_k, top_p=top_p,
                                 min_p=min_p, tokens=tokens, logprobs=logprobs,
                                 return_logprobs=return_logprobs, whole_row=whole_row)
    lib = _lib()
    rows, vocab, stride, code = _scores(logits, "logits")
    dev = logits.device
    if uniforms is None:
        raise TypeError("uniforms must be a torch.Tensor")
    args = (_vector(uniforms, "uniforms", torch.float32, rows, dev),
            _vector(temperature, "temperature", torch.float32, rows, dev),
            _vector(top_k, "top_k", torch.int32, rows, dev),
            _vector(top_p, "top_p", torch.float32, rows, dev),
            _vector(min_p, "min_p", torch.float32, rows, dev))
    tokens = _matrix(tokens, "tokens", torch.int32, (rows,), dev)
    if logprobs is not None or return_logprobs:
        logprobs = _matrix(logprobs, "logprobs", torch.float32, (rows,), dev)
    nbytes = lib.topk_sample_workspace_bytes(rows, vocab)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib.topk_sample(logits.data_ptr(), code, stride, vocab, rows, *args, tokens.data_ptr(),
                           logprobs.data_ptr() if logprobs is not None else None,
                           TOPK_SAMPLE_WHOLE_ROW if whole_row else 0, ws.data_ptr(), nbytes,
                           _raw_stream(dev)))
    return tokens if logprobs is None else (tokens, logprobs)


_SCORING = {"softmax": 0, "sigmoid": TOPK_ROUTE_SIGMOID}
_GROUP_SCORE = {"max": 0, "top2": TOPK_ROUTE_TOP2}


def _route_flags(scoring, group_score, renormalize):
    if scoring not in _SCORING:
        raise ValueError(f"scoring must be one of {sorted(_SCORING)}")
    if group_score not in _GROUP_SCORE:
        raise ValueError(f"group_score must be one of {sorted(_GROUP_SCORE)}")
    return _SCORING[scoring] | _GROUP_SCORE[group_score] | (TOPK_ROUTE_RENORMALIZE if renormalize else 0)


def _route(logits, top_k, bias, num_groups, topk_groups, flags, scale, indices, weights):
    tokens, experts, stride, code = _scores(logits, "logits")
    dev = logits.device
    top_k = _int32(top_k, "top_k")
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    b = _vector(bias, "bias", torch.float32, experts, dev)
    indices = _matrix(indices, "indices", torch.int32, (tokens, top_k), dev)
    weights = _matrix(weights, "weights", torch.float32, (tokens, top_k), dev)
    _check(_lib().topk_route(logits.data_ptr(), code, stride, tokens, experts, top_k, b,
                             _int32(num_groups, "num_groups"), _int32(topk_groups, "topk_groups"),
                             flags, scale, indices.data_ptr(), weights.data_ptr(), _raw_stream(dev)))
    return indices, weights


class _RouteExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, bias, num_groups, topk_groups, flags, scale):
        indices, weights = _route(logits, top_k, bias, num_groups, topk_groups, flags, scale, None,
                                  None)
        ctx.save_for_backward(logits, indices)
        ctx.flags, ctx.scale = flags, scale
        ctx.mark_non_differentiable(indices)
        return indices, weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad_weights):
        logits, indices = ctx.saved_tensors
        return (_route_backward(grad_weights, logits, indices, ctx.flags, ctx.scale, None),
                None, None, None, None, None, None)


def route_experts(logits, top_k, *, scoring="softmax", bias=None, num_groups=1, topk_groups=None,
                  group_score="max", renormalize=True, scale=1.0, indices=None, weights=None,
                  stream=None):
    """The top_k experts of each token and their weights.

    logits [tokens, experts] (float32, bfloat16 or float16); scoring "softmax"
    or "sigmoid"; bias: float32 [experts], added to the scores for the choice
    alone; num_groups equal groups of which the topk_groups best stay (a
    group's score: its largest, or with "top2" its two largest summed);
    renormalize divides the chosen scores by their sum; scale multiplies them.
    Experts at -inf or NaN are never chosen.

    Returns (indices, weights), int32 and float32 [tokens, top_k], best first;
    slots without an expert hold -1 and 0.  The weights are differentiable in
    the logits (a call with stream, indices or weights given is not).  To
    capture forward and backward into a graph, give it logits that no eager
    autograd graph still refers to."""
    flags = _route_flags(scoring, group_score, renormalize)
    scale = float(scale)
    topk_groups = num_groups if topk_groups is None else topk_groups
    guard = _elsewhere(logits, "logits", stream)
    if logits.requires_grad and torch.is_grad_enabled():
        if stream is not None or indices is not None or weights is not None:
            raise ValueError("logits that need a gradient take no stream, indices or weights: "
                             "call under torch.cuda.stream, or detach them")
        if guard is None:
            return _RouteExperts.apply(logits, top_k, bias, num_groups, topk_groups, flags, scale)
        with guard:
            return _RouteExperts.apply(logits, top_k, bias, num_groups, topk_groups, flags, scale)
    if guard is None:
        return _route(logits, top_k, bias, num_groups, topk_groups, flags, scale, indices, weights)
    with guard:
        return _route(logits, top_k, bias, num_groups, topk_groups, flags, scale, indices, weights)


def _route_backward(grad_weights, logits, indices, flags, scale, grad_logits):
    tokens, experts, stride, code = _scores(logits, "logits")
    dev = logits.device
    _tensor(indices, "indices")
    if indices.dim() != 2 or indices.shape[0] != tokens:
        raise ValueError(f"indices must be int32 [{tokens}, top_k]")
    top_k = indices.shape[1]
    indices = _matrix(indices.contiguous(), "indices", torch.int32, (tokens, top_k), dev)
    _tensor(grad_weights, "grad_weights")
    grad_weights = _matrix(grad_weights.contiguous(), "grad_weights", torch.float32,
                           (tokens, top_k), dev)
    grad_logits = _matrix(grad_logits, "grad_logits", logits.dtype, (tokens, experts), dev)
    _check(_lib().topk_route_backward(logits.data_ptr(), code, stride, tokens, experts, top_k, flags,
                                      scale, indices.data_ptr(), grad_weights.data_ptr(),
                                      grad_logits.data_ptr(), experts, _raw_stream(dev)))
    return grad_logits


def route_experts_backward(grad_weights, logits, indices, *, scoring="softmax", renormalize=True,
                           scale=1.0, grad_logits=None, stream=None):
    """Gradient of route_experts' weights in the logits: grad_weights float32
    [tokens, top_k] -> [tokens, experts] in the logits' type.  indices and the
    settings as in the forward call; entries outside [0, experts) have no
    gradient, an expert named twice counts twice."""
    flags = _route_flags(scoring, "max", renormalize)
    guard = _elsewhere(logits, "logits", stream)
    if guard is None:
        return _route_backward(grad_weights, logits, indices, flags, float(scale), grad_logits)
    with guard:
        return _route_backward(grad_weights, logits, indices, flags, float(scale), grad_logits)


def _tables_layout(t):
    _tensor(t, "block_tables")
    if t.dtype != torch.int32:
        raise TypeError(f"block_tables must be torch.int32, got {t.dtype}")
    if t.dim() != 2 or (t.numel() and t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("block_tables must be 2-D with unit inner stride")
    requests, width = t.shape
    _fits("block_tables", requests, width)
    stride = t.stride(0) if requests > 1 else width
    if stride < width:
        raise ValueError("block_tables rows overlap")
    return requests, width, stride


def _slot_dtype(dtype):
    if dtype is None or dtype == torch.int32:
        return torch.int32, 0
    if dtype == torch.int64:
        return torch.int64, 1
    raise TypeError("slots are torch.int32 or torch.int64")


def extend_block_tables(block_tables, kv_lens, new_tokens, free_blocks, free_start, block_size,
                        max_tokens, *, slot_dtype=None, stream=None):
    """Hands out the cache blocks a step needs and maps its new tokens to slots.

    block_tables: int32 [requests, max_blocks], extended in place.  kv_lens,
    new_tokens: int32 [requests], each request's tokens once the step is done
    and how many of them are new.  free_blocks: int32 [n], of which the first
    free_start[0] (int32 [1]) are taken already.  max_tokens: the length of the
    step's token arrays.

    Returns (token_starts [requests + 1], token_requests [max_tokens],
    positions [max_tokens], slots [max_tokens], free_next [1]), int32 (slots
    int64 with slot_dtype=torch.int64).  Entries behind the last token hold -1.
    free_next above len(free_blocks) says that the free list was too short (the
    tokens without a block have slot -1).  At most 4096 requests."""
    guard = _elsewhere(block_tables, "block_tables", stream)
    if guard is not None:
        with guard:
            return extend_block_tables(block_tables, kv_lens, new_tokens, free_blocks, free_start,
                                       block_size, max_tokens, slot_dtype=slot_dtype)
    requests, width, stride = _tables_layout(block_tables)
    dev = block_tables.device
    kv = _vector(_tensor(kv_lens, "kv_lens"), "kv_lens", torch.int32, requests, dev)
    new = _vector(_tensor(new_tokens, "new_tokens"), "new_tokens", torch.int32, requests, dev)
    num_free = free_blocks.numel() if _tensor(free_blocks, "free_blocks").dim() == 1 else -1
    free = _vector(free_blocks, "free_blocks", torch.int32, num_free, dev)
    start = _vector(_tensor(free_start, "free_start"), "free_start", torch.int32, 1, dev)
    max_tokens = _int32(max_tokens, "max_tokens")
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    _, wide = _slot_dtype(slot_dtype)
    # one allocation, each token array on a 16-byte boundary of it
    pad = -max_tokens % 4
    room = [max_tokens, pad, max_tokens, pad, max_tokens << wide, 2 * pad, requests + 1, 1]
    owner, _, positions, _, slots, _, starts, free_next = torch.empty(
        sum(room), dtype=torch.int32, device=dev).split_with_sizes(room)
    if wide:
        slots = slots.view(torch.int64)
    _check(_lib().topk_block_tables(
        block_tables.data_ptr(), stride, width, requests, kv, new, free, num_free, start,
        _int32(block_size, "block_size"), max_tokens, starts.data_ptr(), owner.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), wide, free_next.data_ptr(), _raw_stream(dev)))
    return starts, owner, positions, slots, free_next


def topk_slots(indices, block_tables, block_size, *, next_n=1, row_requests=None, slots=None,
               slot_dtype=None, stream=None):
    """Cache slots of selected positions: int32 [rows, k] local indices, as the
    selection returns them, to table[i // block_size] * block_size + i %
    block_size in the table row of request row_requests[r] (int32 [rows]), or
    r // next_n without it.  -1 (and any index the table does not reach) gives
    -1.  slots may be indices itself (int32)."""
    guard = _elsewhere(indices, "indices", stream)
    if guard is not None:
        with guard:
            return topk_slots(indices, block_tables, block_size, next_n=next_n,
                              row_requests=row_requests, slots=slots, slot_dtype=slot_dtype)
    if indices.dtype != torch.int32:
        raise TypeError(f"indices must be torch.int32, got {indices.dtype}")
    if indices.dim() != 2 or not indices.is_contiguous():
        raise ValueError("indices must be a contiguous int32 [rows, k] tensor")
    rows, k = indices.shape
    _fits("indices", rows, k)
    dev = indices.device
    requests, width, stride = _tables_layout(block_tables)
    if block_tables.device != dev:
        raise ValueError(f"block_tables must be on {dev}")
    next_n = _int32(next_n, "next_n")
    owner = _vector(row_requests, "row_requests", torch.int32, rows, dev)
    if owner is None and next_n >= 1 and requests < (rows + next_n - 1) // next_n:
        raise ValueError(f"block_tables must hold {(rows + next_n - 1) // next_n} requests")
    if slots is not None and slot_dtype is None:
        slot_dtype = slots.dtype
    dt, wide = _slot_dtype(slot_dtype)
    slots = _matrix(slots, "slots", dt, (rows, k), dev)
    _check(_lib().topk_slots(indices.data_ptr(), rows, k, block_tables.data_ptr(), stride, width,
                             requests, owner, next_n, _int32(block_size, "block_size"),
                             slots.data_ptr(), wide, _raw_stream(dev)))
    return slots
