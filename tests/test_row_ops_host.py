"""Refusals of the row operators: the C calls' status codes, decided on the
host before anything touches a device, and the binding's own checks."""
import pytest

ert = pytest.importorskip("exact_row_top_amd")

P = 1 << 20  # a fake, 16-byte aligned "device" address (never dereferenced)
INT = 2 ** 31 - 1


def _sample(logits=P, dtype=0, stride=100, vocab=100, rows=2, u=P, t=P, k=P, p=P, m=P, tokens=2 * P,
            logprobs=3 * P, flags=0, ws=P, ws_bytes=1 << 20):
    return ert.load_library().topk_sample(logits, dtype, stride, vocab, rows, u, t, k, p, m, tokens,
                                          logprobs, flags, ws, ws_bytes, None)


def _route(logits=P, dtype=0, stride=64, tokens=4, experts=64, k=8, bias=P, groups=8, tg=4, flags=0,
           idx=P, w=P):
    return ert.load_library().topk_route(logits, dtype, stride, tokens, experts, k, bias, groups, tg,
                                         flags, 1.0, idx, w, None)


def _grad(logits=P, dtype=0, stride=64, tokens=4, experts=64, k=8, flags=0, idx=P, g=P, out=P,
          out_stride=64):
    return ert.load_library().topk_route_backward(logits, dtype, stride, tokens, experts, k, flags,
                                                  1.0, idx, g, out, out_stride, None)


def _tables(tables=P, stride=10, width=10, requests=3, kv=P, new=P, free=P, num_free=5, start=P,
            bs=16, most=7, starts=P, owner=P, pos=P, slots=P, wide=0, nxt=2 * P):
    return ert.load_library().topk_block_tables(tables, stride, width, requests, kv, new, free, num_free,
                                                start, bs, most, starts, owner, pos, slots, wide, nxt,
                                                None)


def _slots(idx=P, rows=2, k=5, tables=P, stride=10, width=10, requests=2, owner=None, next_n=1, bs=16,
           slots=2 * P, wide=0):
    return ert.load_library().topk_slots(idx, rows, k, tables, stride, width, requests, owner, next_n,
                                         bs, slots, wide, None)


EINVAL, ELAYOUT, EWORKSPACE = 1, 2, 3

REFUSALS = [
    (_sample, EINVAL, [dict(rows=-1), dict(dtype=3), dict(dtype=-1), dict(vocab=0), dict(stride=99),
                       dict(vocab=(1 << 20) + 1, stride=1 << 21), dict(flags=2), dict(logits=None),
                       dict(u=None), dict(tokens=None),
                       dict(rows=INT, vocab=1 << 20, stride=1 << 20), dict(tokens=P), dict(tokens=P + 4),
                       dict(k=2 * P), dict(k=2 * P + 4), dict(logprobs=2 * P + 4), dict(p=3 * P)]),
    (_sample, ELAYOUT, [dict(logits=P + 2), dict(logits=P + 1, dtype=1), dict(u=P + 2), dict(t=P + 1),
                        dict(k=P + 2), dict(p=P + 2), dict(m=P + 3), dict(tokens=P + 2),
                        dict(logprobs=P + 2), dict(ws=P + 8)]),
    (_sample, EWORKSPACE, [dict(ws=None), dict(ws_bytes=1087), dict(ws_bytes=0)]),
    (_route, EINVAL, [dict(tokens=-1), dict(experts=0), dict(experts=1025, stride=2000, groups=1, tg=1),
                      dict(k=0), dict(k=65), dict(experts=4, k=5, groups=1, tg=1), dict(dtype=7),
                      dict(stride=63), dict(groups=0), dict(groups=17), dict(groups=3), dict(tg=0),
                      dict(tg=9), dict(flags=8), dict(logits=None), dict(idx=None), dict(w=None),
                      dict(experts=64, groups=32, tg=2)]),
    (_route, ELAYOUT, [dict(logits=P + 2), dict(bias=P + 2), dict(idx=P + 2), dict(w=P + 1)]),
    (_grad, EINVAL, [dict(tokens=-1), dict(experts=0), dict(k=0), dict(k=65), dict(dtype=3),
                     dict(stride=63), dict(out_stride=63), dict(flags=8), dict(logits=None),
                     dict(idx=None), dict(g=None), dict(out=None)]),
    (_grad, ELAYOUT, [dict(logits=P + 2), dict(idx=P + 2), dict(g=P + 2), dict(out=P + 2),
                      dict(out=P + 1, dtype=1)]),
    (_tables, EINVAL, [dict(requests=-1), dict(requests=4097), dict(width=-1), dict(stride=9),
                       dict(num_free=-1), dict(bs=0), dict(bs=(1 << 30) + 1), dict(most=-1),
                       dict(most=1 << 31), dict(wide=2), dict(start=None), dict(nxt=None),
                       dict(nxt=P), dict(starts=None), dict(kv=None), dict(new=None),
                       dict(tables=None), dict(free=None), dict(owner=None), dict(pos=None),
                       dict(slots=None)]),
    (_tables, ELAYOUT, [dict(tables=P + 2), dict(kv=P + 2), dict(new=P + 2), dict(free=P + 2),
                        dict(start=P + 2), dict(starts=P + 2), dict(owner=P + 2), dict(pos=P + 2),
                        dict(slots=P + 2), dict(slots=P + 4, wide=1), dict(nxt=2 * P + 2)]),
    (_slots, EINVAL, [dict(rows=-1), dict(rows=1 << 31), dict(k=0), dict(width=-1), dict(stride=9),
                      dict(requests=-1), dict(bs=0), dict(next_n=0), dict(wide=-1), dict(idx=None),
                      dict(slots=None), dict(tables=None), dict(slots=P, wide=1)]),
    (_slots, ELAYOUT, [dict(idx=P + 2), dict(tables=P + 2), dict(owner=P + 2), dict(slots=P + 2),
                       dict(slots=P + 4, wide=1)]),
]


@pytest.mark.parametrize("call,status,changes", REFUSALS,
                         ids=[f"{c.__name__}-{s}" for c, s, _ in REFUSALS])
def test_c_refusals(call, status, changes):
    for change in changes:
        assert call(**change) == status, change


def test_c_empty_calls_do_nothing():
    assert _sample(rows=0, logits=None, u=None, tokens=None, ws=None, ws_bytes=0) == 0
    assert _route(tokens=0, logits=None, idx=None, w=None) == 0
    assert _grad(tokens=0, logits=None, idx=None, g=None, out=None) == 0
    assert _slots(rows=0, idx=None, tables=None, slots=None) == 0


def test_sample_workspace_bytes():
    f = ert.load_library().topk_sample_workspace_bytes
    assert f(0, 100) == 0 and f(-1, 100) == 0 and f(1, 0) == 0 and f(1, (1 << 20) + 1) == 0
    one = f(1, 1)
    assert one > 0 and f(2, 2041) == 2 * one and f(1, 2042) > one
    assert f(3, 1 << 20) == 3 * f(1, 1 << 20) > 3 * 512 * 32


def test_binding_refuses_host_tensors_and_wrong_arguments():
    import torch
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        ert.sample_tokens(x, torch.zeros(2))
    with pytest.raises(TypeError):
        ert.sample_tokens([[0.0]], torch.zeros(1))
    from exact_row_top_amd import row_ops
    assert row_ops._int32(-5, "n") == -5
    with pytest.raises(TypeError):
        row_ops._int32(2.0, "n")
    with pytest.raises(ValueError):
        row_ops._int32(1 << 31, "n")
    for shape in ((1 << 31, 1), (1, (1 << 32) + 5)):  # would be cut to 32 bits on the way to the C call
        with pytest.raises(ValueError):
            row_ops._scores(torch.empty(shape, dtype=torch.float16, device="meta"), "logits")
    with pytest.raises(ValueError):
        ert.route_experts(x, 2)
    with pytest.raises(ValueError):
        ert.route_experts(x, 2, scoring="relu")
    with pytest.raises(ValueError):
        ert.route_experts(x, 2, group_score="sum")
    with pytest.raises(ValueError):
        ert.route_experts_backward(torch.zeros(2, 2), x, torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        ert.topk_slots(torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        ert.extend_block_tables(torch.zeros(2, 2, dtype=torch.int32), *[torch.zeros(2, dtype=torch.int32)] * 3,
                                torch.zeros(1, dtype=torch.int32), 16, 4)


@pytest.mark.gpu
def test_binding_refusals_on_the_device():
    import torch
    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")
    x, u = z(4, 100), z(4)
    i32 = torch.int32
    bad_type = [lambda: ert.sample_tokens(x.double(), u), lambda: ert.sample_tokens(x, u.double()),
                lambda: ert.sample_tokens(x, u, top_k=z(4)), lambda: ert.sample_tokens(x, None),
                lambda: ert.sample_tokens(x, u, tokens=z(4)),
                lambda: ert.route_experts(x.long(), 2), lambda: ert.route_experts(x, 2, bias=z(100, dtype=i32)),
                lambda: ert.route_experts_backward(z(4, 2).half(), x, z(4, 2, dtype=i32)),
                lambda: ert.route_experts_backward(z(4, 2), x, z(4, 2, dtype=torch.int64)),
                lambda: ert.route_experts(x, 2.0),
                lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4, dtype=i32), 16.0),
                lambda: ert.topk_slots(x, z(4, 4, dtype=i32), 16),
                lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4), 16),
                lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4, dtype=i32), 16, slot_dtype=torch.int16),
                lambda: ert.extend_block_tables(z(4, 4), *[z(4, dtype=i32)] * 3, z(1, dtype=i32), 16, 4)]
    for f in bad_type:
        with pytest.raises(TypeError):
            f()
    bad_value = [lambda: ert.sample_tokens(x[0], u), lambda: ert.sample_tokens(x.t(), z(100)),
                 lambda: ert.sample_tokens(z(100).expand(4, 100), u), lambda: ert.sample_tokens(x, z(3)),
                 lambda: ert.sample_tokens(x, z(8)[::2]), lambda: ert.sample_tokens(x, u.cpu()),
                 lambda: ert.sample_tokens(x, u, tokens=z(5, dtype=i32)),
                 lambda: ert.route_experts(x, 0), lambda: ert.route_experts(x, 1 << 40),
                 lambda: ert.route_experts(x, 2, bias=z(99)), lambda: ert.route_experts(x, 2, indices=z(4, 3, dtype=i32)),
                 lambda: ert.route_experts_backward(z(4, 3), x, z(4, 2, dtype=i32)),
                 lambda: ert.route_experts_backward(z(4, 2), x, z(3, 2, dtype=i32)),
                 lambda: ert.topk_slots(z(4, 4, dtype=i32)[:, ::2], z(4, 4, dtype=i32), 16),
                 lambda: ert.topk_slots(z(4, 4, dtype=i32), z(3, 4, dtype=i32), 16),
                 lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4, dtype=i32).t()[:, ::2], 16),
                 lambda: ert.extend_block_tables(z(4, 4, dtype=i32), z(3, dtype=i32), z(4, dtype=i32),
                                                 z(4, dtype=i32), z(1, dtype=i32), 16, 4),
                 lambda: ert.extend_block_tables(z(4, 4, dtype=i32), *[z(4, dtype=i32)] * 3, z(1, dtype=i32), 16, -1)]
    for f in bad_value:
        with pytest.raises(ValueError):
            f()
    bad_call = [lambda: ert.sample_tokens(z(1, (1 << 20) + 1), z(1)), lambda: ert.sample_tokens(x[:, :0], u),
                lambda: ert.route_experts(x, 65), lambda: ert.route_experts(x, 2, num_groups=3),
                lambda: ert.route_experts(x, 2, num_groups=4, topk_groups=5), lambda: ert.route_experts(z(4, 1025), 2),
                lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4, dtype=i32), 0),
                lambda: ert.topk_slots(z(4, 4, dtype=i32), z(4, 4, dtype=i32), 16, next_n=0),
                lambda: ert.extend_block_tables(z(4097, 4, dtype=i32), *[z(4097, dtype=i32)] * 3, z(1, dtype=i32), 16, 4)]
    for f in bad_call:
        with pytest.raises(ert.TopKError):
            f()
