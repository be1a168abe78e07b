"""Refusals of a beam search's operators: the C calls' status codes, decided on
the host before anything touches a device, and the binding's own checks."""
import ctypes

import pytest

ert = pytest.importorskip("exact_row_top_amd")

P = 1 << 24          # fake, aligned "device" addresses (never dereferenced), far apart
INT = 2 ** 31 - 1
EINVAL, ELAYOUT, EWORKSPACE = 1, 2, 3


def _at(n):
    return P * (n + 1)


def _beams(logits=_at(0), dtype=0, stride=100, vocab=100, requests=2, beams=4, k=8, scores=_at(1), ended=_at(2), end=3,
           lengths=_at(3), penalty=1.0, out=_at(4), parents=_at(5), tokens=_at(6), ws=_at(7), ws_bytes=1 << 20):
    return ert.load_library().topk_beams(logits, dtype, stride, vocab, requests, beams, k, scores, ended, end, lengths,
                                         penalty, out, parents, tokens, ws, ws_bytes, None)


def _rows(n=1, src=_at(0), dst=_at(1), ss=64, ds=64, size=64, parents=_at(2), requests=2, beams=4, k=4, clear=0):
    arr = lambda t, v: (t * max(n, 1))(*[v] * max(n, 1))  # noqa: E731
    return ert.load_library().topk_reorder_rows(n, arr(ctypes.c_void_p, src), arr(ctypes.c_void_p, dst),
                                                arr(ctypes.c_int64, ss), arr(ctypes.c_int64, ds),
                                                arr(ctypes.c_int64, size), parents, requests, beams, k, clear, None)


def _blocks(tables=_at(0), stride=10, width=10, lens=_at(1), parents=_at(2), requests=2, beams=4, k=4, bs=16, tail=_at(3),
            out=_at(4), out_stride=10, n=1, cache=_at(5), blocks=50, slot=64):
    caches = (ctypes.c_void_p * max(n, 1))(*[cache] * max(n, 1))
    return ert.load_library().topk_reorder_blocks(tables, stride, width, lens, parents, requests, beams, k, bs, tail, out,
                                                  out_stride, n, caches, blocks, slot, None)


def _attend(q=_at(0), dtype=1, qs=1024, qh=128, seqs=6, next_n=1, heads=8, kv=2, dim=128, kc=_at(1), kb=4096, ks=256, kh=128,
            vc=_at(2), vb=4096, vs=256, vh=128, blocks=100, bs=16, st=_at(3), ss=8, sw=8, sl=_at(4), starts=_at(5), groups=3,
            ot=_at(6), os=4, ow=4, ol=_at(7), scale=1.0, ms=0, mo=0, out=_at(8), lse=_at(9), ws=_at(10), ws_bytes=1 << 23):
    return ert.load_library().topk_attend(q, dtype, qs, qh, seqs, next_n, heads, kv, dim, kc, kb, ks, kh, vc, vb, vs, vh,
                                          blocks, bs, st, ss, sw, sl, starts, groups, ot, os, ow, ol, scale, ms, mo, out,
                                          lse, ws, ws_bytes, None)


def _mass(q=_at(0), dtype=1, qs=1024, qh=128, seqs=6, next_n=1, heads=8, kv=2, dim=128, kc=_at(1), kb=4096, ks=256, kh=128,
          blocks=100, bs=16, st=_at(3), ss=8, sw=8, sl=_at(4), starts=_at(5), groups=3, ot=_at(6), os=4, ow=4, ol=_at(7),
          scale=1.0, lse=_at(9), decay=1.0, pm=_at(10), po=_at(11), pn=128, om=_at(12), oo=_at(13), on=64):
    return ert.load_library().topk_attend_mass(q, dtype, qs, qh, seqs, next_n, heads, kv, dim, kc, kb, ks, kh, blocks, bs, st,
                                               ss, sw, sl, starts, groups, ot, os, ow, ol, scale, lse, decay, pm, po, pn, om,
                                               oo, on, None)


def _keep(mass=_at(0), rs=400, hs=200, n=200, requests=2, heads=2, lens=_at(1), budget=50, sinks=4, recent=10, kept=_at(2),
          out=_at(3), width=50, new=_at(4)):
    return ert.load_library().topk_evict_keep(mass, rs, hs, n, requests, heads, lens, budget, sinks, recent, kept, out, width,
                                              new, None)


def _move(kept=_at(0), requests=2, heads=2, budget=50, tables=_at(1), stride=8, width=8, to=_at(2), to_stride=4, to_width=4,
          bs=16, n=1, cache=_at(3), blocks=50, slot=512):
    caches = (ctypes.c_void_p * max(n, 1))(*[cache] * max(n, 1))
    return ert.load_library().topk_evict_move(kept, requests, heads, budget, tables, stride, width, to, to_stride, to_width,
                                              bs, n, caches, blocks, slot, None)


SHAPES = [dict(dtype=0), dict(dtype=3), dict(seqs=-1), dict(next_n=0), dict(next_n=1025), dict(heads=0), dict(kv=0),
          dict(kv=3), dict(dim=96), dict(dim=0), dict(bs=0), dict(bs=(1 << 20) + 1), dict(blocks=-1), dict(groups=-1),
          dict(seqs=INT // 8 + 1), dict(starts=None, seqs=7), dict(scale=-1.0), dict(scale=float("nan")),
          dict(scale=float("inf")), dict(qs=-8), dict(kb=-8), dict(q=None), dict(kc=None), dict(sw=-1), dict(ss=7),
          dict(ow=-1), dict(os=3), dict(st=None), dict(sl=None), dict(ot=None), dict(ol=None),
          dict(sw=1 << 27, ss=1 << 27)]
SHAPES_AT = [dict(q=_at(0) + 8), dict(qs=1028), dict(qh=4), dict(kc=_at(1) + 2), dict(kb=4100), dict(ks=257), dict(kh=4),
             dict(st=_at(3) + 2), dict(sl=_at(4) + 1), dict(ot=_at(6) + 2), dict(ol=_at(7) + 3), dict(starts=_at(5) + 2),
             dict(lse=_at(9) + 2)]
REFUSALS = [
    (_beams, EINVAL, [dict(requests=-1), dict(beams=0), dict(beams=33), dict(k=0), dict(k=65), dict(dtype=3), dict(vocab=0),
                      dict(vocab=(1 << 20) + 1, stride=1 << 21), dict(stride=99), dict(penalty=float("inf")),
                      dict(penalty=float("nan")), dict(end=-1), dict(end=100), dict(logits=None), dict(scores=None),
                      dict(out=None), dict(parents=None), dict(tokens=None), dict(requests=INT // 4, vocab=1 << 20, stride=1 << 20),
                      dict(out=_at(1)), dict(parents=_at(3) + 4), dict(tokens=_at(5) + 32), dict(parents=_at(2))]),
    (_beams, ELAYOUT, [dict(logits=_at(0) + 2), dict(logits=_at(0) + 1, dtype=1), dict(scores=_at(1) + 2),
                       dict(lengths=_at(3) + 2), dict(out=_at(4) + 1), dict(parents=_at(5) + 2), dict(tokens=_at(6) + 2),
                       dict(ws=_at(7) + 8)]),
    (_beams, EWORKSPACE, [dict(ws=None), dict(ws_bytes=0), dict(ws_bytes=3000)]),
    (_rows, EINVAL, [dict(n=-1), dict(requests=-1), dict(beams=0), dict(beams=33), dict(k=0), dict(k=33), dict(clear=2),
                     dict(parents=None), dict(src=None), dict(dst=None), dict(size=-1), dict(ss=63), dict(ds=63),
                     dict(dst=_at(0) + 64), dict(dst=_at(0), ds=128), dict(dst=_at(0), k=3), dict(dst=_at(2)),
                     dict(size=1 << 41, ss=1 << 41, ds=1 << 41), dict(ss=1 << 60), dict(ds=1 << 60),
                     dict(n=2), dict(n=3, dst=_at(0))]),
    (_rows, ELAYOUT, [dict(parents=_at(2) + 2)]),
    (_blocks, EINVAL, [dict(requests=-1), dict(beams=0), dict(beams=33), dict(k=0), dict(k=33), dict(width=-1), dict(stride=9),
                       dict(out_stride=9), dict(bs=0), dict(n=-1), dict(n=65), dict(blocks=-1), dict(slot=-1),
                       dict(tail=None, k=3), dict(lens=None), dict(parents=None), dict(tables=None), dict(out=None),
                       dict(cache=None), dict(out=_at(0) + 16), dict(out=_at(0), out_stride=12), dict(out=_at(1)),
                       dict(out=_at(2)), dict(out=_at(3)), dict(n=2)]),
    (_blocks, ELAYOUT, [dict(tables=_at(0) + 2), dict(lens=_at(1) + 2), dict(parents=_at(2) + 1), dict(tail=_at(3) + 2),
                        dict(out=_at(4) + 2)]),
    (_attend, EINVAL, SHAPES + [dict(out=None), dict(vc=None), dict(vs=-8), dict(ms=-1), dict(mo=-1)]),
    (_attend, ELAYOUT, SHAPES_AT + [dict(vc=_at(2) + 8), dict(vb=4100), dict(out=_at(8) + 8), dict(ws=_at(10) + 4)]),
    (_attend, EWORKSPACE, [dict(ws=None), dict(ws_bytes=100)]),
    (_mass, EINVAL, SHAPES + [dict(lse=None), dict(decay=float("nan")), dict(pn=-1), dict(on=-1), dict(po=None), dict(oo=None),
                              dict(po=_at(10) + 4), dict(oo=_at(12) + 4), dict(oo=_at(11)), dict(po=_at(12)), dict(oo=_at(10)),
                              dict(po=_at(9)), dict(oo=_at(9) + 4)]),
    (_mass, ELAYOUT, SHAPES_AT + [dict(pm=_at(10) + 2), dict(po=_at(11) + 2), dict(om=_at(12) + 2), dict(oo=_at(13) + 1)]),
    (_keep, EINVAL, [dict(requests=-1), dict(heads=0), dict(n=-1), dict(rs=-1), dict(hs=-1), dict(budget=0), dict(sinks=-1),
                     dict(recent=-1), dict(sinks=41), dict(width=49), dict(mass=None), dict(lens=None), dict(kept=None),
                     dict(new=None), dict(new=_at(1)), dict(kept=_at(0) + 8), dict(out=_at(0)), dict(out=_at(2)),
                     dict(new=_at(2)), dict(kept=_at(1)), dict(requests=1 << 30)]),
    (_keep, ELAYOUT, [dict(mass=_at(0) + 2), dict(lens=_at(1) + 2), dict(kept=_at(2) + 2), dict(out=_at(3) + 2),
                      dict(new=_at(4) + 1)]),
    (_move, EINVAL, [dict(requests=-1), dict(heads=0), dict(budget=0), dict(width=-1), dict(stride=7), dict(to_width=-1),
                     dict(to_stride=3), dict(bs=0), dict(n=-1), dict(n=65), dict(blocks=-1), dict(slot=-16), dict(slot=513),
                     dict(slot=48), dict(to=_at(1)), dict(n=2), dict(kept=None), dict(tables=None), dict(to=None), dict(cache=None)]),
    (_move, ELAYOUT, [dict(kept=_at(0) + 2), dict(tables=_at(1) + 2), dict(to=_at(2) + 2), dict(cache=_at(3) + 8)]),
]


@pytest.mark.parametrize("call,status,changes", REFUSALS, ids=[f"{c.__name__}-{s}" for c, s, _ in REFUSALS])
def test_c_refusals(call, status, changes):
    for change in changes:
        assert call(**change) == status, change


def test_c_empty_calls_do_nothing():
    assert _beams(requests=0, logits=None, scores=None, out=None, parents=None, tokens=None, ws=None, ws_bytes=0) == 0
    assert _rows(n=0, parents=None) == 0 and _rows(requests=0, src=None, dst=None, parents=None) == 0
    assert _blocks(requests=0, tables=None, lens=None, parents=None, out=None) == 0
    assert _attend(seqs=0, q=None, out=None, ws=None, ws_bytes=0) == 0
    assert _mass(seqs=0, groups=0, starts=None, q=None, lse=None, pm=None, po=None, om=None, oo=None) == 0
    assert _keep(requests=0, mass=None, lens=None, kept=None, out=None, new=None) == 0
    assert _move(requests=0, kept=None, tables=None, to=None) == 0 and _move(n=0, kept=None) == 0


def test_workspace_bytes():
    f = ert.load_library().topk_beams_workspace_bytes
    assert f(0, 4, 4, 100) == f(1, 0, 4, 100) == f(1, 33, 4, 100) == f(1, 4, 0, 100) == f(1, 4, 65, 100) == 0
    assert f(1, 4, 4, 0) == f(1, 4, 4, (1 << 20) + 1) == 0
    assert 0 < f(1, 1, 1, 1) < f(1, 1, 1, 2049) < f(2, 1, 1, 2049) and f(1, 1, 1, 2048) == f(1, 1, 1, 1)
    g = ert.load_library().topk_attend_workspace_bytes
    assert g(1, 0, 0, 1, 8, 2, 128, 100, 100) == g(1, 4, 0, 1, 8, 3, 128, 100, 100) == g(1, 4, 0, 1, 8, 2, 96, 100, 100) == 0
    assert g(1, 4, 0, 1, 8, 2, 128, 0, 0) >= 0
    # never less than one partial row of each kind for every token and head
    assert g(2, 4, 1, 1, 8, 2, 128, 1000, 100) >= 2 * 4 * 8 * (128 * 4 + 8)


def test_binding_refuses_host_tensors_and_wrong_arguments():
    import torch
    i32 = torch.int32
    x, s, p = torch.zeros(4, 8), torch.zeros(2, 2), torch.zeros(2, 2, dtype=i32)
    with pytest.raises(ValueError):
        ert.select_beams(x, s, 2)
    with pytest.raises(TypeError):
        ert.select_beams([[0.0]], s, 2)
    with pytest.raises(ValueError):
        ert.reorder_beams(x, p)
    with pytest.raises(TypeError):
        ert.reorder_beams(x, [[0]])
    with pytest.raises(ValueError):
        ert.reorder_block_tables(torch.zeros(4, 3, dtype=i32), torch.zeros(2, dtype=i32), p, 16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ert.prefix_attention(q, cache, cache, None, None, p, torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        ert.attention_mass(q, cache, torch.zeros(2, 4), None, None, p, torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        ert.evict_cache(torch.zeros(1, 1, 9), torch.zeros(1, dtype=i32), 4)
    from exact_row_top_amd import search_ops
    with pytest.raises(ValueError):
        search_ops._caches([torch.empty(1 << 31, 1, dtype=torch.uint8, device="meta")], 1, torch.device("meta"))


@pytest.mark.gpu
def test_binding_refusals_on_the_device():
    import torch
    i32, bf = torch.int32, torch.bfloat16

    def z(*shape, dtype=torch.float32):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    x, s, p = z(6, 100), z(2, 3), z(2, 3, dtype=i32)
    q, c = z(6, 4, 64, dtype=bf), z(9, 16, 2, 64, dtype=bf)
    pt, pl, t, n = z(2, 3, dtype=i32), z(2, dtype=i32), z(6, 2, dtype=i32), z(6, dtype=i32)
    m, lens, ot = z(2, 2, 48), z(2, dtype=i32), z(2, 1, dtype=i32)

    def attend(q=q, k=c, v=c, pt=pt, pl=pl, t=t, n=n, **kw):
        return ert.prefix_attention(q, k, v, pt, pl, t, n, **kw)

    def mass(q=q, k=c, lse=z(6, 4), pt=pt, pl=pl, t=t, n=n, **kw):
        return ert.attention_mass(q, k, lse, pt, pl, t, n, **kw)

    def evict(m=m, lens=lens, budget=4, **kw):
        return ert.evict_cache(m, lens, budget, **kw)

    bad_type = [lambda: ert.select_beams(x.double(), s, 2), lambda: ert.select_beams(x, s.double(), 2),
                lambda: ert.select_beams(x, s, 2.0), lambda: ert.select_beams(x, None, 2),
                lambda: ert.select_beams(x, s, 2, ended=s), lambda: ert.select_beams(x, s, 2, lengths=s),
                lambda: ert.reorder_beams(x, p.long()), lambda: ert.reorder_beams([1], p),
                lambda: ert.reorder_block_tables(x, lens, p, 16), lambda: ert.reorder_block_tables(t, lens.long(), p, 16),
                lambda: ert.reorder_block_tables(t, lens, p, 16.0), lambda: ert.reorder_block_tables(t, None, p, 16),
                lambda: attend(q=q.float()), lambda: attend(k=c.half()), lambda: attend(v=c.half()),
                lambda: attend(pt=pt.long()), lambda: attend(n=n.long()), lambda: attend(n=None),
                lambda: attend(next_n=1.0), lambda: attend(group_starts=pl.float()), lambda: mass(lse=z(6, 4).double()),
                lambda: mass(lse=None), lambda: mass(mass=z(6, 2, 32, dtype=bf)), lambda: evict(m=m.half()),
                lambda: evict(lens=lens.long()), lambda: evict(budget=4.0),
                lambda: evict(block_tables=pt, caches=[None])]
    for i, f in enumerate(bad_type):
        with pytest.raises(TypeError):
            f()
            pytest.fail(f"call {i} was taken")
    bad_value = [lambda: ert.select_beams(x, z(2, 4), 2), lambda: ert.select_beams(x, s[0], 2), lambda: ert.select_beams(x, s, 0),
                 lambda: ert.select_beams(x, s.cpu(), 2), lambda: ert.select_beams(x.t(), z(20, 5), 2),
                 lambda: ert.select_beams(x, s, 2, ended=z(2, 2, dtype=torch.bool)), lambda: ert.select_beams(x, s, 1 << 40),
                 lambda: ert.reorder_beams(z(5, 4), p), lambda: ert.reorder_beams(z(6, 4), p[0]),
                 lambda: ert.reorder_beams(z(6, 4, 4).transpose(1, 2), p), lambda: ert.reorder_beams(z(4).expand(6, 4), p),
                 lambda: ert.reorder_beams([x, x], p, out=[x]), lambda: ert.reorder_beams(x, p, out=z(6, 99)),
                 lambda: ert.reorder_beams(x, p, out=z(6, 100, dtype=i32)), lambda: ert.reorder_beams(x.cpu(), p),
                 lambda: ert.reorder_block_tables(z(5, 2, dtype=i32), lens, p, 16),
                 lambda: ert.reorder_block_tables(z(4, 2, dtype=i32), lens, p, 16),
                 lambda: ert.reorder_block_tables(t, z(3, dtype=i32), p, 16),
                 lambda: ert.reorder_block_tables(t, lens, p, 16, caches=[z(4, 8, 2)]),
                 lambda: ert.reorder_block_tables(t, lens, p, 16, caches=[z(4, 16, 2), z(4, 16, 3)]),
                 lambda: ert.reorder_block_tables(t, lens, p, 16, out=z(6, 3, dtype=i32)),
                 lambda: ert.reorder_block_tables(t, lens, p, 16, tail_blocks=z(5, dtype=i32)),
                 lambda: attend(q=q[0]), lambda: attend(q=z(6, 5, 64, dtype=bf)), lambda: attend(q=z(6, 4, 128, dtype=bf)),
                 lambda: attend(v=z(9, 16, 1, 64, dtype=bf)), lambda: attend(t=t[:5]), lambda: attend(n=n[:5]),
                 lambda: attend(next_n=4), lambda: attend(next_n=0), lambda: attend(pt=None),
                 lambda: attend(pt=z(4, 3, dtype=i32), pl=z(4, dtype=i32)), lambda: attend(group_starts=pl),
                 lambda: attend(max_len=-1), lambda: attend(out=z(6, 4, 64, dtype=bf)[:5]),
                 lambda: attend(q=z(6, 4, 128, dtype=bf)[:, :, ::2]), lambda: mass(lse=z(6, 5)), lambda: mass(mass=z(6, 1, 32)),
                 lambda: mass(mass=z(6, 2, 32), out=z(6, 2, 33)), lambda: mass(pt=None, pl=None, prefix_mass=m),
                 lambda: evict(budget=0), lambda: evict(sinks=3, recent=2), lambda: evict(sinks=-1),
                 lambda: evict(lens=lens[:1]), lambda: evict(m=m[0]), lambda: evict(mass_out=z(2, 2, 3)),
                 lambda: evict(caches=[c]), lambda: evict(block_tables=t, caches=[c]),
                 lambda: evict(block_tables=pt, caches=[z(9, 16, 3, 64)]), lambda: evict(block_tables=pt, caches=[z(9, 16, 2, 2)]),
                 lambda: evict(block_tables=pt, caches=[c], out_tables=ot[:1]), lambda: evict(m=z(2, 2, 96)[:, :, ::2])]
    for i, f in enumerate(bad_value):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    bad_call = [lambda: ert.select_beams(x, s, 65), lambda: ert.select_beams(z(33, 10), z(1, 33), 2),
                lambda: ert.select_beams(x, s, 2, length_penalty=float("nan")),
                lambda: ert.select_beams(x, s, 2, ended=z(2, 3, dtype=torch.bool), end_token=100),
                lambda: ert.reorder_beams(z(33, 4), z(1, 33, dtype=i32)), lambda: ert.reorder_beams(z(6, 4), p, beams=0),
                lambda: (lambda b: ert.reorder_beams(b[:6], p, out=b[1:7]))(z(7, 4)),
                lambda: ert.reorder_block_tables(t, lens, p, 0), lambda: attend(scale=-1.0),
                lambda: attend(q=z(6, 4, 96, dtype=bf), k=z(9, 16, 2, 96, dtype=bf), v=z(9, 16, 2, 96, dtype=bf)),
                lambda: attend(q=z(6, 4, 68, dtype=bf)[:, :, 4:]), lambda: mass(decay=float("inf"))]
    for i, f in enumerate(bad_call):
        with pytest.raises((ert.TopKError, ValueError)):
            f()
            pytest.fail(f"call {i} was taken")


def test_c_refusals_of_bounded_mass():
    """The bounds, and the checks that it shares with the call without them."""
    f = ert.load_library().topk_attend_mass_bounded

    def call(ms=0, mo=0, dim=128, lse=_at(9), po=_at(11), q=_at(0), scale=1.0, seqs=6):
        return f(q, 1, 1024, 128, seqs, 1, 8, 2, dim, _at(1), 4096, 256, 128, 100, 16, _at(3), 8, 8, _at(4), _at(5), 3,
                 _at(6), 4, 4, _at(7), scale, ms, mo, lse, 1.0, _at(10), po, 128, _at(12), _at(13), 64, None)

    for change in (dict(ms=-1), dict(mo=-1), dict(dim=96), dict(lse=None), dict(po=None), dict(q=None), dict(scale=-1.0)):
        assert call(**change) == EINVAL, change
    for change in (dict(q=_at(0) + 8), dict(lse=_at(9) + 2), dict(po=_at(11) + 2)):
        assert call(**change) == ELAYOUT, change


def test_inline_assembly_that_uses_m0_says_so():
    """A load to LDS takes its place there from m0: as an operand, or the
    compiler may keep something of its own in it."""
    import glob
    import os
    import re
    found = 0
    for path in glob.glob(os.path.join(os.path.dirname(ert.__file__), "csrc", "*")):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for text in re.findall(r"\basm\b(?:\s+volatile)?\s*\((.*?)\);", src, flags=re.S):
            if re.search(r"\bm0\b|_load_lds|_lds_d", text):
                found += 1
                assert '"{m0}"' in text or '"m0"' in text, (os.path.basename(path), text)
    assert found
