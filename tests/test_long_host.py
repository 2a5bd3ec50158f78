"""Refusals of the operators for long contexts in front of any device work: the C
entries' checks of arguments and the binding's.  CPU only: every call here is
refused, addresses are only looked at."""
import ctypes

import pytest

A, B, C, D = (0x10000 * i for i in range(1, 5))  # 16-byte aligned


def pages_q4(sv, **kw):
    p = dict(k_qs=A, v_qs=B, k_scales=C, v_scales=D, layer_stride=0, n_layers=1, n_pages=4, n_kv_heads=2, page_size=64,
             head_dim=64, n_slots=3, max_pages=2, table=A, refs=B, len=C)
    p.update(kw)
    return sv.spec_pages_q4(*p.values())


def pages(sv, **kw):
    p = dict(k=A, v=B, layer_stride=0, n_layers=1, n_pages=4, n_kv_heads=2, page_size=64, head_dim=64, n_slots=3, max_pages=2,
             table=A, refs=B, len=C)
    p.update(kw)
    return sv.spec_pages(*p.values())


def digest(sv, **kw):
    p = dict(data=A, layer_stride=0, n_layers=1, n_pages=4, n_kv_heads=2, page_size=64, head_dim=64, block=32, n_slots=3,
             max_pages=2, table=A, len=B)
    p.update(kw)
    return sv.spec_digest(*p.values())


def tree(sv, **kw):
    p = dict(n_seq=1, nt=4, n_q_heads=8, window=0, sinks=0, scale=0.0, slots=A, parents=None, n_nodes=None)
    p.update(kw)
    return sv.spec_tree(*p.values())


def ref(x):
    return None if x is None else ctypes.byref(x)


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_round_gb300 as sv
    from speculative_decoding_verification_round_gb300 import _build
    _build.build()
    return sv


BAD_PAGES = [  # a cache's fields, and how they are refused
    (dict(k_qs=None), "INVALID"), (dict(v_qs=None), "INVALID"), (dict(k_scales=None), "INVALID"),
    (dict(v_scales=None), "INVALID"), (dict(k_qs=A + 8), "SHAPE"), (dict(v_scales=D + 2), "SHAPE"),
    (dict(head_dim=48), "SHAPE"), (dict(head_dim=0), "SHAPE"), (dict(head_dim=-32), "SHAPE"), (dict(n_layers=0), "SHAPE"),
    (dict(n_pages=0), "SHAPE"), (dict(n_kv_heads=-1), "SHAPE"), (dict(page_size=0), "SHAPE"),
    (dict(layer_stride=-1), "SHAPE"), (dict(n_layers=2, layer_stride=511), "SHAPE"),
    (dict(layer_stride=1 << 62), "SHAPE"), (dict(n_pages=2 ** 31 - 1, n_kv_heads=4096, page_size=4096), "SHAPE"),
]
BAD_BOOK = [
    (dict(table=None), "INVALID"), (dict(len=None), "INVALID"), (dict(n_slots=0), "SHAPE"), (dict(max_pages=0), "SHAPE"),
    (dict(max_pages=2 ** 26), "SHAPE"),
]


@pytest.mark.parametrize("fields,why", [(None, "INVALID")] + BAD_PAGES + BAD_BOOK)
def test_caches_in_4_bits(sv, fields, why):
    L, want = sv.lib(), getattr(sv, "SPEC_E_" + why)
    kv = None if fields is None else pages_q4(sv, **fields)
    n = ctypes.c_size_t()
    dg = digest(sv)
    calls = [lambda: L.spec_pages_q4_fork(ref(kv), 1, A, B, C, None), lambda: L.spec_pages_q4_free(ref(kv), 1, A, B, None),
             lambda: L.spec_pages_q4_extend(ref(kv), 1, A, B, C, D, None),
             lambda: L.spec_pages_q4_commit(ref(kv), 1, A, 1, A, B, 0, None, C, D + 4096, D, None),
             lambda: L.spec_pages_q4_read(ref(kv), 1, A, 1, A, B, C, D, 0, A, None),
             lambda: L.spec_tree_attn_q4_workspace(ref(kv), 1, 1, 2, ctypes.byref(n)),
             lambda: L.spec_tree_attn_q4(ref(kv), 0, ctypes.byref(tree(sv)), A, 0, B, C, 0, D, A << 8, 1 << 40, A, None),
             lambda: L.spec_block_attn_q4(ref(kv), 0, ctypes.byref(tree(sv)), 32, 2, A, A, 0, B, C, 0, D, A, None)]
    if fields is None or (fields, why) in BAD_PAGES:  # (table and len are not looked at)
        calls += [lambda: L.spec_pages_q4_copy(ref(kv), 1, A, B, None, C, None),
                  lambda: L.spec_block_digest_q4(ctypes.byref(dg), ref(kv), 1, A, None, B, None)]
    for call in calls:
        assert call() == want, sv.last_error()
        assert sv.last_error()


def test_rows_in_and_out(sv):
    L, kv = sv.lib(), ctypes.byref(pages_q4(sv))
    two = ctypes.byref(pages_q4(sv, n_layers=2, layer_stride=512))

    def commit(p=kv, n=1, slots=A, nt=4, k=A, v=B, stride=0, n_path=C, new_len=D, st=A):
        return L.spec_pages_q4_commit(p, n, slots, nt, k, v, stride, None, n_path, new_len, st, None)

    def read(p=kv, n=1, slots=A, nt=4, pos0=A, n_pos=B, k=C, v=D, stride=0, st=A):
        return L.spec_pages_q4_read(p, n, slots, nt, pos0, n_pos, k, v, stride, st, None)

    for f in (commit, read):
        for kw in (dict(slots=None), dict(k=None), dict(v=None), dict(st=None)):
            assert f(**kw) == sv.SPEC_E_INVALID
        for kw in (dict(n=0), dict(nt=0), dict(k=A + 4), dict(v=B + 8), dict(stride=12), dict(n=2 ** 31 - 1, nt=2 ** 31 - 1),
                   dict(p=two, stride=504), dict(p=two, stride=-8), dict(p=two, stride=1 << 60),
                   dict(n=2 ** 20, nt=2 ** 20)):
            assert f(**kw) == sv.SPEC_E_SHAPE, kw
    assert commit(n_path=None) == sv.SPEC_E_INVALID
    assert read(pos0=None) == sv.SPEC_E_INVALID and read(n_pos=None) == sv.SPEC_E_INVALID
    for off in (-8, -4, 4, 8):  # lengths that overlap the cache's without being them
        assert commit(new_len=C + off) == sv.SPEC_E_INVALID and "overlaps" in sv.last_error()


def test_page_lists(sv):
    L, kv = sv.lib(), ctypes.byref(pages_q4(sv))
    fixed = ctypes.byref(pages_q4(sv, refs=None))
    assert L.spec_pages_q4_copy(kv, 0, A, B, None, C, None) == sv.SPEC_E_SHAPE
    assert L.spec_pages_q4_copy(kv, 1, None, B, None, C, None) == sv.SPEC_E_INVALID
    assert L.spec_pages_q4_copy(kv, 1, A, B, None, None, None) == sv.SPEC_E_INVALID
    for f in (lambda p: L.spec_pages_q4_fork(p, 1, A, B, C, None), lambda p: L.spec_pages_q4_free(p, 1, A, B, None),
              lambda p: L.spec_pages_q4_extend(p, 1, A, B, C, D, None)):
        assert f(fixed) == sv.SPEC_E_UNSUPPORTED
    assert L.spec_pages_q4_extend(kv, 1, A, B, None, D, None) == sv.SPEC_E_INVALID
    assert L.spec_pages_q4_extend(kv, -1, A, B, C, D, None) == sv.SPEC_E_SHAPE


def attention_calls(sv):
    L, n = sv.lib(), ctypes.c_size_t()
    kv, f16 = pages_q4(sv), pages(sv)
    assert L.spec_tree_attn_q4_workspace is not None

    def tree_q4(t=None, layer=0, q=A, qs=0, kn=B, vn=C, ks=0, out=D, ws=A << 8, nb=1 << 40, st=A, p=kv, **kw):
        return L.spec_tree_attn_q4(ctypes.byref(p), layer, ctypes.byref(tree(sv, **kw)) if t is None else t, q, qs, kn, vn, ks,
                                   out, ws, nb, st, None)

    def block(q4):
        def f(t=None, layer=0, q=A, qs=0, kn=B, vn=C, ks=0, out=D, st=A, block=32, keep=2, blocks=A << 8, p=None, **kw):
            call = L.spec_block_attn_q4 if q4 else L.spec_block_attn
            return call(ctypes.byref(p or (kv if q4 else f16)), layer, ctypes.byref(tree(sv, **kw)) if t is None else t, block,
                        keep, blocks, q, qs, kn, vn, ks, out, st, None)
        return f
    return tree_q4, block(False), block(True)


def test_attention(sv):
    tree_q4, block, block_q4 = attention_calls(sv)
    for f in (tree_q4, block, block_q4):
        for kw in (dict(slots=None), dict(q=None), dict(kn=None), dict(vn=None), dict(out=None), dict(st=None),
                   dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")),
                   dict(out=A), dict(out=B + 16), dict(out=C - 16)):
            assert f(**kw) == sv.SPEC_E_INVALID, kw
        for kw in (dict(layer=-1), dict(layer=1), dict(n_seq=0), dict(nt=0), dict(nt=65), dict(n_q_heads=7), dict(n_q_heads=0),
                   dict(q=A + 2), dict(kn=B + 8), dict(out=D + 4), dict(qs=504), dict(qs=513), dict(ks=120), dict(ks=-128),
                   dict(qs=1 << 60), dict(n_seq=2 ** 31 - 1)):
            assert f(**kw) == sv.SPEC_E_SHAPE, kw
    assert tree_q4(ws=None) == sv.SPEC_E_INVALID and tree_q4(nb=16) == sv.SPEC_E_SHAPE and tree_q4(ws=(A << 8) + 4) == sv.SPEC_E_SHAPE
    assert tree_q4(ws=D) == sv.SPEC_E_INVALID and tree_q4(ws=A) == sv.SPEC_E_INVALID
    assert tree_q4(p=pages_q4(sv, head_dim=96)) == sv.SPEC_E_UNSUPPORTED
    for f, other in ((block, pages(sv, head_dim=96)), (block_q4, pages_q4(sv, head_dim=96))):
        assert f(window=1) == sv.SPEC_E_UNSUPPORTED and f(p=other) == sv.SPEC_E_UNSUPPORTED
        assert f(blocks=None) == sv.SPEC_E_INVALID and f(out=A << 8) == sv.SPEC_E_INVALID
        for kw in (dict(block=8), dict(block=48), dict(block=128), dict(block=0), dict(block=-16), dict(keep=0), dict(keep=4097)):
            assert f(**kw) == sv.SPEC_E_SHAPE, kw


BAD_DIGESTS = [(dict(data=None), "INVALID"), (dict(table=None), "INVALID"), (dict(len=None), "INVALID"),
               (dict(data=A + 8), "SHAPE"), (dict(n_layers=0), "SHAPE"), (dict(n_pages=0), "SHAPE"), (dict(n_kv_heads=0), "SHAPE"),
               (dict(page_size=0), "SHAPE"), (dict(n_slots=0), "SHAPE"), (dict(max_pages=0), "SHAPE"),
               (dict(head_dim=32), "UNSUPPORTED"), (dict(block=24), "SHAPE"), (dict(block=128), "SHAPE"), (dict(block=0), "SHAPE"),
               (dict(layer_stride=4), "SHAPE"), (dict(n_layers=2, layer_stride=2040), "SHAPE"), (dict(max_pages=2 ** 26), "SHAPE"),
               (dict(layer_stride=1 << 60), "SHAPE"),
               (dict(n_pages=2 ** 31 - 1, n_kv_heads=4096, page_size=4096, max_pages=1), "SHAPE")]


@pytest.mark.parametrize("fields,why", [(None, "INVALID")] + BAD_DIGESTS)
def test_digests(sv, fields, why):
    L, want = sv.lib(), getattr(sv, "SPEC_E_" + why)
    dg = None if fields is None else digest(sv, **fields)
    assert L.spec_block_digest(ref(dg), ctypes.byref(pages(sv)), 1, A, None, B, None) == want
    assert L.spec_block_digest_q4(ref(dg), ctypes.byref(pages_q4(sv)), 1, A, None, B, None) == want
    assert L.spec_block_scores(ref(dg), 0, 1, A, 1, None, 2, A, 0, B, 8, C, None) == want


def test_digest_calls(sv):
    L, dg = sv.lib(), ctypes.byref(digest(sv))
    for f, make in ((L.spec_block_digest, pages), (L.spec_block_digest_q4, pages_q4)):
        kv = ctypes.byref(make(sv))
        assert f(dg, None, 1, A, None, B, None) == sv.SPEC_E_INVALID
        assert f(dg, kv, 1, None, None, B, None) == f(dg, kv, 1, A, None, None, None) == sv.SPEC_E_INVALID
        assert f(dg, kv, 0, A, None, B, None) == f(dg, kv, 2 ** 30, A, None, B, None) == sv.SPEC_E_SHAPE
        for kw in (dict(n_layers=2, layer_stride=1 << 20), dict(n_pages=5), dict(n_kv_heads=1), dict(page_size=32),
                   dict(head_dim=128)):
            assert f(dg, ctypes.byref(make(sv, **kw)), 1, A, None, B, None) == sv.SPEC_E_SHAPE, kw
    two = ctypes.byref(digest(sv, n_layers=2, layer_stride=2048))
    kv = ctypes.byref(pages(sv, n_layers=2, layer_stride=4 * 2 * 64 * 64 + 8))
    assert L.spec_block_digest(two, kv, 1, A, None, B, None) == sv.SPEC_E_SHAPE and "whole rows" in sv.last_error()


def test_scores(sv):
    L, dg = sv.lib(), ctypes.byref(digest(sv))

    def f(layer=0, n_seq=1, slots=A, nt=4, nq=8, q=A, qs=0, scores=B, ld=8, st=C):
        return L.spec_block_scores(dg, layer, n_seq, slots, nt, None, nq, q, qs, scores, ld, st, None)
    for kw in (dict(slots=None), dict(q=None), dict(scores=None), dict(st=None)):
        assert f(**kw) == sv.SPEC_E_INVALID, kw
    for kw in (dict(layer=1), dict(layer=-1), dict(n_seq=0), dict(nt=0), dict(nt=65), dict(nq=0), dict(nq=7), dict(q=A + 8),
               dict(scores=B + 2), dict(qs=504), dict(qs=516), dict(qs=-512), dict(ld=0), dict(ld=-1), dict(ld=2 ** 31 + 1),
               dict(n_seq=2 ** 31 - 1, nt=64, nq=128)):
        assert f(**kw) == sv.SPEC_E_SHAPE, kw
    assert f(nq=2 * 65) == sv.SPEC_E_UNSUPPORTED


def test_selection(sv):
    L = sv.lib()

    def f(lens=A, n_slots=2, block=16, n_seq=1, slots=A, nt=4, nkv=2, scores=B, ld=8, keep=4, first=1, last=1, out=C, st=D):
        return L.spec_block_select(lens, n_slots, block, n_seq, slots, nt, None, nkv, scores, ld, keep, first, last, out, st,
                                   None)
    for kw in (dict(lens=None), dict(slots=None), dict(scores=None), dict(out=None), dict(st=None)):
        assert f(**kw) == sv.SPEC_E_INVALID, kw
    for kw in (dict(n_slots=0), dict(block=8), dict(block=256), dict(n_seq=0), dict(nt=0), dict(nt=65), dict(nkv=0),
               dict(keep=0), dict(keep=4097), dict(first=-1), dict(last=-1), dict(first=3, last=2),
               dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(scores=B + 2), dict(out=C + 1), dict(ld=0),
               dict(ld=2 ** 31 + 1), dict(n_seq=2 ** 31 - 1, nt=64)):
        assert f(**kw) == sv.SPEC_E_SHAPE, kw


def test_the_bindings_own_checks(sv):
    import torch
    codes = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    half = lambda *s: torch.zeros(s, dtype=torch.float16)  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = (codes(2, 4, 2, 8, 2, 16), codes(2, 4, 2, 8, 2, 16), half(2, 4, 2, 8, 2), half(2, 4, 2, 8, 2))
    kv = sv.KVPagesQ4(*good, i32(3, 2), i32(3), i32(4))
    p = kv.pages
    assert (p.n_layers, p.n_pages, p.n_kv_heads, p.page_size, p.head_dim, p.n_slots, p.max_pages, p.layer_stride) == (
        2, 4, 2, 8, 64, 3, 2, 64)
    assert kv.device == -2  # host memory that is not pinned
    for i, t in ((0, codes(2, 4, 2, 8, 2, 8)), (1, good[0].transpose(1, 2)), (0, half(2, 4, 2, 8, 2, 16)),
                 (2, torch.zeros((2, 4, 2, 8, 2), dtype=torch.bfloat16)), (3, half(2, 4, 2, 8, 1)),
                 (1, codes(2, 5, 2, 8, 2, 16)[:, :4])):  # (the last: another layer stride)
        with pytest.raises(ValueError):
            sv.KVPagesQ4(*good[:i], t, *good[i + 1:])
    for book in ((i32(3, 2), i32(2), None), (i32(3, 2).long(), i32(3), None), (i32(3, 2), i32(3), i32(3)),
                 (i32(2, 3).T, i32(3), None)):
        with pytest.raises(ValueError):
            sv.KVPagesQ4(*good, *book)
    wide = [torch.zeros((2, 5) + t.shape[2:], dtype=t.dtype)[:, :4] for t in good]  # layers apart, alike in all four
    assert sv.KVPagesQ4(*wide).pages.layer_stride == 80
    dg = sv.KVDigest(half(2, 4, 2, 2, 2, 64), 16, i32(3, 2), i32(3))
    assert (dg.pages.page_size, dg.pages.block, dg.pages.layer_stride) == (32, 16, 4 * 2 * 2 * 2 * 64)
    for bad in (half(2, 4, 2, 2, 3, 64), torch.zeros((2, 4, 2, 2, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 4, 2, 2, 2, 64)),
                half(2, 4, 2, 2, 2, 128)[..., :64]):
        with pytest.raises(ValueError):
            sv.KVDigest(bad, 16, i32(3, 2), i32(3))
    # one kind of cache in another's place
    f16 = sv.KVPages(half(2, 4, 2, 8, 64), half(2, 4, 2, 8, 64), i32(3, 2), i32(3))
    for x, kinds in ((f16, sv.KVPagesQ4), (dg, sv.KVPagesQ4), (kv, sv.KVDigest), (dg, (sv.KVPages, sv.KVPagesQ4)), (None, sv.KVDigest)):
        with pytest.raises(TypeError):
            sv._struct(x, kinds)
    with pytest.raises(TypeError):
        sv.spec_tree_attn_q4_workspace(f16, 1, 1, 2)
    for x in (kv, dg):
        with pytest.raises(AttributeError):
            sv.spec_tree_attn_workspace(x, 1, 1, 2)
        assert not hasattr(x, "at") and not hasattr(x, "ref")  # what the fp16 cache's calls take
    with pytest.raises(ValueError):
        sv._struct(kv, sv.KVPagesQ4, 0)  # not pinned
    for scores in (half(1, 1, 2, 8), torch.zeros((1, 1, 8, 2)).transpose(2, 3), i32(1, 1, 2, 8)):
        with pytest.raises(ValueError):
            sv._rows_of_scores(scores)
