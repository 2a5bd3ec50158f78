"""Pins of the drafted-tree reference (oracle/tree.py) against library
routines, closed forms and brute force, and the host-side refusals of the
entry points.  CPU only."""
import ctypes
import math

import numpy as np
import pytest

from oracle import tree


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------
def test_chain_is_causal_attention(orc):
    """A chain over a context is plain causal attention (the existing oracle,
    itself pinned to a library routine)."""
    g = np.random.default_rng(1)
    nq, nkv, hd, n, m = 6, 2, 16, 9, 5
    f16 = lambda *s: g.standard_normal(s).astype(np.float16)  # noqa: E731
    k, v, q = f16(n + m, nkv, hd), f16(n + m, nkv, hd), f16(m, nq, hd)
    out, _, _ = tree.tree_attention(q, k[:n], v[:n], k[n:], v[n:], [-1, 0, 1, 2, 3])
    bits = lambda a: np.ascontiguousarray(a).view(np.uint16)  # noqa: E731
    ref = orc.attention(bits(q), bits(k.transpose(1, 0, 2)), bits(v.transpose(1, 0, 2)), np.arange(n, n + m))
    assert np.array_equal(out.astype(np.float16).view(np.uint16), ref)


def test_siblings_do_not_see_each_other_and_match_their_own_chain():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((7, 1, 8)), g.standard_normal((7, 1, 8))
    kn, vn, q = g.standard_normal((5, 1, 8)), g.standard_normal((5, 1, 8)), g.standard_normal((5, 2, 8))
    parents = [-1, 0, 0, 1, 2]
    out, _, _ = tree.tree_attention(q, k, v, kn, vn, parents)
    for i in range(5):
        path = tree.chains(parents)[i]
        one, _, _ = tree.tree_attention(q[path], k, v, kn[path], vn[path], list(range(-1, len(path) - 1)))
        assert np.allclose(one[-1], out[i], rtol=0, atol=1e-14)


@pytest.mark.parametrize("n_past,window,sinks", [(0, 1, 0), (10, 4, 2), (10, 1, 3), (3, 8, 0), (12, 12, 5)])
def test_window_and_sinks_by_hand(n_past, window, sinks):
    parents = [-1, 0, 0, 2]
    for i, depth in enumerate([0, 1, 1, 2]):
        cached, nodes = tree.visible(n_past, parents, i, window, sinks)
        at = n_past + depth
        assert cached == [p for p in range(n_past) if p < sinks or at - p < window]
        assert i in nodes and all(at - (n_past + len(tree.chains(parents)[j]) - 1) < window
                                  or n_past + len(tree.chains(parents)[j]) - 1 < sinks for j in nodes)


def test_accept_tree_on_a_chain_is_the_chain_rule(orc):
    g = np.random.default_rng(3)
    for _ in range(200):
        d = int(g.integers(0, 8))
        am, draft = g.integers(0, 3, d + 1), g.integers(0, 3, d)
        path, em = tree.accept_tree(am, [99, *draft], list(range(-1, d)))
        n, ref = orc.accept_greedy(am[None].astype(np.int32), draft[None].astype(np.int32))
        assert len(path) == n[0] + 1 and em == ref[0][:n[0] + 1].tolist() and path == list(range(n[0] + 1))


def test_accept_tree_takes_the_longest_agreeing_path():
    """Distinct sibling tokens: the accepted path is the only maximal path all
    of whose nodes carry their parent's argmax, found by brute force."""
    g = np.random.default_rng(4)
    for _ in range(200):
        m = int(g.integers(1, 12))
        parents = [-1] + [int(g.integers(max(0, i - 4), i)) for i in range(1, m)]
        tokens, seen = [0] * m, {}
        for i in range(1, m):
            tokens[i] = seen.setdefault(parents[i], 0)
            seen[parents[i]] += 1
        am = g.integers(0, 3, m)
        path, em = tree.accept_tree(am, tokens, parents)
        good = [c for c in tree.chains(parents) if c[0] == 0 and all(tokens[b] == am[a] for a, b in zip(c, c[1:]))]
        assert path == max(good, key=len) and em == [am[j] for j in path]


def test_sampling_without_filters_is_the_exact_pick(orc):
    g = np.random.default_rng(5)
    for _ in range(50):
        l = (g.standard_normal(40) * 3).astype(np.float32)
        T, u = float(np.float32(g.uniform(0.3, 2))), int(g.integers(0, 2 ** 32))
        W, S = orc.row_weights(l, T)
        tok, ids = tree.sample_row(l, orc.row_weights, u, T)
        assert tok == orc.weight_pick(W, S, u) and ids == list(range(40))


def test_filters_against_a_softmax(orc):
    """The kept sets are those of the textbook rules on a fp64 softmax,
    wherever those rules are not within 1e-6 of a border."""
    from scipy.special import softmax
    g = np.random.default_rng(6)
    checked = 0
    for _ in range(200):
        l = (g.standard_normal(60) * 2).astype(np.float32)
        T = float(np.float32(g.uniform(0.5, 1.5)))
        k, p, m = int(g.integers(1, 60)), float(g.uniform(0.2, 0.99)), float(g.uniform(0, 0.2))
        probs = softmax(l.astype(np.float64) / T)
        order = np.argsort(-probs, kind="stable")[:k]
        cum = np.cumsum(probs[order]) / probs[order].sum()
        before = np.concatenate([[0], cum[:-1]])
        ratio = probs[order] / probs.max()
        if np.min(np.abs(before - p)) < 1e-6 or np.min(np.abs(ratio - m)) < 1e-6:
            continue
        keep = order[(before < p) & (ratio >= m)]
        assert tree.sample_row(l, orc.row_weights, 7, T, k, p, m)[1] == sorted(keep.tolist())
        checked += 1
    assert checked > 150


def test_sampling_frequencies_are_the_filtered_softmax(orc):
    """Over an even grid of u every token comes up in proportion to its weight."""
    l = np.array([1.0, 3.0, 2.0, 3.0, -1.0, 0.5], np.float32)
    n = 4096
    got = np.bincount([tree.sample_row(l, orc.row_weights, i * (2 ** 32 // n), 0.8, 4, 0.99, 0.0)[0]
                       for i in range(n)], minlength=6) / n
    e = np.exp((l.astype(np.float64) - 3) / 0.8)
    e[[4, 5]] = 0
    assert np.max(np.abs(got - e / e.sum())) <= 1.0 / n + 1e-6


def test_book_small_story():
    """Fork, copy on write, commit and free, followed by hand."""
    b = tree.Book(n_slots=4, max_pages=4, n_pages=6, page=4)
    assert b.extend([0], [6]) == ([0], [(-1, -1)]) and b.table[0] == [0, 1, -1, -1]
    assert b.commit([0], [list(range(6))], [6], lambda i, n: n) == [0] and b.len[0] == 6
    assert b.fork([0, 0], [1, 2]) == [0, 0] and b.refs == [3, 3, 0, 0, 0, 0]
    # both branches and the parent write behind position 6: the last keeps page 1
    st, cp = b.extend([1, 2, 0], [1, 3, 1])
    assert st == [0, 0, 0] and cp == [(1, 2), (1, 3), (-1, -1)] and b.refs == [3, 1, 1, 1, 1, 0]
    assert b.table[1][:2] == [0, 2] and b.table[2][:3] == [0, 3, 4] and b.rows[(2, 1)] == 5
    assert b.commit([2], [[2, 0, 1]], [2], lambda i, n: ("n", n)) == [0]
    assert b.rows[(3, 2)] == ("n", 2) and b.rows[(3, 3)] == ("n", 0) and b.len[2] == 8
    assert b.extend([1], [100])[0] == [tree.ST_FULL] and b.extend([1], [9])[0] == [tree.ST_FULL]
    assert b.free([2, 1]) == [0, 0] and b.refs == [1, 1, 0, 0, 0, 0]


# ---------------------------------------------------------------------------
# refusals on the host (no device work, no GPU)
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_round_gb300 as sv
    from speculative_decoding_verification_round_gb300 import _build
    _build.build()
    return sv


A = 1 << 20  # a 16-byte aligned address that nothing reads


def pages(sv, **kw):
    d = dict(k=A, v=A, layer_stride=2 * 8 * 64 * 128, n_layers=2, n_pages=8, n_kv_heads=2, page_size=64,
             head_dim=128, n_slots=3, max_pages=4, table=A, refs=A, len=A)
    d["layer_stride"] = 8 * 2 * 64 * 128
    d.update(kw)
    return sv.spec_pages(**d)


def test_binding_structs_match_the_header(sv):
    """Field offsets of the two structs as the C compiler lays them out."""
    assert ctypes.sizeof(sv.spec_pages) == 80 and sv.spec_pages.table.offset == 56
    assert ctypes.sizeof(sv.spec_tree) == 48 and sv.spec_tree.slots.offset == 24
    assert sv.SPEC_FILTERED == float(np.finfo(np.float32).min)


BAD_PAGES = [(dict(k=None), "INVALID"), (dict(v=A + 8), "SHAPE"), (dict(n_layers=0), "SHAPE"),
             (dict(n_pages=0), "SHAPE"), (dict(page_size=0), "SHAPE"), (dict(head_dim=12), "SHAPE"),
             (dict(layer_stride=8), "SHAPE"), (dict(layer_stride=8 * 2 * 64 * 128 + 4), "SHAPE"),
             (dict(table=None), "INVALID"), (dict(len=None), "INVALID"), (dict(n_slots=0), "SHAPE"),
             (dict(max_pages=1 << 26), "SHAPE"), (dict(n_pages=2 ** 31 - 1, page_size=2 ** 31 - 1), "SHAPE")]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_bad_pages_are_refused_by_every_call(sv, kw, code):
    L, kv = sv.lib(), ctypes.byref(pages(sv, **kw))
    rc = getattr(sv, "SPEC_E_" + code)
    assert L.spec_pages_fork(kv, 1, A, A, A, None) == rc
    assert L.spec_pages_extend(kv, 1, A, A, A, A, None) == rc
    assert L.spec_pages_commit(kv, 1, A, 4, A, A, 0, A, A, None, A, None) == rc
    assert L.spec_pages_free(kv, 1, A, A, None) == rc
    b = ctypes.c_size_t()
    assert L.spec_tree_attn_workspace(kv, 1, 4, 4, ctypes.byref(b)) == rc


def test_page_calls_refuse_bad_arguments(sv):
    L, kv = sv.lib(), ctypes.byref(pages(sv))
    fixed = ctypes.byref(pages(sv, refs=None))
    for bad in (0, -1):
        assert L.spec_pages_copy(kv, bad, A, A, None, A, None) == sv.SPEC_E_SHAPE
        assert L.spec_pages_free(kv, bad, A, A, None) == sv.SPEC_E_SHAPE
    assert L.spec_pages_copy(kv, 1, None, A, None, A, None) == sv.SPEC_E_INVALID
    assert L.spec_pages_copy(kv, 1, A, A, None, None, None) == sv.SPEC_E_INVALID
    assert L.spec_pages_copy(kv, 2 ** 31 - 1, A, A, None, A, None) == sv.SPEC_E_SHAPE
    assert L.spec_pages_fork(fixed, 1, A, A, A, None) == sv.SPEC_E_UNSUPPORTED
    assert L.spec_pages_extend(fixed, 1, A, A, A, A, None) == sv.SPEC_E_UNSUPPORTED
    assert L.spec_pages_free(fixed, 1, A, A, None) == sv.SPEC_E_UNSUPPORTED
    assert L.spec_pages_extend(kv, 1025, A, A, A, A, None) == sv.SPEC_E_SHAPE
    assert L.spec_pages_extend(kv, 1, A, None, A, A, None) == sv.SPEC_E_INVALID
    commit = lambda nt=4, k=A, stride=0, np_=A, new=None: L.spec_pages_commit(  # noqa: E731
        kv, 1, A, nt, k, A, stride, A, np_, new, A, None)
    assert commit(nt=0) == sv.SPEC_E_SHAPE and commit(k=A + 2) == sv.SPEC_E_SHAPE
    assert commit(stride=8) == sv.SPEC_E_SHAPE and commit(np_=None) == sv.SPEC_E_INVALID
    assert commit(new=A + 4) == sv.SPEC_E_INVALID  # half over len
    assert L.spec_model_pages(None, kv) == sv.SPEC_E_INVALID


def test_tree_attention_refuses_bad_arguments(sv):
    L, kv = sv.lib(), pages(sv)

    def call(layer=0, n_seq=1, nt=4, nq=4, window=0, sinks=0, scale=0.0, slots=A, q=A, qs=0, kvs=0, out=A,
             ws=A, nbytes=1 << 40, status=A, kv=kv):
        t = sv.spec_tree(n_seq, nt, nq, window, sinks, scale, slots, None, None)
        return L.spec_tree_attn(ctypes.byref(kv), layer, ctypes.byref(t), q, qs, A, A, kvs, out, ws, nbytes,
                                status, None)
    for kw in (dict(slots=None), dict(q=None), dict(out=None), dict(ws=None), dict(status=None), dict(window=-1),
               dict(sinks=-1), dict(scale=math.inf), dict(scale=math.nan)):
        assert call(**kw) == sv.SPEC_E_INVALID, kw
    for kw in (dict(layer=2), dict(layer=-1), dict(n_seq=0), dict(nt=0), dict(nt=65), dict(nq=3), dict(nq=0),
               dict(q=A + 8), dict(out=A + 2), dict(qs=4 * 128 + 4), dict(qs=128), dict(kvs=8), dict(qs=-512),
               dict(nbytes=16), dict(ws=A + 8)):
        assert call(**kw) == sv.SPEC_E_SHAPE, kw
    # out over q (A is k_new and v_new, too), workspace over them, workspace over out
    far, farther = A + (1 << 30), A + (1 << 34)
    for kw in (dict(ws=farther), dict(ws=farther, out=A + 2048), dict(out=far, q=farther), dict(ws=far, out=far, nbytes=1 << 24)):
        assert call(**kw) == sv.SPEC_E_INVALID and "overlap" in sv.last_error(), kw
    odd = pages(sv, head_dim=96, layer_stride=8 * 2 * 64 * 96)
    assert call(kv=odd) == sv.SPEC_E_UNSUPPORTED
    assert L.spec_accept_tree(A, A, A, None, 1, 65, A, A, A, None) == sv.SPEC_E_SHAPE
    assert L.spec_accept_tree(A, A, A, None, 0, 4, A, A, A, None) == sv.SPEC_E_SHAPE
    assert L.spec_accept_tree(A, A, None, None, 1, 4, A, A, A, None) == sv.SPEC_E_INVALID


def test_sample_refuses_bad_arguments(sv):
    L = sv.lib()

    def call(logits=A, R=2, V=100, ld=0, u=A, token=A, filtered=None, ldf=0):
        return L.spec_sample(logits, R, V, ld, u, None, None, None, None, token, None, filtered, ldf, None, 0, None)
    for kw in (dict(logits=None), dict(u=None), dict(token=None)):
        assert call(**kw) == sv.SPEC_E_INVALID
    for kw in (dict(R=0), dict(V=0), dict(V=1048513, ld=1 << 21), dict(ld=99), dict(filtered=A + (1 << 16), ldf=50), dict(logits=A + 2)):
        assert call(**kw) == sv.SPEC_E_SHAPE, kw
    assert call(R=192, V=248320) == sv.SPEC_E_SHAPE and "workspace" in sv.last_error()
    assert sv.spec_sample_workspace(1, 151936) == 0 and sv.spec_sample_workspace(192, 248320) > 0
    assert call(filtered=A + 4) == sv.SPEC_E_INVALID  # half over the logits
    assert call(filtered=A, ld=100, ldf=104) == sv.SPEC_E_INVALID  # the logits with another stride


def test_pages_of_other_tensors_are_refused():
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    ok = torch.zeros((2, 4, 2, 8, 64), dtype=torch.float16)
    sv.KVPages(ok, ok.clone(), torch.zeros((3, 2), dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    for k, v in ((ok.bfloat16(), ok.bfloat16()), (ok.float(), ok.float()), (ok, ok[:1]), (ok, ok.bfloat16()),
                 (ok.transpose(2, 3), ok.transpose(2, 3))):
        with pytest.raises(ValueError):
            sv.KVPages(k, v)
    for kw in (dict(table=torch.zeros((3, 2), dtype=torch.int64)), dict(lens=torch.zeros(2, dtype=torch.int32)),
               dict(refs=torch.zeros(3, dtype=torch.int32))):
        args = dict(table=torch.zeros((3, 2), dtype=torch.int32), lens=torch.zeros(3, dtype=torch.int32))
        with pytest.raises(ValueError):
            sv.KVPages(ok, ok.clone(), **{**args, **kw})


def test_tensors_that_a_kernel_cannot_read_are_refused(sv, monkeypatch):
    """Host tensors, and tensors of another device than the current one, in
    every call of the drafted-tree operators and in KVPages: refused in front
    of the library."""
    import torch
    host = lambda *shape: torch.zeros(shape, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros((1, 4, 1, 8, 64), dtype=torch.float16)
    on_host = sv.KVPages(cache, cache, host(3, 2), host(3), host(4))

    class Device:  # a tensor of device 0, as far as the binding looks
        is_cuda = True
        device = "cuda:0"

        def __init__(self, t, index=0):
            self.t, self.index, self.shape, self.dtype = t, index, t.shape, t.dtype

        def __getattr__(self, name):
            return getattr(self.t, name)

        def __getitem__(self, i):
            return self.t[i]

        def get_device(self):
            return self.index

        def data_ptr(self):
            return A
    on0 = lambda *shape: Device(host(*shape))  # noqa: E731
    kv = sv.KVPages(Device(cache), Device(cache), on0(3, 2), on0(3), on0(4))
    for other in (host(3), Device(host(3), 1)):
        with pytest.raises(ValueError):
            sv.KVPages(Device(cache), Device(cache), on0(3, 2), other, on0(4))
    half = Device(torch.zeros(4096, dtype=torch.float16))
    n = on0(1)
    calls = {  # the arguments that are tensors, by name
        sv.spec_pages_copy: (dict(kv=kv, n=1), dict(src=n, dst=n, status=n, n_pos=n)),
        sv.spec_pages_fork: (dict(kv=kv, n=1), dict(src=n, dst=n, status=n)),
        sv.spec_pages_extend: (dict(kv=kv, n=1), dict(slots=n, n_new=n, copies=n, status=n)),
        sv.spec_pages_commit: (dict(kv=kv, n=1, nt=1), dict(slots=n, k_new=half, v_new=half, path=n, n_path=n, status=n,
                                                         new_len=n)),
        sv.spec_pages_free: (dict(kv=kv, n=1), dict(slots=n, status=n)),
        sv.spec_tree_attn: (dict(kv=kv, layer=0, n_seq=1, nt=1, n_q_heads=1),
                            dict(slots=n, q=half, k_new=half, v_new=half, out=half, workspace=half, status=n, parents=n,
                                 n_nodes=n)),
        sv.spec_accept_tree: (dict(n_seq=1, nt=1), dict(argmax=n, tokens=n, parents=n, n_nodes=n, path=n, n_path=n,
                                                        emitted=n)),
        sv.spec_sample: (dict(R=1, V=8), dict(logits=half, u=n, token=n, temperature=half, top_k=n, top_p=half, min_p=half,
                                              n_kept=n, filtered=half, workspace=half)),
    }
    here = lambda d: monkeypatch.setattr(sv, "_here", lambda stream: (d, None))  # noqa: E731

    class Library:
        def __getattr__(self, name):
            return lambda *args: pytest.fail("a refused call reached the library")
    monkeypatch.setattr(sv, "lib", Library)
    for call, (plain, tensors) in calls.items():
        for name, good in tensors.items():
            for bad in (good.t, Device(good.t, 1)):
                here(0)
                with pytest.raises(ValueError):
                    call(**plain, **{**tensors, name: bad})
        if "kv" in plain:
            with pytest.raises(ValueError):
                call(**{**plain, "kv": on_host}, **tensors)
        here(1)  # everything on device 0, device 1 current
        with pytest.raises(ValueError):
            call(**plain, **tensors)
