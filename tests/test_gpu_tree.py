"""spec_tree_attn on the GPU against the plain 64-bit tree attention of
oracle/tree.py, its edges and refusals, and a run of the drafted-tree
operators together."""
import numpy as np
import pytest

from oracle import tree
from test_gpu_attn import attn_model
from util import small_decoder  # noqa: F401  (the suite's helpers are importable)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def random_parents(g, nt, kind="tree"):
    if kind == "chain":
        return list(range(-1, nt - 1))
    if kind == "flat":  # all children of the context
        return [-1] * nt
    return [-1] + [int(g.integers(max(-1 if kind == "forest" else 0, i - 6), i)) for i in range(1, nt)]


class Case:
    """Inputs of one call, fp16 on the host (float16 arrays) and the device."""

    def __init__(self, sv, dev, g, nq, nkv, hd, lens, nt, page, window=0, sinks=0, counts=None, kind="tree", layers=2,
                 scale=None, amp=1.0):
        import torch
        self.sv, self.dev, self.nq, self.nkv, self.hd, self.nt = sv, dev, nq, nkv, hd, nt
        self.window, self.sinks, self.page, self.scale = window, sinks, page, scale
        n = self.n = len(lens)
        self.lens = list(lens)
        f16 = lambda *s: (g.standard_normal(s) * amp).astype(np.float16)  # noqa: E731
        max_pages = max(1, -(-max(self.lens) // page)) + 1
        n_pages = n * max_pages + 2
        self.layer = int(g.integers(0, layers))
        self.k, self.v = f16(layers, n_pages, nkv, page, hd), f16(layers, n_pages, nkv, page, hd)
        order = g.permutation(n_pages)
        self.table = np.full((n + 1, max_pages), -1, np.int32)
        self.slots = g.permutation(n + 1)[:n].astype(np.int32)
        self.slot_len = np.zeros(n + 1, np.int32)
        for b in range(n):
            held = -(-self.lens[b] // page)
            self.table[self.slots[b], :held] = order[b * max_pages:b * max_pages + held]
            self.slot_len[self.slots[b]] = self.lens[b]
        self.parents = np.array([random_parents(g, nt, kind) for _ in range(n)], np.int32)
        self.counts = np.full(n, nt, np.int32) if counts is None else np.asarray(counts, np.int32)
        self.q, self.kn, self.vn = f16(n, nt, nq, hd), f16(n, nt, nkv, hd), f16(n, nt, nkv, hd)
        self.T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)

    def cached(self, which, b):
        """[len][nkv][hd] of sequence b; zeros where a position has no page."""
        pool, out = (self.k, self.v)[which][self.layer], np.zeros((self.lens[b], self.nkv, self.hd), np.float16)
        for p in range(self.lens[b]):
            pg = self.table[self.slots[b], p // self.page]
            if pg >= 0:
                out[p] = pool[pg, :, p % self.page]
        return out

    def pool(self):
        return self.sv.KVPages(self.T(self.k), self.T(self.v), self.T(self.table), self.T(self.slot_len))

    def call(self, kv=None, status_only=False, chain=False, counts=True, **kw):
        import torch
        kv = kv or self.pool()
        self.out = torch.full((self.n, self.nt, self.nq, self.hd), 7.0, dtype=torch.float16, device=self.dev)
        self.status = torch.full((self.n,), 99, dtype=torch.int32, device=self.dev)
        ws = torch.full((self.sv.spec_tree_attn_workspace(kv, self.n, self.nt, self.nq),), 0xFF, dtype=torch.uint8,
                        device=self.dev)  # NaN everywhere
        args = dict(q=self.T(self.q), k_new=self.T(self.kn), v_new=self.T(self.vn))
        args.update(kw)
        self.sv.spec_tree_attn(kv, self.layer, self.n, self.T(self.slots), self.nt, self.nq, out=self.out,
                               workspace=ws, status=self.status, parents=None if chain else self.T(self.parents),
                               n_nodes=self.T(self.counts) if counts else None, window=self.window, sinks=self.sinks,
                               scale=self.scale or 0.0, **args)
        torch.cuda.synchronize()
        return self.out.cpu().numpy()

    def check(self, got, seqs=None):
        """Against the reference.  The bound: half an fp16 step of the result
        (2^-11 relative, 2^-25 absolute below the normals); the scores' error
        ds (hd products summed in fp32, at most one unit in the last place,
        2^-23, of the sum of magnitudes a step, then two roundings), which
        moves every weight by a factor within exp(+-2 ds); exp2 and the hi + lo
        split of the weights, 2^-20; and fp32 sums over the keys, one unit per
        step of 8 keys: all times the |v| average of the row.  With more than
        32 query rows a kv head the weights are rounded once to fp16: half a
        step, 2^-11, or 2^-25 below the normals, where a row's largest weight
        is at least 2^6."""
        for b in range(self.n) if seqs is None else seqs:
            m = int(self.counts[b])
            assert (got[b, m:] == np.float16(7.0)).all(), b  # rows of no node
            if m == 0:
                continue
            ref, mag, dots = tree.tree_attention(self.q[b, :m], self.cached(0, b), self.cached(1, b), self.kn[b, :m],
                                                 self.vn[b, :m], self.parents[b, :m].tolist(), self.window, self.sinks,
                                                 self.scale)
            scale = self.scale or self.hd ** -0.5
            ds = (self.hd + 4) * 2.0 ** -23 * abs(scale) * dots
            rel = np.expm1(2 * ds) + 2.0 ** -20 + ((self.lens[b] + m) / 8 + 64) * 2.0 ** -23
            if self.nt * self.nq // self.nkv > 32:
                rel = rel + 2.0 ** -11 + (self.lens[b] + m) * 2.0 ** -31
            bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[..., None] * mag
            err = np.abs(got[b, :m].astype(np.float64) - ref)
            assert np.isfinite(got[b, :m]).all() and (err <= bound).all(), (b, float(np.max(err - bound)))


SHAPES = [
    # nq, nkv, hd, lens, nt, page, window, sinks, counts, kind
    (32, 8, 128, [300], 8, 64, 0, 0, None, "tree"),           # GQA 4, 32 rows
    (40, 8, 128, [512, 37, 500], 16, 64, 0, 0, None, "tree"),   # GQA 5, 80 rows: two row blocks
    (4, 4, 64, [0, 1, 2], 1, 16, 0, 0, None, "chain"),         # no context, one position; one row a head
    (14, 2, 64, [4000, 17], 1, 16, 0, 0, None, "chain"),       # a draft model's decode step
    (14, 2, 64, [257, 64, 65], 3, 24, 0, 0, [3, 1, 0], "tree"), # odd pages; a sequence without nodes
    (8, 1, 128, [700], 63, 100, 0, 0, None, "tree"),           # 504 rows of one head
    (6, 1, 128, [190, 63, 0], 64, 7, 0, 0, [64, 33, 64], "forest"),
    (5, 5, 64, [128, 129, 127], 64, 128, 0, 0, None, "flat"),
    (32, 8, 128, [5000, 3], 2, 1000, 0, 0, None, "chain"),
    (16, 2, 64, [1000, 900, 0, 63], 5, 16, 100, 4, [5, 5, 5, 2], "tree"),
    (8, 8, 128, [2000, 64, 10], 12, 64, 64, 0, None, "tree"),  # the window is a tile
    (8, 2, 128, [513, 65, 1], 20, 32, 1, 0, None, "tree"),     # every node sees itself alone
    (8, 2, 128, [513, 65, 1], 20, 32, 3, 200, None, "chain"),  # sinks past the window
    (4, 2, 64, [3000, 500], 33, 48, 777, 65, None, "forest"),
    (4, 1, 64, [300], 4, 64, 2 ** 31 - 1, 2 ** 31 - 1, None, "tree"),
]


@pytest.mark.parametrize("nq,nkv,hd,lens,nt,page,window,sinks,counts,kind", SHAPES)
def test_matches_the_reference(dev, nq, nkv, hd, lens, nt, page, window, sinks, counts, kind):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(nq * 1000 + nt * 7 + len(lens))
    c = Case(sv, dev, g, nq, nkv, hd, lens, nt, page, window, sinks, counts, kind)
    got = c.call(chain=kind == "chain", counts=counts is not None)
    assert c.status.tolist() == [0] * c.n
    c.check(got)
    assert np.array_equal(c.call(chain=kind == "chain").view(np.uint16), got.view(np.uint16))  # the same bits


def test_many_ragged_sequences(dev):
    """More sequences than a CTA scans at once, lengths and node counts from
    zero up, slots named more than once."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(5)
    n = 300
    lens = [int(x) for x in g.choice([0, 1, 16, 17, 40, 130], n)]
    c = Case(sv, dev, g, 4, 2, 64, lens, 6, 16, counts=g.integers(0, 7, n))
    c.slots[7], c.lens[7] = c.slots[3], c.lens[3]
    c.slots[299], c.lens[299] = c.slots[3], c.lens[3]
    got = c.call()
    assert c.status.tolist() == [0] * n
    c.check(got)


@pytest.mark.parametrize("nq,nkv,hd,n,longest,nt", [(32, 8, 128, 2, 9001, 16), (16, 8, 64, 3, 7000, 40),
                                                    (32, 8, 128, 500, 290, 16), (40, 8, 128, 300, 140, 16),
                                                    (8, 2, 64, 700, 200, 64)])
def test_repeated_calls_agree(dev, nq, nkv, hd, n, longest, nt):
    """No result depends on how the streams of a CTA run against each other:
    pieces of one tile and of many, sequences that begin in the middle of a
    CTA, the same call forty times, bit by bit."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([31, nq, n])
    lens = g.integers(0, longest + 1, n)
    lens[:2] = longest
    c = Case(sv, dev, g, nq, nkv, hd, lens.tolist(), nt, 64, layers=1)
    first = c.call()
    c.check(first, range(0, n, max(1, n // 12)))
    out, kv, slots, parents, counts = c.out, c.pool(), c.T(c.slots), c.T(c.parents), c.T(c.counts)
    q, kn, vn, want = c.T(c.q), c.T(c.kn), c.T(c.vn), c.out.clone()
    ws = torch.empty(sv.spec_tree_attn_workspace(kv, n, nt, nq), dtype=torch.uint8, device=dev)
    for _ in range(40):
        out.fill_(7.0)
        sv.spec_tree_attn(kv, 0, n, slots, nt, nq, q, kn, vn, out, ws, c.status, parents=parents, n_nodes=counts)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("nt", [16, 32])
def test_repeated_calls_over_a_long_context_agree(dev, nt):
    """Two sequences of 131071 positions: the streams of a CTA get far apart
    on the way, and the second sequence begins in the middle of one."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    gen = torch.Generator(device=dev)
    gen.manual_seed(nt)
    rnd = lambda *s: torch.randn(s, generator=gen, device=dev, dtype=torch.float16)  # noqa: E731
    nq, nkv, hd, page, ctx, n = 32, 8, 128, 256, 131071, 2
    pages = -(-ctx // page)
    k, v = rnd(1, n * pages, nkv, page, hd), rnd(1, n * pages, nkv, page, hd)
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.arange(n * pages, **i32).view(n, pages)
    lens, slots = torch.full((n,), ctx, **i32), torch.arange(n, **i32)
    q, kn, vn = rnd(n, nt, nq, hd), rnd(n, nt, nkv, hd), rnd(n, nt, nkv, hd)
    out, status = torch.empty((n, nt, nq, hd), dtype=torch.float16, device=dev), torch.full((n,), 9, **i32)
    pool = sv.KVPages(k, v, table, lens)
    ws = torch.empty(sv.spec_tree_attn_workspace(pool, n, nt, nq), dtype=torch.uint8, device=dev)
    want = None
    for _ in range(60):  # a chain, with no parents given
        sv.spec_tree_attn(pool, 0, n, slots, nt, nq, q, kn, vn, out, ws, status)
        want = out.clone() if want is None else want
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    assert status.tolist() == [0, 0]
    g = nq // nkv
    for b, h in ((0, 0), (0, 7), (1, 0), (1, 3)):
        kk = torch.cat([k[0, b * pages:(b + 1) * pages, h].reshape(-1, hd)[:ctx], kn[b, :, h]]).double()
        vv = torch.cat([v[0, b * pages:(b + 1) * pages, h].reshape(-1, hd)[:ctx], vn[b, :, h]]).double()
        s = torch.einsum("ngd,kd->ngk", q[b, :, h * g:(h + 1) * g].double(), kk) * hd ** -0.5
        s[:, :, ctx:].masked_fill_(torch.ones(nt, nt, device=dev).triu(1).bool()[:, None], -float("inf"))
        w = torch.softmax(s, -1)
        ref, mag = torch.einsum("ngk,kd->ngd", w, vv), torch.einsum("ngk,kd->ngd", w, vv.abs())
        # (the bound of Case.check; |q . k| sums are below 2 hd here)
        rel = np.expm1(2 * (hd + 4) * 2.0 ** -23 * hd ** -0.5 * 2 * hd) + 2.0 ** -20 + (
            (ctx + nt) / 8 + 64) * 2.0 ** -23 + 2.0 ** -11 + (ctx + nt) * 2.0 ** -31
        err = (out[b, :, h * g:(h + 1) * g].double() - ref).abs()
        assert (err <= 2.0 ** -11 * ref.abs() + 2.0 ** -25 + 1.01 * rel * mag).all()


def test_large_scores_and_a_given_scale(dev):
    """Scores far apart (weights underflow, the running maximum moves) and a
    scale of the caller's, negative too."""
    import speculative_decoding_verification_round_gb300 as sv
    for scale, amp in ((0.5, 2.0), (-0.25, 1.0), (3.0, 0.5)):
        g = np.random.default_rng(int(amp * 10))
        c = Case(sv, dev, g, 8, 2, 64, [600, 90], 9, 32, scale=scale, amp=amp)
        c.check(c.call())


def test_strided_rows_of_a_fused_qkv_buffer(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(3)
    nq, nkv, hd, nt = 8, 2, 64, 5
    c = Case(sv, dev, g, nq, nkv, hd, [100, 33], nt, 16)
    row = (nq + 2 * nkv) * hd + 24
    buf = torch.full((2 * nt, row), float("nan"), dtype=torch.float16, device=dev)
    buf[:, :nq * hd] = c.T(c.q).view(2 * nt, -1)
    buf[:, nq * hd:(nq + nkv) * hd] = c.T(c.kn).view(2 * nt, -1)
    buf[:, (nq + nkv) * hd:(nq + 2 * nkv) * hd] = c.T(c.vn).view(2 * nt, -1)
    flat = buf.view(-1)
    got = c.call(q=flat, k_new=flat[nq * hd:], v_new=flat[(nq + nkv) * hd:], q_stride=row, kv_stride=row)
    c.check(got)


@pytest.mark.parametrize("hd,nq", [(64, 2), (128, 8), (128, 40)])
def test_nothing_of_what_is_masked_gets_in(dev, hd, nq):
    """Infinities and NaN in rows of V and K that a row does not see -- behind
    the length, in front of the window, in other branches, past the node
    count -- leave it exactly as it is without them."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(4)
    c = Case(sv, dev, g, nq, 2, hd, [300, 90], 8, 32, window=50, sinks=3, counts=[8, 6])
    c.parents[:] = [-1, 0, 0, 1, 2, 2, 4, 0]
    clean = c.call()
    c.check(clean)
    held = {}
    for b in range(2):
        for p in range(c.lens[b]):
            held[(int(c.table[c.slots[b], p // 32]), p % 32)] = (b, p)
    for pg in range(c.k.shape[1]):
        for at in range(32):
            b, p = held.get((pg, at), (None, None))
            if b is None or 3 <= p < c.lens[b] - 49:  # no node sees it
                c.k[:, pg, :, at], c.v[:, pg, :, at] = np.nan, np.inf
    c.kn[1, 6:], c.vn[1, 6:] = np.inf, np.nan
    c.vn[0, 5], c.kn[0, 5] = -np.inf, np.nan  # a leaf: nobody else sees it
    c.vn[1, 3] = np.nan
    got = c.call()
    same = np.ones((2, 8), bool)
    same[0, 5] = same[1, 3] = False
    # (the poisoned tiles add their rows one by one: the last bits may differ)
    assert np.isfinite(got[same]).all() and not np.isfinite(got[0, 5]).any() and not np.isfinite(got[1, 3]).any()
    d = np.abs(got[same].astype(np.float64) - clean[same].astype(np.float64))
    # both are within the bound of check() of the same reference; an fp16 step of the value covers twice that
    assert (d <= 2.0 ** -10 * np.abs(clean[same].astype(np.float64)) + 2.0 ** -13).all()


def test_pages_out_of_sight_may_be_gone(dev):
    """With a window, pages wholly between the sinks and the window need not
    be there."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(6)
    c = Case(sv, dev, g, 8, 2, 64, [1000, 700], 7, 16, window=100, sinks=20)
    for b in range(2):
        c.table[c.slots[b], 2:(c.lens[b] - 99) // 16] = -1
    got = c.call()
    assert c.status.tolist() == [0, 0]
    c.check(got)
    c.table[c.slots[1], 1] = -1  # positions 16..19 are sinks
    got = c.call()
    assert c.status.tolist() == [0, tree.ST_PAGE] and np.isnan(got[1]).all()
    c.check(got, [0])


def test_refused_sequences(dev):
    """Each sequence in error is NaN with its status; the others are served."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(7)
    c = Case(sv, dev, g, 8, 2, 64, [100, 90, 80, 70, 60, 50, 40, 30], 6, 16, counts=[6, 6, 6, 6, 4, 7, 6, 5])
    c.slots[1] = 99
    c.table[c.slots[2], 3] = 10 ** 6
    c.slot_len[c.slots[3]] = c.table.shape[1] * 16 + 1
    c.parents[4, 3] = 3
    c.table[c.slots[6], 0] = -7
    c.parents[7, 5] = 5  # not a node of this sequence (5 nodes): not looked at
    got = c.call()
    assert c.status.tolist() == [0, tree.ST_SLOT, tree.ST_PAGE, tree.ST_PAGE, tree.ST_TREE, tree.ST_TREE, tree.ST_PAGE, 0]
    c.parents[7, 5] = 0
    c.check(got, [0, 7])
    for b, m in ((1, 6), (2, 6), (3, 6), (4, 6), (5, 6), (6, 6)):
        rows = got[b, :4] if b == 4 else got[b, :m]
        assert np.isnan(rows).all(), b
    c.slot_len[c.slots[3]] = -1
    got = c.call()
    assert c.status.tolist()[3] == tree.ST_PAGE and np.isnan(got[3]).all()


@pytest.mark.parametrize("nq,nkv,nt", [(8, 2, 6), (8, 1, 12)])
def test_rows_behind_a_refused_sequence_stay(dev, nq, nkv, nt):
    """Whatever a sequence is refused for, only its first n_nodes rows are NaN;
    all of them if the count is what is wrong."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(12)
    c = Case(sv, dev, g, nq, nkv, 64, [100, 90, 80, 70, 60, 50, 0], nt, 16, counts=[4, 3, 4, 4, nt + 1, -1, 2])
    c.parents[0, 3] = 3              # a node that is its own parent
    c.slots[1] = -1
    c.table[c.slots[2], 1] = -3
    c.parents[3, 2], c.table[c.slots[3], 0] = -2, 10 ** 6
    c.parents[6, 1] = 1
    got = c.call()
    assert c.status.tolist() == [tree.ST_TREE, tree.ST_SLOT, tree.ST_PAGE, tree.ST_TREE | tree.ST_PAGE, tree.ST_TREE,
                                 tree.ST_TREE, tree.ST_TREE]
    for b, m in enumerate([4, 3, 4, 4, nt, nt, 2]):
        assert np.isnan(got[b, :m]).all() and (got[b, m:] == 7.0).all(), b


def test_graph_replay_and_two_streams(dev):
    """A captured call replayed over new lengths, trees and rows; and two calls
    at once on two streams, each with a workspace of its own."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(8)
    cs = [Case(sv, dev, g, 8, 2, 128, [700, 300], 10, 32) for _ in range(2)]
    want = [c.call() for c in cs]
    kv = cs[0].pool()
    T = cs[0].T
    d = dict(q=T(cs[0].q), k_new=T(cs[0].kn), v_new=T(cs[0].vn), parents=T(cs[0].parents), n_nodes=T(cs[0].counts))
    slots, out = T(cs[0].slots), torch.zeros((2, 10, 8, 128), dtype=torch.float16, device=dev)
    st = torch.zeros(2, dtype=torch.int32, device=dev)
    ws = torch.empty(sv.spec_tree_attn_workspace(kv, 2, 10, 8), dtype=torch.uint8, device=dev)
    k, v, table, lens, _ = kv._keep
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_tree_attn(kv, cs[0].layer, 2, slots, 10, 8, out=out, workspace=ws, status=st, **d)
    c1 = cs[1]
    for c, w in ((cs[0], want[0]), (c1, want[1]), (cs[0], want[0])):
        for dst, src in ((k[cs[0].layer], c.k[c.layer]), (v[cs[0].layer], c.v[c.layer]), (table, c.table),
                         (lens, c.slot_len), (slots, c.slots), (d["q"], c.q), (d["k_new"], c.kn), (d["v_new"], c.vn),
                         (d["parents"], c.parents)):
            dst.copy_(T(src))
        graph.replay()
        assert np.array_equal(out.cpu().numpy().view(np.uint16), w.view(np.uint16))
    # two streams, many calls in flight on each
    sides = []
    for c in cs:
        p = c.pool()
        sides.append(dict(st=torch.cuda.Stream(), kv=p, ws=torch.empty_like(ws), c=c, outs=[], keep=[
            c.T(a) for a in (c.slots, c.q, c.kn, c.vn, c.parents)], status=torch.zeros_like(st)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s in sides:
            o = torch.zeros_like(out)
            s["outs"].append(o)
            s["st"].wait_stream(torch.cuda.current_stream())
            slots_, q_, kn_, vn_, par_ = s["keep"]
            sv.spec_tree_attn(s["kv"], s["c"].layer, 2, slots_, 10, 8, q_, kn_, vn_, o, s["ws"], s["status"],
                              parents=par_, stream=s["st"])
    torch.cuda.synchronize()
    for s, w in zip(sides, want):
        for o in s["outs"]:
            assert np.array_equal(o.cpu().numpy().view(np.uint16), w.view(np.uint16))


def test_offsets_past_32_bits(dev):
    """A pool of more than 2^31 elements: the pages at its end."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(9)
    nkv, hd, page, n_pages = 8, 128, 256, 8400  # 2.2e9 elements
    c = Case(sv, dev, g, 8, nkv, hd, [600], 4, page, layers=1)
    k = torch.empty((1, n_pages, nkv, page, hd), dtype=torch.float16, device=dev)
    v = torch.empty_like(k)
    table = c.table.copy()
    for j in range(3):
        table[c.slots[0], j] = n_pages - 1 - j
        k[0, n_pages - 1 - j] = c.T(c.k[0, c.table[c.slots[0], j]])
        v[0, n_pages - 1 - j] = c.T(c.v[0, c.table[c.slots[0], j]])
    kv = sv.KVPages(k, v, c.T(table), c.T(c.slot_len))
    c.check(c.call(kv))
    # and a copy and a commit there
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    sv.spec_pages_copy(kv, 1, i32([n_pages - 1]), i32([n_pages - 5]), st)
    assert st.item() == 0 and torch.equal(k[0, n_pages - 5], k[0, n_pages - 1])
    n_path = i32([2])
    sv.spec_pages_commit(kv, 1, c.T(c.slots), 4, c.T(c.kn), c.T(c.vn), i32([[1, 3, 0, 0]]), n_path, st)
    assert st.item() == 0
    assert torch.equal(k[0, n_pages - 3, :, 600 - 512], c.T(c.kn)[0, 1])
    assert torch.equal(v[0, n_pages - 3, :, 601 - 512], c.T(c.vn)[0, 3])


# ---------------------------------------------------------------------------
# the model's own cache, and the operators together
# ---------------------------------------------------------------------------
def test_the_models_cache_as_pages(dev):
    """A chain over the model's slot cache agrees with spec_verify_attn on the
    same cache; commit advances the model's n_past; slots are copied."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(11)
    nq, nkv, hd, nt, max_ctx = 8, 2, 128, 7, 200
    m = attn_model(sv, dev, g, nq, nkv, hd, max_ctx, nt, 3)
    kv = sv.spec_model_pages(m)
    f16 = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float16)).to(dev)  # noqa: E731
    kc, vc = f16(nkv, 150, hd), f16(nkv, 150, hd)
    sv.spec_kv_fill(m, 0, 1, 0, 150, kc, vc)
    sv.spec_state_set(m, [1], n_past=[150], anchor=[3])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    st, ws = i32([9]), torch.empty(sv.spec_tree_attn_workspace(kv, 1, nt, nq), dtype=torch.uint8, device=dev)
    # a fork of the slot: its first 150 positions and its state
    sv.spec_pages_copy(kv, 1, i32([1]), i32([2]), st, n_pos=i32([150]))
    sv.spec_state_set(m, [2], n_past=[150], anchor=[3])
    q, kn, vn = f16(nt, nq, hd), f16(nt, nkv, hd), f16(nt, nkv, hd)
    outs = []
    for slot in (1, 2):
        o = torch.zeros((nt, nq * hd), dtype=torch.float16, device=dev)
        sv.spec_tree_attn(kv, 0, 1, i32([slot]), nt, nq, q, kn, vn, o, ws, st)
        assert st.item() == 0
        outs.append(o)
    assert torch.equal(outs[0], outs[1])
    ref = torch.zeros_like(outs[0])
    sv.spec_verify_attn(m, 0, 1, i32([1]), nt, q, kn, vn, ref)
    assert sv.spec_error_check(m) == 0
    # each within half an fp16 step (and the far smaller fp32 error) of the same value
    err = (outs[0].double() - ref.double()).abs()
    assert (err <= 2.0 ** -10 * ref.double().abs() + 2.0 ** -16).all()
    # commit of rows 0, 2, 5 into slot 2
    sv.spec_pages_commit(kv, 1, i32([2]), nt, kn, vn, i32([[0, 2, 5, -1, -1, -1, -1]]), i32([3]), st)
    assert st.item() == 0 and sv.spec_state_get(m, [0, 1, 2])[0] == [0, 150, 153]
    k2, v2 = torch.empty((nkv, 153, hd), dtype=torch.float16, device=dev), torch.empty((nkv, 153, hd), dtype=torch.float16, device=dev)
    sv.spec_kv_read(m, 0, 2, 0, 153, k2, v2)
    torch.cuda.synchronize()
    assert torch.equal(k2[:, :150], kc) and torch.equal(v2[:, 150:].transpose(0, 1), vn[[0, 2, 5]])
    assert torch.equal(k2[:, 150:].transpose(0, 1), kn[[0, 2, 5]])
    # past max_ctx: refused, nothing changes
    sv.spec_state_set(m, [2], n_past=[max_ctx - 2])
    sv.spec_pages_commit(kv, 1, i32([2]), nt, kn, vn, None, i32([3]), st)
    assert st.item() == tree.ST_FULL and sv.spec_state_get(m, [2])[0] == [max_ctx - 2]
    for call in (lambda: sv.spec_pages_free(kv, 1, i32([2]), st), lambda: sv.spec_pages_fork(kv, 1, i32([1]), i32([2]), st)):
        with pytest.raises(sv.SpecError) as e:
            call()
        assert e.value.code == sv.SPEC_E_UNSUPPORTED


def test_a_commit_into_the_models_cache_advances_n_past_alone(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(16)
    m = attn_model(sv, dev, g, 4, 2, 128, 100, 7, 3)
    kv = sv.spec_model_pages(m)
    sv.spec_state_set(m, [0, 1, 2], n_past=[5, 6, 7], emit_idx=[8, 9, 10], anchor=[1, 2, 3])
    kn = torch.ones((1, 4, 2, 128), dtype=torch.float16, device=dev)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    st = i32([9])
    sv.spec_pages_commit(kv, 1, i32([1]), 4, kn, kn, None, i32([3]), st)
    assert st.item() == 0 and sv.spec_state_get(m, [0, 1, 2]) == ([5, 9, 7], [8, 9, 10], [1, 2, 3])


def test_rounds_of_a_tree_drafting_decoder(orc, dev):
    """The operators as a tree-drafting program uses them, over a small
    attention model whose logits are a fixed projection of the attention
    output: prompts appended to a paged cache and forked into branches; every
    round candidates sampled under filters, the tree's nodes evaluated in
    every layer, the greedy path accepted and committed.  The emitted tokens
    are those of a plain sequential decode in 64 bits wherever that decode's
    margins are not within the fp16 noise, and the cache ends as the
    sequential one."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(21)
    layers, nq, nkv, hd, V, nt, rounds = 2, 4, 2, 64, 40, 9, 4
    n_prompt, n_seq = [21, 5], 4
    page, max_pages = 8, 16
    E = (g.standard_normal((V, nq * hd)) * 1.0).astype(np.float16)      # token -> hidden
    Wk = g.standard_normal((layers, V, nkv, hd)).astype(np.float16)     # token -> key, value (no positions)
    Wv = g.standard_normal((layers, V, nkv, hd)).astype(np.float16)
    Wo = (g.standard_normal((nq * hd, V)) * 0.5).astype(np.float32)
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    Ed, Wkd, Wvd, Wod = T(E), T(Wk), T(Wv), T(Wo)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731

    def plain_logits(context):
        """fp64 logits behind a list of tokens."""
        h = np.zeros(nq * hd)
        for l in range(layers):
            k, v = Wk[l, context], Wv[l, context]
            q = E[context[-1]].reshape(1, nq, hd)
            o, _, _ = tree.tree_attention(q, k[:-1], v[:-1], k[-1:], v[-1:], [-1])
            h += o.reshape(-1)
        return h @ Wo.astype(np.float64)

    n_pages = 60
    kc = torch.zeros((layers, n_pages, nkv, page, hd), dtype=torch.float16, device=dev)
    vc = torch.zeros_like(kc)
    table, lens, refs = i32([[-1] * max_pages] * n_seq), i32([0] * n_seq), i32([0] * n_pages)
    kv = sv.KVPages(kc, vc, table, lens, refs)
    st, cp = i32([9] * n_seq), i32([[9, 9]] * n_seq)
    texts = [[int(x) for x in g.integers(0, V, n)] for n in n_prompt]
    for s, text in enumerate(texts):  # the prompt but its last token, which is the first anchor
        n = len(text) - 1
        sv.spec_pages_extend(kv, 1, i32([s]), i32([n]), cp[:1], st[:1])
        sv.spec_pages_commit(kv, 1, i32([s]), n, Wkd[:, text[:-1]].unsqueeze(1).contiguous(),
                             Wvd[:, text[:-1]].unsqueeze(1).contiguous(), None, i32([n]), st[:1])
        assert st[0].item() == 0
    sv.spec_pages_fork(kv, 2, i32([0, 1]), i32([2, 3]), st[:2])
    assert st[:2].tolist() == [0, 0]
    texts += [list(t) for t in texts]
    texts[2][-1], texts[3][-1] = (texts[2][-1] + 1) % V, (texts[3][-1] + 7) % V  # branches with anchors of their own
    slots = i32(list(range(n_seq)))
    ws = torch.empty(sv.spec_tree_attn_workspace(kv, n_seq, nt, nq), dtype=torch.uint8, device=dev)
    ambiguous = [False] * n_seq
    emitted_total = 0
    for rnd in range(rounds):
        # ---- draft: per node two sampled children, from noisy logits of the sequence's true ones
        parents = np.array([-1, 0, 0, 1, 1, 2, 3, 3, 6], np.int32)
        tokens = np.zeros((n_seq, nt), np.int32)
        for s in range(n_seq):
            tokens[s, 0] = texts[s][-1]
        paths = tree.chains(parents.tolist())
        for i in range(1, nt):
            lg = np.stack([plain_logits(texts[s][:-1] + [int(tokens[s, j]) for j in paths[i][:-1]])
                           for s in range(n_seq)]).astype(np.float32)
            u = g.integers(0, 2 ** 32, n_seq, dtype=np.uint64).astype(np.uint32)
            tok = i32([9] * n_seq)
            sv.spec_sample(T(lg), n_seq, V, T(u.view(np.int32)), tok, temperature=T(np.full(n_seq, 0.7, np.float32)),
                           top_k=i32([3] * n_seq), top_p=T(np.full(n_seq, 0.95, np.float32)))
            tokens[:, i] = tok.cpu().numpy()
            for s in range(n_seq):
                assert tokens[s, i] == tree.sample_row(lg[s], orc.row_weights, u[s], float(np.float32(0.7)), 3, 0.95)[0]
        # ---- the target pass over the tree
        td = T(tokens).long()
        sv.spec_pages_extend(kv, n_seq, slots, i32([nt] * n_seq), cp, st)
        assert st.tolist() == [0] * n_seq
        kn, vn = Wkd[:, td].contiguous(), Wvd[:, td].contiguous()  # [layers][n_seq][nt][nkv][hd]
        q = Ed[td].contiguous()
        h = torch.zeros((n_seq, nt, nq * hd), dtype=torch.float64, device=dev)
        par = T(np.tile(parents, (n_seq, 1)))
        for l in range(layers):
            o = torch.zeros((n_seq, nt, nq * hd), dtype=torch.float16, device=dev)
            sv.spec_tree_attn(kv, l, n_seq, slots, nt, nq, q, kn[l], vn[l], o, ws, st, parents=par)
            h += o.double()
        logits = h @ Wod.double()
        am = logits.argmax(2).to(torch.int32)
        path, n_path, em = i32([[9] * nt] * n_seq), i32([9] * n_seq), i32([[9] * nt] * n_seq)
        sv.spec_accept_tree(am, T(tokens), par, None, n_seq, nt, path, n_path, em)
        sv.spec_pages_commit(kv, n_seq, slots, nt, kn, vn, path, n_path, st)
        assert st.tolist() == [0] * n_seq
        # ---- against the sequential decode
        for s in range(n_seq):
            new = em[s, :n_path[s].item()].tolist()
            for t in new:
                lg = plain_logits(texts[s])
                top2 = np.partition(lg, -2)[-2:]
                # an output is off by at most half an fp16 step, |o| < 4: 2^-9 a layer and weight
                noise = 2 * layers * 2.0 ** -9 * np.abs(Wo).sum(0).max()
                if top2[1] - top2[0] > noise or int(np.argmax(lg)) == t:
                    assert int(np.argmax(lg)) == t
                else:
                    ambiguous[s] = True
                texts[s].append(t)
            emitted_total += len(new)
            assert lens[s].item() == len(texts[s]) - 1
    assert emitted_total > n_seq * rounds  # some drafts were accepted
    # ---- the cache holds the texts' keys and values
    for s in range(n_seq):
        for p, t in enumerate(texts[s][:-1]):
            pg = table[s, p // page].item()
            assert torch.equal(kc[:, pg, :, p % page], Wkd[:, t]) and torch.equal(vc[:, pg, :, p % page], Wvd[:, t])


# ---------------------------------------------------------------------------
# the weights' precision
# ---------------------------------------------------------------------------
def check_tight(c, got, floor):
    """As Case.check, without a rounding of the weights to fp16 for any number
    of rows.  Weights, relative to themselves: the split into two fp16 numbers
    2^-21 (hi cut off behind 11 bits, lo rounded to half a step of its own) and
    2^-22 (that much of hi more in lo), exp2 2^-22, the rounding of its
    argument, up to 16 in magnitude where a weight counts, 2^-21: together less
    than 2^-19.  Relative to the row's
    largest weight, 1: `floor`, where hi and lo leave fp16's normal numbers.
    Plus the scores' error and fp32 sums as there."""
    for b in range(c.n):
        m = int(c.counts[b])
        if m == 0:
            continue
        k, v = c.cached(0, b), c.cached(1, b)
        ref, mag, dots = tree.tree_attention(c.q[b, :m], k, v, c.kn[b, :m], c.vn[b, :m], c.parents[b, :m].tolist(),
                                             c.window, c.sinks, c.scale)
        scale = c.scale or c.hd ** -0.5
        ds = (c.hd + 4) * 2.0 ** -23 * abs(scale) * dots
        rel = np.expm1(2 * ds) + 2.0 ** -19 + ((c.lens[b] + m) / 8 + 64) * 2.0 ** -23
        g = c.nq // c.nkv
        v_sum = np.abs(v.astype(np.float64)).sum(0) + np.abs(c.vn[b, :m].astype(np.float64)).sum(0)  # [nkv][hd]
        bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * (rel[..., None] * mag + floor * np.repeat(v_sum, g, 0))
        err = np.abs(got[b, :m].astype(np.float64) - ref)
        assert np.isfinite(got[b, :m]).all() and (err <= bound).all(), (b, float(np.max(err - bound)))


WEIGHT_FLOOR = 2.0 ** -36  # of the kernel for many rows: 2^-25 twice over a factor of 2^12


@pytest.mark.parametrize("nq,nkv,hd,lens,nt", [(8, 2, 64, [500, 90], 3), (8, 2, 128, [500, 90], 8),
                                               (32, 8, 128, [300, 77], 16), (40, 8, 128, [512, 260], 16),
                                               (8, 2, 64, [900, 130], 32), (8, 1, 128, [700], 63), (16, 2, 64, [128], 64)])
def test_weights_are_not_rounded_to_fp16(dev, nq, nkv, hd, lens, nt):
    """Keys of score 0 and value 1 against as many of a score a little below
    and value -1: the output is half the difference of the two weights, a few
    roundings of one fp16 number, and the scores are too small to be off.  With
    any number of rows."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([41, nq, nt])
    c = Case(sv, dev, g, nq, nkv, hd, lens, nt, 64, scale=1.0)
    c.q[:] = 0
    c.q[..., 0] = g.uniform(0.5, 2.0, c.q.shape[:3])
    for k, v in ((c.k, c.v), (c.kn, c.vn)):
        low = g.integers(0, 2, k.shape[:-1]).astype(bool)
        k[:], v[:] = 0, np.where(low, -1.0, 1.0)[..., None]
        k[..., 0] = np.where(low, -0.0011, 0.0)
    check_tight(c, c.call(), WEIGHT_FLOOR)


@pytest.mark.parametrize("window,sinks", [(0, 0), (2000, 4)])
@pytest.mark.parametrize("nt", [4, 8, 16, 32, 64])
def test_keys_far_below_a_dominant_one(dev, nt, window, sinks):
    """A first position whose score stands 8 to 18 nats above thousands of
    nearly equal ones and whose value is 0: the output is what those add up
    to.  16, 32, 64, 128 and 256 rows a kv head."""
    import speculative_decoding_verification_round_gb300 as sv
    hd, n = 64, 3000
    for nats in (8.0, 14.0, 16.0, 18.0):
        g = np.random.default_rng([43, nt, int(nats)])
        c = Case(sv, dev, g, 4, 1, hd, [n], nt, 64, window, sinks, layers=1)
        c.q[:] = 1.0 + 0.01 * g.standard_normal(c.q.shape)
        for a in (c.k, c.kn):
            a[:] = 0.01 * g.standard_normal(a.shape)
        for a in (c.v, c.vn):
            a[:] = g.uniform(0.5, 1.5, a.shape)
        first = c.table[c.slots[0], 0]
        c.k[0, first, 0, 0], c.v[0, first, 0, 0] = nats / np.sqrt(hd), 0.0
        check_tight(c, c.call(), WEIGHT_FLOOR)


@pytest.mark.parametrize("nq,nkv,hd,nt", [(4, 2, 64, 3), (8, 1, 128, 4), (8, 2, 128, 16), (8, 2, 64, 32), (4, 1, 128, 64)])
def test_infinite_values_that_are_seen(dev, nq, nkv, hd, nt):
    """Infinities in V at positions that every row sees: infinite outputs of
    their sign, NaN where both signs meet or a NaN is, and nothing elsewhere."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([53, nt])
    c = Case(sv, dev, g, nq, nkv, hd, [600, 140], nt, 32)
    clean = c.call()
    for b in range(2):
        for p, d, x in ((3, 0, np.inf), (100, 1, -np.inf), (40, 2, np.inf), (90, 2, -np.inf), (7, 3, np.nan), (20, 4, np.inf),
                        (127, 4, np.inf)):
            c.v[c.layer, c.table[c.slots[b], p // 32], :, p % 32, d] = x
    got = c.call()
    assert (got[..., [0, 4]] == np.inf).all() and (got[..., 1] == -np.inf).all() and np.isnan(got[..., 2:4]).all()
    assert np.array_equal(got[..., 5:].view(np.uint16), clean[..., 5:].view(np.uint16))


# ---------------------------------------------------------------------------
# waits that give up
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("nq,nkv,hd,lens,nt", [(32, 8, 128, [900, 0, 37, 400, 5], 16), (40, 8, 128, [600, 0, 1, 200, 9], 16),
                                               (8, 2, 64, [700, 0, 130, 65, 20000], 63), (16, 2, 64, [40, 0, 300, 9, 128], 12),
                                               (6, 1, 128, [30000, 0, 2, 70, 7], 64)])
def test_a_wait_that_gives_up_fails_closed(dev, nq, nkv, hd, lens, nt):
    """Every CTA's first wait given up at once: the call ends, the sequences
    with nodes are NaN with SPEC_ST_TIMEOUT beside a status of their own, rows
    of no node stay; with the budget restored the next calls are right, bit by
    bit as before."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([47, nq, nt])
    c = Case(sv, dev, g, nq, nkv, hd, lens, nt, 32, window=0, sinks=0, counts=[nt, nt, nt - 1, 0, 5])
    c.slots[2] = 77
    c.v[c.layer, c.table[c.slots[0], 0]] = np.inf  # (behind a masked tile's marks, too: a window)
    good = c.call()
    assert c.status.tolist() == [0, 0, tree.ST_SLOT, 0, 0]
    try:
        for window in (0, 20, 0):
            sv.spec_tree_set_wait_budget(0)
            c.window, c.sinks = window, window // 5
            got = c.call()
            assert c.status.tolist() == [sv.SPEC_ST_TIMEOUT] * 2 + [tree.ST_SLOT, 0, sv.SPEC_ST_TIMEOUT]
            for b, m in enumerate(c.counts):
                assert np.isnan(got[b, :m]).all() and (got[b, m:] == 7.0).all(), b
            c.window = c.sinks = 0
            sv.spec_tree_set_wait_budget(131072)
            assert np.array_equal(c.call().view(np.uint16), good.view(np.uint16))
            assert c.status.tolist() == [0, 0, tree.ST_SLOT, 0, 0]
        for bad in (-1, 131073):
            with pytest.raises(sv.SpecError):
                sv.spec_tree_set_wait_budget(bad)
    finally:
        sv.spec_tree_set_wait_budget(131072)
