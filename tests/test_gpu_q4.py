"""The cache in 4 bits on the GPU: commit, reading back and pages bit by bit
against oracle/long_context.py, attention over it against the plain 64-bit tree
attention of oracle/tree.py on the values that the codes stand for."""
import numpy as np
import pytest

from oracle import long_context as lc
from oracle import tree
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def random_rows(g, shape, amp=1.0):
    """fp16 rows with a few channels larger than the others."""
    x = g.standard_normal(shape) * np.where(g.random(shape[-1]) < 0.06, 4.0, 1.0) * amp
    return x.astype(np.float16)


def random_cache(g, shape):
    """Codes, scales (eight significant bits, of either sign, some 0) and their values."""
    codes = g.integers(0, 256, shape[:-1] + (shape[-1] // 32, 16)).astype(np.uint8)
    s = np.exp2(g.uniform(-4, 0, shape[:-1] + (shape[-1] // 32,)))
    m, e = np.frexp(s)
    s = np.ldexp(np.rint(m * 256) / 256, e) * np.where(g.random(s.shape) < 0.5, -1, 1) * (g.random(s.shape) > 0.02)
    s = s.astype(np.float16)
    return codes, s, lc.values(codes, s).astype(np.float16)


class Q4Case(Case):
    """test_gpu_tree's inputs over a cache in 4 bits; self.k, self.v are its values (exact in fp16)."""

    def __init__(self, sv, dev, g, *args, **kw):
        super().__init__(sv, dev, g, *args, **kw)
        self.kc, self.ks, self.k = random_cache(g, self.k.shape)
        self.vc, self.vs, self.v = random_cache(g, self.v.shape)

    def pool(self):
        return self.sv.KVPagesQ4(*(self.T(a) for a in (self.kc, self.vc, self.ks, self.vs, self.table, self.slot_len)))

    def call(self, kv=None, chain=False, counts=True, **kw):
        import torch
        kv = kv or self.pool()
        self.out = torch.full((self.n, self.nt, self.nq, self.hd), 7.0, dtype=torch.float16, device=self.dev)
        self.status = torch.full((self.n,), 99, dtype=torch.int32, device=self.dev)
        ws = torch.full((self.sv.spec_tree_attn_q4_workspace(kv, self.n, self.nt, self.nq),), 0xFF, dtype=torch.uint8,
                        device=self.dev)
        args = dict(q=self.T(self.q), k_new=self.T(self.kn), v_new=self.T(self.vn))
        args.update(kw)
        self.sv.spec_tree_attn_q4(kv, self.layer, self.n, self.T(self.slots), self.nt, self.nq, out=self.out,
                                  workspace=ws, status=self.status, parents=None if chain else self.T(self.parents),
                                  n_nodes=self.T(self.counts) if counts else None, window=self.window,
                                  sinks=self.sinks, scale=self.scale or 0.0, **args)
        torch.cuda.synchronize()
        return self.out.cpu().numpy()

    def check(self, got, seqs=None):
        """The bound of Case.check with the scores' error of this path.  A block of 32
        sums products of q with codes u in [0, 15], from -8 sum q on: its magnitudes are at
        most 23 |q|_1 of the block, a unit of 2^-23 of them for each of its 32 + 2 terms,
        and with the scale two roundings more; the sum over blocks adds one a
        block, of values that are smaller.  With |s| the block's scale that is 40 x 24 x 2^-23
        sum |q_b|_1 |s_b|.  Weights are pairs of fp16 numbers at any number of rows: 2^-36
        of the largest for each key."""
        for b in range(self.n) if seqs is None else seqs:
            m = int(self.counts[b])
            assert (got[b, m:] == np.float16(7.0)).all(), b  # rows of no node
            if m == 0:
                continue
            kc = self.cached(0, b)
            ref, mag, dots = tree.tree_attention(self.q[b, :m], kc, self.cached(1, b), self.kn[b, :m],
                                                 self.vn[b, :m], self.parents[b, :m].tolist(), self.window, self.sinks,
                                                 self.scale)
            scale = self.scale or self.hd ** -0.5
            ds = (self.hd + 4) * 2.0 ** -23 * abs(scale) * dots
            if kc.size:
                q1 = np.abs(self.q[b, :m].astype(np.float64)).reshape(m, self.nkv, -1, self.hd // 32, 32).sum(-1)
                pg = [(self.table[self.slots[b], p // self.page], p % self.page) for p in range(self.lens[b])]
                s = np.stack([np.abs(self.ks[self.layer, e, :, at].astype(np.float64)) for e, at in pg if e >= 0])
                worst = np.einsum("mhgb,phb->mhgp", q1, np.nan_to_num(s)).max(-1).reshape(m, self.nq)
                ds = ds + 40 * 24 * 2.0 ** -23 * abs(scale) * worst
            rel = np.expm1(2 * ds) + 2.0 ** -20 + ((self.lens[b] + m) / 8 + 64) * 2.0 ** -23
            rel = rel + (self.lens[b] + m) * 2.0 ** -36
            bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[..., None] * mag
            err = np.abs(got[b, :m].astype(np.float64) - ref)
            assert np.isfinite(got[b, :m]).all() and (err <= bound).all(), (b, float(np.max(err - bound)))


SHAPES = [
    # nq, nkv, hd, lens, nt, page, window, sinks, counts, kind
    (4, 4, 64, [0, 1, 2], 1, 16, 0, 0, None, "chain"),           # no context, one position; one row a head
    (8, 1, 128, [0, 33, 31, 32], 1, 16, 0, 0, None, "chain"),    # around a warp's positions
    (32, 8, 128, [300], 1, 64, 0, 0, None, "chain"),             # GQA 4: 4 rows
    (14, 2, 64, [4000, 17], 1, 16, 0, 0, None, "chain"),         # a draft model's decode step
    (32, 8, 128, [300, 129], 4, 64, 0, 0, None, "tree"),         # 16 rows
    (32, 8, 128, [300], 8, 64, 0, 0, None, "tree"),              # 32 rows
    (40, 8, 128, [512, 37, 500], 16, 64, 0, 0, None, "tree"),    # GQA 5, 80 rows
    (14, 2, 64, [257, 64, 65], 3, 24, 0, 0, [3, 1, 0], "tree"),  # odd pages; a sequence without nodes
    (8, 1, 128, [700], 63, 100, 0, 0, None, "tree"),             # 504 rows of one head
    (6, 1, 128, [190, 63, 0], 64, 7, 0, 0, [64, 33, 64], "forest"),
    (5, 5, 64, [128, 129, 127], 64, 128, 0, 0, None, "flat"),
    (32, 8, 128, [5000, 3], 2, 1000, 0, 0, None, "chain"),
    (16, 2, 64, [1000, 900, 0, 63], 2, 16, 100, 4, [2, 2, 2, 1], "tree"),
    (16, 2, 64, [1000, 900, 0, 63], 5, 16, 100, 4, [5, 5, 5, 2], "tree"),
    (8, 8, 128, [2000, 64, 10], 12, 64, 64, 0, None, "tree"),
    (8, 2, 128, [513, 65, 1], 3, 32, 1, 0, None, "tree"),        # every node sees itself alone
    (8, 2, 128, [513, 65, 1], 20, 32, 3, 200, None, "chain"),    # sinks past the window
    (4, 2, 64, [3000, 500], 33, 48, 777, 65, None, "forest"),
    (4, 1, 64, [300], 4, 64, 2 ** 31 - 1, 2 ** 31 - 1, None, "tree"),
]


@pytest.mark.parametrize("nq,nkv,hd,lens,nt,page,window,sinks,counts,kind", SHAPES)
def test_attention_matches_the_reference(dev, nq, nkv, hd, lens, nt, page, window, sinks, counts, kind):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(nq * 1000 + nt * 7 + len(lens))
    c = Q4Case(sv, dev, g, nq, nkv, hd, lens, nt, page, window, sinks, counts, kind)
    got = c.call(chain=kind == "chain", counts=counts is not None)
    assert c.status.tolist() == [0] * c.n
    c.check(got)
    assert np.array_equal(c.call(chain=kind == "chain").view(np.uint16), got.view(np.uint16))  # the same bits


def test_many_ragged_sequences(dev):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(5)
    n = 300
    lens = [int(x) for x in g.choice([0, 1, 16, 17, 40, 130], n)]
    c = Q4Case(sv, dev, g, 4, 2, 64, lens, 6, 16, counts=g.integers(0, 7, n))
    c.slots[7], c.lens[7] = c.slots[3], c.lens[3]
    got = c.call()
    assert c.status.tolist() == [0] * n
    c.check(got)


def test_large_scores_and_a_given_scale(dev):
    import speculative_decoding_verification_round_gb300 as sv
    for scale, amp in ((0.5, 2.0), (-0.25, 1.0), (3.0, 0.5)):
        for nt in (1, 9):
            g = np.random.default_rng(int(amp * 10))
            c = Q4Case(sv, dev, g, 8, 2, 64, [600, 90], nt, 32, scale=scale, amp=amp)
            c.check(c.call())


@pytest.mark.parametrize("hd,nq,nt", [(64, 2, 1), (128, 8, 4), (128, 8, 8), (128, 40, 8), (64, 16, 8), (64, 16, 64)])
def test_nothing_of_what_is_masked_gets_in(dev, hd, nq, nt):
    """Rows that a row does not see -- behind the length, in front of the window,
    in other branches, past the node count -- may hold NaN scales, infinities and NaN."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(4)
    c = Q4Case(sv, dev, g, nq, 2, hd, [300, 90], nt, 32, window=50, sinks=3)
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
                c.ks[:, pg, :, at], c.vs[:, pg, :, at] = np.nan, np.inf
    depth = [len(x) - 1 for x in tree.chains(c.parents[0].tolist())]
    p = c.lens[0] - 49  # seen by the nodes of depth 0 alone
    c.vs[:, c.table[c.slots[0], p // 32], :, p % 32] = np.nan
    got = c.call()
    same = np.ones((2, nt), bool)
    same[0] = [d > 0 for d in depth]
    assert np.isfinite(got[same]).all() and np.isnan(got[~same]).all()
    d = np.abs(got[same].astype(np.float64) - clean[same].astype(np.float64))
    # both are within the bound of check() of the same reference; an fp16 step of the value covers twice that
    assert (d <= 2.0 ** -10 * np.abs(clean[same].astype(np.float64)) + 2.0 ** -13).all()
    # a NaN in a key that is seen is seen
    c = Q4Case(sv, dev, g, nq, 2, hd, [300, 90], nt, 32)
    c.ks[:, c.table[c.slots[1], 1], 0, 5] = np.nan
    got = c.call()
    assert np.isfinite(got[0]).all() and np.isnan(got[1, :, :nq // 2]).all() and np.isfinite(got[1, :, nq // 2:]).all()


@pytest.mark.parametrize("hd,nt", [(64, 1), (128, 4), (64, 8), (128, 9), (64, 40)])
def test_strides_and_other_rows_queries(dev, hd, nt):
    """Rows of q, k_new and v_new apart, and planes whose layers are apart, with NaN
    between; a NaN in one row's query is that row's alone."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([hd, nt])
    c = Q4Case(sv, dev, g, 8, 2, hd, [300, 0, 77], nt, 16, counts=[nt, nt, max(1, nt - 1)])
    want = c.call()
    c.check(want)

    def apart(x, row):
        buf = torch.full((c.n * nt, row), float("nan"), dtype=torch.float16, device=dev)
        buf[:, :x[0, 0].size] = c.T(x).view(c.n * nt, -1)
        return buf
    qs, ks = 8 * hd + 24, 2 * hd + 8
    layers = [torch.full((t.shape[0], t.shape[1] + 3, *t.shape[2:]), 0x7F if t.dtype == torch.uint8 else float("nan"), dtype=t.dtype,
                         device=dev)[:, :t.shape[1]] for t in c.pool()._keep[:4]]
    for a, b in zip(layers, c.pool()._keep):
        a.copy_(b)
    kv = sv.KVPagesQ4(*layers, c.T(c.table), c.T(c.slot_len))
    got = c.call(kv, q=apart(c.q, qs), k_new=apart(c.kn, ks), v_new=apart(c.vn, ks), q_stride=qs, kv_stride=ks)
    assert c.status.tolist() == [0] * 3 and np.array_equal(got.view(np.uint16), want.view(np.uint16))
    q = c.q.copy()
    q[0, nt - 1, 3, 5], q[2, 0, 6, hd - 1] = np.nan, np.inf
    got = c.call(q=c.T(q))
    odd = np.zeros(got.shape[:3], bool)
    odd[0, nt - 1, 3] = odd[2, 0, 6] = True
    assert np.isnan(got[odd]).all() and np.array_equal(got[~odd].view(np.uint16), want[~odd].view(np.uint16))


def test_infinities_of_the_trees_own_rows(dev):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(14)
    for nt in (4, 8, 20):
        c = Q4Case(sv, dev, g, 8, 2, 128, [70, 90], nt, 32, counts=[nt, nt - 1])
        c.parents[:, 1:] = 0
        c.kn[1, nt - 1], c.vn[1, nt - 1] = np.inf, np.nan
        c.vn[0, nt - 1] = -np.inf
        got = c.call()
        assert np.isfinite(got[0, :nt - 1]).all() and np.isfinite(got[1, :nt - 1]).all()
        assert np.isneginf(got[0, nt - 1]).all()
        c.vn[0, nt - 1] = 0
        c.check(c.call())


@pytest.mark.parametrize("nq,nkv,hd,n,longest,nt", [(32, 8, 128, 2, 9001, 16), (16, 8, 64, 3, 7000, 40),
                                                    (32, 8, 128, 500, 290, 16), (40, 8, 128, 300, 140, 16),
                                                    (8, 2, 64, 700, 200, 64), (32, 8, 128, 40, 3000, 1), (16, 2, 64, 60, 2000, 2)])
def test_repeated_calls_agree(dev, nq, nkv, hd, n, longest, nt):
    """No result depends on how the warps of a CTA run against each other: the same
    call forty times, bit by bit."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([31, nq, n])
    lens = g.integers(0, longest + 1, n)
    lens[:2] = longest
    c = Q4Case(sv, dev, g, nq, nkv, hd, lens.tolist(), nt, 64, layers=1)
    first = c.call()
    c.check(first, range(0, n, max(1, n // 12)))
    out, kv, slots, parents, counts = c.out, c.pool(), c.T(c.slots), c.T(c.parents), c.T(c.counts)
    q, kn, vn, want = c.T(c.q), c.T(c.kn), c.T(c.vn), c.out.clone()
    ws = torch.empty(sv.spec_tree_attn_q4_workspace(kv, n, nt, nq), dtype=torch.uint8, device=dev)
    for _ in range(40):
        out.fill_(7.0)
        sv.spec_tree_attn_q4(kv, 0, n, slots, nt, nq, q, kn, vn, out, ws, c.status, parents=parents, n_nodes=counts)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_two_streams_at_once(dev):
    """Calls of all three kernels, two of each at a time with workspaces of their own."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    for nq, lens, nt in ((8, [300, 90], 1), (16, [20000, 90], 3), (40, [900, 130], 9)):
        sides = []
        for i in range(2):
            c = Q4Case(sv, dev, np.random.default_rng([nt, i]), nq, 2, 128, lens, nt, 32, layers=1)
            want = c.call()
            c.check(want)
            kv = c.pool()
            ws = torch.empty(sv.spec_tree_attn_q4_workspace(kv, 2, nt, nq), dtype=torch.uint8, device=dev)
            args = [c.T(a) for a in (c.slots, c.q, c.kn, c.vn, c.parents)]
            sides.append((kv, ws, args, c.out.clone(), torch.zeros_like(c.out), c.status, torch.cuda.Stream()))
        torch.cuda.synchronize()
        for _ in range(20):
            for kv, ws, (slots, q, kn, vn, par), want, out, st, stream in sides:
                sv.spec_tree_attn_q4(kv, 0, 2, slots, nt, nq, q, kn, vn, out, ws, st, parents=par, stream=stream)
        torch.cuda.synchronize()
        for _, _, _, want, out, st, _ in sides:
            assert torch.equal(out, want) and st.tolist() == [0, 0]


def test_waits_that_give_up(dev):
    """Every CTA's first wait for scores gives up at once: its sequences are NaN
    with SPEC_ST_TIMEOUT, and the next call is served."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(16)
    try:
        for nq, hd, nt in ((8, 64, 16), (8, 128, 24), (16, 128, 40)):
            c = Q4Case(sv, dev, g, nq, 2, hd, [900, 130, 0], nt, 32)
            good = c.call()
            c.check(good)
            sv.spec_tree_set_wait_budget(0)
            got = c.call()
            assert c.status.tolist() == [sv.SPEC_ST_TIMEOUT] * 3 and np.isnan(got).all()
            sv.spec_tree_set_wait_budget(131072)
            assert np.array_equal(c.call().view(np.uint16), good.view(np.uint16))
            assert c.status.tolist() == [0, 0, 0]
    finally:
        sv.spec_tree_set_wait_budget(131072)


def test_scales_of_any_size(dev):
    """Values from fp16's smallest to near its largest."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(15)
    for e, nt in ((-24, 1), (-20, 4), (-16, 8), (-13, 1), (11, 4), (12, 12), (-24, 16), (12, 40)):
        c = Q4Case(sv, dev, g, 8, 2, 64, [300, 90], nt, 32)
        c.vs[:] = np.sign(c.vs) * np.exp2(e) * (1 if e < -18 else 1.9921875)
        c.v = lc.values(c.vc, c.vs).astype(np.float16)
        assert (c.v == lc.values(c.vc, c.vs)).all()
        c.vn[:] = c.vn * np.float16(2.0 ** max(e, -20))
        c.check(c.call())


def test_refused_sequences(dev):
    import speculative_decoding_verification_round_gb300 as sv
    for nt in (2, 6):
        g = np.random.default_rng(7)
        c = Q4Case(sv, dev, g, 8, 2, 64, [100, 90, 80, 70, 60, 50, 40, 30], nt, 16, counts=[nt] * 5 + [nt + 1, nt, nt])
        c.slots[1] = 99
        c.table[c.slots[2], 3] = 10 ** 6
        c.slot_len[c.slots[3]] = c.table.shape[1] * 16 + 1
        c.parents[4, 1] = 3
        c.table[c.slots[6], 0] = -7
        got = c.call()
        assert c.status.tolist() == [0, tree.ST_SLOT, tree.ST_PAGE, tree.ST_PAGE, tree.ST_TREE, tree.ST_TREE, tree.ST_PAGE, 0]
        c.check(got, [0, 7])
        assert np.isnan(got[1:7]).all()


@pytest.mark.parametrize("nt,longest", [(20, 400), (2, 20000), (4, 20000)])
def test_refused_sequences_of_large_calls(dev, nt, longest):
    """The same of the kernels for many rows and for long tables."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(19)
    c = Q4Case(sv, dev, g, 8, 2, 64, [longest, 190, 200, 70, 60, 130], nt, 64, counts=[nt, nt, nt, nt, nt + 1, nt - 1], layers=1)
    c.slots[1] = -1
    c.table[c.slots[2], 3] = -5
    c.slot_len[c.slots[3]] = -1
    c.parents[5, nt - 2] = nt - 2
    got = c.call()
    assert c.status.tolist() == [0, tree.ST_SLOT, tree.ST_PAGE, tree.ST_PAGE, tree.ST_TREE, tree.ST_TREE]
    c.check(got, [0])
    assert np.isnan(got[1:5]).all() and np.isnan(got[5, :nt - 1]).all()
    c.parents[5, nt - 2] = -1
    c.table[c.slots[0], longest // 128] = 10 ** 6  # in the middle of the long one
    got = c.call()
    assert c.status.tolist() == [tree.ST_PAGE, tree.ST_SLOT, tree.ST_PAGE, tree.ST_PAGE, tree.ST_TREE, 0]
    c.check(got, [5])
    assert np.isnan(got[:5]).all()


# ---------------------------------------------------------------------------
# rows into the cache and out of it
# ---------------------------------------------------------------------------
class Planes:
    """A cache in 4 bits on the host and the device, filled with noise."""

    def __init__(self, sv, dev, g, layers, n_pages, nkv, page, hd, table, lens, refs=None):
        import torch
        self.g = g
        shape = (layers, n_pages, nkv, page, hd)
        self.host = []
        for _ in range(2):
            codes, scales, _v = random_cache(g, shape)
            self.host += [codes, scales]
        self.table, self.lens, self.refs = (None if a is None else np.asarray(a, np.int32) for a in (table, lens, refs))
        self.T = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev)
        kc, ks, vc, vs = (self.T(a) for a in self.host)
        self.kv = sv.KVPagesQ4(kc, vc, ks, vs, self.T(self.table), self.T(self.lens), self.T(self.refs))

    def planes(self):
        kc, vc, ks, vs = (t.cpu().numpy() for t in self.kv._keep[:4])
        return kc, ks, vc, vs

    def book(self):
        return tuple(None if t is None else t.cpu().numpy() for t in self.kv._keep[4:])


def same_planes(got, want):
    for a, b in zip(got, want):
        if a.dtype == np.float16:
            a, b = a.view(np.uint16), b.view(np.uint16)
            a, b = np.where(a == 0x8000, 0, a), np.where(b == 0x8000, 0, b)  # (a scale of zero has no sign)
        assert np.array_equal(a, b)


@pytest.mark.parametrize("hd,nkv,page,nt,with_path", [(128, 8, 16, 9, True), (64, 2, 24, 70, False), (32, 1, 7, 3, True),
                                                     (96, 3, 5, 130, False)])
def test_commit_and_read(dev, hd, nkv, page, nt, with_path):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([hd, nt])
    layers, n = 2, 3
    lens = np.array([5, 0, 2 * page, 1], np.int32)
    max_pages = -(-(2 * page + nt) // page) + 1
    table = g.permutation(4 * max_pages).reshape(4, max_pages).astype(np.int32)
    c = Planes(sv, dev, g, layers, 4 * max_pages, nkv, page, hd, table, lens)
    rows = [random_rows(g, (layers, n, nt, nkv, hd)) for _ in range(2)]
    for x in rows:  # ties, zeros, the largest, the smallest, what is not finite
        x[0, 0, 0, 0, :32] = np.where(np.arange(32) % 2 == 0, 1.5, -1.5)
        x[0, 0, 1, 0, :32] = 0
        x[0, 0, 2, 0, :32] = np.linspace(-65504, 65504, 32)
        x[0, 1, 0, 0, :32] = np.arange(32) * 2.0 ** -24
        x[0, 1, 1, 0, :32] = np.arange(32) * 2.0 ** -16
        x[0, 1, 2, 0, :32] = np.arange(32) / 4.0 - 3.875  # halves of the scale
        x[1, 0, 0, 0, 3], x[1, 0, 1, 0, 7] = np.inf, np.nan
    slots = np.array([2, 0, 3], np.int32)
    n_path = np.array([nt, max(0, nt - 2), 1], np.int32)
    path = np.sort(np.stack([g.permutation(nt) for _ in range(n)]), 1).astype(np.int32) if with_path else None
    if with_path:
        path[0] = path[0][::-1]
    st = torch.full((n,), 9, dtype=torch.int32, device=dev)
    new_len = torch.full((4,), -5, dtype=torch.int32, device=dev)
    sv.spec_pages_q4_commit(c.kv, n, c.T(slots), nt, c.T(rows[0]), c.T(rows[1]), c.T(path), c.T(n_path), st, new_len=new_len)
    assert st.tolist() == [0] * n
    want = [a.copy() for a in c.host]
    back = [np.full((layers, n, nt, nkv, hd), 3.0, np.float16) for _ in range(2)]
    for i in range(n):
        for j in range(n_path[i]):
            pos = lens[slots[i]] + j
            pg, at = table[slots[i], pos // page], pos % page
            for w in range(2):
                codes, scales = lc.pack(*lc.quantise(rows[w][:, i, j if path is None else path[i, j]]))
                want[2 * w][:, pg, :, at], want[2 * w + 1][:, pg, :, at] = codes, scales
                back[w][:, i, j] = lc.values(codes, scales)
    got = c.planes()
    for a, b in zip(got, want):  # NaN scales as such
        if a.dtype == np.float16:
            assert np.array_equal(np.isnan(a), np.isnan(b))
            a[np.isnan(a)], b[np.isnan(b)] = 1, 1
    same_planes(got, want)
    assert new_len.tolist() == [int(lens[s] + n_path[list(slots).index(s)]) if s in slots else -5 for s in range(4)]
    out = [torch.full((layers, n, nt, nkv, hd), 3.0, dtype=torch.float16, device=dev) for _ in range(2)]
    sv.spec_pages_q4_read(c.kv, n, c.T(slots), nt, c.T(lens[slots]), c.T(n_path), out[0], out[1], st)
    assert st.tolist() == [0] * n
    for a, b in zip(out, back):
        a = a.cpu().numpy()
        assert np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(a[~np.isnan(b)], b[~np.isnan(b)])
    # the lengths in place
    sv.spec_pages_q4_commit(c.kv, n, c.T(slots), nt, c.T(rows[0]), c.T(rows[1]), c.T(path), c.T(n_path), st)
    assert st.tolist() == [0] * n
    assert c.kv._keep[5].tolist() == [int(lens[s] + (n_path[list(slots).index(s)] if s in slots else 0)) for s in range(4)]


def test_commit_and_read_refusals(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(1)
    layers, nkv, page, hd, nt = 2, 2, 4, 32, 3
    table = np.array([[0, 1], [2, -1], [3, 99], [4, 5], [6, 7], [8, 9], [8, 10]], np.int32)
    lens = np.array([3, 3, 3, 7, 2, 1, 0], np.int32)
    refs = np.array([1] * 8 + [2] + [1] * 3, np.int32)
    c = Planes(sv, dev, g, layers, 12, nkv, page, hd, table, lens, refs)
    before, book = c.planes(), c.book()
    n = 9
    slots = np.array([1, 2, 3, 4, 5, -1, 7, 0, 0], np.int32)
    path = np.tile(np.array([0, 1, 2], np.int32), (n, 1))
    path[3, 1] = 3
    n_path = np.array([3, 2, 3, 3, 1, 1, 1, 1, 1], np.int32)
    rows = random_rows(g, (layers, n, nt, nkv, hd))
    st = torch.full((n,), 9, dtype=torch.int32, device=dev)
    sv.spec_pages_q4_commit(c.kv, n, c.T(slots), nt, c.T(rows), c.T(rows), c.T(path), c.T(n_path), st)
    assert st.tolist() == [tree.ST_PAGE, tree.ST_PAGE, tree.ST_FULL, tree.ST_TREE, tree.ST_SHARED, tree.ST_SLOT, tree.ST_SLOT,
                           tree.ST_SLOT, tree.ST_SLOT]
    same_planes(c.planes(), before)
    assert all(np.array_equal(a, b) for a, b in zip(c.book(), book))
    out = torch.full((layers, n, nt, nkv, hd), 3.0, dtype=torch.float16, device=dev)
    pos0 = np.array([3, 2, 6, 2, -1, 0, 0, 0, 1], np.int32)
    n_pos = np.array([3, 3, 3, 4, 1, 1, 1, 1, 0], np.int32)
    sv.spec_pages_q4_read(c.kv, n, c.T(slots), nt, c.T(pos0), c.T(n_pos), out, out.clone(), st)
    assert st.tolist() == [tree.ST_PAGE, tree.ST_PAGE, tree.ST_FULL, tree.ST_TREE, tree.ST_FULL, tree.ST_SLOT, tree.ST_SLOT, 0, 0]
    assert (out[:, :7] == 3.0).all() and (out[:, 8] == 3.0).all() and (out[:, 7, 1:] == 3.0).all()
    want = lc.values(before[0][:, 0, :, 0], before[1][:, 0, :, 0])
    assert np.array_equal(out[:, 7, 0].cpu().numpy().astype(np.float64), want)


def test_rows_with_layers_apart(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(3)
    layers, n, nt, nkv, hd, page = 3, 2, 40, 2, 64, 16
    table = g.permutation(8).reshape(2, 4).astype(np.int32)
    c = Planes(sv, dev, g, layers, 8, nkv, page, hd, table, [3, 9])
    rows = [random_rows(g, (layers, n, nt, nkv, hd)) for _ in range(2)]
    step = n * nt * nkv * hd + 80
    bufs = [torch.full((layers, step), float("nan"), dtype=torch.float16, device=dev) for _ in range(4)]
    for b, x in zip(bufs, rows):
        b[:, :step - 80] = c.T(x).view(layers, -1)
    slots, n_path, st = c.T(np.array([1, 0], np.int32)), c.T(np.array([nt, 33], np.int32)), c.T(np.array([9, 9], np.int32))
    pos0 = c.T(np.array([9, 3], np.int32))
    sv.spec_pages_q4_commit(c.kv, n, slots, nt, bufs[0], bufs[1], None, n_path, st, new_layer_stride=step)
    assert st.tolist() == [0, 0] and c.kv._keep[5].tolist() == [36, 49]
    sv.spec_pages_q4_read(c.kv, n, slots, nt, pos0, n_path, bufs[2], bufs[3], st, layer_stride=step)
    assert st.tolist() == [0, 0]
    for w in range(2):
        got = bufs[2 + w].cpu().numpy()
        assert np.isnan(got[:, step - 80:]).all()
        got = got[:, :step - 80].reshape(layers, n, nt, nkv, hd)
        want = lc.values(*lc.pack(*lc.quantise(rows[w])))
        assert np.array_equal(got[:, 0], want[:, 0]) and np.array_equal(got[:, 1, :33], want[:, 1, :33])
        assert np.isnan(got[:, 1, 33:]).all()


@pytest.mark.parametrize("hd,nkv,page", [(64, 2, 48), (96, 1, 100)])
def test_prompts_in_and_out(dev, hd, nkv, page):
    """Rows enough for several waves of CTAs."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(hd)
    layers, n, nt = 8, 2, 2003
    max_pages = -(-nt // page) + 1
    table = g.permutation(2 * max_pages).reshape(2, max_pages).astype(np.int32)
    c = Planes(sv, dev, g, layers, 2 * max_pages, nkv, page, hd, table, [3, 0])
    rows = [random_rows(g, (layers, n, nt, nkv, hd)) for _ in range(2)]
    n_path = np.array([nt, 1500], np.int32)
    slots, st = c.T(np.array([1, 0], np.int32)), c.T(np.array([9, 9], np.int32))
    sv.spec_pages_q4_commit(c.kv, n, slots, nt, c.T(rows[0]), c.T(rows[1]), None, c.T(n_path), st)
    assert st.tolist() == [0, 0]
    out = [torch.full((layers, n, nt, nkv, hd), 3.0, dtype=torch.float16, device=dev) for _ in range(2)]
    sv.spec_pages_q4_read(c.kv, n, slots, nt, c.T(np.array([0, 3], np.int32)), c.T(n_path), out[0], out[1], st)
    assert st.tolist() == [0, 0]
    for w in range(2):
        want = lc.values(*lc.pack(*lc.quantise(rows[w]))).astype(np.float16)
        want[:, 1, 1500:] = 3.0
        assert np.array_equal(out[w].cpu().numpy(), want)


@pytest.mark.parametrize("hd,nkv,page", [(128, 8, 64), (64, 1, 5), (32, 3, 16)])
def test_copies_of_pages(dev, hd, nkv, page):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(page)
    c = Planes(sv, dev, g, 2, 9, nkv, page, hd, None, None)
    src, dst = np.array([0, 1, 1, 8, 3, 20], np.int32), np.array([4, 5, 6, 8, 5, 2], np.int32)
    n_pos = np.array([page, page // 2, 0, 1, 1, 1], np.int32)
    for counts in (n_pos, None):
        before = c.planes()
        st = torch.full((6,), 9, dtype=torch.int32, device=dev)
        sv.spec_pages_q4_copy(c.kv, 6, c.T(src), c.T(dst), st, n_pos=c.T(counts))
        assert st.tolist() == [0, tree.ST_SLOT, 0, tree.ST_SLOT, tree.ST_SLOT, tree.ST_SLOT]
        for i in (0, 2):
            m = page if counts is None else n_pos[i]
            for a in before:
                a[:, dst[i], :, :m] = a[:, src[i], :, :m]
        same_planes(c.planes(), before)


def test_branches(dev):
    """Fork, extension with copies of shared pages, release: as spec_pages_* do it."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(2)
    page, max_pages = 6, 4
    book = tree.Book(6, max_pages, 14, page)
    book.len[0], book.table[0][:3] = 15, [7, 2, 9]
    for p in (7, 2, 9):
        book.refs[p] = 1
    c = Planes(sv, dev, g, 2, 14, 2, page, 64, book.table, book.len, book.refs)
    want = [a.copy() for a in c.host]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    st, copies = i32([9] * 3), i32([[9, 9]] * 3)
    sv.spec_pages_q4_fork(c.kv, 2, i32([0, 0]), i32([3, 5]), st[:2])
    assert st.tolist()[:2] == book.fork([0, 0], [3, 5])
    sv.spec_pages_q4_extend(c.kv, 3, i32([5, 0, 3]), i32([4, 1, 9]), copies, st)
    status, cp = book.extend([5, 0, 3], [4, 1, 9])
    assert st.tolist() == status == [0, 0, 0]
    assert [tuple(x) for x in copies.tolist()] == [tuple(x) if x is not None else (-1, -1) for x in cp]
    for x in cp:
        if x is not None and x[0] >= 0:
            for a in want:
                a[:, x[1], :, :3] = a[:, x[0], :, :3]
    same_planes(c.planes(), want)
    table, lens, refs = c.book()
    assert table.tolist() == book.table and lens.tolist() == book.len and refs.tolist() == book.refs
    sv.spec_pages_q4_free(c.kv, 2, i32([0, 3]), st[:2])
    assert st.tolist()[:2] == [0, 0]
    table, lens, refs = c.book()
    assert (table[[0, 3]] == -1).all() and lens.tolist() == [0, 0, 0, 0, 0, 15] and refs.sum() == (table >= 0).sum()
