"""Selected blocks on the GPU: digests and selections bit by bit, scores and
attention against 64 bits (oracle/long_context.py, oracle/tree.py), in fp16 and in
4 bits, their edges and refusals, and a run of all of them together."""
import numpy as np
import pytest

from oracle import long_context as lc
from oracle import tree
from test_gpu_attn import attn_model
from test_gpu_q4 import Q4Case
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def make(sv, dev, g, q4, *args, **kw):
    return (Q4Case if q4 else Case)(sv, dev, g, *args, **kw)


class Blocks:
    """Digests, scores and lists of a test case's cache."""

    def __init__(self, c, block, ld=None):
        import torch
        self.c, self.block, self.per = c, block, c.page // block
        layers, n_pages = c.k.shape[:2]
        self.data = torch.full((layers, n_pages, c.nkv, self.per, 2, c.hd), 5.0, dtype=torch.float16, device=c.dev)
        self.kv = c.pool()
        self.dg = c.sv.KVDigest(self.data, block, self.kv._keep[-3], self.kv._keep[-2])
        self.nb = [-(-n // block) for n in c.lens]
        self.ld = ld or max(1, max(self.nb))
        self.scores = torch.full((c.n, c.nt, c.nkv, self.ld), 9.0, device=c.dev)
        self.status = torch.full((c.n,), 99, dtype=torch.int32, device=c.dev)

    def digests(self, pos0=None):
        c = self.c
        c.sv.spec_block_digest(self.dg, self.kv, c.n, c.T(c.slots), self.status,
                               pos0=None if pos0 is None else c.T(np.asarray(pos0, np.int32)))
        return self.data.cpu().numpy()

    def want_digests(self, before, pos0=None):
        c, out = self.c, before.copy()
        for layer in range(c.k.shape[0]):
            for b in range(c.n):
                first = 0 if pos0 is None else pos0[b] // self.block
                for j in range(first, self.nb[b]):
                    p0, p1 = j * self.block, min(c.lens[b], (j + 1) * self.block)
                    pg, at = c.table[c.slots[b], p0 // c.page], p0 % c.page
                    if not 0 <= pg < c.k.shape[1]:
                        continue
                    for h in range(c.nkv):
                        out[layer, pg, h, at // self.block] = lc.digest(c.k[layer, pg, h, at:at + p1 - p0])
        return out

    def score(self, counts=True, q=None, **kw):
        c = self.c
        c.sv.spec_block_scores(self.dg, c.layer, c.n, c.T(c.slots), c.nt, c.nq, c.T(c.q) if q is None else q, self.scores,
                               self.status, n_nodes=c.T(c.counts) if counts else None, **kw)
        return self.scores.cpu().numpy()

    def check_scores(self, got, data):
        """A sum of 2 hd products in fp32: one unit of 2^-23 of their magnitudes each."""
        c, G = self.c, self.c.nq // self.c.nkv
        for b in range(c.n):
            assert (got[b, c.counts[b]:] == 9.0).all() and (got[b, :, :, self.nb[b]:] == 9.0).all()
            for i in range(c.counts[b]):
                for h in range(c.nkv):
                    for j in range(self.nb[b]):
                        pg, at = c.table[c.slots[b], j // self.per], j % self.per
                        want, mag = lc.score(c.q[b, i, h * G:(h + 1) * G], data[c.layer, pg, h, at])
                        assert abs(got[b, i, h, j] - want) <= 2 * c.hd * 2.0 ** -23 * mag, (b, i, h, j)

    def lists(self, g, keep):
        """Lists in any order, with gaps."""
        c = self.c
        out = np.full((c.n, c.nt, c.nkv, keep), -1, np.int32)
        for b in range(c.n):
            for i in range(c.nt):
                for h in range(c.nkv):
                    ids = g.permutation(self.nb[b])[:g.integers(0, keep + 1)]
                    out[b, i, h, np.sort(g.permutation(keep)[:len(ids)])] = ids
        return out

    def attend(self, lists, chain=False, counts=True, **kw):
        import torch
        c = self.c
        c.out = torch.full((c.n, c.nt, c.nq, c.hd), 7.0, dtype=torch.float16, device=c.dev)
        self.st = torch.full((c.n, c.nt, c.nkv), 99, dtype=torch.int32, device=c.dev)
        args = dict(q=c.T(c.q), k_new=c.T(c.kn), v_new=c.T(c.vn))
        args.update(kw)
        c.sv.spec_block_attn(self.kv, c.layer, c.n, c.T(c.slots), c.nt, c.nq, self.block, lists.shape[-1], c.T(lists),
                             out=c.out, status=self.st, parents=None if chain else c.T(c.parents),
                             n_nodes=c.T(c.counts) if counts else None, scale=c.scale or 0.0, **args)
        torch.cuda.synchronize()
        return c.out.cpu().numpy()

    def check_attention(self, got, lists, rows=None):
        """Case.check's bound (Q4Case's scores error for codes)."""
        c, G = self.c, self.c.nq // self.c.nkv
        q4 = isinstance(c, Q4Case)
        for b in range(c.n):
            assert (got[b, c.counts[b]:] == np.float16(7.0)).all()
            if c.counts[b] == 0:
                continue
            paths = tree.chains(c.parents[b, :c.counts[b]].tolist())
            kk, vv = c.cached(0, b).astype(np.float64), c.cached(1, b).astype(np.float64)
            for i in range(c.counts[b]):
                for h in range(c.nkv):
                    if rows is not None and not rows(b, i, h):
                        continue
                    at = [p for j in lists[b, i, h] if j >= 0
                          for p in range(j * self.block, min(c.lens[b], (j + 1) * self.block))]
                    k = np.concatenate([kk[at, h], c.kn[b, paths[i], h].astype(np.float64)])
                    v = np.concatenate([vv[at, h], c.vn[b, paths[i], h].astype(np.float64)])
                    q = c.q[b, i, h * G:(h + 1) * G].astype(np.float64)
                    scale = c.scale or c.hd ** -0.5
                    s = q @ k.T * scale
                    p = np.exp(s - s.max(1, keepdims=True))
                    p /= p.sum(1, keepdims=True)
                    ref, mag = p @ v, p @ np.abs(v)
                    ds = (c.hd + 4) * 2.0 ** -23 * abs(scale) * (np.abs(q) @ np.abs(k).T).max(1)
                    if q4 and at:
                        sc = np.stack([np.abs(c.ks[c.layer, c.table[c.slots[b], x // c.page], h, x % c.page].astype(np.float64))
                                       for x in at])
                        ds = ds + 40 * 24 * 2.0 ** -23 * abs(scale) * (
                            np.abs(q).reshape(G, c.hd // 32, 32).sum(-1) @ sc.T).max(1)
                    rel = np.expm1(2 * ds) + 2.0 ** -20 + (len(at) / 8 + 128) * 2.0 ** -23 + (len(at) + 64) * 2.0 ** -36
                    bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[:, None] * mag
                    err = np.abs(got[b, i, h * G:(h + 1) * G].astype(np.float64) - ref)
                    assert (err <= bound).all(), (b, i, h, float(np.max(err - bound)))


SHAPES = [
    # nq, nkv, hd, lens, nt, page, block, counts, kind, keep
    (32, 8, 128, [700], 1, 64, 64, None, "chain", 5),
    (14, 2, 64, [1000, 17, 0, 16], 3, 16, 16, [3, 2, 3, 0], "tree", 20),
    (40, 8, 128, [500, 130], 4, 256, 32, None, "tree", 9),
    (8, 8, 64, [64, 63, 65], 2, 128, 128, None, "flat", 2),
    (6, 1, 128, [900], 64, 96, 16, None, "chain", 7),
    (16, 1, 64, [2500, 3], 2, 1024, 64, None, "tree", 40),
    (20, 1, 128, [300], 5, 32, 32, None, "forest", 3),
    (64, 1, 64, [200], 2, 48, 16, None, "tree", 13),
]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("nq,nkv,hd,lens,nt,page,block,counts,kind,keep", SHAPES)
def test_each_step(dev, q4, nq, nkv, hd, lens, nt, page, block, counts, kind, keep):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([nq, nt, block, q4])
    c = make(sv, dev, g, q4, nq, nkv, hd, lens, nt, page, counts=counts, kind=kind)
    x = Blocks(c, block)
    before = x.data.cpu().numpy()
    data = x.digests()
    assert x.status.tolist() == [0] * c.n
    assert np.array_equal(data, x.want_digests(before))
    got = x.score(counts=counts is not None)
    assert x.status.tolist() == [0] * c.n
    x.check_scores(got, data)
    for keep_, first, last in ((keep, 1, 1), (keep, 0, 0), (1, 0, 1)):
        blocks = torch.full((c.n, nt, nkv, keep_), 77, dtype=torch.int32, device=dev)
        sv.spec_block_select(c.T(c.slot_len), block, c.n, c.T(c.slots), nt, nkv, x.scores, keep_, blocks, x.status,
                             n_nodes=c.T(c.counts), n_first=first, n_last=last)
        assert x.status.tolist() == [0] * c.n
        for b in range(c.n):
            assert (blocks[b, c.counts[b]:] == 77).all()
            for i in range(c.counts[b]):
                for h in range(nkv):
                    want = lc.select(got[b, i, h], x.nb[b], keep_, first, last)
                    assert blocks[b, i, h].tolist() == want + [-1] * (keep_ - len(want))
    lists = x.lists(g, keep)
    out = x.attend(lists, chain=kind == "chain", counts=counts is not None)
    for b in range(c.n):
        assert (x.st[b, :c.counts[b]] == 0).all() and (x.st[b, c.counts[b]:] == 99).all()
    x.check_attention(out, lists)
    assert np.array_equal(x.attend(lists).view(np.uint16), out.view(np.uint16))  # the same bits


def test_digests_from_a_position_on(dev):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(1)
    for q4 in (False, True):
        c = make(sv, dev, g, q4, 4, 2, 64, [300, 90, 5, 64], 1, 64)
        c.table[c.slots[1], 0] = -1
        x = Blocks(c, 16)
        before = x.data.cpu().numpy()
        pos0 = [160, 0, 5, 70]
        assert np.array_equal(x.digests(pos0), x.want_digests(before, pos0))
        assert x.status.tolist() == [0, tree.ST_PAGE, 0, 0]
        c.slots[3] = 77
        x.digests([0, 64, -1, 0])
        assert x.status.tolist() == [0, 0, tree.ST_FULL, tree.ST_SLOT]


def test_digests_and_scores_of_what_is_not_finite(dev):
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(2)
    c = Case(sv, dev, g, 4, 2, 64, [128], 2, 32)
    pg = c.table[c.slots[0]]
    c.k[c.layer, pg[0], 0, 3, 5] = np.nan
    c.k[c.layer, pg[1], 0, 4, 6] = np.inf
    c.k[c.layer, pg[2], 1, 0] = 0
    x = Blocks(c, 32)
    before = x.data.cpu().numpy()
    data = x.digests()
    want = x.want_digests(before)
    assert np.array_equal(np.isnan(data), np.isnan(want)) and np.array_equal(data[~np.isnan(want)], want[~np.isnan(want)])
    got = x.score()
    assert np.isnan(got[0, :, 0, 0]).all() and not np.isfinite(got[0, :, 0, 1]).any()
    assert np.isfinite(got[0, :, 1]).all() and np.isfinite(got[0, :, 0, 2:]).all()


def test_scores_of_strided_queries_and_refusals(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(3)
    c = Case(sv, dev, g, 8, 2, 64, [100, 90, 80, 70, 60], 5, 16, counts=[5, 4, 5, 6, 5])
    row = 8 * 64 + 40
    buf = torch.full((c.n * 5, row), float("nan"), dtype=torch.float16, device=dev)
    buf[:, :512] = c.T(c.q).view(-1, 512)
    x = Blocks(c, 16, ld=9)
    data = x.digests()
    c.slots[1], c.slot_len[c.slots[4]], c.table[c.slots[2], 1] = -1, 150, -1
    y = Blocks(c, 16, ld=9)
    y.data.copy_(x.data)
    got = y.score(q=buf, q_stride=row)
    assert y.status.tolist() == [0, tree.ST_SLOT, tree.ST_PAGE, tree.ST_TREE, tree.ST_FULL]
    assert (got[[1, 3, 4]] == 9.0).all()
    assert np.isneginf(got[2, :, :, 1]).all() and np.isfinite(got[2, :, :, :1]).all() and np.isfinite(got[2, :, :, 2:5]).all()
    c.counts[1:], x.nb[1:] = 0, [0] * 4
    want = got.copy()
    want[1:] = 9.0
    x.check_scores(want, data)


@pytest.mark.parametrize("nb,keep", [(7, 3), (128, 64), (1024, 100), (1025, 2), (4097, 256), (20000, 4096), (40000, 333)])
def test_selections(dev, nb, keep):
    """Equal scores, infinities, NaN, both zeros, rows that are all alike; rows past
    what the registers hold."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(nb)
    n, nt, nkv = 2, 3, 2
    x = g.standard_normal((n, nt, nkv, nb + 3)).astype(np.float32)
    x[0, 0, 0] = np.round(x[0, 0, 0])           # many equal ones
    x[0, 0, 1] = 0
    x[0, 0, 1, ::3] = -0.0
    x[0, 1, 0] = -np.inf
    x[0, 1, 1, ::2] = np.nan
    x[0, 2, 0, 1::7] = np.inf
    x[0, 2, 1] = np.where(g.random(nb + 3) < 0.01, 1.0, -2.5)
    x[1, 0, 0] = np.float32(1.0) + np.arange(nb + 3)[::-1] * np.float32(2.0 ** -23)
    lens = np.array([4, nb * 16, nb * 16 - 15], np.int32)
    slots = np.array([1, 2], np.int32)
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    st = torch.full((n,), 9, dtype=torch.int32, device=dev)
    for first, last in ((1, 1), (0, 0), (min(2, keep), 0), (0, min(keep, 5))):
        out = torch.full((n, nt, nkv, keep), 77, dtype=torch.int32, device=dev)
        sv.spec_block_select(T(lens), 16, n, T(slots), nt, nkv, T(x), keep, out, st, n_first=first, n_last=last)
        assert st.tolist() == [0, 0]
        got = out.cpu().numpy()
        for b in range(n):
            for i in range(nt):
                for h in range(nkv):
                    assert got[b, i, h].tolist() == lc.select(x[b, i, h] + np.float32(0), nb, keep, first, last), (b, i, h)


@pytest.mark.parametrize("n,nt,nkv,nb,keep", [(1, 2, 3, 700, 30), (2, 2, 2, 3000, 64), (4, 9, 6, 77, 5), (5, 8, 8, 500, 64),
                                             (4, 16, 5, 1000, 9), (3, 64, 2, 2040, 200), (6, 12, 4, 4090, 33)])
def test_selections_of_few_and_many_rows(dev, n, nt, nkv, nb, keep):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([nb, n])
    x = np.round(20 + 3 * g.standard_normal((n, nt, nkv, nb)) ** 3, 2).astype(np.float32)
    lens = g.integers(0, nb * 32 + 1, n).astype(np.int32)
    lens[0] = nb * 32
    counts = g.integers(0, nt + 1, n).astype(np.int32)
    counts[0] = nt
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    st = torch.full((n,), 9, dtype=torch.int32, device=dev)
    out = torch.full((n, nt, nkv, keep), 77, dtype=torch.int32, device=dev)
    sv.spec_block_select(T(lens), 32, n, T(np.arange(n, dtype=np.int32)), nt, nkv, T(x), keep, out, st, n_nodes=T(counts))
    assert st.tolist() == [0] * n
    got = out.cpu().numpy()
    for b in range(n):
        assert (got[b, counts[b]:] == 77).all()
        blocks = -(-int(lens[b]) // 32)
        for i in range(counts[b]):
            for h in range(nkv):
                want = lc.select(x[b, i, h], blocks, keep, 1, 1)
                assert got[b, i, h].tolist() == want + [-1] * (keep - len(want)), (b, i, h)


def test_selection_refusals(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    T = lambda a, d=np.int32: torch.from_numpy(np.ascontiguousarray(np.asarray(a, d))).to(dev)  # noqa: E731
    x = T(np.arange(5 * 2 * 10).reshape(5, 2, 1, 10), np.float32)
    out, st = torch.full((5, 2, 1, 3), 77, dtype=torch.int32, device=dev), T([9] * 5)
    sv.spec_block_select(T([100, 161, -1, 33]), 16, 5, T([0, 4, 1, 2, 3]), 2, 1, x, 3, out, st, n_nodes=T([1, 2, 2, 2, 3]))
    assert st.tolist() == [0, tree.ST_SLOT, tree.ST_FULL, tree.ST_FULL, tree.ST_TREE]
    assert out[0].tolist() == [[[0, 5, 6]], [[77, 77, 77]]] and (out[1:] == -1).all()


def test_attention_refusals(dev):
    """Each row in error is NaN with its status, the others are served."""
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng(7)
        c = make(sv, dev, g, q4, 8, 2, 64, [100, 90, 80, 70, 60, 50, 40], 4, 16, counts=[4, 4, 4, 4, 4, 5, 3])
        x = Blocks(c, 16)
        lists = x.lists(g, 4)
        lists[0, 1, 0, 2], lists[0, 2, 1, 0] = 7, -2  # 100 positions: blocks 0-6
        lists[1], lists[6, 0, 1, 3] = [0, 1, 5, -1], 2
        c.table[c.slots[1], 1] = -1
        c.slots[2] = 99
        c.slot_len[c.slots[3]] = -4
        c.parents[4, 3] = 3
        c.table[c.slots[6], 2] = 10 ** 6
        x = Blocks(c, 16)
        out = x.attend(lists)
        st = x.st.cpu().numpy()
        want = np.zeros((7, 4, 2), np.int32)
        want[0, 1, 0] = want[0, 2, 1] = 64
        want[1] = tree.ST_PAGE
        want[2], want[3], want[4], want[5] = tree.ST_SLOT, tree.ST_PAGE, tree.ST_TREE, tree.ST_TREE
        for i in range(3):
            for h in range(2):
                if 2 in lists[6, i, h]:
                    want[6, i, h] = tree.ST_PAGE
        want[6, 3] = 99
        assert np.array_equal(st, want)
        for b in range(7):
            for i in range(4):
                for h in range(2):
                    rows = out[b, i, 4 * h:4 * h + 4]
                    if want[b, i, h] not in (0, 99):
                        assert np.isnan(rows).all(), (b, i, h)
                    elif want[b, i, h] == 99:
                        assert (rows == 7.0).all()
                    else:
                        assert np.isfinite(rows).all()
        c.counts[1:] = 0
        clean = out.copy()
        clean[1:] = 7.0
        x.check_attention(clean, lists, rows=lambda b, i, h: want[b, i, h] == 0)


def test_what_is_not_selected_may_be_anything(dev):
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng(8)
        c = make(sv, dev, g, q4, 8, 2, 128, [300, 90], 5, 64)
        x = Blocks(c, 32)
        lists = np.full((2, 5, 2, 4), -1, np.int32)
        lists[0], lists[1] = [1, 4, 9, -1], [0, 2, -1, -1]
        clean = x.attend(lists)
        x.check_attention(clean, lists)
        seen = {(int(c.table[c.slots[b], p // 64]), p % 64) for b in range(2) for j in lists[b, 0, 0] if j >= 0
                for p in range(32 * j, min(c.lens[b], 32 * j + 32))}
        for pg in range(c.k.shape[1]):
            for at in range(64):
                if (pg, at) not in seen:
                    if q4:
                        c.ks[:, pg, :, at], c.vs[:, pg, :, at] = np.nan, np.inf
                    else:
                        c.k[:, pg, :, at], c.v[:, pg, :, at] = np.nan, np.inf
        c.parents[:] = [-1, 0, 0, 0, 0]
        x = Blocks(c, 32)
        ref = x.attend(lists)
        c.kn[:, 4], c.vn[:, 4] = np.nan, np.inf
        c.counts[1] = 4
        got = x.attend(lists)
        assert np.isfinite(ref).all() and np.array_equal(got[:, :4].view(np.uint16), ref[:, :4].view(np.uint16))
        assert np.isnan(got[0, 4]).all() and (got[1, 4] == 7.0).all()


@pytest.mark.parametrize("hd,nq,scale", [(64, 8, -0.25), (128, 24, 0.3), (128, 8, None)])
def test_strides_scales_and_a_block_named_twice(dev, hd, nq, scale):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng([hd, nq, q4])
        c = make(sv, dev, g, q4, nq, 2, hd, [310, 64], 5, 32, scale=scale, counts=[5, 4])
        x = Blocks(c, 16)
        lists = x.lists(g, 7)
        lists[0, 2, 0, :5] = [3, 19, 3, 3, 0]  # (19: six positions)
        want = x.attend(lists)
        assert (x.st[0] == 0).all() and (x.st[1, :4] == 0).all()
        x.check_attention(want, lists)

        def apart(a, row):
            buf = torch.full((c.n * c.nt, row), float("nan"), dtype=torch.float16, device=dev)
            buf[:, :a[0, 0].size] = c.T(a).view(c.n * c.nt, -1)
            return buf
        qs, ks = nq * hd + 8, 2 * hd + 40
        got = x.attend(lists, q=apart(c.q, qs), k_new=apart(c.kn, ks), v_new=apart(c.vn, ks), q_stride=qs, kv_stride=ks)
        assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
        q = c.q.copy()
        q[0, 1, 2, 3] = np.nan
        got = x.attend(lists, q=c.T(q))
        odd = np.zeros(got.shape[:3], bool)
        odd[0, 1, 2] = True
        assert np.isnan(got[odd]).all() and np.array_equal(got[~odd].view(np.uint16), want[~odd].view(np.uint16))


@pytest.mark.parametrize("hd,nq,nt", [(128, 20, 64), (128, 8, 17), (64, 8, 1)])
def test_the_longest_lists(dev, hd, nq, nt):
    """4096 places, most of them empty, the blocks anywhere."""
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng([hd, nt])
        c = make(sv, dev, g, q4, nq, 1, hd, [700], nt, 32, layers=1)
        x = Blocks(c, 16)
        lists = np.full((1, nt, 1, 4096), -1, np.int32)
        for i in range(nt):
            ids = g.permutation(44)[:i % 7 + 1]
            lists[0, i, 0, g.permutation(4096)[:len(ids)]] = ids
        lists[0, 0, 0, [0, 4095]] = [0, 43]
        got = x.attend(lists, chain=False)
        assert (x.st == 0).all()
        x.check_attention(got, lists)


def test_digests_of_copied_pages(dev):
    """A branch whose shared last page is copied when it grows: digests of the copy
    from the page's start on, the other branch's as they were."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(13)
    layers, nkv, page, block, hd, n_pages = 2, 2, 32, 16, 64, 9
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    shape = (layers, n_pages, nkv, page, hd // 32)
    planes = [torch.zeros(shape + (16,), dtype=torch.uint8, device=dev) for _ in range(2)] + [
        torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(2)]
    table, lens, refs = i32([[-1] * 4] * 2), i32([0, 0]), i32([0] * n_pages)
    kv = sv.KVPagesQ4(*planes, table, lens, refs)
    data = torch.full((layers, n_pages, nkv, page // block, 2, hd), 5.0, dtype=torch.float16, device=dev)
    dg = sv.KVDigest(data, block, table, lens)
    st, copies = i32([9]), i32([[9, 9]])

    def grow(slot, rows, pos0):
        k = torch.from_numpy(g.standard_normal((layers, 1, rows, nkv, hd)).astype(np.float16)).to(dev)
        sv.spec_pages_q4_extend(kv, 1, i32([slot]), i32([rows]), copies, st)
        assert st.tolist() == [0]
        sv.spec_pages_q4_commit(kv, 1, i32([slot]), rows, k, k.flip(2), None, i32([rows]), st)
        assert st.tolist() == [0]
        sv.spec_block_digest(dg, kv, 1, i32([slot]), st, pos0=i32([pos0]))
        assert st.tolist() == [0]

    def check(slot):
        n = lens[slot].item()
        rows = [torch.zeros((layers, 1, n, nkv, hd), dtype=torch.float16, device=dev) for _ in range(2)]
        sv.spec_pages_q4_read(kv, 1, i32([slot]), n, i32([0]), i32([n]), rows[0], rows[1], st)
        assert st.tolist() == [0]
        k, d, t = rows[0][:, 0].cpu().numpy(), data.cpu().numpy(), table[slot].tolist()
        for layer in range(layers):
            for h in range(nkv):
                for j in range(-(-n // block)):
                    got = d[layer, t[j * block // page], h, j * block % page // block]
                    assert np.array_equal(got, lc.digest(k[layer, j * block:(j + 1) * block, h])), (slot, layer, h, j)

    grow(0, 70, 0)
    check(0)
    sv.spec_pages_q4_fork(kv, 1, i32([0]), i32([1]), st)
    assert st.tolist() == [0]
    check(1)
    grow(1, 20, 64)  # 70 positions: the copied page begins with 64
    assert copies[0, 0].item() == table[0, 2].item() and copies[0, 1].item() == table[1, 2].item()
    check(0), check(1)
    grow(0, 30, 64)
    check(0), check(1)


def test_the_models_own_cache(dev):
    """A model's slots as pages: digests beside them, a selection, attention over lists of
    all blocks as tree attention."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(18)
    nq, nkv, hd, nt, max_ctx, block, n = 8, 2, 128, 7, 224, 32, 150
    m = attn_model(sv, dev, g, nq, nkv, hd, max_ctx, nt, 3)
    kv = sv.spec_model_pages(m)
    f16 = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float16)).to(dev)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    kc, vc = f16(nkv, n, hd), f16(nkv, n, hd)
    sv.spec_kv_fill(m, 0, 1, 0, n, kc, vc)
    sv.spec_state_set(m, [1], n_past=[n], anchor=[3])
    layers = kv.pages.n_layers
    data = torch.zeros((layers, 3, nkv, max_ctx // block, 2, hd), dtype=torch.float16, device=dev)
    lens, slots, st = i32([0, n, 0]), i32([1]), i32([9])
    dg = sv.KVDigest(data, block, i32([[0], [1], [2]]), lens)
    sv.spec_block_digest(dg, kv, 1, slots, st)
    assert st.item() == 0
    k = kc.cpu().numpy()
    for h in range(nkv):
        for j in range(5):
            assert np.array_equal(data[0, 1, h, j].cpu().numpy(), lc.digest(k[h, block * j:block * (j + 1)]))
    q, kn, vn = f16(1, nt, nq, hd), f16(1, nt, nkv, hd), f16(1, nt, nkv, hd)
    scores = torch.zeros((1, nt, nkv, max_ctx // block), device=dev)
    blocks, row_st = i32(np.zeros((1, nt, nkv, 5)).tolist()), i32(np.zeros((1, nt, nkv)).tolist())
    sv.spec_block_scores(dg, 0, 1, slots, nt, nq, q, scores, st)
    sv.spec_block_select(lens, block, 1, slots, nt, nkv, scores, 5, blocks, st)
    assert st.item() == 0 and (blocks == i32([0, 1, 2, 3, 4])).all()
    outs = [torch.zeros((1, nt, nq, hd), dtype=torch.float16, device=dev) for _ in range(2)]
    sv.spec_block_attn(kv, 0, 1, slots, nt, nq, block, 5, blocks, q, kn, vn, outs[0], row_st)
    ws = torch.empty(sv.spec_tree_attn_workspace(kv, 1, nt, nq), dtype=torch.uint8, device=dev)
    sv.spec_tree_attn(kv, 0, 1, slots, nt, nq, q, kn, vn, outs[1], ws, st)
    assert st.item() == 0 and (row_st == 0).all()
    # each within half an fp16 step (and the far smaller fp32 error) of the same value
    err = (outs[0].double() - outs[1].double()).abs()
    assert (err <= 2.0 ** -10 * outs[1].double().abs() + 2.0 ** -16).all()


def test_captured_rounds(dev):
    """Rounds whose lengths grow on the device, captured once: commit in place, digests
    of what is new, scores, selection, both attentions; replayed, they are the eager ones."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    nq, nkv, hd, page, block, nt, n, keep, max_pages, layers = 8, 2, 128, 64, 32, 5, 2, 4, 6, 2
    g = np.random.default_rng(17)
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    f16 = lambda *s: T(g.standard_normal(s).astype(np.float16))  # noqa: E731
    prompt, kn, vn, q = f16(layers, n, 200, nkv, hd), f16(layers, n, nt, nkv, hd), f16(layers, n, nt, nkv, hd), f16(n, nt, nq, hd)
    pages = g.permutation(n * max_pages).reshape(n, max_pages).astype(np.int32)

    class Run:
        def __init__(self):
            shape = (layers, n * max_pages, nkv, page, hd // 32)
            planes = [torch.zeros(shape + (16,), dtype=torch.uint8, device=dev) for _ in range(2)] + [
                torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(2)]
            self.lens, self.st = T(np.zeros(n, np.int32)), T(np.full(n, 9, np.int32))
            self.kv = sv.KVPagesQ4(*planes, T(pages), self.lens)
            self.dg = sv.KVDigest(torch.zeros((layers, n * max_pages, nkv, page // block, 2, hd), dtype=torch.float16, device=dev), block,
                                  self.kv._keep[4], self.lens)
            self.slots, self.n_path, self.path = T(np.array([1, 0], np.int32)), T(np.array([3, 2], np.int32)), T(
                np.array([[0, 2, 4, 0, 0], [0, 1, 0, 0, 0]], np.int32))
            self.pos0 = torch.zeros(n, dtype=torch.int32, device=dev)
            self.scores = torch.zeros((n, nt, nkv, max_pages * 2), device=dev)
            self.blocks = torch.zeros((n, nt, nkv, keep), dtype=torch.int32, device=dev)
            self.outs = [torch.zeros((n, nt, nq, hd), dtype=torch.float16, device=dev) for _ in range(2)]
            self.row_st = torch.zeros((n, nt, nkv), dtype=torch.int32, device=dev)
            self.ws = torch.empty(sv.spec_tree_attn_q4_workspace(self.kv, n, nt, nq), dtype=torch.uint8, device=dev)
            self.bad = torch.zeros((), dtype=torch.int32, device=dev)
            sv.spec_pages_q4_commit(self.kv, n, self.slots, 200, prompt, prompt, None, T(np.array([200, 61], np.int32)), self.st)
            sv.spec_block_digest(self.dg, self.kv, n, self.slots, self.st)

        def round(self):
            a = (n, self.slots, nt)
            self.pos0.copy_(self.lens.index_select(0, self.slots))
            sv.spec_pages_q4_commit(self.kv, n, self.slots, nt, kn, vn, self.path, self.n_path, self.st)
            self.bad |= self.st.max()
            sv.spec_block_digest(self.dg, self.kv, n, self.slots, self.st, pos0=self.pos0)
            self.bad |= self.st.max()
            sv.spec_block_scores(self.dg, 1, *a, nq, q, self.scores, self.st)
            self.bad |= self.st.max()
            sv.spec_block_select(self.lens, block, *a, nkv, self.scores, keep, self.blocks, self.st)
            self.bad |= self.st.max()
            sv.spec_block_attn(self.kv, 1, *a, nq, block, keep, self.blocks, q, kn[1], vn[1], self.outs[0], self.row_st)
            self.bad |= self.row_st.max()
            sv.spec_tree_attn_q4(self.kv, 1, *a, nq, q, kn[1], vn[1], self.outs[1], self.ws, self.st)
            self.bad |= self.st.max()

    eager, replayed, first = Run(), Run(), Run()
    first.round()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        replayed.round()
    assert replayed.lens.tolist() == [61, 200]  # (captured, not run)
    for step in range(1, 5):
        eager.round()
        graph.replay()
        assert eager.lens.tolist() == replayed.lens.tolist() == [61 + 2 * step, 200 + 3 * step]
        assert eager.bad.item() == replayed.bad.item() == 0
        for a, b in zip(eager.outs + [eager.scores, eager.blocks], replayed.outs + [replayed.scores, replayed.blocks]):
            assert torch.equal(a, b) and (a.dtype != torch.float16 or torch.isfinite(a).all())


def test_all_blocks_are_the_whole_context(dev):
    """Lists that name every block: the attention of spec_tree_attn."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(9)
    for q4 in (False, True):
        c = make(sv, dev, g, q4, 8, 2, 64, [333, 64, 0], 6, 32)
        x = Blocks(c, 16)
        lists = np.full((3, 6, 2, 21), -1, np.int32)
        for b in range(3):
            lists[b, :, :, :x.nb[b]] = np.arange(x.nb[b])
        a = x.attend(lists)
        c.check(a)
        c.check(c.call())


@pytest.mark.parametrize("n,nt,nq,nkv,keep", [(1, 1, 8, 1, 40), (1, 1, 32, 8, 290), (3, 2, 32, 8, 33), (9, 7, 16, 8, 11)])
def test_any_number_of_ctas_a_row(dev, n, nt, nq, nkv, keep):
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng([n, keep])
        c = make(sv, dev, g, q4, nq, nkv, 64, [4800 - 7 * b for b in range(n)], nt, 48, layers=1)
        x = Blocks(c, 16)
        lists = np.sort(np.stack([g.permutation(295)[:keep] for _ in range(n * nt * nkv)]), 1).reshape(n, nt, nkv, keep)
        lists = lists.astype(np.int32)
        got = x.attend(lists)
        x.check_attention(got, lists, rows=lambda b, i, h: (b + i + h) % 3 == 0)
        for _ in range(10):
            assert np.array_equal(x.attend(lists).view(np.uint16), got.view(np.uint16))


def test_offsets_past_32_bits(dev):
    """Pools of more than 2^31 elements: the pages at their end."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(10)
    nkv, hd, page, n_pages = 8, 128, 256, 8400
    for q4 in (False, True):
        c = make(sv, dev, g, q4, 8, nkv, hd, [600], 4, page, layers=1)
        small = c.pool()._keep
        big = [torch.empty((1, n_pages, *t.shape[2:]), dtype=t.dtype, device=dev) for t in small[:4 if q4 else 2]]
        table = c.table.copy()
        for j in range(3):
            table[c.slots[0], j] = n_pages - 1 - j
            for a, t in zip(big, small):
                a[0, n_pages - 1 - j] = t[c.layer, c.table[c.slots[0], j]]
        x = Blocks(c, 64)
        lists = np.tile(np.array([0, 3, 9, -1], np.int32), (1, 4, nkv, 1))
        want = x.attend(lists)
        x.kv = (sv.KVPagesQ4 if q4 else sv.KVPages)(*big, c.T(table), c.T(c.slot_len))
        assert np.array_equal(x.attend(lists).view(np.uint16), want.view(np.uint16))
        data = torch.zeros((1, n_pages, nkv, 4, 2, hd), dtype=torch.float16, device=dev)
        dg = sv.KVDigest(data, 64, c.T(table), c.T(c.slot_len))
        sv.spec_block_digest(dg, x.kv, 1, c.T(c.slots), x.status)
        assert x.status.tolist() == [0]
        if q4:
            assert np.array_equal(c.call(x.kv).view(np.uint16), c.call().view(np.uint16))
            n_path = torch.tensor([2], dtype=torch.int32, device=dev)
            sv.spec_pages_q4_commit(x.kv, 1, c.T(c.slots), 4, c.T(c.kn[None]), c.T(c.vn[None]), None, n_path, x.status)
            assert x.status.tolist() == [0]
            codes, scales = lc.pack(*lc.quantise(c.kn[0, :2]))
            assert np.array_equal(big[0][0, n_pages - 3, :, 600 - 512:602 - 512].cpu().numpy(), codes.swapaxes(0, 1))


def test_graph_replay_and_two_streams(dev):
    """All steps captured once and replayed over other rows; two at once."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    for q4 in (False, True):
        g = np.random.default_rng(11)
        cs = [make(sv, dev, g, q4, 8, 2, 128, [700, 300], 3, 32) for _ in range(2)]
        sides = []
        for c in cs:
            x = Blocks(c, 32)
            blocks = torch.zeros((2, 3, 2, 6), dtype=torch.int32, device=dev)
            out = torch.zeros((2, 3, 8, 128), dtype=torch.float16, device=dev)
            sides.append(dict(c=c, x=x, blocks=blocks, out=out, st=torch.zeros((2, 3, 2), dtype=torch.int32, device=dev),
                              slots=c.T(c.slots), q=c.T(c.q), kn=c.T(c.kn), vn=c.T(c.vn), par=c.T(c.parents),
                              lens=c.T(c.slot_len), stream=torch.cuda.Stream()))

        def steps(s, stream=None):
            x, c = s["x"], s["c"]
            sv.spec_block_digest(x.dg, x.kv, 2, s["slots"], x.status, stream=stream)
            sv.spec_block_scores(x.dg, c.layer, 2, s["slots"], 3, 8, s["q"], x.scores, x.status, stream=stream)
            sv.spec_block_select(s["lens"], 32, 2, s["slots"], 3, 2, x.scores, 6, s["blocks"], x.status, stream=stream)
            sv.spec_block_attn(x.kv, c.layer, 2, s["slots"], 3, 8, 32, 6, s["blocks"], s["q"], s["kn"], s["vn"], s["out"],
                               s["st"], parents=s["par"], stream=stream)

        for s in sides:
            steps(s)
        torch.cuda.synchronize()
        want = [s["out"].clone() for s in sides]
        for s in sides:
            s["x"].check_attention(s["out"].cpu().numpy(), s["blocks"].cpu().numpy())
            s["q2"] = s["q"].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps(sides[0])
        sides[0]["q"].copy_(sides[0]["q2"].flip(0))
        graph.replay()
        other = sides[0]["out"].clone()
        sides[0]["q"].copy_(sides[0]["q2"])
        graph.replay()
        assert torch.equal(sides[0]["out"], want[0]) and not torch.equal(other, want[0])
        torch.cuda.synchronize()
        for _ in range(20):
            for s in sides:
                steps(s, stream=s["stream"])
        torch.cuda.synchronize()
        for s, w in zip(sides, want):
            assert torch.equal(s["out"], w)


def test_a_decoding_loop_over_a_cache_in_4_bits(dev):
    """Prompts committed, then rounds of trees: digests of what is new, scores,
    selection, attention over the lists, the accepted path committed."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(12)
    nq, nkv, hd, page, block, nt, n, keep, layers = 8, 2, 64, 32, 16, 5, 3, 6, 2
    max_pages = 12
    book = tree.Book(n, max_pages, n * max_pages, page)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    T = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    shape = (layers, n * max_pages, nkv, page, hd // 32)
    planes = [torch.zeros(shape + (16,), dtype=torch.uint8, device=dev) for _ in range(2)] + [
        torch.zeros(shape, dtype=torch.float16, device=dev) for _ in range(2)]
    table, lens, refs = i32(book.table), i32(book.len), i32(book.refs)
    kv = sv.KVPagesQ4(*planes, table, lens, refs)
    data = torch.zeros((layers, n * max_pages, nkv, page // block, 2, hd), dtype=torch.float16, device=dev)
    dg = sv.KVDigest(data, block, table, lens)
    slots, st, copies = i32([2, 0, 1]), i32([9] * n), i32([[0, 0]] * n)
    held = [np.zeros((layers, 0, nkv, hd)) for _ in range(2 * n)]  # what the cache stands for, k and v of every entry

    def commit(kn, vn, path, n_path):
        rows = kn.shape[2]
        sv.spec_pages_q4_extend(kv, n, slots, T(n_path), copies, st)
        assert st.tolist() == [0] * n
        p0 = lens[slots.long()].clone()
        sv.spec_pages_q4_commit(kv, n, slots, rows, T(kn), T(vn), None if path is None else T(path), T(n_path), st)
        assert st.tolist() == [0] * n
        sv.spec_block_digest(dg, kv, n, slots, st, pos0=p0)
        assert st.tolist() == [0] * n
        for b in range(n):
            ids = np.arange(n_path[b]) if path is None else path[b, :n_path[b]]
            for w, x in enumerate((kn, vn)):
                held[2 * b + w] = np.concatenate([held[2 * b + w], lc.values(*lc.pack(*lc.quantise(x[:, b, ids])))], 1)

    prompt = np.array([150, 97, 16], np.int32)
    f16 = lambda *s: g.standard_normal(s).astype(np.float16)  # noqa: E731
    commit(f16(layers, n, 150, nkv, hd), f16(layers, n, 150, nkv, hd), None, prompt)
    for step in range(4):
        kn, vn, q = f16(layers, n, nt, nkv, hd), f16(layers, n, nt, nkv, hd), f16(layers, n, nt, nq, hd)
        par = np.array([[-1, 0, 0, 1, 3]] * n, np.int32)
        nb = [-(-held[2 * b].shape[1] // block) for b in range(n)]
        for layer in range(layers):
            scores = torch.zeros((n, nt, nkv, max_pages * 2), device=dev)
            blocks = torch.zeros((n, nt, nkv, keep), dtype=torch.int32, device=dev)
            out, row_st = torch.zeros((n, nt, nq, hd), dtype=torch.float16, device=dev), i32(np.full((n, nt, nkv), 9).tolist())
            sv.spec_block_scores(dg, layer, n, slots, nt, nq, T(q[layer]), scores, st)
            sv.spec_block_select(lens, block, n, slots, nt, nkv, scores, keep, blocks, st)
            sv.spec_block_attn(kv, layer, n, slots, nt, nq, block, keep, blocks, T(q[layer]), T(kn[layer]), T(vn[layer]), out,
                               row_st, parents=T(par))
            assert st.tolist() == [0] * n and (row_st == 0).all()
            got, lists, sc = out.cpu().numpy().astype(np.float64), blocks.cpu().numpy(), scores.cpu().numpy()
            for b in range(n):
                k, v = held[2 * b][layer], held[2 * b + 1][layer]
                for i, path in enumerate(tree.chains(par[b].tolist())):
                    for h in range(nkv):
                        qq = q[layer, b, i, 4 * h:4 * h + 4].astype(np.float64)
                        for j in range(nb[b]):
                            want, mag = lc.score(qq, lc.digest(k[block * j:block * (j + 1), h]))
                            assert abs(sc[b, i, h, j] - want) <= 2 * hd * 2.0 ** -23 * mag
                        ids = lc.select(sc[b, i, h], nb[b], keep, 1, 1)
                        assert lists[b, i, h].tolist() == ids + [-1] * (keep - len(ids))
                        at = [p for j in ids for p in range(block * j, min(len(k), block * (j + 1)))]
                        kk = np.concatenate([k[at, h], kn[layer, b, path, h]])
                        vv = np.concatenate([v[at, h], vn[layer, b, path, h]])
                        s = qq @ kk.T / 8.0
                        p = np.exp(s - s.max(1, keepdims=True))
                        p /= p.sum(1, keepdims=True)
                        # half a step of the result, and fp32's and the weights' part (Blocks.check_attention
                        # derives it) below 2^-10 of the values' average here: |scores' error| <= 40 x 24 x 2^-23 x
                        # sum |q_b| |s_b| / 8, sums below 64 x 3.5 x 0.6
                        ref, mag = p @ vv, p @ np.abs(vv)
                        assert (np.abs(got[b, i, 4 * h:4 * h + 4] - ref) <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (
                            np.expm1(2 * 960 * 2.0 ** -23 * 64 * 3.5 * 0.6 / 8) + 2.0 ** -16) * mag).all()
        commit(kn, vn, np.array([[0, 1, 3, 4, 0], [0, 2, 0, 0, 0], [0, 1, 3, 0, 0]], np.int32),
               np.array([4, 2, 3], np.int32))
    # the cache read back is what it stands for
    total = [x.shape[1] for x in held[::2]]
    most = max(total)
    back = [torch.zeros((layers, n, most, nkv, hd), dtype=torch.float16, device=dev) for _ in range(2)]
    sv.spec_pages_q4_read(kv, n, slots, most, i32([0] * n), i32(total), back[0], back[1], st)
    assert st.tolist() == [0] * n
    for b in range(n):
        for w in range(2):
            assert np.array_equal(back[w][:, b, :total[b]].cpu().numpy().astype(np.float64), held[2 * b + w])
