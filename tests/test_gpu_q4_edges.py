"""Attention over a cache in 4 bits where its kernels differ: every form of them
(clusters of CTAs a unit, the cut over all CTAs, tcgen05), named by the launches of
a captured call, on inputs in which a position too few or too many shows."""
import re

import numpy as np
import pytest

from captured import launches
from oracle import long_context as lc
from oracle import tree
from test_gpu_q4 import Planes, Q4Case, random_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def kernel_of(c):
    """The attention kernel of a case's call: its name and the numbers of its template."""
    import torch
    sv, kv = c.sv, c.pool()
    slots, q, kn, vn, parents, counts = (c.T(a) for a in (c.slots, c.q, c.kn, c.vn, c.parents, c.counts))
    out = torch.zeros((c.n, c.nt, c.nq, c.hd), dtype=torch.float16, device=c.dev)
    ws = torch.empty(sv.spec_tree_attn_q4_workspace(kv, c.n, c.nt, c.nq), dtype=torch.uint8, device=c.dev)
    st = torch.zeros(c.n, dtype=torch.int32, device=c.dev)
    name = launches(lambda: sv.spec_tree_attn_q4(kv, c.layer, c.n, slots, c.nt, c.nq, q, kn, vn, out, ws, st, parents=parents,
                                                 n_nodes=counts, window=c.window, sinks=c.sinks, scale=c.scale or 0.0))[0][0]
    for kernel in ("q4_unit_kernel", "q4_attn_kernel", "tree_attn_tc_kernel"):
        if kernel in name:
            return (kernel, *(int(x) for x in re.search(kernel + r"ILi(\d+)ELi(\d+)E", name).groups()))
    raise AssertionError(name)


# kernel, hd, tiles of 8 rows (tcgen05: rows), query heads over 2, nodes
UNIT = [("q4_unit_kernel", 64, 1, 2, 1), ("q4_unit_kernel", 64, 1, 4, 4), ("q4_unit_kernel", 64, 2, 8, 4),
        ("q4_unit_kernel", 64, 4, 8, 7), ("q4_unit_kernel", 128, 1, 8, 2), ("q4_unit_kernel", 128, 2, 8, 4),
        ("q4_unit_kernel", 128, 4, 8, 8)]
CUT = [("q4_attn_kernel", 64, 1, 14, 1), ("q4_attn_kernel", 64, 2, 8, 4), ("q4_attn_kernel", 64, 4, 8, 8),
       ("q4_attn_kernel", 128, 1, 8, 2), ("q4_attn_kernel", 128, 2, 10, 3), ("q4_attn_kernel", 128, 4, 8, 8)]
TC = [("tree_attn_tc_kernel", 64, 64, 16, 8), ("tree_attn_tc_kernel", 64, 256, 8, 64), ("tree_attn_tc_kernel", 128, 64, 10, 9),
      ("tree_attn_tc_kernel", 128, 128, 16, 16), ("tree_attn_tc_kernel", 128, 256, 16, 32)]
FORMS = UNIT + CUT + TC
KEYS = "kernel,hd,rows,nq,nt"


def case_of(dev, g, kernel, hd, rows, nq, nt, window=True, long=(9000, 300), **kw):
    """A case that runs on that kernel: two sequences, with a window and sinks or without."""
    import speculative_decoding_verification_round_gb300 as sv
    cut = kernel == "q4_attn_kernel"  # (tables of more than 64 warps' three steps, and a window of more)
    lens = list(long) if cut else [300, 90]
    c = Q4Case(sv, dev, g, nq, 2, hd, lens, nt, kw.pop("page", 32), window=(6300 if cut else 50) if window else 0,
               sinks=3 if window else 0, layers=1, **kw)
    assert kernel_of(c) == (kernel, hd, rows)
    return c


@pytest.mark.parametrize(KEYS, FORMS)
def test_scales_whose_values_pass_fp16(dev, kernel, hd, rows, nq, nt):
    """Finite scales above 8188 make values that are infinite in fp16: those of hidden
    positions are nobody's, those that are seen are rounded as everywhere."""
    g = np.random.default_rng([hd, nt])
    c = case_of(dev, g, kernel, hd, rows, nq, nt)
    clean = c.call()
    c.check(clean)
    for b in range(2):
        lo = c.lens[b] - c.window + 1  # (the first position that a node of depth 0 sees)
        for p in range(3, max(3, lo)):
            pg, at = c.table[c.slots[b], p // 32], p % 32
            c.vs[:, pg, :, at] = np.float16(g.choice([8192, -8192, 10000, -40000, 65504]))
            c.vc[:, pg, :, at, :, ::5] = 0x00  # -8, -8
    got = c.call()
    assert c.status.tolist() == [0, 0]
    c.check(got)
    # one that the nodes of depth 0 see, the others not
    p = c.lens[0] - c.window + 1
    pg, at = c.table[c.slots[0], p // 32], p % 32
    c.vs[:, pg, :, at] = np.float16(10008)
    c.vc[:, pg, :, at] = (g.integers(3, 14, c.vc[:, pg, :, at].shape) * 17).astype(np.uint8)
    v = lc.values(c.vc[:, pg, :, at], c.vs[:, pg, :, at])
    c.v[:, pg, :, at] = v.astype(np.float16)
    assert np.isfinite(c.v).all() and (c.v[:, pg, :, at] != v).any()
    got = c.call()
    c.check(got)
    # and past fp16's range in one channel of each kv head
    c.vc[:, pg, :, at, 1, 2] = 0x88 & 0xF0  # element 34: -8
    over = c.call()
    depth = np.array([len(x) - 1 for x in tree.chains(c.parents[0].tolist())])
    sees = np.zeros(got.shape, bool)
    sees[0, depth == 0, :, 34] = True
    assert np.isneginf(over[sees]).all()
    same = ~sees
    same[0, depth == 0, :, 50] = False  # (the byte's other element)
    assert np.array_equal(over[same].view(np.uint16), got[same].view(np.uint16))


@pytest.mark.parametrize(KEYS, FORMS)
def test_values_are_rounded_to_fp16(dev, kernel, hd, rows, nq, nt):
    """No scores, and values of 0 but for the window's first position and the last two: their
    mean over what is seen, each of them rounded to fp16 first."""
    g = np.random.default_rng([hd, nt, 2])
    c = case_of(dev, g, kernel, hd, rows, nq, nt)
    if kernel == "q4_attn_kernel":
        c.lens = [6400, 300]
        c.slot_len[c.slots] = c.lens
    c.q[:], c.vn[:], c.parents[:] = 0, 0, -1
    for b in range(2):
        for p in range(max(0, c.lens[b] - c.window + 1), c.lens[b]):
            pg, at = c.table[c.slots[b], p // 32], p % 32
            if p < c.lens[b] - 2 and p != c.lens[b] - c.window + 1:
                c.vs[:, pg, :, at] = 0
            else:
                c.vs[:, pg, :, at] = np.float16(10008 if g.random() < 0.5 else 9992)
                c.vc[:, pg, :, at] = (g.integers(3, 14, c.vc[:, pg, :, at].shape) * 17).astype(np.uint8)
        for p in range(3):  # the sinks
            c.vs[:, c.table[c.slots[b], p // 32], :, p % 32] = 0
    c.v = lc.values(c.vc, c.vs).astype(np.float16)
    got = c.call()
    assert c.status.tolist() == [0, 0]
    for b in range(2):
        v = c.cached(1, b).astype(np.float64)
        lo = max(0, c.lens[b] - c.window + 1)
        seen = v[lo:].sum(0) + v[:min(3, lo)].sum(0)
        count = c.lens[b] - lo + min(3, lo) + 1
        want = np.repeat(seen / count, nq // 2, 0)[None]
        mag = np.repeat((np.abs(v[lo:]).sum(0) + np.abs(v[:min(3, lo)]).sum(0)) / count, nq // 2, 0)[None]
        # sums of a few fp16 values times 2^12 are exact in fp32; a weight's two parts are 2^-22 of it more,
        # which round the additions -- by 2^-24 of a partial sum, up to the sum of magnitudes, where the values
        # cancel -- then the reciprocal and the product once each
        low, high = ((want + e * mag).astype(np.float16) for e in (-2.0 ** -20, 2.0 ** -20))
        assert ((got[b] >= low) & (got[b] <= high)).all()

# ---------------------------------------------------------------------------
# every position counts
# ---------------------------------------------------------------------------
LONGER = [(*f, long) for f in FORMS for long in ([(5000, 2900)] if f in UNIT else [(1500, 700)] if f in TC else [(9000, 300)])]


class Edges(Q4Case):
    """Long contexts, in which a row's weights go further down."""

    def check(self, got, seqs=None):
        """Q4Case.check's bound but for what a pair of fp16 numbers loses of a weight w: two
        numbers of 2^12 w, each off by up to 2^-25 (half of fp16's smallest step), together 2^-36 of the
        row's largest, for each key, however small its w is.  It counts times the key's own |v|, not
        times the row's weighted |v|: where the keys of almost all of the weight have zeros
        in a channel, the latter is next to nothing."""
        for b in range(self.n) if seqs is None else seqs:
            m = int(self.counts[b])
            assert (got[b, m:] == np.float16(7.0)).all(), b
            kc, vc = self.cached(0, b), self.cached(1, b)
            ref, mag, dots = tree.tree_attention(self.q[b, :m], kc, vc, self.kn[b, :m], self.vn[b, :m],
                                                 self.parents[b, :m].tolist(), self.window, self.sinks, self.scale)
            scale = abs(self.scale or self.hd ** -0.5)
            q1 = np.abs(self.q[b, :m].astype(np.float64)).reshape(m, self.nkv, -1, self.hd // 32, 32).sum(-1)
            at = np.arange(self.lens[b])
            s = np.abs(self.ks[self.layer][self.table[self.slots[b], at // self.page], :, at % self.page].astype(np.float64))
            worst = np.einsum("mhgb,phb->mhgp", q1, np.nan_to_num(s)).max(-1).reshape(m, self.nq)
            ds = (self.hd + 4) * 2.0 ** -23 * scale * dots + 40 * 24 * 2.0 ** -23 * scale * worst
            rel = np.expm1(2 * ds) + 2.0 ** -20 + ((self.lens[b] + m) / 8 + 64) * 2.0 ** -23
            far = 2.0 ** -36 * (np.abs(vc.astype(np.float64)).sum(0) + np.abs(self.vn[b, :m].astype(np.float64)).sum(0))
            bound = 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 1.01 * rel[..., None] * mag + np.repeat(
                far, self.nq // self.nkv, 0)[None]
            err = np.abs(got[b, :m].astype(np.float64) - ref)
            assert np.isfinite(got[b, :m]).all() and (err <= bound).all(), (b, float(np.max(err - bound)))


def long_case(dev, g, kernel, hd, rows, nq, nt, long, windowed, **kw):
    """A long context; with a window, tiles of sinks and of the window and whole ones between them that nobody sees."""
    import speculative_decoding_verification_round_gb300 as sv
    cut = kernel == "q4_attn_kernel"
    c = Edges(sv, dev, g, nq, 2, hd, list(long), nt, 64 if windowed else 48, window=(6250 if cut else 450) if windowed else 0,
               sinks=170 if windowed else 0, layers=1, **kw)
    assert kernel_of(c) == (kernel, hd, rows)
    return c


@pytest.mark.parametrize("windowed", [False, True])
@pytest.mark.parametrize(KEYS + ",long", LONGER)
def test_values_of_all_positions(dev, kernel, hd, rows, nq, nt, long, windowed):
    """No scores: every row is the mean of what it sees.  Each position has a value in one
    channel of one kv head alone, so that one that is left out, counted twice or seen by the wrong
    rows moves a channel by far more than a rounding."""
    g = np.random.default_rng([hd, nt, 3])
    c = long_case(dev, g, kernel, hd, rows, nq, nt, long, windowed, counts=[nt, max(1, nt - 1)])
    c.q[:], c.vn[:] = 0, 0
    c.vc[:], c.vs[:] = 0x88, 1
    for b in range(2):
        where = g.permutation(np.arange(c.lens[b]) % (2 * hd))  # [positions] -> kv head and channel
        for p, (h, d) in enumerate(zip(where // hd, where % hd)):
            u = int(g.integers(9, 16))
            c.vc[0, c.table[c.slots[b], p // c.page], h, p % c.page, d // 32, d % 16] = u | 0x80 if d % 32 < 16 else u << 4 | 8
    c.v = lc.values(c.vc, c.vs).astype(np.float16)
    got = c.call()
    assert c.status.tolist() == [0, 0]
    for b in range(2):
        v = c.cached(1, b).astype(np.float64)
        for i in range(int(c.counts[b])):
            cached, nodes = tree.visible(c.lens[b], c.parents[b, :c.counts[b]].tolist(), i, c.window, c.sinks)
            want = np.repeat(v[cached].sum(0) / (len(cached) + len(nodes)), nq // 2, 0)
            # whole numbers times 2^12, exact in fp32, but for 2^-22 of them (the weights' two parts), which
            # round up to 70 products and 100 sums of warps and CTAs by 2^-23 each
            bound = (2.0 ** -11 + 2.0 ** -15) * np.abs(want) + 2.0 ** -25
            assert (np.abs(got[b, i].astype(np.float64) - want) <= bound).all(), (b, i)
        assert (got[b, c.counts[b]:] == 7.0).all()


@pytest.mark.parametrize("windowed", [False, True])
@pytest.mark.parametrize(KEYS + ",long", LONGER)
def test_keys_at_the_edges(dev, kernel, hd, rows, nq, nt, long, windowed):
    """Each row's query has one channel; a hundred positions around the edges of warps' steps, tiles, pages,
    sinks, window and length have keys in one, which weigh e^16 times what the others do."""
    g = np.random.default_rng([hd, nt, 4])
    c = long_case(dev, g, kernel, hd, rows, nq, nt, long, windowed, counts=[nt, max(1, nt - 1)], scale=1.0)
    c.kc[:], c.ks[:], c.kn[:], c.q[:] = 0x88, -0.5, 0, 0
    dims = np.stack([g.permutation(hd)[:rows_] for rows_ in [min(8, nt * nq // 2)] * 2])  # of each kv head
    for i in range(nt):
        for h in range(nq):
            of = dims[h // (nq // 2)]
            c.q[:, i, h, of[(i * (nq // 2) + h) % len(of)]] = 4
    for b in range(2):
        n = c.lens[b]
        lo = n - c.window + 1 if c.window else n // 2
        edges = {0, 32, 128, c.page, 2 * c.page, c.sinks, c.sinks + 32, lo, lo + 1, lo + 2, lo // 32 * 32, lo // 128 * 128, lo // c.page * c.page,
                 lo // 128 * 128 + 128, n // 32 * 32, n // 128 * 128, n // c.page * c.page, n, n // 2 // 32 * 32, (n + lo) // 2 // c.page * c.page}
        at = sorted({p for e in edges for p in (e - 1, e, e + 1) if 0 <= p < n} | set(g.integers(0, n, 30).tolist()))
        for j, p in enumerate(g.permutation(at)):
            for h in range(2):
                d = dims[h][j % dims.shape[1]]
                c.kc[0, c.table[c.slots[b], p // c.page], h, p % c.page, d // 32, d % 16] = 0x80 if d % 32 < 16 else 0x08
    c.k = lc.values(c.kc, c.ks).astype(np.float16)
    got = c.call()
    assert c.status.tolist() == [0, 0]
    c.check(got)


@pytest.mark.parametrize(KEYS, FORMS)
def test_pages_that_nobody_sees_may_be_gone(dev, kernel, hd, rows, nq, nt):
    """Between the sinks and the window a table may hold anything; a missing page that is seen is reported."""
    g = np.random.default_rng([hd, nt, 9])
    c = case_of(dev, g, kernel, hd, rows, nq, nt)
    want = c.call()
    c.check(want)
    lo = c.lens[0] - c.window + 1
    row = c.table[c.slots[0]]
    row[1:lo // 32] = np.where(np.arange(1, lo // 32) % 2 == 0, -1, 10 ** 6)
    got = c.call()
    assert c.status.tolist() == [0, 0] and np.array_equal(got.view(np.uint16), want.view(np.uint16))
    for e, page in ((lo // 32, -1), (0, 10 ** 6), ((c.lens[0] - 1) // 32, -3)):
        held, row[e] = row[e], page
        got = c.call()
        row[e] = held
        assert c.status.tolist() == [tree.ST_PAGE, 0] and np.isnan(got[0]).all()
        assert np.array_equal(got[1].view(np.uint16), want[1].view(np.uint16))


@pytest.mark.parametrize(KEYS, [UNIT[2], UNIT[4], *CUT[:2], *CUT[4:], TC[1], TC[2], TC[4]])
def test_planes_of_more_than_4_gigabytes(dev, kernel, hd, rows, nq, nt):
    """Pages behind 2^32 bytes of codes: attention, copies, commit and reading back."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([hd, nt, 10])
    c = case_of(dev, g, kernel, hd, rows, nq, nt)
    want = c.call()
    c.check(want)
    used = c.ks.shape[1]
    first = (1 << 32) // (2 * 32 * hd // 2) + 5
    big = [torch.empty((1, first + used, *a.shape[2:]), dtype=torch.uint8 if a.dtype == np.uint8 else torch.float16, device=dev)
           for a in (c.kc, c.vc, c.ks, c.vs)]
    for t, a in zip(big, (c.kc, c.vc, c.ks, c.vs)):
        t[:, :used] = c.T(a)
    assert big[0].numel() > 1 << 32
    # every page to the end, by the operator
    st = torch.full((used,), 9, dtype=torch.int32, device=dev)
    ids = torch.arange(used, dtype=torch.int32, device=dev)
    table = c.T(np.where(c.table >= 0, c.table + first, c.table).astype(np.int32))
    kv = sv.KVPagesQ4(*big, table, c.T(c.slot_len))
    sv.spec_pages_q4_copy(kv, used, ids, ids + first, st)
    assert (st == 0).all()
    for t in big:
        t[:, :used] = 0
    got = c.call(kv)
    assert c.status.tolist() == [0, 0] and np.array_equal(got.view(np.uint16), want.view(np.uint16))
    # the last positions read back, then written over with the nodes' rows
    n = c.lens[0]
    pos0, n_pos = (torch.tensor([x], dtype=torch.int32, device=dev) for x in (n - 40, 40))
    out = [torch.zeros((1, 1, 40, 2, hd), dtype=torch.float16, device=dev) for _ in range(2)]
    slot = c.T(c.slots[:1])
    sv.spec_pages_q4_read(kv, 1, slot, 40, pos0, n_pos, out[0], out[1], st)
    assert int(st[0]) == 0
    for o, which in zip(out, (0, 1)):
        assert np.array_equal(o[0, 0].cpu().numpy(), c.cached(which, 0)[n - 40:])
    m = min(nt, n - n // 32 * 32)  # (no page is missing)
    kv._keep[-2][int(c.slots[0])] = n - m
    count = torch.tensor([m], dtype=torch.int32, device=dev)
    sv.spec_pages_q4_commit(kv, 1, slot, nt, c.T(c.kn[None, :1]), c.T(c.vn[None, :1]), None, count, st)
    assert int(st[0]) == 0 and int(kv._keep[-2][int(c.slots[0])]) == n
    sv.spec_pages_q4_read(kv, 1, slot, 40, pos0, n_pos, out[0], out[1], st)
    for o, x, which in zip(out, (c.kn, c.vn), (0, 1)):
        rows_ = np.concatenate([c.cached(which, 0)[n - 40:n - m].astype(np.float64), lc.values(*lc.pack(*lc.quantise(x[0, :m])))])
        assert np.array_equal(o[0, 0].cpu().numpy().astype(np.float64), rows_)


# ---------------------------------------------------------------------------
# the cut on what the other forms are tested with in test_gpu_q4.py
# ---------------------------------------------------------------------------
@pytest.mark.parametrize(KEYS, CUT)
def test_the_cut_matches_the_reference(dev, kernel, hd, rows, nq, nt):
    """Without and with a window and sinks, chains and trees, a negative scale, values near both ends of fp16."""
    g = np.random.default_rng([hd, nt, 5])
    for windowed, kind, scale in ((False, "tree", None), (True, "tree", None), (True, "chain", -0.25), (False, "forest", 0.5)):
        c = long_case(dev, g, kernel, hd, rows, nq, nt, (9000, 300), windowed, counts=[nt, max(1, nt - 1)], kind=kind,
                      scale=scale)
        got = c.call()
        assert c.status.tolist() == [0, 0]
        c.check(got)
        assert np.array_equal(c.call().view(np.uint16), got.view(np.uint16))
    for e in (-24, -16, 12):
        c.vs[:] = np.sign(c.vs) * np.exp2(e) * (1 if e < -18 else 1.9921875)
        c.v = lc.values(c.vc, c.vs).astype(np.float16)
        c.vn[:] = (c.vn / np.abs(c.vn.astype(np.float64)).max() * 2.0 ** max(e, -20)).astype(np.float16)
        c.check(c.call())


@pytest.mark.parametrize(KEYS, CUT)
def test_nothing_masked_gets_into_the_cut(dev, kernel, hd, rows, nq, nt):
    """Scales of NaN and infinity behind the length, in front of the window and between sinks and window; infinities
    of other branches' rows; a NaN that the first nodes see."""
    g = np.random.default_rng([hd, nt, 6])
    c = long_case(dev, g, kernel, hd, rows, nq, nt, (9000, 300), True, counts=[nt, max(1, nt - 1)])
    if nt > 1:
        c.parents[:, 1:] = 0
    c.check(c.call())
    seen = np.zeros(c.ks.shape[1:4:2], bool)
    for b in range(2):
        for p in range(c.lens[b]):
            if p < 170 or p > c.lens[b] - c.window:
                seen[c.table[c.slots[b], p // 64], p % 64] = True
    c.ks[:, :, :] = np.where(seen[None, :, None, :, None], c.ks, np.float16(np.nan))
    c.vs[:, :, :] = np.where(seen[None, :, None, :, None], c.vs, np.float16(np.inf))
    good = c.call()
    c.check(good)
    last = int(c.counts[0]) - 1
    if nt > 1:  # a row of its own, of which the others know nothing
        kn, vn = c.kn.copy(), c.vn.copy()
        c.vn[0, last], c.kn[1, 0] = -np.inf, np.nan
        got = c.call()
        assert np.isneginf(got[0, last]).all()
        assert np.isnan(got[1, :c.counts[1]]).all()  # (everyone's root)
        c.kn, c.vn = kn, vn
        got[0, last], got[1] = good[0, last], good[1]
        c.check(got)
    p = c.lens[0] - c.window + 1
    c.vs[:, c.table[c.slots[0], p // 64], :, p % 64] = np.nan
    got = c.call()
    assert np.isnan(got[0, 0]).all()  # (the others are one deeper)
    assert np.array_equal(got[0, 1:].view(np.uint16), good[0, 1:].view(np.uint16))
    assert np.array_equal(got[1].view(np.uint16), good[1].view(np.uint16))


@pytest.mark.parametrize(KEYS, CUT)
def test_strides_of_the_cut(dev, kernel, hd, rows, nq, nt):
    """Rows of q, k_new and v_new apart, with NaN between; a NaN in one row's query is that row's alone."""
    import torch
    g = np.random.default_rng([hd, nt, 7])
    c = long_case(dev, g, kernel, hd, rows, nq, nt, (9000, 300), False)
    want = c.call()
    c.check(want)

    def apart(x, row):
        buf = torch.full((c.n * nt, row), float("nan"), dtype=torch.float16, device=dev)
        buf[:, :x[0, 0].size] = c.T(x).view(c.n * nt, -1)
        return buf
    qs, ks = nq * hd + 24, 2 * hd + 8
    got = c.call(q=apart(c.q, qs), k_new=apart(c.kn, ks), v_new=apart(c.vn, ks), q_stride=qs, kv_stride=ks)
    assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    q = c.q.copy()
    q[0, nt - 1, 1, 5], q[1, 0, nq - 1, hd - 1] = np.nan, np.inf
    got = c.call(q=c.T(q))
    odd = np.zeros(got.shape[:3], bool)
    odd[0, nt - 1, 1] = odd[1, 0, nq - 1] = True
    assert np.isnan(got[odd]).all()
    got[odd] = want[odd]
    c.check(got)


# ---------------------------------------------------------------------------
# rows into the cache
# ---------------------------------------------------------------------------
def test_a_scale_of_zero_is_positive(dev):
    """Blocks of zeros of either sign, and of values whose scale rounds to 0, get the same bits
    whatever the blocks beside them hold."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(8)
    nt, nkv, hd, page = 6, 4, 128, 8
    rows = random_rows(g, (1, 1, nt, nkv, hd))
    blocks = rows.reshape(nt, nkv * hd // 32, 32)
    blocks[0, ::2] = 0
    blocks[1, ::2] = -0.0
    blocks[2, ::2, ::3] = 0
    blocks[2, ::2, 1::3] = blocks[2, ::2, 2::3] = -0.0
    blocks[3, ::2] = 2.0 ** -24 * g.integers(-3, 4, blocks[3, ::2].shape)
    blocks[4:, ::4] = 0
    blocks[5, 2::4] = -0.0
    blocks[1::2, 1::2] = np.where(np.arange(32) % 2 == 0, 1.5, -1.5)  # (a tie of both signs)
    c = Planes(sv, dev, g, 1, 1, nkv, page, hd, [[0]], [0])
    st = torch.full((1,), 9, dtype=torch.int32, device=dev)
    sv.spec_pages_q4_commit(c.kv, 1, c.T(np.array([0], np.int32)), nt, c.T(rows), c.T(rows), None,
                            c.T(np.array([nt], np.int32)), st)
    assert st.tolist() == [0]
    codes, scales = lc.pack(*lc.quantise(rows[0, 0]))
    zero = (scales == 0).swapaxes(0, 1)
    assert zero.sum() == 4 * 8 + 4 + 8
    for got, scale in zip(c.planes()[::2], c.planes()[1::2]):
        assert np.array_equal(got[0, 0, :, :nt], codes.swapaxes(0, 1))
        assert (scale[0, 0, :, :nt].view(np.uint16)[zero] == 0).all()
