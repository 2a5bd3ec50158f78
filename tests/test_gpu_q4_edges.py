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
