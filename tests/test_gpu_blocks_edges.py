"""Attention over selected blocks: the shape of a launch against what an SM holds, and
inputs in which a position too few or too many shows."""
import numpy as np
import pytest

from captured import launches
from oracle import tree
from test_gpu_blocks import Blocks, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


@pytest.mark.parametrize("hd,nq,nt,keeps", [(128, 8, 1, (319, 320, 321, 352, 353)), (128, 9, 4, (64, 4096)),
                                            (64, 8, 2, (300, 4096)), (128, 8, 64, (64, 200))])
def test_clusters_of_sixteen_have_two_ctas_an_sm(dev, hd, nq, nt, keeps):
    """Sixteen CTAs of a unit, where an SM holds two of them, and otherwise eight: 16 SMs may be more than
    a GPC has.  The list's 8 bytes a block decide it."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    for keep in keeps:
        g = np.random.default_rng([hd, keep])
        c = make(sv, dev, g, False, nq, 1, hd, [5000], nt, 64, layers=1)
        x = Blocks(c, 64)
        lists = np.full((1, nt, 1, keep), -1, np.int32)
        for i in range(nt):
            lists[0, i, 0, g.permutation(keep)[:40]] = g.permutation(x.nb[0])[:40]
        got = x.attend(lists)
        assert (x.st == 0).all()
        x.check_attention(got, lists, rows=lambda b, i, h: i < 2)
        args = [c.T(a) for a in (c.slots, lists, c.q, c.kn, c.vn, c.parents)]
        out = torch.zeros_like(c.out)
        (name, ctas, _, fit), = launches(lambda: sv.spec_block_attn(
            x.kv, 0, 1, args[0], nt, nq, 64, keep, args[1], args[2], args[3], args[4], out, x.st, parents=args[5]))
        assert "block_attn_kernel" in name
        units = nt * (1 if nq <= 8 else -(-nq // 16))
        want = 16 if fit >= 2 else 8
        sms = torch.cuda.get_device_properties(dev).multi_processor_count
        while units * want > min(fit, 2) * sms:
            want //= 2
        assert ctas == units * want, (keep, ctas, fit)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("hd,nq,nt,keep,block,page", [(128, 8, 1, 70, 64, 192), (64, 5, 2, 130, 16, 48), (128, 12, 3, 9, 32, 32),
                                                      (64, 16, 40, 21, 128, 128), (128, 4, 64, 6, 16, 16)])
def test_each_listed_position_counts_once(dev, q4, hd, nq, nt, keep, block, page):
    """No scores: every row is the mean of the listed positions' values, each of which is in one channel of one
    kv head alone, and of zeros.  One that is left out or counted twice moves a channel by far more than a rounding."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng([hd, keep])
    c = make(sv, dev, g, q4, 2 * nq, 2, hd, [4801, 95], nt, page, layers=1, counts=[nt, max(1, nt - 1)])
    c.q[:], c.vn[:], c.v[:] = 0, 0, 0
    if q4:
        c.vc[:], c.vs[:] = 0x88, 1
    for b in range(2):
        where = g.permutation(np.arange(c.lens[b]) % (2 * hd))
        for p, (h, d) in enumerate(zip(where // hd, where % hd)):
            u, pg, at = int(g.integers(1, 8)), c.table[c.slots[b], p // page], p % page
            c.v[0, pg, h, at, d] = u
            if q4:
                c.vc[0, pg, h, at, d // 32, d % 16] = u + 8 | 0x80 if d % 32 < 16 else u + 8 << 4 | 8
    x = Blocks(c, block)
    lists = x.lists(g, keep)
    lists[0, 0, 0] = -1
    lists[0, 0, 0, :keep] = np.resize(g.permutation(x.nb[0]), keep)  # (twice where there are no more)
    lists[0, 0, 1, 0] = x.nb[0] - 1  # the last one, partly filled
    lists[1, 0, :, 0] = x.nb[1] - 1
    got = x.attend(lists)
    paths = [[len(p) for p in tree.chains(c.parents[b, :c.counts[b]].tolist())] for b in range(2)]
    for b in range(2):
        v = c.cached(1, b).astype(np.float64)
        for i in range(int(c.counts[b])):
            assert (x.st[b, i] == 0).all()
            for h in range(2):
                at = [p for j in lists[b, i, h] if j >= 0 for p in range(j * block, min(c.lens[b], (j + 1) * block))]
                want = v[at, h].sum(0) / (len(at) + paths[b][i])
                # whole numbers times 2^12, exact in fp32, but for 2^-22 of them (the weights' two parts), which
                # round up to 80 products and 24 sums of warps and CTAs by 2^-23 each
                bound = (2.0 ** -11 + 2.0 ** -16) * np.abs(want) + 2.0 ** -25
                err = np.abs(got[b, i, h * nq:(h + 1) * nq].astype(np.float64) - want)
                assert (err <= bound).all(), (b, i, h)
        assert (got[b, c.counts[b]:] == 7.0).all()
