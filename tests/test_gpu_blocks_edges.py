"""Attention over selected blocks: the shape of a launch against what an SM holds."""
import numpy as np
import pytest

from captured import launches
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
