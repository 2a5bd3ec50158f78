"""spec_sample on the GPU against the plain rules of oracle/tree.py: tokens,
counts and filtered logits, all exactly."""
import numpy as np
import pytest

from oracle import tree

pytestmark = pytest.mark.gpu

LOW = np.finfo(np.float32).min


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


def run(dev, logits, u, T=None, k=None, p=None, m=None, ld=0, off=0, in_place=False, filtered=True, stream=None):
    """The call on rows of stride ld that start `off` floats into a buffer."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    R, V = logits.shape
    ld = ld or V
    mk = lambda: torch.full((off + R * ld + 8,), 123.0, device=dev)  # noqa: E731
    buf = mk()
    rows = buf[off:off + R * ld].view(R, ld)
    rows[:, :V] = torch.from_numpy(logits).to(dev)
    fbuf = buf if in_place else mk()
    t = lambda a, d: None if a is None else torch.from_numpy(np.asarray(a)).to(d).to(dev)  # noqa: E731
    token = torch.full((R,), 99, dtype=torch.int32, device=dev)
    kept = torch.full((R,), 99, dtype=torch.int32, device=dev)
    uu = torch.from_numpy(np.asarray(u, np.uint32).view(np.int32)).to(dev)
    sv.spec_sample(rows, R, V, uu, token, temperature=t(T, torch.float32), top_k=t(k, torch.int32),
                   top_p=t(p, torch.float32), min_p=t(m, torch.float32), n_kept=kept,
                   filtered=fbuf[off:] if filtered else None, ld=ld, ld_filtered=ld, stream=stream)
    out = fbuf[off:off + R * ld].view(R, ld)
    assert (fbuf[:off] == 123.0).all() and (out[:, V:] == 123.0).all() and (fbuf[off + R * ld:] == 123.0).all()
    return token.cpu().numpy(), kept.cpu().numpy(), out[:, :V].cpu().numpy()


def check(orc, dev, logits, u, T=None, k=None, p=None, m=None, **kw):
    R = logits.shape[0]
    tok, kept, filt = run(dev, logits, u, T, k, p, m, **kw)
    at = lambda a, r, d: d if a is None else a[r]  # noqa: E731
    for r in range(R):
        ref, ids = tree.sample_row(logits[r], orc.row_weights, u[r], float(np.float32(at(T, r, 1.0))),
                                   int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0))
        assert (tok[r], kept[r]) == (ref, len(ids)), (r, at(T, r, 1.0), at(k, r, 0), at(p, r, 1.0), at(m, r, 0.0))
        want = np.full_like(logits[r], LOW)
        want[ids] = logits[r, ids]
        if kw.get("filtered", True):
            assert np.array_equal(filt[r].view(np.uint32), want.view(np.uint32)), r


def settings(g, R, V):
    """Rows of all kinds: each filter alone, together, at its ends."""
    T = g.choice([0.0, 0.3, 0.7, 1.0, 1.7, 30.0], R).astype(np.float32)
    k = g.choice([0, 1, 2, 5, 50, 1000, V - 1, V, V + 1, 2 ** 31 - 1], R).clip(0).astype(np.int32)
    p = g.choice([0.0, 1e-6, 0.3, 0.9, 0.999, 1.0, 1.0], R).astype(np.float32)
    m = g.choice([0.0, 0.0, 1e-9, 0.05, 1.0], R).astype(np.float32)
    return T, k, p, m


@pytest.mark.parametrize("V,R,ld,off", [(1, 8, 0, 0), (2, 40, 3, 1), (16, 60, 0, 0), (33, 60, 0, 3), (1000, 60, 1001, 2),
                                        (4096, 20, 0, 0), (4097, 30, 0, 1), (9000, 24, 0, 0), (32000, 24, 0, 0),
                                        (32001, 16, 32004, 0), (151936, 6, 0, 0), (248320, 6, 0, 0)])
def test_rows_of_every_kind(orc, dev, V, R, ld, off):
    g = np.random.default_rng(V)
    logits = (g.standard_normal((R, V)) * g.choice([0.1, 2.0, 8.0], (R, 1))).astype(np.float32)
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    u[:4] = [0, 2 ** 32 - 1, 1, 2 ** 31][:min(4, R)]
    check(orc, dev, logits, u, *settings(g, R, V), ld=ld, off=off)


@pytest.mark.parametrize("V,levels", [(50, 2), (3000, 1), (3000, 3), (40000, 1), (40000, 7), (248320, 2)])
def test_equal_logits(orc, dev, V, levels):
    """Ties go to the lowest id, within bins of far more tokens than are
    ranked at once, at cuts inside a tie of counts and of masses."""
    g = np.random.default_rng(V + levels)
    R = 24 if V < 100000 else 4
    logits = (g.integers(0, levels, (R, V)) * 0.125 - 3.0).astype(np.float32)
    logits[logits == 0] *= g.choice([1.0, -1.0])  # zeros of both signs are equal
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    check(orc, dev, logits, u, *settings(g, R, V))


def test_nearly_equal_logits(orc, dev):
    """Logits a few ulps apart: one step of z holds them all, their order keys
    differ in the last bits; and a crowd around zero, where keys are dense."""
    g = np.random.default_rng(8)
    V, R = 20000, 24
    near = (np.float32(1.0) + g.integers(0, 3000, (R // 2, V)).astype(np.float32) * np.float32(2 ** -23))
    zero = (g.standard_normal((R // 2, V)) * 1e-30).astype(np.float32)
    logits = np.concatenate([near, zero]).astype(np.float32)
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    check(orc, dev, logits, u, *settings(g, R, V))


def test_masked_logits(orc, dev):
    """-infinity and the type's lowest value where a grammar forbids tokens,
    down to one token that is allowed; none of -infinity is ever kept."""
    g = np.random.default_rng(9)
    V, R = 10000, 40
    logits = (g.standard_normal((R, V)) * 2).astype(np.float32)
    for r in range(R):
        gone = g.permutation(V)[:[V - 1, V - 2, V // 2, 10][r % 4]]
        logits[r, gone] = [-np.inf, LOW][r // 4 % 2]
    T, k, p, m = settings(g, R, V)
    T = np.where(T == 0, np.float32(0), np.maximum(T, np.float32(1.0)))  # LOW / T stays finite
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    check(orc, dev, logits, u, T, k, p, m)
    # a row of the lowest value alone is even; with T < 1 it overflows and is refused
    flat = np.full((2, 64), LOW, np.float32)
    tok, kept, _ = run(dev, flat, [2 ** 31, 5], T=np.array([1.0, 0.5], np.float32))
    assert tok.tolist() == [32, -1] and kept.tolist() == [64, 0]


def test_refused_rows(orc, dev):
    """A bad row gets -1, 0 and NaN; its neighbours are served."""
    g = np.random.default_rng(10)
    V, R = 5000, 12
    logits = g.standard_normal((R, V)).astype(np.float32)
    logits[1, 4999] = np.nan
    logits[2, 0] = np.inf
    logits[3, :] = -np.inf
    T, k = np.ones(R, np.float32), np.full(R, 40, np.int32)
    p, m = np.full(R, 0.9, np.float32), np.zeros(R, np.float32)
    T[4], T[5], T[6], k[7], p[8], p[9], m[10] = -1, np.nan, np.inf, -1, 1.5, np.nan, -0.1
    tok, kept, filt = run(dev, logits, np.arange(R), T, k, p, m)
    assert (tok[1:11] == -1).all() and (kept[1:11] == 0).all() and np.isnan(filt[1:11]).all()
    for r in (0, 11):
        ref, ids = tree.sample_row(logits[r], orc.row_weights, r, 1.0, 40, 0.9)
        assert (tok[r], kept[r]) == (ref, len(ids)) and np.isfinite(filt[r]).all()


def test_quotients_at_the_end_of_the_range(orc, dev):
    """Largest logits whose l / T is finite by a unit or two in the last place
    while l (1 / T) overflows; few rows and many."""
    g = np.random.default_rng(15)
    ends = []
    with np.errstate(over="ignore"):
        for T in g.uniform(0.05, 0.999, 400).astype(np.float32):
            l = np.float32(np.finfo(np.float32).max * T)
            for _ in range(6):
                if np.isfinite(l / T) and not np.isfinite(l * (np.float32(1) / T)):
                    ends.append((T, l))
                l = np.nextafter(l, np.float32(0))
    ends = ends[:24]
    assert len(ends) == 24
    for V, R in ((500, 24), (100003, 24)):
        logits = g.standard_normal((R, V)).astype(np.float32)
        for r, (T, l) in enumerate(ends):
            at = g.permutation(V)[:9]
            logits[r, at[:5]] = l
            logits[r, at[5]] = np.nextafter(l, np.float32(0))
            logits[r, at[6:]] = -l
            if r % 6 == 5:  # everything at the other end
                logits[r] = -l
        T = np.array([t for t, _ in ends])
        kinds = np.arange(R) % 4
        check(orc, dev, logits, g.integers(0, 2 ** 32, R, dtype=np.uint64), T,
              np.where(kinds == 1, 3, 0).astype(np.int32), np.where(kinds >= 2, 0.6, 1.0).astype(np.float32),
              np.where(kinds == 3, 0.01, 0.0).astype(np.float32))


def test_in_place_without_outputs_on_a_stream_and_replayed(orc, dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(11)
    V, R = 33000, 10
    logits = (g.standard_normal((R, V)) * 2).astype(np.float32)
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    T, k, p, m = settings(g, R, V)
    check(orc, dev, logits, u, T, k, p, m, in_place=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        check(orc, dev, logits, u, T, k, p, m, filtered=False)
    ld, token = torch.from_numpy(logits).to(dev), torch.zeros(R, dtype=torch.int32, device=dev)
    ud = torch.from_numpy(u.astype(np.uint32).view(np.int32)).to(dev)
    kd = torch.from_numpy(k).to(dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_sample(ld, R, V, ud, token, top_k=kd)
    for r in range(3):  # new words and settings in the same arrays
        u2 = g.integers(0, 2 ** 32, R, dtype=np.uint64)
        k2 = g.integers(0, 60, R).astype(np.int32)
        ud.copy_(torch.from_numpy(u2.astype(np.uint32).view(np.int32)))
        kd.copy_(torch.from_numpy(k2))
        graph.replay()
        assert token.tolist() == [tree.sample_row(logits[i], orc.row_weights, u2[i], 1.0, int(k2[i]))[0] for i in range(R)]


def test_rows_beyond_shared_memory(orc, dev):
    """A vocabulary that a cluster's shared memory does not hold whole."""
    g = np.random.default_rng(12)
    V, R = 600001, 3
    logits = (g.standard_normal((R, V)) * 2).astype(np.float32)
    u = g.integers(0, 2 ** 32, R, dtype=np.uint64)
    T, k = np.array([0.8, 1.0, 1.0], np.float32), np.array([40, 0, 0], np.int32)
    p, m = np.array([0.9, 0.95, 1.0], np.float32), np.array([0, 0.01, 0], np.float32)
    check(orc, dev, logits, u, T, k, p, m)
    check(orc, dev, logits, u, T, k, p, m, in_place=True, off=1)


def many(g, R, V, scale=2.0):
    logits = (g.standard_normal((R, V)) * scale).astype(np.float32)
    return logits, g.integers(0, 2 ** 32, R, dtype=np.uint64)


@pytest.mark.parametrize("R,V,ld,off,in_place", [(126, 40003, 0, 0, False), (304, 16500, 16501, 1, True),
                                                 (3, 1000001, 0, 2, True), (158, 32000, 32004, 0, True),
                                                 (16, 151936, 0, 0, False), (5, 500002, 0, 0, True)])
def test_many_long_rows(orc, dev, R, V, ld, off, in_place):
    """Enough logits for passes over all rows: kinds mixed, strides and
    alignments, the last segment and the last group of 128 cut short."""
    import speculative_decoding_verification_round_gb300 as sv
    assert sv.spec_sample_workspace(R, V) > 0
    g = np.random.default_rng([20, V])
    logits, u = many(g, R, V)
    logits *= g.choice([0.1, 1.0, 3.0], (R, 1)).astype(np.float32)  # flat rows, too: long lists
    T, k, p, m = settings(g, R, V)
    T[:2], k[:2], p[:2], m[:2] = 1, [0, 2000], [0.9999, 1.0], 0
    check(orc, dev, logits, u, T, k, p, m, ld=ld, off=off, in_place=in_place)


def test_many_long_rows_of_equal_masked_and_bad_logits(orc, dev):
    """Rows whose tokens do not fit the list (all of them equal, or of two
    values, or with all large ones in one place), rows with one token left,
    and refused ones between."""
    g = np.random.default_rng(21)
    R, V = 140, 36000
    logits, u = many(g, R, V)
    T, k, p, m = settings(g, R, V)
    T = np.where(T == 0, np.float32(0), np.maximum(T, np.float32(1.0)))
    for r in range(0, R, 2):
        if r % 14 == 0:
            logits[r] = 1.5
        elif r % 14 == 2:
            logits[r] = g.integers(0, 2, V)
        elif r % 14 == 4:
            logits[r].sort()
        elif r % 14 == 6:
            logits[r, g.permutation(V)[:V - 1]] = [-np.inf, LOW][r // 14 % 2]
        elif r % 14 == 8:
            logits[r, :V - 5000] = -np.inf
        elif r % 14 == 10:
            logits[r, g.permutation(V)[:200]] = [0.0, -0.0] * 100
            logits[r] = np.minimum(logits[r], 0)
    check(orc, dev, logits, u, T, k, p, m)
    good = run(dev, logits, u, T, k, p, m)
    bad = [1, 17, 39, 61, 83, 111]
    logits[1, V - 1], logits[17, 0], logits[39] = np.nan, np.inf, -np.inf
    T[61], k[83], p[111] = -1, -1, np.nan
    tok, kept, filt = run(dev, logits, u, T, k, p, m)
    assert (tok[bad] == -1).all() and (kept[bad] == 0).all() and np.isnan(filt[bad]).all()
    rest = np.setdiff1d(np.arange(R), bad)
    assert np.array_equal(tok[rest], good[0][rest]) and np.array_equal(kept[rest], good[1][rest])
    assert np.array_equal(filt[rest], good[2][rest])


def test_many_long_rows_replayed_and_on_two_streams(orc, dev):
    """Two graphs with a workspace each, replayed at once on two streams; and
    calls without one, whose workspace is the allocator's."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(22)
    R, V = 158, 31999
    sides = []
    for s in range(2):
        logits, u = many(g, R, V)
        T, k, p, m = settings(g, R, V)
        want = [tree.sample_row(logits[r], orc.row_weights, u[r], float(T[r]), int(k[r]), p[r], m[r])[0] for r in range(R)]
        c = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        x = (c(logits), R, V, c(u.astype(np.uint32).view(np.int32)), torch.zeros(R, dtype=torch.int32, device=dev),
             c(T), c(k), c(p), c(m))
        ws = torch.empty(sv.spec_sample_workspace(R, V), dtype=torch.uint8, device=dev)
        st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=st):
            sv.spec_sample(*x, workspace=ws)
        sides.append((x, ws, st, graph, want))
    for _ in range(5):
        for x, _, st, graph, _ in sides:
            with torch.cuda.stream(st):
                x[4].zero_()
                graph.replay()
    torch.cuda.synchronize()
    assert all(x[4].tolist() == want for x, _, _, _, want in sides)
    for x, _, st, _, _ in sides:
        with torch.cuda.stream(st):
            x[4].zero_()
            sv.spec_sample(*x)
    for x, _, st, _, _ in sides:  # the stream as an argument
        x[4].record_stream(st)
        sv.spec_sample(*x, stream=st)
    torch.cuda.synchronize()
    assert all(x[4].tolist() == want for x, _, _, _, want in sides)


@pytest.mark.parametrize("R,V,step", [(2, 1048512, 1), (300, 20000, 100), (1000, 65536, 20), (45, 131073, 15),
                                      (12, 524289, 3)])
def test_many_rows_and_few_agree(dev, R, V, step):
    """All rows at once (in passes) and a few at a time (in clusters): the
    same tokens, counts and filtered logits, with ties and settings of all
    kinds, up to the longest row."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    assert sv.spec_sample_workspace(R, V) > 0 == sv.spec_sample_workspace(step, V)
    gen = torch.Generator(device=dev)
    gen.manual_seed(V)
    rnd = lambda: torch.rand((R,), generator=gen, device=dev)  # noqa: E731
    x = torch.randn((R, V), generator=gen, device=dev) * torch.rand((R, 1), generator=gen, device=dev) * 4
    x[::7] = (x[::7] * 2).round() / 2
    u = torch.randint(-2 ** 31, 2 ** 31, (R,), generator=gen, device=dev).to(torch.int32)
    one, none = torch.ones(R, device=dev), torch.zeros(R, device=dev)
    T = torch.where(rnd() < 0.3, one, rnd() * 1.5 + 0.1)
    k = torch.where(rnd() < 0.5, none, 10 ** (rnd() * 5)).to(torch.int32)
    p, m = torch.where(rnd() < 0.5, one, rnd()), torch.where(rnd() < 0.7, none, rnd() * 0.1)

    def call(s):
        n = x[s].shape[0]
        token, kept = torch.zeros(n, dtype=torch.int32, device=dev), torch.zeros(n, dtype=torch.int32, device=dev)
        out = torch.empty_like(x[s])
        sv.spec_sample(x[s], n, V, u[s], token, temperature=T[s], top_k=k[s], top_p=p[s], min_p=m[s], n_kept=kept,
                       filtered=out)
        return token, kept, out
    all_rows = call(slice(0, R))
    assert (all_rows[0] >= 0).all()
    for i in range(0, R, step):
        s = slice(i, min(R, i + step))
        assert all(torch.equal(a[s], b) for a, b in zip(all_rows, call(s))), i


def test_filtered_logits_feed_the_rejection_sampler(orc, dev):
    """Drafts sampled under filters, target rows filtered alike: the accept of
    the filtered rows is the oracle's, and no emitted token was filtered out."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(13)
    n_seq, d, V, T = 6, 5, 3000, 0.8
    q = (g.standard_normal((n_seq, d, V)) * 2).astype(np.float32)
    p = np.concatenate([q, q[:, :1]], 1) + (g.standard_normal((n_seq, d + 1, V)) * 0.5).astype(np.float32)
    full = lambda n, v, t: np.full(n, v, t)  # noqa: E731

    def filt(x, u):
        R = x.shape[0] * x.shape[1]
        return run(dev, x.reshape(R, V), u, full(R, T, np.float32), full(R, 30, np.int32), full(R, 0.9, np.float32))
    draft, _, qf = filt(q, g.integers(0, 2 ** 32, n_seq * d, dtype=np.uint64))
    _, kept, pf = filt(p, g.integers(0, 2 ** 32, n_seq * (d + 1), dtype=np.uint64))
    assert (kept <= 30).all()
    qf, pf, draft = qf.reshape(q.shape), pf.reshape(p.shape), draft.reshape(n_seq, d)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    em = torch.zeros((n_seq, d + 1), dtype=torch.int32, device=dev)
    n_acc = torch.zeros(n_seq, dtype=torch.int32, device=dev)
    idx = torch.zeros(n_seq, dtype=torch.int64, device=dev)
    sv.spec_accept_stochastic(t(pf), t(qf), t(draft), n_seq, d, V, T, 5, t(np.arange(n_seq, dtype=np.int32)), idx,
                              n_acc, em)
    assert sv.spec_error_check(None) == 0
    n_ref, em_ref, _ = orc.accept_stochastic(pf, qf, draft, T, 5, list(range(n_seq)), np.zeros(n_seq, np.uint64))
    assert np.array_equal(n_acc.cpu().numpy(), n_ref) and np.array_equal(em.cpu().numpy(), em_ref)
    for s in range(n_seq):
        for i in range(n_ref[s] + 1):
            assert pf[s, i, em_ref[s, i]] > LOW
    # a refused row fails the accept closed
    bad = t(pf)
    bad[0] = float("nan")
    sv.spec_accept_stochastic(bad, t(qf), t(draft), n_seq, d, V, T, 5, t(np.arange(n_seq, dtype=np.int32)), idx,
                              n_acc, em)
    assert sv.spec_error_check(None) != 0 and (n_acc == -1).all()
