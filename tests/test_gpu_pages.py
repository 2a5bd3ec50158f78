"""The pages of a KV cache on the GPU (spec_pages_*) against the plain
bookkeeping of oracle/tree.py: tables, counts, lengths, copies and the rows'
bits, all exactly; and spec_accept_tree."""
import numpy as np
import pytest

from oracle import tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available()
    return torch.device("cuda:0")


class Pool:
    """A paged cache on the device beside its plain book; every row of every
    page starts with a value of its own."""

    def __init__(self, sv, dev, n_slots, max_pages, n_pages, page, layers=2, nkv=2, hd=64, pad=0):
        import torch
        self.sv, self.dev = sv, dev
        self.book = tree.Book(n_slots, max_pages, n_pages, page)
        g = torch.Generator(device=dev).manual_seed(n_pages * 131 + page)
        n = n_pages * nkv * page * hd
        mk = lambda: torch.randint(-32768, 32767, (layers, n + pad), generator=g, device=dev,  # noqa: E731
                                   dtype=torch.int16)[:, :n].view(layers, n_pages, nkv, page, hd)
        self.k, self.v = mk(), mk()
        self.start = (self.k.clone(), self.v.clone())
        self.table = torch.full((n_slots, max_pages), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
        self.kv = sv.KVPages(self.k, self.v, self.table, self.lens, self.refs)
        self.want = [t.clone() for t in self.start]  # the plain cache
        self.calls = 0

    def i32(self, v):
        import torch
        return torch.tensor(v, dtype=torch.int32, device=self.dev)

    def check(self):
        import torch
        assert self.table.tolist() == self.book.table
        assert self.refs.tolist() == self.book.refs
        assert self.lens.tolist() == self.book.len
        assert torch.equal(self.k, self.want[0]) and torch.equal(self.v, self.want[1])

    def fork(self, src, dst):
        st = self.i32([77] * len(src))
        self.sv.spec_pages_fork(self.kv, len(src), self.i32(src), self.i32(dst), st)
        assert st.tolist() == self.book.fork(src, dst)
        return st.tolist()

    def extend(self, slots, n_new):
        n = len(slots)
        st, cp = self.i32([77] * n), self.i32([[7, 7]] * n)
        fills = [self.book.len[s] % self.book.page if 0 <= s < len(self.book.len) else 0 for s in slots]
        self.sv.spec_pages_extend(self.kv, n, self.i32(slots), self.i32(n_new), cp, st)
        want, copies = self.book.extend(slots, n_new)
        assert st.tolist() == want and [tuple(c) for c in cp.tolist()] == copies
        for (a, b), f in zip(copies, fills):
            if a >= 0:
                for t in self.want:
                    t[:, b, :, :f] = t[:, a, :, :f]
        return want

    def commit(self, slots, path, n_path, nt, use_path=True):
        import torch
        n, shape = len(slots), self.k.shape
        self.calls += 1
        g = torch.Generator(device=self.dev).manual_seed(self.calls)
        kn, vn = (torch.randint(-32768, 32767, (shape[0], n, nt, shape[2], shape[4]), generator=g, device=self.dev,
                                dtype=torch.int16) for _ in range(2))
        st = self.i32([77] * n)
        before = list(self.book.len)
        self.sv.spec_pages_commit(self.kv, n, self.i32(slots), nt, kn, vn, self.i32(path) if use_path else None,
                                  self.i32(n_path), st)
        want = self.book.commit(slots, path, n_path, lambda i, node: None)
        assert st.tolist() == want
        for i, s in enumerate(slots):
            if want[i] == 0:
                for j in range(n_path[i]):
                    pos = before[s] + j
                    pg = self.book.table[s][pos // self.book.page]
                    for t, new in zip(self.want, (kn, vn)):
                        t[:, pg, :, pos % self.book.page] = new[:, i, path[i][j]]
        return want

    def free(self, slots):
        st = self.i32([77] * len(slots))
        self.sv.spec_pages_free(self.kv, len(slots), self.i32(slots), st)
        assert st.tolist() == self.book.free(slots)
        return st.tolist()


@pytest.mark.parametrize("seed,page,hd,nkv,layers,n_pages", [
    (0, 4, 64, 2, 2, 40), (1, 16, 128, 1, 3, 24), (2, 5, 8, 3, 1, 64), (3, 1, 64, 2, 2, 90), (4, 24, 128, 2, 2, 5000)])
def test_random_lives_of_branches(dev, seed, page, hd, nkv, layers, n_pages):
    """Random calls, refused entries among them; after each the whole state
    equals the plain book's."""
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(seed)
    n_slots, max_pages = 12, -(-60 // page)
    p = Pool(sv, dev, n_slots, max_pages, n_pages, page, layers, nkv, hd, pad=16 * seed)
    done = set()
    for _ in range(60):
        op = g.choice(["extend", "commit", "fork", "free", "step"])
        n = int(g.integers(1, 6))
        slots = [int(s) for s in g.permutation(n_slots)[:n]]
        if op == "fork":
            src = [int(s) for s in g.integers(0, n_slots, n)]
            done |= set(p.fork(src, slots))
        elif op == "free":
            p.free(slots[:2])
        elif op == "extend":
            done |= set(p.extend(slots, [int(x) for x in g.integers(0, 20, n)]))
        elif op == "commit":  # mostly without room for it
            nt = int(g.integers(1, 9))
            path = [sorted(g.permutation(nt).tolist()) for _ in range(n)]
            done |= set(p.commit(slots, path, [int(x) for x in g.integers(0, nt + 1, n)], nt))
        else:  # a round: room for nt nodes, then the accepted path of each
            nt = int(g.integers(1, 9))
            st = p.extend(slots, [nt] * n)
            ok = [s for s, x in zip(slots, st) if x == 0]
            if ok:
                path, n_path = [], []
                for _ in ok:
                    m = int(g.integers(1, nt + 1))
                    keep = sorted(int(x) for x in g.permutation(nt)[:m])
                    path.append(keep + [-1] * (nt - m))
                    n_path.append(m)
                p.commit(ok, path, n_path, nt)
        p.check()
    assert {0, tree.ST_SLOT} <= done


def test_an_exhausted_pool_gives_nothing_out(dev):
    """Fresh pages and copies that do not all fit: no entry gets any, those
    with errors of their own keep them, and the next call that fits is served."""
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 6, 8, 10, 4)
    p.extend([0], [18])
    p.commit([0], [list(range(18))], [18], 18)   # five pages, the last half full
    p.fork([0, 0], [1, 2])
    p.check()
    full = tree.ST_FULL
    assert p.extend([1, 2, 0, 3], [1, 3, 1, 8]) == [0] * 4    # two copies, one more page, two pages: all ten are held
    p.check()
    assert p.extend([4, 5, 5, 1], [4, 4, 1, 100]) == [full, 1, 1, full]  # (slot 1 asks for more than its table holds)
    p.check()
    assert p.extend([4, 9], [4, 1]) == [full, tree.ST_SLOT]
    p.free([3])
    assert p.extend([4, 5], [4, 8]) == [full, full] and p.extend([4, 5], [4, 4]) == [0, 0]
    p.check()


def test_many_entries_and_a_large_pool(dev):
    """1024 branches extended in one call (the limit), free pages far into the
    pool, every branch of one parent copying its tail but the parent."""
    import speculative_decoding_verification_round_gb300 as sv
    n = 1023
    p = Pool(sv, dev, n + 1, 8, 20011, 8, layers=1, nkv=1, hd=8)
    p.extend([0], [20])
    p.commit([0], [list(range(20))], [20], 20, use_path=False)
    p.fork([0] * n, list(range(1, n + 1)))
    st = p.extend(list(range(1, n + 1)) + [0], [9] * n + [9])
    assert st == [0] * (n + 1) and p.refs[2].item() == 1 and p.table[0, 2].item() == 2
    p.check()
    p.free(list(range(0, n + 1, 2)))
    p.extend(list(range(0, n + 1, 2)), [60] * 512)
    p.check()


def test_wanted_pages_that_sum_up_past_32_bits(dev):
    """1024 entries, each of which its table has room for: the sum of the pages
    that they want is 2^32, and 2^31 and a little; none gets any."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    n, n_pages, i32 = 1024, 1500, dict(dtype=torch.int32, device=dev)
    table = torch.full((n, 2 ** 22), -1, **i32)
    lens, refs = torch.zeros(n, **i32), torch.zeros(n_pages, **i32)
    k = torch.zeros((1, n_pages, 1, 1, 8), dtype=torch.int16, device=dev)
    kv = sv.KVPages(k, k.clone(), table, lens, refs)
    slots = torch.arange(n, **i32)
    for want in (2 ** 22, 2 ** 21 + 1):
        st, cp = torch.full((n,), 77, **i32), torch.full((n, 2), 7, **i32)
        sv.spec_pages_extend(kv, n, slots, torch.full((n,), want, **i32), cp, st)
        assert (st == tree.ST_FULL).all() and (cp == -1).all()
        assert not refs.any() and (table == -1).all()
    sv.spec_pages_extend(kv, n, slots, torch.ones(n, **i32), cp, st)
    assert not st.any() and (refs[:n] == 1).all() and not refs[n:].any()
    assert torch.equal(table[:, 0], slots) and (table[:, 1] == -1).all()


def test_the_largest_pool(dev):
    """2^31 - 1 pages: the last one is found, and when it is taken the call ends."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    n_pages, i32 = 2 ** 31 - 1, dict(dtype=torch.int32, device=dev)
    k = torch.empty((1, n_pages, 1, 1, 8), dtype=torch.int16, device=dev)
    refs = torch.ones(n_pages, **i32)
    refs[-1] = 0
    table, lens = torch.full((1, 4), -1, **i32), torch.zeros(1, **i32)
    kv = sv.KVPages(k, k, table, lens, refs)
    one, st, cp = torch.ones(1, **i32), torch.full((1,), 77, **i32), torch.full((1, 2), 7, **i32)
    sv.spec_pages_extend(kv, 1, torch.zeros(1, **i32), one, cp, st)
    assert st.item() == 0 and table.tolist() == [[n_pages - 1, -1, -1, -1]] and refs[-1].item() == 1
    sv.spec_pages_extend(kv, 1, torch.zeros(1, **i32), one * 2, cp, st)
    assert st.item() == tree.ST_FULL and table.tolist() == [[n_pages - 1, -1, -1, -1]] and cp.tolist() == [[-1, -1]]


def test_a_long_prompt_is_appended_in_place(dev):
    """path NULL, more rows than a CTA's share, several pages, an odd start;
    then new_len apart from len."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 3, 40, 90, 24, layers=2, nkv=2, hd=64)
    p.extend([1, 2], [7, 500])
    p.commit([1], [list(range(7))], [7], 7, use_path=False)
    p.extend([1], [301])
    p.commit([1, 2], [list(range(301))] * 2, [301, 0], 301, use_path=False)
    p.check()
    new = p.i32([-5, -5, -5])
    k = torch.zeros((2, 1, 4, 2, 64), dtype=torch.int16, device=dev)
    st = p.i32([9])
    p.extend([2], [4])
    sv.spec_pages_commit(p.kv, 1, p.i32([2]), 4, k, k, None, p.i32([3]), st, new_len=new)
    assert st.tolist() == [0] and new.tolist() == [-5, -5, 3] and p.lens.tolist() == [0, 308, 0]


def test_refused_entries_change_nothing(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 4, 4, 16, 4)
    p.extend([0, 1], [9, 3])
    p.commit([0, 1], [[0] * 9] * 2, [9, 3], 9)
    p.check()
    assert p.fork([0, 0, 0], [2, 3, 3]) == [0, tree.ST_SLOT, tree.ST_SLOT]
    assert p.fork([0, -1, 4], [2, 3, 0]) == [tree.ST_SLOT] * 3  # not empty; out of range; out of range
    assert p.fork([2, 0], [3, 2]) == [tree.ST_SLOT] * 2        # a branch of what is made in the same call
    assert p.commit([0], [[0]], [1], 1) == [tree.ST_SHARED]    # slot 2 holds the page too
    assert p.commit([3], [[0]], [1], 1) == [tree.ST_PAGE]      # no page there
    assert p.commit([1], [[1]], [1], 1) == [tree.ST_TREE]      # a row that is none
    assert p.commit([1], [[0]], [2], 1) == [tree.ST_TREE]
    assert p.commit([1, 1], [[0], [0]], [1, 1], 1) == [tree.ST_SLOT] * 2
    assert p.commit([1], [[0] * 20], [14], 20) == [tree.ST_FULL]
    assert p.extend([1, 1, 4], [1, 1, 1]) == [tree.ST_SLOT] * 3
    assert p.extend([1], [-1]) == [tree.ST_PAGE]
    assert p.free([1, 1, -1]) == [tree.ST_SLOT] * 3
    p.check()
    # a length lowered by the caller below a shared page
    p.lens[2] = p.book.len[2] = 3
    assert p.extend([2], [4]) == [tree.ST_SHARED]
    p.check()
    # ids out of range in a table are dropped when the slot is freed
    p.table[3, 0] = 99
    st = p.i32([0])
    sv.spec_pages_free(p.kv, 1, p.i32([3]), st)
    assert st.tolist() == [tree.ST_PAGE]
    p.check()
    assert torch.equal(p.table[3].cpu(), torch.full((4,), -1, dtype=torch.int32))


def test_ids_below_minus_one_are_out_of_range_too(dev):
    """A slot whose row holds one is emptied, and told."""
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 3, 4, 16, 4)
    p.extend([0, 1], [9, 9])
    p.commit([0, 1], [[0] * 9] * 2, [9, 9], 9)
    held = p.book.table[1][1]
    p.table[1, 1] = -2
    st = p.i32([77, 77, 77])
    sv.spec_pages_free(p.kv, 3, p.i32([0, 1, 2]), st)
    assert st.tolist() == [0, tree.ST_PAGE, 0]
    assert (p.table == -1).all() and not p.lens.any()
    assert p.refs.tolist() == [int(i == held) for i in range(16)]  # the page whose id was lost stays taken


@pytest.mark.parametrize("page,hd,nkv,layers", [(4, 64, 2, 3), (300, 128, 8, 2), (1, 8, 1, 1)])
def test_copies(dev, page, hd, nkv, layers):
    """Whole pages and prefixes of them (of zero positions too), a page larger
    than one CTA's share, a source named several times; entries that write
    what others touch are refused."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 1, 1, 12, page, layers, nkv, hd, pad=8)
    kv = sv.KVPages(p.k, p.v)
    src, dst = [3, 3, 0, 7, 8], [1, 2, 4, 5, 5]
    st = p.i32([9] * 5)
    sv.spec_pages_copy(kv, 5, p.i32(src), p.i32(dst), st)
    assert st.tolist() == [0, 0, 0, 1, 1]
    for a, b in ((3, 1), (3, 2), (0, 4)):
        for t in p.want:
            t[:, b] = t[:, a]
    p.check()
    n_pos = [0, page, max(1, page // 3), page + 1, -1, 1]
    src, dst = [0, 3, 7, 0, 0, 12], [6, 8, 9, 10, 11, 2]
    st = p.i32([9] * 6)
    sv.spec_pages_copy(kv, 6, p.i32(src), p.i32(dst), st, n_pos=p.i32(n_pos))
    assert st.tolist() == [0, 0, 0, tree.ST_PAGE, tree.ST_PAGE, tree.ST_SLOT]
    for a, b, n in ((3, 8, page), (7, 9, max(1, page // 3))):
        for t in p.want:
            t[:, b, :, :n] = t[:, a, :, :n]
    p.check()
    st = p.i32([9, 9, 9])
    sv.spec_pages_copy(kv, 3, p.i32([0, 1, 5]), p.i32([1, 2, 5]), st)  # 1 is written and read; 5 onto itself
    assert st.tolist() == [1, 1, 1]
    p.check()
    assert torch.equal(p.k, p.want[0])


def test_a_captured_round_replays(dev):
    """free + fork + extend + commit as one graph, replayed: each replay gives
    the state of the plain book after the same calls."""
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    p = Pool(sv, dev, 5, 6, 40, 8)
    p.extend([0], [13])
    p.commit([0], [list(range(13))], [13], 13)
    kids, src = [1, 2, 3], [0, 0, 0]
    kn = torch.randint(-99, 99, (2, 3, 4, 2, 64), dtype=torch.int16, device=dev)
    slots, par, four = p.i32(kids), p.i32(src), p.i32([4, 4, 4])
    path, n_path = p.i32([[0, 2, 3, -1], [0, -1, -1, -1], [0, 1, 2, 3]]), p.i32([3, 1, 4])
    st, cp = p.i32([[9] * 3] * 4), p.i32([[9, 9]] * 3)

    def calls():
        sv.spec_pages_free(p.kv, 3, slots, st[0])
        sv.spec_pages_fork(p.kv, 3, par, slots, st[1])
        sv.spec_pages_extend(p.kv, 3, slots, four, cp, st[2])
        sv.spec_pages_commit(p.kv, 3, slots, 4, kn, kn, path, n_path, st[3])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        st.fill_(9)
        graph.replay()
        assert st.tolist() == [p.book.free(kids), p.book.fork(src, kids), p.book.extend(kids, [4] * 3)[0],
                               p.book.commit(kids, path.tolist(), [3, 1, 4], lambda i, n: (i, n))]
        assert p.table.tolist() == p.book.table and p.refs.tolist() == p.book.refs
        assert p.lens.tolist() == p.book.len == [13, 16, 14, 17, 0]
        for s, i in ((1, 0), (2, 1), (3, 2)):
            for pos in range(13, p.book.len[s]):
                row = p.k[:, p.book.table[s][pos // 8], :, pos % 8]
                assert torch.equal(row, kn[:, i, path[i][pos - 13]])
            for pos in range(13):
                a, b = (p.k[:, p.book.table[x][pos // 8], :, pos % 8] for x in (0, s))
                assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# acceptance along a tree
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("nt,n_seq,vocab", [(1, 3, 5), (2, 40, 2), (8, 200, 3), (33, 129, 3), (63, 64, 2), (64, 300, 4)])
def test_accept_tree(dev, nt, n_seq, vocab):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    g = np.random.default_rng(nt)
    parents = np.array([[-1] + [int(g.integers(max(-1, i - 5), i)) for i in range(1, nt)] for _ in range(n_seq)])
    parents[0] = np.arange(-1, nt - 1)  # a chain
    tokens, am = g.integers(0, vocab, (n_seq, nt)), g.integers(0, vocab, (n_seq, nt))
    am[0, :-1] = tokens[0, 1:]          # accepted to its end
    counts = g.integers(0, nt + 1, n_seq)
    counts[0] = nt
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(dev)  # noqa: E731
    path, n_path, em = t(np.full((n_seq, nt), 9)), t(np.full(n_seq, 9)), t(np.full((n_seq, nt), 9))
    for n_nodes in (counts, None):
        sv.spec_accept_tree(t(am), t(tokens), t(parents), None if n_nodes is None else t(n_nodes), n_seq, nt, path,
                            n_path, em)
        for s in range(n_seq):
            m = nt if n_nodes is None else int(n_nodes[s])
            rp, re = tree.accept_tree(am[s], tokens[s, :m], parents[s, :m]) if m else ([], [])
            pad = [-1] * (nt - len(rp))
            assert n_path[s].item() == len(rp)
            assert path[s].tolist() == rp + pad and em[s].tolist() == re + pad
    assert n_path[0].item() == nt


def test_accept_tree_refuses_what_is_no_tree(dev):
    import torch
    import speculative_decoding_verification_round_gb300 as sv
    parents = [[-1, 0, 1, 2], [-1, 1, 0, 0], [0, 0, 0, 0], [-1, -2, 0, 0], [-1, 0, 0, 3], [-1, 0, 0, 3], [-1, 0, 0, 9]]
    counts = [5, 4, 4, 4, 4, 3, 3]  # the last two are trees: their bad node is not counted
    n = len(counts)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    path, n_path, em = t([[9] * 4] * n), t([9] * n), t([[9] * 4] * n)
    zeros = t([[0] * 4] * n)
    sv.spec_accept_tree(zeros, zeros, t(parents), t(counts), n, 4, path, n_path, em)
    assert n_path.tolist() == [-1] * 5 + [2, 2]
    assert path[:5].tolist() == em[:5].tolist() == [[-1] * 4] * 5 and path[5].tolist() == [0, 1, -1, -1]
