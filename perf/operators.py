"""What is measured of the tree-drafting operators: attention of a tree of
drafted tokens over a paged cache (with a sliding window and sink positions),
the pages of that cache (fork, copy on write, commit of an accepted path,
copies), filtered sampling from given random numbers, and greedy acceptance
along a tree.  Each case is one call (or the few calls that belong together)
of a speculative-decoding round; the plain forms below say what it computes.

`own` false: the plain form in elementary torch operations; true: the calls of
the package."""
import math

import torch

own = False

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # the 8-layer decoder's verify step with the chain of 8 rows replaced by a tree of 8 nodes:
        # one sequence, 4096 cached positions, one page per slot (the model's own cache)
        dict(name="tree_attn_one", op="attn", n_seq=1, nt=8, nq=32, nkv=8, hd=128, ctx=4096, page=4352,
             window=0, sinks=0, ragged=False),
        # the batched 40-layer decoder's verify step: 12 sequences around 512 positions, 16 nodes, GQA 5
        dict(name="tree_attn_batch", op="attn", n_seq=12, nt=16, nq=40, nkv=8, hd=128, ctx=512, page=64,
             window=0, sinks=0, ragged=True),
        # wide trees (63 nodes, an odd count) of four users over long odd contexts: many rows a head
        dict(name="tree_attn_wide", op="attn", n_seq=4, nt=63, nq=32, nkv=8, hd=128, ctx=8191, page=64,
             window=0, sinks=0, ragged=True),
        # two very long contexts: the cache is all of the work
        dict(name="tree_attn_long", op="attn", n_seq=2, nt=16, nq=32, nkv=8, hd=128, ctx=131071, page=256,
             window=0, sinks=0, ragged=False),
        # a 0.5B-class draft model (14 query heads over 2, head dimension 64) decoding single tokens
        # with a sliding window and four sink positions: latency counts
        dict(name="window_decode", op="attn", n_seq=16, nt=1, nq=14, nkv=2, hd=64, ctx=32768, page=16,
             window=4096, sinks=4, ragged=True),
        # each of 12 prompts forked into four branches, each branch given room for 16 drafted positions
        # (the filled part of its last page copied): one step of a branching decode, 40 layers
        dict(name="pages_branch", op="branch", n_parents=12, n_children=4, nt=16, layers=40, nkv=8, hd=128,
             ctx=550, page=64),
        # the accepted path of 12 sequences' 16-node trees into the cache, 40 layers
        dict(name="pages_commit", op="commit", n_seq=12, nt=16, layers=40, nkv=8, hd=128, ctx=512, page=64),
        # whole pages moved in bulk (a batch of sequences brought back from parked pages)
        dict(name="pages_copy", op="copy", n_copy=96, layers=40, nkv=8, hd=128, page=64),
        # one user's next token, every filter on
        dict(name="sample_one", op="sample", rows=1, vocab=151936, filtered=False, mix="all"),
        # a batched round's 12 x 16 target rows, each with its own settings, and the filtered logits that
        # the rejection sampler reads
        dict(name="sample_rows", op="sample", rows=192, vocab=248320, filtered=True, mix="mixed"),
        # one sequence's 8-node tree, and a server's full batch of 63-node trees
        dict(name="accept_one", op="accept", n_seq=1, nt=8, vocab=32000),
        dict(name="accept_batch", op="accept", n_seq=512, nt=63, vocab=151936),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "branch", "commit", "copy", "sample", "sample", "accept"])
    if op == "attn":
        nq, nkv, hd = rng.choice([(32, 8, 128), (40, 8, 128), (14, 2, 64), (8, 8, 128), (16, 2, 64), (6, 1, 128)])
        n_seq, nt = _log(rng, 1, 32), _log(rng, 1, 64)
        most = min(131072, (1 << 30) // (n_seq * nkv * hd * 4), (1 << 27) // (n_seq * nt * nq))
        return dict(op=op, n_seq=n_seq, nt=nt, nq=nq, nkv=nkv, hd=hd, ctx=_log(rng, 1, max(2, most)),
                    page=rng.choice([16, 24, 64, 128, 256, 1000]),
                    window=rng.choice([0, 0, rng.randint(1, 5000)]), sinks=rng.choice([0, 4, rng.randint(0, 200)]),
                    ragged=rng.random() < 0.7)
    layers = rng.randint(1, 40)
    nkv, hd, page = rng.choice([1, 2, 8]), rng.choice([64, 128]), rng.choice([16, 24, 64, 128])
    if op == "branch":
        return dict(op=op, n_parents=rng.randint(1, 12), n_children=rng.randint(1, 5), nt=rng.randint(1, 64),
                    layers=layers, nkv=nkv, hd=hd, ctx=rng.randint(1, 700), page=page)
    if op == "commit":
        return dict(op=op, n_seq=_log(rng, 1, 32), nt=rng.randint(1, 64), layers=layers, nkv=nkv, hd=hd,
                    ctx=rng.randint(1, 700), page=page)
    if op == "copy":
        return dict(op=op, n_copy=_log(rng, 1, 96), layers=layers, nkv=nkv, hd=hd, page=min(page, 64))
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 192), vocab=_log(rng, 16, 248320), filtered=rng.random() < 0.5,
                    mix=rng.choice(["all", "mixed", "top_k", "top_p", "none"]))
    return dict(op=op, n_seq=_log(rng, 1, 512), nt=rng.randint(1, 64), vocab=rng.choice([32000, 151936]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)


def _ints(g, lo, hi, shape):
    """Whole numbers of [lo, hi] (hi included)."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _tree(g, n_seq, nt):
    """Drafted trees: node 0 is the anchor, every other node hangs on one of the eight before it."""
    i = torch.arange(nt, device="cuda", dtype=torch.int32)
    back = _ints(g, 1, 8, (n_seq, nt))
    return torch.where(i > 0, (i - back).clamp(min=0), -1).to(torch.int32).contiguous()


def _pool(g, layers, n_pages, nkv, page, hd):
    shape = (layers, n_pages, nkv, page, hd)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float16),
            torch.randn(shape, generator=g, device="cuda", dtype=torch.float16))


def _shuffled_table(g, lens, page, room, n_pages, max_pages):
    """Pages of a random order for the positions [0, len + room) of every slot; -1 elsewhere."""
    need = (lens.long() + room + page - 1) // page
    first = torch.cumsum(need, 0) - need
    order = torch.randperm(n_pages, generator=g, device="cuda")
    j = torch.arange(max_pages, device="cuda")
    return torch.where(j < need[:, None], order[(first[:, None] + j).clamp(max=n_pages - 1)], -1).to(torch.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(op=op, case=case)
    if op == "attn":
        n, nt, ctx, page = case["n_seq"], case["nt"], case["ctx"], case["page"]
        s["lens"] = _ints(g, max(0, ctx - ctx // 8), ctx, (n,)) if case["ragged"] else torch.full(
            (n,), ctx, device="cuda", dtype=torch.int32)
        max_pages = -(-(ctx + nt) // page)
        n_pages = n * max_pages
        s["k"], s["v"] = _pool(g, 1, n_pages, case["nkv"], page, case["hd"])
        s["table"] = _shuffled_table(g, s["lens"], page, 0, n_pages, max_pages)
        s["slots"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        s["parents"] = _tree(g, n, nt)
        s["n_nodes"] = _ints(g, max(1, nt - nt // 4), nt, (n,)) if case["ragged"] else torch.full(
            (n,), nt, device="cuda", dtype=torch.int32)
        half = lambda *sh: torch.randn(sh, generator=g, device="cuda", dtype=torch.float16)  # noqa: E731
        s["q"] = half(n, nt, case["nq"], case["hd"])
        s["k_new"], s["v_new"] = half(n, nt, case["nkv"], case["hd"]), half(n, nt, case["nkv"], case["hd"])
        s["out"] = torch.zeros((n, nt, case["nq"], case["hd"]), device="cuda", dtype=torch.float16)
        s["status"] = torch.zeros(n, device="cuda", dtype=torch.int32)
    elif op == "branch":
        par, ch, page = case["n_parents"], case["n_children"], case["page"]
        n_slots, kids = par * (1 + ch), par * ch
        plens = _ints(g, max(1, case["ctx"] - 8), case["ctx"], (par,))
        max_pages = -(-(case["ctx"] + case["nt"]) // page)
        n_pages = par * max_pages + kids * (1 + -(-case["nt"] // page)) + 3
        s["k"], s["v"] = _pool(g, case["layers"], n_pages, case["nkv"], page, case["hd"])
        s["lens"] = torch.cat([plens, torch.zeros(kids, device="cuda", dtype=torch.int32)])
        s["table"] = torch.full((n_slots, max_pages), -1, device="cuda", dtype=torch.int32)
        s["table"][:par] = _shuffled_table(g, plens, page, 0, n_pages, max_pages)
        used = s["table"].flatten()
        s["refs"] = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
        s["refs"][used[used >= 0].long()] = 1
        s["src"] = torch.arange(par, device="cuda", dtype=torch.int32).repeat_interleave(ch).contiguous()
        s["kids"] = torch.arange(par, n_slots, device="cuda", dtype=torch.int32)
        s["n_new"] = torch.full((kids,), case["nt"], device="cuda", dtype=torch.int32)
        s["status"] = torch.zeros((3, kids), device="cuda", dtype=torch.int32)
        s["copies"] = torch.zeros((kids, 2), device="cuda", dtype=torch.int32)
    elif op == "commit":
        n, nt, page = case["n_seq"], case["nt"], case["page"]
        s["lens"] = _ints(g, max(0, case["ctx"] - 12), case["ctx"], (n,))
        max_pages = -(-(case["ctx"] + nt) // page)
        n_pages = n * max_pages
        s["k"], s["v"] = _pool(g, case["layers"], n_pages, case["nkv"], page, case["hd"])
        s["table"] = _shuffled_table(g, s["lens"], page, nt, n_pages, max_pages)
        used = s["table"].flatten()
        s["refs"] = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
        s["refs"][used[used >= 0].long()] = 1
        s["slots"] = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
        shape = (case["layers"], n, nt, case["nkv"], case["hd"])
        s["k_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
        s["v_new"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
        # accepted paths: the anchor, then each later node with the workloads' agreement rate's spacing
        step = _ints(g, 1, 3, (n, nt))
        step[:, 0] = 0
        path = torch.cumsum(step, 1)
        s["n_path"] = (path < nt).sum(1).to(torch.int32)
        s["path"] = torch.where(path < nt, path, -1).to(torch.int32).contiguous()
        s["new_len"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["status"] = torch.zeros(n, device="cuda", dtype=torch.int32)
    elif op == "copy":
        n = case["n_copy"]
        n_pages = 2 * n + 5
        s["k"], s["v"] = _pool(g, case["layers"], n_pages, case["nkv"], case["page"], case["hd"])
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        s["src"], s["dst"] = order[:n].contiguous(), order[n:2 * n].contiguous()
        s["status"] = torch.zeros(n, device="cuda", dtype=torch.int32)
    elif op == "sample":
        r, v, mix = case["rows"], case["vocab"], case["mix"]
        s["logits"] = torch.randn((r, v), generator=g, device="cuda") * 2.0
        uni = lambda lo, hi: torch.rand(r, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
        on = lambda p: torch.rand(r, generator=g, device="cuda") < p  # noqa: E731
        t, k = uni(0.6, 1.2), _ints(g, 1, min(v, 1000), (r,))
        p, m = uni(0.8, 0.98), uni(0.001, 0.05)
        use = dict(all=(1.0, 1.0, 1.0, 1.0), mixed=(0.9, 0.5, 0.6, 0.3), top_k=(1.0, 1.0, 0.0, 0.0),
                   top_p=(1.0, 0.0, 1.0, 0.0), none=(1.0, 0.0, 0.0, 0.0))[mix]
        s["temperature"] = torch.where(on(use[0]), t, 0.0)
        s["top_k"] = torch.where(on(use[1]), k, 0).to(torch.int32)
        s["top_p"] = torch.where(on(use[2]), p, 1.0)
        s["min_p"] = torch.where(on(use[3]), m, 0.0)
        s["u"] = torch.randint(-(1 << 31), 1 << 31, (r,), generator=g, device="cuda").to(torch.int32)
        s["token"] = torch.zeros(r, device="cuda", dtype=torch.int32)
        s["n_kept"] = torch.zeros(r, device="cuda", dtype=torch.int32)
        s["filtered"] = torch.zeros((r, v), device="cuda") if case["filtered"] else None
    else:
        n, nt, v = case["n_seq"], case["nt"], case["vocab"]
        s["parents"] = _tree(g, n, nt)
        s["tokens"] = _ints(g, 0, v - 1, (n, nt))
        s["n_nodes"] = _ints(g, max(1, nt - nt // 4), nt, (n,))
        s["argmax"] = _ints(g, 0, v - 1, (n, nt))
        # the target agrees with one child of a node (the last drawn) at the workloads' rate
        i = torch.arange(nt, device="cuda")
        child = torch.where(s["parents"][:, None, :] == i[None, :, None], i, -1).max(2).values  # a node's last child
        agree = (torch.rand((n, nt), generator=g, device="cuda") < 0.74) & (child >= 0)
        tok = torch.gather(s["tokens"], 1, child.clamp(min=0))
        s["argmax"] = torch.where(agree, tok, s["argmax"]).to(torch.int32).contiguous()
        s["path"] = torch.zeros((n, nt), device="cuda", dtype=torch.int32)
        s["n_path"] = torch.zeros(n, device="cuda", dtype=torch.int32)
        s["emitted"] = torch.zeros((n, nt), device="cuda", dtype=torch.int32)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _closure(parents):
    """[n, nt, nt] whether node j is node i or one of its ancestors, and every node's depth."""
    n, nt = parents.shape
    i = torch.arange(nt, device=parents.device)
    up = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    reach = up
    for _ in range(6):  # paths of up to 64 nodes, by doubling
        reach = (torch.bmm(reach, reach) > 0).float()
    return reach > 0, (reach.sum(2) - 1).long()


def _plain_attn(s):
    c = s["case"]
    n, nt, nq, nkv, hd = c["n_seq"], c["nt"], c["nq"], c["nkv"], c["hd"]
    g = nq // nkv
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    table = s["table"][slots].long().clamp(min=0)
    # the cache of every sequence, [n, nkv, positions, hd], its nodes behind it
    ctx = lambda pool, new: torch.cat([  # noqa: E731
        pool[0][table].permute(0, 2, 1, 3, 4).reshape(n, nkv, -1, hd), new.permute(0, 2, 1, 3)], 2).float()
    k, v = ctx(s["k"], s["k_new"]), ctx(s["v"], s["v_new"])
    cap = k.shape[2] - nt
    reach, depth = _closure(s["parents"])
    pos = torch.arange(cap, device="cuda")
    at = lens[:, None] + depth  # [n, nt] the nodes' positions
    seen = (pos < lens[:, None, None]).expand(n, nt, cap)
    if c["window"] > 0:
        seen = seen & ((pos < c["sinks"]) | (pos > at[:, :, None] - c["window"]))
        reach = reach & ((at[:, None, :] < c["sinks"]) | (at[:, None, :] > at[:, :, None] - c["window"]))
    seen = torch.cat([seen, reach], 2)
    seen = seen[:, None, :, None, :].expand(n, 1, nt, g, cap + nt).reshape(n, 1, nt * g, cap + nt)
    q = s["q"].float().view(n, nt, nkv, g, hd).permute(0, 2, 1, 3, 4).reshape(n, nkv, nt * g, hd)
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(hd))
    x = torch.where(seen, x, -math.inf)
    p = torch.exp(x - x.max(3, keepdim=True).values)
    o = torch.matmul(p, v) / p.sum(3, keepdim=True)
    o = o.view(n, nkv, nt, g, hd).permute(0, 2, 1, 3, 4).reshape(n, nt, nq, hd).to(torch.float16)
    live = torch.arange(nt, device="cuda") < s["n_nodes"][:, None]
    return torch.where(live[:, :, None, None], o, s["out"]), torch.zeros_like(s["status"])


def _plain_branch(s):
    c = s["case"]
    table, refs, lens, kids, src = s["table"], s["refs"], s["lens"], s["kids"].long(), s["src"].long()
    page, j = c["page"], torch.arange(table.shape[1], device="cuda")

    def count(pages, by):  # refs of every page in `pages` (-1: none) changed by `by`
        refs.index_add_(0, pages.flatten().long().clamp(min=0),
                        torch.where(pages.flatten() >= 0, by, 0).to(torch.int32))

    # free: what the branches of the last step held
    count(table[kids], -1)
    table[kids] = -1
    lens[kids] = 0
    # fork: a branch shares its parent's pages
    held = (lens[src].long() + page - 1) // page
    table[kids] = torch.where(j < held[:, None], table[src], -1)
    count(table[kids], 1)
    lens[kids] = lens[src]
    # extend: the filled part of a shared last page is copied (the last of its holders keeps it), and
    # the lowest free pages become the copies and the room behind, branch by branch
    ln = lens[kids].long()
    tail = table[kids, (ln // page).clamp(max=table.shape[1] - 1)]
    part = (ln % page) > 0
    same = (tail[:, None] == tail[None, :]) & part[:, None] & part[None, :]
    before = torch.tril(same, -1).sum(1)
    copy = part & (refs[tail.long().clamp(min=0)] - before > 1)
    want = (ln + s["n_new"].long() + page - 1) // page
    need = copy.long() + (want - held)
    free = torch.sort((refs != 0).long(), stable=True).indices  # free pages first, in order
    first = torch.cumsum(need, 0) - need
    fresh = free[(first[:, None] + j).clamp(max=free.shape[0] - 1)].to(torch.int32)
    row = torch.where((j >= held[:, None]) & (j < want[:, None]),
                      torch.gather(fresh, 1, (j - held[:, None] + copy.long()[:, None]).clamp(min=0, max=j.shape[0] - 1)),
                      table[kids])
    row = torch.where((j == (ln // page)[:, None]) & copy[:, None], fresh[:, :1], row)
    count(torch.where(copy, tail, -1), -1)
    count(torch.where(j < need[:, None], fresh, -1), 1)
    table[kids] = row
    s["copies"][:, 0] = torch.where(copy, tail, -1)
    s["copies"][:, 1] = torch.where(copy, fresh[:, 0], -1)
    i, at = torch.nonzero(copy[:, None] & (torch.arange(page, device="cuda") < (ln % page)[:, None]), as_tuple=True)
    a, b = tail[i].long(), fresh[i, 0].long()
    s["k"][:, b, :, at] = s["k"][:, a, :, at]
    s["v"][:, b, :, at] = s["v"][:, a, :, at]
    s["status"].zero_()
    return table, refs, lens, s["copies"], s["status"], s["k"], s["v"]


def _plain_commit(s):
    c = s["case"]
    n, nt, page = c["n_seq"], c["nt"], c["page"]
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    i, j = torch.nonzero(torch.arange(nt, device="cuda") < s["n_path"][:, None], as_tuple=True)
    pos = lens[i] + j
    pg, at, node = s["table"][slots[i], pos // page].long(), pos % page, s["path"][i, j].long()
    s["k"][:, pg, :, at] = s["k_new"][:, i, node].transpose(0, 1)
    s["v"][:, pg, :, at] = s["v_new"][:, i, node].transpose(0, 1)
    s["new_len"][slots] = (lens + s["n_path"]).to(torch.int32)
    s["status"].zero_()
    return s["new_len"], s["status"], s["k"], s["v"]


def _plain_copy(s):
    a, b = s["src"].long(), s["dst"].long()
    s["k"][:, b] = s["k"][:, a]
    s["v"][:, b] = s["v"][:, a]
    s["status"].zero_()
    return s["status"], s["k"], s["v"]


def _weights(x):
    """floor(exp(x) * 2^32) for x <= 0 by the sampler's own exp: fixed fp32 operations, each rounded."""
    f = lambda h: float.fromhex(h)  # noqa: E731
    n = torch.round(x * f("0x1.715476p+0"))
    r = x - n * f("0x1.62e4p-1")
    r = r - n * f("0x1.7f7d1cp-20")
    p = torch.full_like(x, f("0x1.a01a02p-13"))
    for a in ("0x1.6c16c2p-10", "0x1.111112p-7", "0x1.555556p-5", "0x1.555556p-3", "0x1p-1", "0x1p+0", "0x1p+0"):
        p = p * r
        p = p + f(a)
    e = n.clamp(min=-200).to(torch.int32) + 32
    two = ((e.clamp(min=0) + 127) << 23).view(torch.float32)
    return torch.where((x >= -87.0) & (e >= 0), p * two, 0.0).to(torch.int64)


def _scaled(a, b, up):
    """floor (up: ceil) of a * b / 2^32 for 0 <= a < 2^32 and 0 <= b < 2^51, in 64 bits."""
    a1, a0, bh, bl = a >> 16, a & 0xFFFF, b >> 32, b & 0xFFFFFFFF
    mid = a1 * bl + ((a0 * bl) >> 16)
    rest = (((mid & 0xFFFF) << 16) | ((a0 * bl) & 0xFFFF)) != 0
    return a * bh + (mid >> 16) + (rest.long() if up else 0)


def _plain_sample(s):
    l = s["logits"]
    v = l.shape[1]
    t = s["temperature"][:, None]
    greedy = t == 0
    z = l / torch.where(greedy, 1.0, t)
    w = _weights(z - z.max(1, keepdim=True).values)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    rank = torch.arange(v, device="cuda")
    k = torch.where(s["top_k"] > 0, s["top_k"], v)[:, None]
    k = torch.where(greedy, 1, k)
    ws = torch.gather(w, 1, order) * (rank < k)
    cum = torch.cumsum(ws, 1)
    p = torch.floor(s["top_p"].double() * 4294967296.0).long()[:, None]
    need = _scaled(p.clamp(max=(1 << 32) - 1), cum[:, -1:], True)
    keep = (rank < k) & ((p >= 1 << 32) | (cum - ws < need) | (rank == 0))
    m = torch.floor(s["min_p"].double() * 4294967296.0).long()[:, None]
    keep = keep & (ws >= m)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    cum = torch.cumsum(w * kept, 1)
    at = _scaled(s["u"].long()[:, None] & 0xFFFFFFFF, cum[:, -1:], False)
    token = (cum <= at).sum(1).to(torch.int32)
    filtered = None if s["filtered"] is None else torch.where(kept, l, torch.finfo(torch.float32).min)
    return token, kept.sum(1).to(torch.int32), filtered


def _plain_accept(s):
    parents, nt = s["parents"], s["case"]["nt"]
    i = torch.arange(nt, device="cuda")
    up = parents.long().clamp(min=0)
    live = i < s["n_nodes"][:, None]
    hit = live & (parents >= 0) & (s["tokens"] == torch.gather(s["argmax"], 1, up))
    # the first child that agrees, of every node
    older = hit[:, None, :] & (parents[:, :, None] == parents[:, None, :]) & (i < i[:, None])
    step = (hit & ~older.any(2)) | (i == 0)
    reach, _ = _closure(parents)
    on = live & ~(reach & ~step[:, None, :]).any(2)
    n_path = on.sum(1)
    path = torch.sort(torch.where(on, i, nt), 1).values
    back = torch.where(i < n_path[:, None], path, -1).to(torch.int32)
    nxt = torch.gather(torch.cat([path, torch.full_like(path[:, :1], nt)], 1), 1, (i + 1).expand_as(path))
    tok = torch.gather(s["tokens"], 1, nxt.clamp(max=nt - 1))
    last = torch.gather(s["argmax"], 1, path.clamp(max=nt - 1))
    em = torch.where(i < n_path[:, None] - 1, tok, torch.where(i == n_path[:, None] - 1, last, -1))
    return back, n_path.to(torch.int32), em.to(torch.int32)


def _pool_of(s, sv):
    """The handle that a program keeps beside its cache."""
    if "pool" not in s:
        s["pool"] = sv.KVPages(s["k"], s["v"], s.get("table"), s.get("lens"), s.get("refs"))
    return s["pool"]


def run(s):
    op = s["op"]
    if not own:
        return dict(attn=_plain_attn, branch=_plain_branch, commit=_plain_commit, copy=_plain_copy,
                    sample=_plain_sample, accept=_plain_accept)[op](s)
    import speculative_decoding_verification_round_gb300 as sv
    c = s["case"]
    if op == "attn":
        pool = _pool_of(s, sv)
        if "workspace" not in s:
            s["workspace"] = torch.empty(sv.spec_tree_attn_workspace(pool, c["n_seq"], c["nt"], c["nq"]),
                                         device="cuda", dtype=torch.uint8)
        sv.spec_tree_attn(pool, 0, c["n_seq"], s["slots"], c["nt"], c["nq"], s["q"], s["k_new"], s["v_new"],
                          s["out"], s["workspace"], s["status"], parents=s["parents"], n_nodes=s["n_nodes"],
                          window=c["window"], sinks=c["sinks"])
        return s["out"], s["status"]
    if op == "branch":
        pool, n = _pool_of(s, sv), c["n_parents"] * c["n_children"]
        sv.spec_pages_free(pool, n, s["kids"], s["status"][0])
        sv.spec_pages_fork(pool, n, s["src"], s["kids"], s["status"][1])
        sv.spec_pages_extend(pool, n, s["kids"], s["n_new"], s["copies"], s["status"][2])
        return s["table"], s["refs"], s["lens"], s["copies"], s["status"], s["k"], s["v"]
    if op == "commit":
        sv.spec_pages_commit(_pool_of(s, sv), c["n_seq"], s["slots"], c["nt"], s["k_new"], s["v_new"], s["path"],
                             s["n_path"], s["status"], new_len=s["new_len"])
        return s["new_len"], s["status"], s["k"], s["v"]
    if op == "copy":
        sv.spec_pages_copy(_pool_of(s, sv), c["n_copy"], s["src"], s["dst"], s["status"])
        return s["status"], s["k"], s["v"]
    if op == "sample":
        sv.spec_sample(s["logits"], c["rows"], c["vocab"], s["u"], s["token"], temperature=s["temperature"],
                       top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], n_kept=s["n_kept"],
                       filtered=s["filtered"])
        return s["token"], s["n_kept"], s["filtered"]
    sv.spec_accept_tree(s["argmax"], s["tokens"], s["parents"], s["n_nodes"], c["n_seq"], c["nt"], s["path"],
                        s["n_path"], s["emitted"])
    return s["path"], s["n_path"], s["emitted"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c, op = case, case["op"]
    if op == "attn":
        row = c["nkv"] * c["hd"] * 2
        seen = c["ctx"] if c["window"] == 0 else min(c["ctx"], c["window"] + c["sinks"])
        ctx = seen - (min(c["ctx"] // 16, seen // 16) if c["ragged"] and seen == c["ctx"] else 0)  # the mean length
        nodes = c["n_seq"] * (c["nt"] - (c["nt"] // 8 if c["ragged"] else 0))
        return {"bytes": c["n_seq"] * ctx * 2 * row + nodes * (2 * row + 4 * c["nq"] * c["hd"]),
                "flops": 4.0 * nodes * c["nq"] * c["hd"] * (ctx + c["nt"] / 2)}
    row = c["layers"] * c["nkv"] * c["hd"] * 4 if "layers" in c else 0  # K and V of a position, all layers
    if op == "branch":  # at most a page's filled part a branch, read and written, and the bookkeeping
        kids = c["n_parents"] * c["n_children"]
        tail = c["ctx"] % c["page"]
        entries = kids * (c["ctx"] // c["page"] + 1)
        return {"bytes": kids * tail * row + min(c["n_parents"], kids) * tail * row + entries * 20 + 100, "flops": 0}
    if op == "commit":
        return {"bytes": 2 * c["n_seq"] * ((c["nt"] + 1) // 2) * row + 12 * c["n_seq"], "flops": 0}
    if op == "copy":
        return {"bytes": 2 * c["n_copy"] * c["page"] * row, "flops": 0}
    if op == "sample":
        return {"bytes": c["rows"] * c["vocab"] * (8 if c["filtered"] else 4), "flops": 25.0 * c["rows"] * c["vocab"]}
    return {"bytes": 20 * c["n_seq"] * c["nt"] + 8 * c["n_seq"], "flops": 0}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------


def _exact_attn(s):
    c = s["case"]
    out = s["out"].double()
    g = c["nq"] // c["nkv"]
    for b in range(c["n_seq"]):
        slot, m = int(s["slots"][b]), int(s["n_nodes"][b])
        ln = int(s["lens"][slot])
        pg = s["table"][slot, :-(-ln // c["page"])].long()
        k = s["k"][0, pg].transpose(1, 2).reshape(-1, c["nkv"], c["hd"])[:ln]
        v = s["v"][0, pg].transpose(1, 2).reshape(-1, c["nkv"], c["hd"])[:ln]
        k = torch.cat([k, s["k_new"][b, :m]]).double().repeat_interleave(g, 1)
        v = torch.cat([v, s["v_new"][b, :m]]).double().repeat_interleave(g, 1)
        parents = s["parents"][b].tolist()
        depth, chain = [], []
        for i in range(m):
            up = parents[i]
            chain.append(([] if up < 0 else chain[up]) + [i])
            depth.append(len(chain[i]) - 1)
        place = torch.arange(ln + m, device="cuda")
        place[ln:] = ln + torch.tensor(depth, device="cuda")
        for i in range(m):
            see = torch.zeros(ln + m, dtype=torch.bool, device="cuda")
            see[:ln] = True
            see[[ln + j for j in chain[i]]] = True
            if c["window"] > 0:
                see &= (place < c["sinks"]) | (place > ln + depth[i] - c["window"])
            at = torch.nonzero(see).flatten()
            x = torch.einsum("hd,lhd->hl", s["q"][b, i].double(), k[at]) / math.sqrt(c["hd"])
            out[b, i] = torch.einsum("hl,lhd->hd", torch.softmax(x, 1), v[at])
    return out, torch.zeros_like(s["status"])


def _exact_branch(s):
    c = s["case"]
    page, table, refs, lens = c["page"], s["table"].cpu(), s["refs"].cpu(), s["lens"].cpu()
    src, kids, copies = s["src"].tolist(), s["kids"].tolist(), torch.full_like(s["copies"], -1)
    for a, b in zip(src, kids):
        for e in range(-(-int(lens[a]) // page)):
            table[b, e] = table[a, e]
            refs[table[a, e]] += 1
        lens[b] = lens[a]
    taken = iter([x for x in range(len(refs)) if refs[x] == 0])
    for i, b in enumerate(kids):
        ln = int(lens[b])
        if ln % page and refs[table[b, ln // page]] > 1:
            old, new = int(table[b, ln // page]), next(taken)
            refs[old] -= 1
            refs[new] = 1
            table[b, ln // page] = new
            copies[i, 0], copies[i, 1] = old, new
            s["k"][:, new, :, :ln % page] = s["k"][:, old, :, :ln % page]
            s["v"][:, new, :, :ln % page] = s["v"][:, old, :, :ln % page]
        for e in range(-(-ln // page), -(-(ln + c["nt"]) // page)):
            new = next(taken)
            refs[new] = 1
            table[b, e] = new
    return table.cuda(), refs.cuda(), lens.cuda(), copies, s["status"], s["k"], s["v"]


def _exact_commit(s):
    c = s["case"]
    for b in range(c["n_seq"]):
        slot = int(s["slots"][b])
        ln, n = int(s["lens"][slot]), int(s["n_path"][b])
        for j, node in enumerate(s["path"][b, :n].tolist()):
            pg, at = int(s["table"][slot, (ln + j) // c["page"]]), (ln + j) % c["page"]
            s["k"][:, pg, :, at] = s["k_new"][:, b, node]
            s["v"][:, pg, :, at] = s["v_new"][:, b, node]
        s["new_len"][slot] = ln + n
    return s["new_len"], s["status"], s["k"], s["v"]


def _exact_copy(s):
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        s["k"][:, b] = s["k"][:, a]
        s["v"][:, b] = s["v"][:, a]
    return s["status"], s["k"], s["v"]


def _exact_sample(s):
    import numpy as np
    f32 = np.float32
    low = np.finfo(f32).min
    logits = s["logits"].cpu().numpy()
    tokens, counts, filt = [], [], None if s["filtered"] is None else np.full_like(logits, low)
    coef = [1.0 / math.factorial(a) for a in range(8)]
    for r in range(logits.shape[0]):
        l, t = logits[r], f32(s["temperature"][r].item())
        k, p, m = int(s["top_k"][r]), float(s["top_p"][r]), float(s["min_p"][r])
        if t == 0:
            t, k = f32(1), 1
        z = l / t
        x = z - z.max()
        n = np.rint(x * f32(1.0 / math.log(2.0)))
        # ln 2 in two parts: its first fifteen bits, and the rest
        hi = f32(math.floor(math.log(2.0) * 32768) / 32768)
        red = (x - n * hi) - n * f32(math.log(2.0) - float(hi))
        y = np.full_like(red, f32(coef[7]))
        for a in range(6, -1, -1):
            y = y * red + f32(coef[a])
        w = np.where((n >= -32) & (x >= -87), np.floor(np.ldexp(y.astype(np.float64), n.astype(np.int64) + 32)), 0)
        w = w.astype(np.int64)
        order = np.argsort(-l, kind="stable")
        if k > 0:
            order = order[:k]
        if p < 1.0:
            cum = np.cumsum(w[order])
            num = int(math.floor(p * 2.0 ** 32)) * int(cum[-1])
            need = -(-num // 2 ** 32)
            order = order[:max(1, int(np.searchsorted(cum, need, side="left")) + 1)]
        order = order[w[order] >= int(math.floor(m * 2.0 ** 32))]
        ids = np.sort(order)
        cum = np.cumsum(w[ids])
        at = (int(s["u"][r].item()) & 0xFFFFFFFF) * int(cum[-1]) // 2 ** 32
        tokens.append(int(ids[np.searchsorted(cum, at, side="right")]))
        counts.append(len(ids))
        if filt is not None:
            filt[r, ids] = l[ids]
    back = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    return back(tokens), back(counts), None if filt is None else torch.from_numpy(filt).cuda()


def _exact_accept(s):
    n, nt = s["case"]["n_seq"], s["case"]["nt"]
    parents, tokens, top, count = (s[k].tolist() for k in ("parents", "tokens", "argmax", "n_nodes"))
    paths, lens, emitted = [], [], []
    for b in range(n):
        path, em = [0], []
        while True:
            em.append(top[b][path[-1]])
            nxt = [j for j in range(count[b]) if parents[b][j] == path[-1] and tokens[b][j] == em[-1]]
            if not nxt:
                break
            path.append(nxt[0])
        paths.append(path + [-1] * (nt - len(path)))
        lens.append(len(path))
        emitted.append(em + [-1] * (nt - len(em)))
    back = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    return back(paths), back(lens), back(emitted)


def exact(case, seed):
    s = prepare(case, seed)
    return dict(attn=_exact_attn, branch=_exact_branch, commit=_exact_commit, copy=_exact_copy, sample=_exact_sample,
                accept=_exact_accept)[case["op"]](s)
