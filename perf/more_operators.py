"""What is measured of the operators for long contexts: a KV cache held in 4 bits
(rows committed into it and read back, attention of drafted trees and single
tokens over it), and attention over the blocks of a cache that a cheap score
selects for each query (digests of the blocks with the scores, the selection,
the attention).  Each case is one call, or the few calls that belong together,
of a decoding step; the plain forms below say what it computes.

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
        # the accepted paths of 12 sequences' 16-node trees, 40 layers: every round of the batched decoder
        dict(name="commit_step", op="commit", n_seq=12, nt=16, layers=40, nkv=8, hd=128, ctx=512, page=64, path=True),
        # two prompts of an odd length into eight layers of the cache
        dict(name="commit_prompt", op="commit", n_seq=2, nt=4097, layers=8, nkv=8, hd=128, ctx=0, page=256, path=False),
        # one user's next token over a middling context: latency counts
        dict(name="q4_one", op="attn", n_seq=1, nt=1, nq=32, nkv=8, hd=128, ctx=8191, page=64, window=0, sinks=0,
             ragged=False),
        # a 0.5B-class draft model's single tokens with a sliding window and sinks, small pages
        dict(name="q4_window", op="attn", n_seq=16, nt=1, nq=14, nkv=2, hd=64, ctx=32768, page=16, window=4096, sinks=4,
             ragged=True),
        # chains of four drafts of four users over very long contexts: the cache is all of the work
        dict(name="q4_long", op="attn", n_seq=4, nt=4, nq=32, nkv=8, hd=128, ctx=131071, page=256, window=0, sinks=0,
             ragged=False),
        # wide trees (63 nodes) of four users: many query rows a head
        dict(name="q4_wide", op="attn", n_seq=4, nt=63, nq=32, nkv=8, hd=128, ctx=8191, page=64, window=0, sinks=0,
             ragged=True),
        # the blocks that the last round filled, and every block's score for the next token of two long contexts
        dict(name="scores_step", op="scores", n_seq=2, nt=1, nq=32, nkv=8, hd=128, ctx=131071, page=256, block=64, new=70,
             q4=False),
        # prompts just committed (all of their blocks are new), trees of 16 nodes, a cache in 4 bits
        dict(name="scores_prompt", op="scores", n_seq=12, nt=16, nq=40, nkv=8, hd=128, ctx=4095, page=64, block=32, new=4095,
             q4=True),
        # one token's blocks out of 8192 small ones
        dict(name="select_one", op="select", n_seq=1, nt=1, nkv=8, ctx=131071, block=16, keep=256, ragged=False),
        # a batched round's 12 x 16 nodes, 2048 blocks each
        dict(name="select_batch", op="select", n_seq=12, nt=16, nkv=8, ctx=131071, block=64, keep=64, ragged=True),
        # one token over 64 of 2048 blocks
        dict(name="blocks_one", op="blocks", n_seq=1, nt=1, nq=32, nkv=8, hd=128, ctx=131071, page=256, block=64, keep=64,
             q4=False, ragged=False),
        # trees of 8 nodes of 12 users, a list for every node and head, a cache in 4 bits
        dict(name="blocks_batch", op="blocks", n_seq=12, nt=8, nq=40, nkv=8, hd=128, ctx=32767, page=64, block=32, keep=64,
             q4=True, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["commit", "attn", "attn", "attn", "scores", "select", "blocks", "blocks"])
    nq, nkv, hd = rng.choice([(32, 8, 128), (40, 8, 128), (14, 2, 64), (8, 8, 128), (16, 2, 64), (6, 1, 128)])
    page = rng.choice([16, 32, 64, 128, 256, 1024])
    if op == "commit":
        layers, path = rng.randint(1, 40), rng.random() < 0.5
        n_seq = _log(rng, 1, 32)
        nt = rng.randint(1, 64) if path else _log(rng, 1, max(1, 65536 // (n_seq * layers)))
        return dict(op=op, n_seq=n_seq, nt=nt, layers=layers, nkv=nkv, hd=hd, ctx=rng.randint(0, 700),
                    page=rng.choice([16, 24, 64, 100]), path=path)
    n_seq, nt = _log(rng, 1, 32), _log(rng, 1, 64)
    if op == "attn":
        most = min(131072, (1 << 29) // (n_seq * nkv * hd * 2), (1 << 26) // (n_seq * nt * nq))
        return dict(op=op, n_seq=n_seq, nt=nt, nq=nq, nkv=nkv, hd=hd, ctx=_log(rng, 1, max(2, most)),
                    page=rng.choice([16, 24, 64, 128, 256, 1000]), window=rng.choice([0, 0, rng.randint(1, 5000)]),
                    sinks=rng.choice([0, 4, rng.randint(0, 200)]), ragged=rng.random() < 0.7)
    block = rng.choice([b for b in (16, 32, 64, 128) if page % b == 0])
    if op == "scores":
        n_seq, nt = _log(rng, 1, 16), _log(rng, 1, 16)
        most = min(131072, (1 << 28) // (n_seq * nkv * hd), (1 << 26) // (n_seq * nt * nq) * 16)
        ctx = _log(rng, 1, max(2, most))
        return dict(op=op, n_seq=n_seq, nt=nt, nq=nq, nkv=nkv, hd=hd, ctx=ctx, page=page, block=block,
                    new=rng.choice([1, 5, min(ctx, 100), ctx]), q4=rng.random() < 0.5)
    ctx = _log(rng, 1, 131072)
    if op == "select":
        most = max(1, (1 << 22) // (n_seq * nkv * -(-ctx // block)))
        return dict(op=op, n_seq=n_seq, nt=_log(rng, 1, min(64, most)), nkv=nkv, ctx=ctx, block=block,
                    keep=_log(rng, 2, 256), ragged=rng.random() < 0.7)
    n_seq, nt = _log(rng, 1, 16), _log(rng, 1, 16)
    ctx = min(ctx, (1 << 28) // (n_seq * nkv * hd))
    keep = min(_log(rng, 2, 256), max(2, (1 << 27) // (n_seq * nt * nkv * hd * block)))
    return dict(op=op, n_seq=n_seq, nt=nt, nq=nq, nkv=nkv, hd=hd, ctx=ctx, page=page, block=block, keep=keep,
                q4=rng.random() < 0.5, ragged=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# the 4-bit format: blocks of 32 elements of a row
# ---------------------------------------------------------------------------


def _quantise(x):
    """[..., hd] fp16 -> codes [..., hd / 32, 16] (element j of a block in the low nibble of byte j, element
    16 + j in the high one, each q + 8) and fp16 scales [..., hd / 32].  The scale is -1/8 of the element of
    the largest magnitude (the first of several), rounded to eight significant bits, at most 8160; q = x /
    scale rounded to a whole number of [-8, 7].  A block that is not finite gets a NaN for a scale."""
    b = x.float().unflatten(-1, (-1, 32))
    top = torch.gather(b, -1, b.abs().argmax(-1, keepdim=True))
    d = (top * -0.125).to(torch.bfloat16).to(torch.float16).float().clamp(-8160.0, 8160.0)
    fine = torch.isfinite(b).all(-1, keepdim=True)
    q = torch.round(b / torch.where(d == 0, 1.0, d)).clamp(-8, 7)
    q = torch.where((d == 0) | ~fine, 0.0, q).to(torch.int32) + 8
    codes = (q[..., :16] | (q[..., 16:] << 4)).to(torch.uint8)
    return codes, torch.where(fine, d, math.nan).squeeze(-1).to(torch.float16)


def _values(codes, scales):
    """[..., hd] fp32 of what the codes stand for."""
    q = torch.cat([codes & 15, codes >> 4], -1).float() - 8.0
    return (q * scales.float()[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 23)


def _ints(g, lo, hi, shape):
    """Whole numbers of [lo, hi] (hi included)."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64).to(torch.int32)


def _half(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)


def _i32(*shape):
    return torch.zeros(shape, device="cuda", dtype=torch.int32)


def _pool(g, layers, n_pages, nkv, page, hd, keys):
    """Rows of a cache; keys have a few channels that are larger than the others, as a model's have."""
    x = _half(g, layers, n_pages, nkv, page, hd)
    if keys:
        x *= torch.where(torch.rand(hd, generator=g, device="cuda") < 0.06, 4.0, 1.0).to(torch.float16)
    return x


def _cache(s, g, layers, n_pages, nkv, page, hd, q4):
    for which in ("k", "v"):
        x = _pool(g, layers, n_pages, nkv, page, hd, which == "k")
        if not q4:
            s[which] = x
            continue
        parts = [_quantise(p) for p in x.split(max(1, (1 << 25) // (nkv * page * hd * layers)), 1)]
        s[which + "_qs"], s[which + "_scales"] = (torch.cat([p[i] for p in parts], 1) for i in (0, 1))


def _shuffled_table(g, lens, page, room, n_pages, max_pages):
    """Pages of a random order for the positions [0, len + room) of every slot; -1 elsewhere."""
    need = (lens.long() + room + page - 1) // page
    first = torch.cumsum(need, 0) - need
    order = torch.randperm(n_pages, generator=g, device="cuda")
    j = torch.arange(max_pages, device="cuda")
    return torch.where(j < need[:, None], order[(first[:, None] + j).clamp(max=n_pages - 1)], -1).to(torch.int32)


def _lens(g, case):
    n, ctx = case["n_seq"], case["ctx"]
    if case.get("ragged"):
        return _ints(g, max(0, ctx - ctx // 8), ctx, (n,))
    return torch.full((n,), ctx, device="cuda", dtype=torch.int32)


def _tree(s, g, case):
    """Drafted trees: node 0 is the anchor, every other node hangs on one of the eight before it."""
    n, nt, hd = case["n_seq"], case["nt"], case["hd"]
    i = torch.arange(nt, device="cuda", dtype=torch.int32)
    s["parents"] = torch.where(i > 0, (i - _ints(g, 1, 8, (n, nt))).clamp(min=0), -1).to(torch.int32).contiguous()
    s["n_nodes"] = _ints(g, max(1, nt - nt // 4), nt, (n,)) if case["ragged"] else torch.full(
        (n,), nt, device="cuda", dtype=torch.int32)
    s["q"] = _half(g, n, nt, case["nq"], hd)
    s["k_new"], s["v_new"] = _half(g, n, nt, case["nkv"], hd), _half(g, n, nt, case["nkv"], hd)
    s["out"] = torch.zeros((n, nt, case["nq"], hd), device="cuda", dtype=torch.float16)


def prepare(case, seed):
    g, op, n, nt = _gen(seed), case["op"], case["n_seq"], case["nt"]
    s = dict(op=op, case=case, slots=torch.randperm(n, generator=g, device="cuda").to(torch.int32), status=_i32(n))
    if op == "select":
        s["lens"] = _lens(g, case)
        nb = -(-case["ctx"] // case["block"])
        # bounds of a row's logits: a level of its own, a tail of blocks that matter
        x = torch.randn((n, nt, case["nkv"], nb), generator=g, device="cuda")
        s["scores"] = 20.0 + 3.0 * x + 0.5 * x * x
        s["blocks"] = _i32(n, nt, case["nkv"], case["keep"])
        return s
    nkv, hd, page = case["nkv"], case["hd"], case["page"]
    if op == "commit":
        layers = case["layers"]
        s["lens"] = _ints(g, max(0, case["ctx"] - 12), case["ctx"], (n,))
        max_pages = -(-(case["ctx"] + nt) // page)
        n_pages = n * max_pages
        s["table"] = _shuffled_table(g, s["lens"], page, nt, n_pages, max_pages)
        s["refs"] = _i32(n_pages)
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        rows = (layers, n_pages, nkv, page, hd // 32)
        for which in ("k", "v"):
            s[which + "_qs"] = torch.zeros(rows + (16,), device="cuda", dtype=torch.uint8)
            s[which + "_scales"] = torch.zeros(rows, device="cuda", dtype=torch.float16)
            s[which + "_new"] = _pool(g, layers, n, nt, nkv, hd, which == "k")
            s[which + "_back"] = torch.zeros((layers, n, nt, nkv, hd), device="cuda", dtype=torch.float16)
        if case["path"]:  # accepted paths: the anchor, then later nodes
            step = _ints(g, 1, 3, (n, nt))
            step[:, 0] = 0
            path = torch.cumsum(step, 1)
            s["n_path"] = (path < nt).sum(1).to(torch.int32)
            s["path"] = torch.where(path < nt, path, -1).to(torch.int32).contiguous()
        else:
            s["n_path"], s["path"] = _ints(g, max(1, nt - nt // 8), nt, (n,)), None
        s["new_len"], s["status_read"] = _i32(n), _i32(n)
        s["pos0"] = s["lens"][s["slots"].long()]
        return s
    s["lens"] = _lens(g, case)
    max_pages = -(-(case["ctx"] + nt) // page)
    n_pages = n * max_pages
    s["table"] = _shuffled_table(g, s["lens"], page, 0, n_pages, max_pages)
    _cache(s, g, 1, n_pages, nkv, page, hd, case.get("q4", op == "attn"))
    if op == "scores":
        s["q"] = _half(g, n, nt, case["nq"], hd)
        s["pos0"] = (s["lens"][s["slots"].long()] - case["new"]).clamp(min=0)
        # the digests of the blocks before these positions
        k = _rows(s, "k").unflatten(3, (-1, case["block"]))
        s["digest"] = torch.stack([k.amin(4), k.amax(4)], 4).to(torch.float16)
        s["scores"] = torch.zeros((n, nt, nkv, -(-case["ctx"] // case["block"])), device="cuda")
        s["status_digest"] = _i32(n)
    else:
        _tree(s, g, case)
    if op == "blocks":
        # ascending lists: the first block, the last one and others, as a selection gives them
        nb = -(-s["lens"][s["slots"].long()] // case["block"])
        most = -(-case["ctx"] // case["block"])
        j = torch.arange(most, device="cuda")
        rank = torch.rand((n, nt, nkv, most), generator=g, device="cuda")
        rank = torch.where((j == 0) | (j == (nb - 1)[:, None, None, None]), 2.0, rank)
        rank = torch.where(j < nb[:, None, None, None], rank, -1.0)
        keep = min(case["keep"], most)
        at = torch.sort(rank, dim=3, descending=True).indices[..., :keep]
        at = torch.sort(torch.where(torch.gather(rank, 3, at) >= 0, at, most), 3).values
        s["blocks"] = torch.full((n, nt, nkv, case["keep"]), -1, device="cuda", dtype=torch.int32)
        s["blocks"][..., :keep] = torch.where(at < most, at, -1).to(torch.int32)
        s["status"] = _i32(n, nt, nkv)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _rows(s, which):
    """The cache's rows as fp32, [layers, pages, heads, page, hd]."""
    return s[which].float() if which in s else _values(s[which + "_qs"], s[which + "_scales"])


def _plain_commit(s):
    c = s["case"]
    nt, page = c["nt"], c["page"]
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    i, j = torch.nonzero(torch.arange(nt, device="cuda") < s["n_path"][:, None], as_tuple=True)
    pos = lens[i] + j
    pg, at = s["table"][slots[i], pos // page].long(), pos % page
    node = j if s["path"] is None else s["path"][i, j].long()
    for which in ("k", "v"):
        codes, scales = _quantise(s[which + "_new"][:, i, node])
        s[which + "_qs"][:, pg, :, at] = codes.transpose(0, 1)
        s[which + "_scales"][:, pg, :, at] = scales.transpose(0, 1)
        back = _values(s[which + "_qs"][:, pg, :, at], s[which + "_scales"][:, pg, :, at])
        s[which + "_back"][:, i, j] = back.transpose(0, 1).to(torch.float16)
    s["new_len"][slots] = (lens + s["n_path"]).to(torch.int32)
    s["status"].zero_()
    s["status_read"].zero_()
    return s["new_len"], s["status"], s["status_read"], s["k_back"], s["v_back"]


def _closure(parents):
    """[n, nt, nt] whether node j is node i or one of its ancestors, and every node's depth."""
    i = torch.arange(parents.shape[1], device=parents.device)
    reach = ((parents[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(6):  # paths of up to 64 nodes, by doubling
        reach = (torch.bmm(reach, reach) > 0).float()
    return reach > 0, (reach.sum(2) - 1).long()


def _attend(q, k, v, seen):
    x = torch.matmul(q, k.transpose(-2, -1)) * (1.0 / math.sqrt(q.shape[-1]))
    x = torch.where(seen, x, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True)


def _finished(s, o):
    live = torch.arange(s["case"]["nt"], device="cuda") < s["n_nodes"][:, None]
    return torch.where(live[:, :, None, None], o.to(torch.float16), s["out"]), torch.zeros_like(s["status"])


def _plain_attn(s):
    c = s["case"]
    n, nt, nq, nkv, hd = c["n_seq"], c["nt"], c["nq"], c["nkv"], c["hd"]
    g = nq // nkv
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    table = s["table"][slots].long().clamp(min=0)
    ctx = lambda which: torch.cat([  # noqa: E731  the cache of every sequence, [n, nkv, positions, hd], its nodes behind it
        _values(s[which + "_qs"][0][table], s[which + "_scales"][0][table]).transpose(1, 2).reshape(n, nkv, -1, hd),
        s[which + "_new"].permute(0, 2, 1, 3).float()], 2)
    k, v = ctx("k"), ctx("v")
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
    o = _attend(q, k, v, seen)
    return _finished(s, o.view(n, nkv, nt, g, hd).permute(0, 2, 1, 3, 4).reshape(n, nt, nq, hd))


def _plain_scores(s):
    """The digests (least and largest value of every channel) of the blocks that hold positions [pos0, len),
    then for every block a bound of any of the group's logits: max over the heads of sum_d max(q lo, q hi)."""
    c = s["case"]
    n, nt, nkv, hd, block, page = c["n_seq"], c["nt"], c["nkv"], c["hd"], c["block"], c["page"]
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    nb, per = -(-lens // block), page // block
    j = torch.arange(s["scores"].shape[3], device="cuda")
    here = j < nb[:, None]
    i, b = torch.nonzero(here & (j >= (s["pos0"].long() // block)[:, None]), as_tuple=True)
    pg = s["table"][slots[i], b // per].long()
    cut = lambda x: x[0].unflatten(2, (per, block))[pg, :, b % per]  # noqa: E731  [blocks, nkv, block, ...]
    k = cut(s["k"]).float() if "k" in s else _values(cut(s["k_qs"]), cut(s["k_scales"]))
    full = (b[:, None] * block + torch.arange(block, device="cuda") < lens[i][:, None])[:, None, :, None]
    s["digest"][0, pg, :, b % per, 0] = torch.where(full, k, math.inf).amin(2).to(torch.float16)
    s["digest"][0, pg, :, b % per, 1] = torch.where(full, k, -math.inf).amax(2).to(torch.float16)
    d = s["digest"][0][s["table"][slots].long().clamp(min=0)]  # [n, pages, nkv, per, 2, hd]
    d = d.permute(0, 2, 4, 1, 3, 5).reshape(n, nkv, 2, -1, hd)[:, :, :, :j.shape[0]].float()
    q = s["q"].float().view(n, nt, nkv, -1, hd).transpose(1, 2).flatten(2, 3)  # [n, nkv, nt g, hd]
    x = torch.matmul(q.clamp(max=0.0), d[:, :, 0].transpose(2, 3)) + torch.matmul(q.clamp(min=0.0), d[:, :, 1].transpose(2, 3))
    x = x.unflatten(2, (nt, -1)).amax(3).transpose(1, 2)  # [n, nt, nkv, blocks]
    s["scores"] = torch.where(here[:, None, None, :], x, s["scores"])
    s["status"].zero_()
    s["status_digest"].zero_()
    return s["digest"], s["scores"], s["status"], s["status_digest"]


def _plain_select(s):
    """Of a row's blocks the first, the last and those with the largest scores (equal ones: the lowest), in order."""
    c = s["case"]
    keep, most = c["keep"], s["scores"].shape[3]
    nb = -(-s["lens"][s["slots"].long()].long() // c["block"])[:, None, None, None]
    j = torch.arange(most, device="cuda")
    x = torch.where((j < 1) | (j >= nb - 1), math.inf, s["scores"])
    x = torch.where(j < nb, x, -math.inf)
    at = torch.sort(x, dim=3, descending=True, stable=True).indices[..., :keep]
    at = torch.sort(torch.where(at < nb, at, most), 3).values
    out = torch.full_like(s["blocks"], -1)
    out[..., :at.shape[3]] = torch.where(at < most, at, -1).to(torch.int32)
    s["status"].zero_()
    return out, s["status"]


def _plain_blocks(s):
    c = s["case"]
    n, nt, nq, nkv, hd, block, page = c["n_seq"], c["nt"], c["nq"], c["nkv"], c["hd"], c["block"], c["page"]
    slots = s["slots"].long()
    lens = s["lens"][slots].long()
    pos = (s["blocks"].long()[..., None] * block + torch.arange(block, device="cuda")).flatten(3)  # [n, nt, nkv, keys]
    see = (s["blocks"] >= 0).repeat_interleave(block, 3) & (pos < lens[:, None, None, None])
    pos = pos.clamp(min=0, max=s["table"].shape[1] * page - 1)
    pg = s["table"][slots[:, None, None, None], pos // page].long().clamp(min=0)
    head = torch.arange(nkv, device="cuda")[:, None]
    at = ((pg * nkv + head) * page + pos % page).flatten()

    def rows(which):
        flat = lambda x: x.flatten(0, 3)[at]  # noqa: E731
        x = flat(s[which]).float() if which in s else _values(flat(s[which + "_qs"]), flat(s[which + "_scales"]))
        fresh = s[which + "_new"].float().permute(0, 2, 1, 3)[:, None].expand(n, nt, nkv, nt, hd)
        return torch.cat([x.view(n, nt, nkv, -1, hd), fresh], 3)

    reach, _ = _closure(s["parents"])
    seen = torch.cat([see, reach[:, :, None, :].expand(n, nt, nkv, nt)], 3)
    o = _attend(s["q"].float().view(n, nt, nkv, -1, hd), rows("k"), rows("v"), seen[:, :, :, None])
    return _finished(s, o.reshape(n, nt, nq, hd))


def _handles(s, sv):
    """The handles that a program keeps beside its cache."""
    if "kv" not in s:
        table, lens, refs = s["table"], s["lens"], s.get("refs")
        if "k" in s:
            s["kv"] = sv.KVPages(s["k"], s["v"], table, lens, refs)
        else:
            s["kv"] = sv.KVPagesQ4(s["k_qs"], s["v_qs"], s["k_scales"], s["v_scales"], table, lens, refs)
        if "digest" in s:
            s["dg"] = sv.KVDigest(s["digest"], s["case"]["block"], table, lens)
    return s["kv"]


def run(s):
    op = s["op"]
    if not own:
        return dict(commit=_plain_commit, attn=_plain_attn, scores=_plain_scores, select=_plain_select,
                    blocks=_plain_blocks)[op](s)
    import speculative_decoding_verification_round_gb300 as sv
    c = s["case"]
    n, nt = c["n_seq"], c["nt"]
    if op == "select":
        sv.spec_block_select(s["lens"], c["block"], n, s["slots"], nt, c["nkv"], s["scores"], c["keep"], s["blocks"],
                             s["status"], n_first=1, n_last=1)
        return s["blocks"], s["status"]
    kv = _handles(s, sv)
    if op == "commit":
        sv.spec_pages_q4_commit(kv, n, s["slots"], nt, s["k_new"], s["v_new"], s["path"], s["n_path"], s["status"],
                                new_len=s["new_len"])
        sv.spec_pages_q4_read(kv, n, s["slots"], nt, s["pos0"], s["n_path"], s["k_back"], s["v_back"], s["status_read"])
        return s["new_len"], s["status"], s["status_read"], s["k_back"], s["v_back"]
    if op == "attn":
        if "workspace" not in s:
            s["workspace"] = torch.empty(sv.spec_tree_attn_q4_workspace(kv, n, nt, c["nq"]), device="cuda",
                                         dtype=torch.uint8)
        sv.spec_tree_attn_q4(kv, 0, n, s["slots"], nt, c["nq"], s["q"], s["k_new"], s["v_new"], s["out"],
                             s["workspace"], s["status"], parents=s["parents"], n_nodes=s["n_nodes"],
                             window=c["window"], sinks=c["sinks"])
        return s["out"], s["status"]
    if op == "scores":
        sv.spec_block_digest(s["dg"], kv, n, s["slots"], s["status_digest"], pos0=s["pos0"])
        sv.spec_block_scores(s["dg"], 0, n, s["slots"], nt, c["nq"], s["q"], s["scores"], s["status"])
        return s["digest"], s["scores"], s["status"], s["status_digest"]
    sv.spec_block_attn(kv, 0, n, s["slots"], nt, c["nq"], c["block"], c["keep"], s["blocks"], s["q"], s["k_new"],
                       s["v_new"], s["out"], s["status"], parents=s["parents"], n_nodes=s["n_nodes"])
    return s["out"], s["status"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    c, op = case, case["op"]
    n, nt, nkv = c["n_seq"], c["nt"], c["nkv"]
    if op == "select":
        nb = -(-c["ctx"] // c["block"])
        return {"bytes": n * nt * nkv * 4.0 * (nb + min(nb, c["keep"])), "flops": 0}
    hd = c["hd"]
    row4, row16 = hd / 2 + hd / 16, 2 * hd  # bytes of a head's row in 4 bits, in fp16
    if op == "commit":  # fp16 in, 4 bits out; 4 bits in, fp16 out
        rows = n * ((nt + 1) // 2 if c["path"] else nt - nt // 16) * c["layers"] * nkv * 2
        return {"bytes": 2.0 * rows * (row16 + row4), "flops": 0}
    nodes = n * (nt - (nt // 8 if c.get("ragged") else 0))
    ends = nodes * (2.0 * nkv * row16 + 2.0 * c["nq"] * row16)  # the nodes' rows, queries and results
    short = c["ctx"] // 16 if c.get("ragged") else 0
    if op == "attn":
        seen = c["ctx"] - short
        if c["window"] > 0:
            seen = min(seen, c["window"] + c["sinks"])
        return {"bytes": n * seen * nkv * 2.0 * row4 + ends,
                "flops": 4.0 * nodes * c["nq"] * hd * (seen + nt / 2)}
    row = row4 if c["q4"] else row16
    if op == "scores":
        nb = -(-c["ctx"] // c["block"])
        fresh = min(c["ctx"], c["new"] + c["block"])
        return {"bytes": n * nkv * (fresh * float(row) + 2.0 * row16 * nb + nt * nb * 4.0) + nodes * c["nq"] * 2.0 * hd,
                "flops": 4.0 * nodes * c["nq"] * hd * nb}
    keys = min(c["ctx"] - short, c["keep"] * c["block"])
    # the lists of a sequence's nodes may name the same blocks: no block need be read twice
    return {"bytes": n * nkv * min(nt * keys, c["ctx"] - short) * 2.0 * row + ends + nodes * nkv * c["keep"] * 4.0,
            "flops": 4.0 * nodes * c["nq"] * hd * (keys + nt / 2)}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------


def _exact_rows(codes, scales):
    """The codes' values in 64 bits."""
    out = torch.empty(scales.shape + (32,), dtype=torch.float64, device=codes.device)
    out[..., :16] = (codes % 16).double()
    out[..., 16:] = torch.div(codes, 16, rounding_mode="floor").double()
    return ((out - 8.0) * scales.double().unsqueeze(-1)).reshape(scales.shape[:-1] + (-1,))


def _exact_commit(s):
    c = s["case"]
    for b in range(c["n_seq"]):
        slot, m = int(s["slots"][b]), int(s["n_path"][b])
        s["new_len"][slot] = int(s["lens"][slot]) + m
        node = list(range(m)) if s["path"] is None else s["path"][b, :m].tolist()
        for which in ("k", "v"):
            x = s[which + "_new"][:, b, node].double().unflatten(-1, (-1, 32))
            most = x.abs().max(-1, keepdim=True).values
            first = (x.abs() == most).int().argmax(-1, keepdim=True)
            d = -torch.gather(x, -1, first) / 8.0
            # eight significant bits, nothing below 2^-24
            step = torch.exp2(torch.floor(torch.log2(d.abs().clamp(min=1e-300))) - 7.0)
            d = torch.round(torch.round(d / step) * step * 2.0 ** 24) / 2.0 ** 24
            d = d.clamp(-8160.0, 8160.0)
            q = torch.where(d == 0, 0.0, torch.round(x / torch.where(d == 0, 1.0, d)).clamp(-8, 7))
            s[which + "_back"][:, b, :m] = (q * d).flatten(-2).to(torch.float16)
    return s["new_len"], s["status"], s["status_read"], s["k_back"].double(), s["v_back"].double()


def _exact_ctx(s, which, slot, h, pos):
    """Rows of one head at the positions `pos` of a slot, in 64 bits."""
    pg, at = s["table"][slot, pos // s["case"]["page"]].long(), pos % s["case"]["page"]
    if which in s:
        return s[which][0, pg, h, at].double()
    return _exact_rows(s[which + "_qs"][0, pg, h, at], s[which + "_scales"][0, pg, h, at])


def _paths(parents):
    chain = []
    for i, up in enumerate(parents):
        chain.append(([] if up < 0 else chain[up]) + [i])
    return chain


def _exact_attn(s):
    c = s["case"]
    out, g, cached = s["out"].double(), c["nq"] // c["nkv"], s["op"] == "attn"
    if c["n_seq"] * c["nt"] * c["nkv"] > 8192:
        return None, torch.zeros_like(s["status"])
    for b in range(c["n_seq"]):
        slot, m = int(s["slots"][b]), int(s["n_nodes"][b])
        ln = int(s["lens"][slot])
        chain = _paths(s["parents"][b].tolist())
        every = torch.arange(ln, device="cuda")
        for h in range(c["nkv"]):
            kn, vn = s["k_new"][b, :m, h].double(), s["v_new"][b, :m, h].double()
            if cached:
                k, v = _exact_ctx(s, "k", slot, h, every), _exact_ctx(s, "v", slot, h, every)
            for i in range(m):
                nodes = torch.tensor(chain[i], device="cuda")
                if cached:
                    at = ln + len(chain[i]) - 1
                    near = lambda p: (p < c["sinks"]) | (p > at - c["window"]) if c["window"] > 0 else p >= 0  # noqa: E731
                    old = near(every)
                    nodes = nodes[near(ln + torch.arange(len(chain[i]), device="cuda"))]
                    ki, vi = (k, v) if c["window"] == 0 else (k[old], v[old])
                else:
                    b0 = s["blocks"][b, i, h].long()
                    pos = (b0[b0 >= 0][:, None] * c["block"] + torch.arange(c["block"], device="cuda")).flatten()
                    pos = pos[pos < ln]
                    ki, vi = _exact_ctx(s, "k", slot, h, pos), _exact_ctx(s, "v", slot, h, pos)
                q = s["q"][b, i, h * g:(h + 1) * g].double()
                x = torch.cat([q @ ki.T, q @ kn[nodes].T], 1) / math.sqrt(c["hd"])
                p = torch.softmax(x, 1)
                out[b, i, h * g:(h + 1) * g] = p[:, :ki.shape[0]] @ vi + p[:, ki.shape[0]:] @ vn[nodes]
    return out, torch.zeros_like(s["status"])


def _exact_scores(s):
    c = s["case"]
    block, per = c["block"], c["page"] // c["block"]
    scores, dig, g = s["scores"].double(), s["digest"].double(), c["nq"] // c["nkv"]
    for b in range(c["n_seq"]):
        slot = int(s["slots"][b])
        ln = int(s["lens"][slot])
        for h in range(c["nkv"]):
            first = int(s["pos0"][b]) // block
            k = _exact_ctx(s, "k", slot, h, torch.arange(first * block, ln, device="cuda"))
            whole = k.shape[0] // block
            lo, hi = [], []
            if whole:
                part = k[:whole * block].view(whole, block, -1)
                lo, hi = [part.min(1).values], [part.max(1).values]
            if k.shape[0] % block:
                lo.append(k[whole * block:].min(0, keepdim=True).values)
                hi.append(k[whole * block:].max(0, keepdim=True).values)
            if lo:
                j = torch.arange(first, first + sum(x.shape[0] for x in lo), device="cuda")
                pg = s["table"][slot, j // per].long()
                dig[0, pg, h, j % per, 0], dig[0, pg, h, j % per, 1] = torch.cat(lo), torch.cat(hi)
            j = torch.arange(-(-ln // block), device="cuda")
            d = dig[0, s["table"][slot, j // per].long(), h, j % per]
            for i in range(c["nt"]):
                q = s["q"][b, i, h * g:(h + 1) * g].double()
                top = [torch.maximum(q[e] * d[:, 0], q[e] * d[:, 1]).sum(1) for e in range(g)]
                scores[b, i, h, :j.shape[0]] = torch.stack(top).max(0).values
    return dig, scores, s["status"], s["status_digest"]


def _exact_select(s):
    import numpy as np
    c = s["case"]
    x, lens, slots = s["scores"].cpu().numpy(), s["lens"].tolist(), s["slots"].tolist()
    out = np.full(tuple(s["blocks"].shape), -1, np.int32)
    for b in range(c["n_seq"]):
        nb = -(-lens[slots[b]] // c["block"])
        for i in range(c["nt"]):
            for h in range(c["nkv"]):
                ids = list(range(nb))
                if nb > c["keep"]:
                    order = 1 + np.argsort(-x[b, i, h, 1:nb - 1], kind="stable")
                    ids = sorted([0, nb - 1] + order[:c["keep"] - 2].tolist())
                out[b, i, h, :len(ids)] = ids
    return torch.from_numpy(out).cuda(), s["status"]


def exact(case, seed):
    s = prepare(case, seed)
    return dict(commit=_exact_commit, attn=_exact_attn, scores=_exact_scores, select=_exact_select,
                blocks=_exact_attn)[case["op"]](s)
