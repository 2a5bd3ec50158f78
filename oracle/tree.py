"""Plain reference of the drafted-tree operators, one step at a time and in
64 bits: attention of a tree over a cache (sliding window, sinks), the
bookkeeping of a paged cache, filtered sampling on the sampler's integer
weights, greedy acceptance along a tree.  Shares no code with the CUDA path.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

ST_SLOT, ST_PAGE, ST_SHARED, ST_FULL, ST_TREE = 1, 2, 4, 8, 16


# ---------------------------------------------------------------------------
# trees
# ---------------------------------------------------------------------------
def chains(parents):
    """Every node's path from its root, itself last."""
    out = []
    for i, p in enumerate(parents):
        assert -1 <= p < i
        out.append((out[p] if p >= 0 else []) + [i])
    return out


def visible(n_past, parents, i, window=0, sinks=0):
    """(cached positions, nodes) that node i sees."""
    paths = chains(parents)
    at = n_past + len(paths[i]) - 1
    near = lambda p: window == 0 or p < sinks or p > at - window  # noqa: E731
    return ([p for p in range(n_past) if near(p)],
            [j for j in paths[i] if near(n_past + len(paths[j]) - 1)])


def tree_attention(q, k, v, k_new, v_new, parents, window=0, sinks=0, scale=None):
    """q [nodes][nq][hd]; k, v [n_past][nkv][hd] the cached positions; k_new,
    v_new [nodes][nkv][hd].  Returns (out [nodes][nq][hd] fp64, the same with
    |v| for v, the largest sum of |q_d k_d| over the visible keys of a row)."""
    q, k, v, kn, vn = (np.asarray(a, np.float64) for a in (q, k, v, k_new, v_new))
    n, nq, hd = q.shape
    g = nq // kn.shape[1]
    scale = 1.0 / math.sqrt(hd) if scale is None else scale
    out, mag, dots = np.zeros_like(q), np.zeros_like(q), np.zeros((n, nq))
    for i in range(n):
        cached, nodes = visible(k.shape[0], parents, i, window, sinks)
        for h in range(nq):
            kk = np.concatenate([k[cached, h // g], kn[nodes, h // g]])
            vv = np.concatenate([v[cached, h // g], vn[nodes, h // g]])
            s = kk @ q[i, h] * scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h], mag[i, h] = p @ vv, p @ np.abs(vv)
            dots[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h]))
    return out, mag, dots


def accept_tree(argmax, tokens, parents):
    """(path, emitted) of one sequence's tree: both of the path's length."""
    path, emitted = [0], []
    while True:
        emitted.append(int(argmax[path[-1]]))
        for j in range(len(parents)):
            if parents[j] == path[-1] and tokens[j] == emitted[-1]:
                path.append(j)
                break
        else:
            return path, emitted


# ---------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------
class Book:
    """Tables, reference counts and lengths of a paged cache, and what each
    call does to them; `rows` maps (page, position in it) to what is stored
    there (anything)."""

    def __init__(self, n_slots, max_pages, n_pages, page):
        self.table = [[-1] * max_pages for _ in range(n_slots)]
        self.refs, self.len = [0] * n_pages, [0] * n_slots
        self.page, self.rows = page, {}

    def _slot(self, s):
        return 0 <= s < len(self.table)

    def fork(self, src, dst):
        status = []
        empty = [all(e < 0 for e in row) and n == 0 for row, n in zip(self.table, self.len)]
        for i, (a, b) in enumerate(zip(src, dst)):
            st = 0
            if not (self._slot(a) and self._slot(b)) or dst.count(b) > 1 or b in src or a in dst:
                st |= ST_SLOT
            elif not empty[b]:
                st |= ST_SLOT
            if st == 0:
                held = -(-self.len[a] // self.page)
                if any(not 0 <= e < len(self.refs) for e in self.table[a][:held]):
                    st |= ST_PAGE
            status.append(st)
        for a, b, st in zip(src, dst, status):
            if st == 0:
                held = -(-self.len[a] // self.page)
                self.table[b][:held] = self.table[a][:held]
                for e in self.table[a][:held]:
                    self.refs[e] += 1
                self.len[b] = self.len[a]
        return status

    def extend(self, slots, n_new):
        """(status, copies); moves the copied rows too."""
        status, plan = [], []
        left = list(self.refs)
        for s, add in zip(slots, n_new):
            st, need, copy = 0, [], None
            if not self._slot(s) or slots.count(s) > 1:
                st |= ST_SLOT
            elif add < 0 or self.len[s] < 0:
                st |= ST_PAGE
            elif -(-(self.len[s] + add) // self.page) > len(self.table[s]):
                st |= ST_FULL
            else:
                n, row = self.len[s], self.table[s]
                for e in range(n // self.page, -(-(n + add) // self.page)):
                    if e == n // self.page and n % self.page:
                        if not 0 <= row[e] < len(self.refs):
                            st |= ST_PAGE
                        elif add > 0 and left[row[e]] > 1:
                            copy = e
                    elif row[e] < 0:
                        need.append(e)
                    elif row[e] >= len(self.refs) or need:
                        st |= ST_PAGE
                    elif self.refs[row[e]] > 1:
                        st |= ST_SHARED
            if st == 0 and copy is not None:
                left[self.table[s][copy]] -= 1
            status.append(st)
            plan.append((copy, need) if st == 0 else (None, []))
        copies = [(-1, -1)] * len(slots)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        if sum((c is not None) + len(n) for c, n in plan) > len(free):
            return [st or ST_FULL for st in status], copies
        moves = []
        for i, (s, (copy, need)) in enumerate(zip(slots, plan)):
            if copy is not None:
                old, new = self.table[s][copy], free.pop(0)
                copies[i] = (old, new)
                moves += [((new, r), self.rows.get((old, r))) for r in range(self.len[s] % self.page)]
                self.refs[old] -= 1
                self.refs[new] = 1
                self.table[s][copy] = new
            for e in need:
                self.table[s][e] = free.pop(0)
                self.refs[self.table[s][e]] = 1
        self.rows.update(moves)
        return status, copies

    def commit(self, slots, path, n_path, value):
        """value(i, node): what row `node` of entry i holds."""
        status = []
        for i, s in enumerate(slots):
            st, nt = 0, len(path[i])
            if not self._slot(s) or slots.count(s) > 1:
                st |= ST_SLOT
            if not 0 <= n_path[i] <= nt:
                st |= ST_TREE
            if st == 0:
                n, m = self.len[s], n_path[i]
                if n + m > len(self.table[s]) * self.page:
                    st |= ST_FULL
                else:
                    held = {self.table[s][p // self.page] for p in range(n, n + m)}
                    if any(not 0 <= e < len(self.refs) for e in held):
                        st |= ST_PAGE
                    if any(0 <= e < len(self.refs) and self.refs[e] != 1 for e in held):
                        st |= ST_SHARED
                    if any(not 0 <= j < nt for j in path[i][:m]):
                        st |= ST_TREE
            status.append(st)
            if st == 0:
                for j, node in enumerate(path[i][:m]):
                    self.rows[(self.table[s][(n + j) // self.page], (n + j) % self.page)] = value(i, node)
                self.len[s] += m
        return status

    def free(self, slots):
        status = []
        for s in slots:
            if not self._slot(s) or slots.count(s) > 1:
                status.append(ST_SLOT)
                continue
            for e in self.table[s]:
                if e >= 0:
                    self.refs[e] -= 1
            self.table[s] = [-1] * len(self.table[s])
            self.len[s] = 0
            status.append(0)
        return status


# ---------------------------------------------------------------------------
# filtered sampling
# ---------------------------------------------------------------------------
def kept_tokens(logits, W, top_k=0, top_p=1.0, min_p=0.0):
    """The ids that stay, in the order (logit descending, id ascending).
    W: integer weights as Python or numpy integers."""
    logits = np.asarray(logits, np.float32)
    order = [int(v) for v in np.lexsort((np.arange(len(logits)), -logits)) if logits[v] > -np.inf]
    if top_k > 0:
        order = order[:top_k]
    P = int(math.floor(Fraction(float(np.float32(top_p))) * 2 ** 32))
    if P < 2 ** 32:
        total, before, keep = sum(int(W[v]) for v in order), 0, []
        for v in order:
            if keep and not before * 2 ** 32 < P * total:
                break
            keep.append(v)
            before += int(W[v])
        order = keep
    M = int(math.floor(Fraction(float(np.float32(min_p))) * 2 ** 32))
    return [v for v in order if int(W[v]) >= M]


def sample_row(logits, row_weights, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, kept ids in id order).  row_weights(logits, T): the integer
    weights and their sum (the rejection sampler's)."""
    logits = np.asarray(logits, np.float32)
    if T == 0.0:
        T, top_k = 1.0, 1
    finite = np.where(np.isfinite(logits), logits, np.finfo(np.float32).min).astype(np.float32)
    W, _ = row_weights(finite, T)
    W = np.where(np.isfinite(logits), W, 0).astype(np.uint64)
    ids = sorted(kept_tokens(logits, W, top_k, top_p, min_p))
    total = sum(int(W[v]) for v in ids)
    at, run = int(u) * total // 2 ** 32, 0
    for v in ids:
        run += int(W[v])
        if run > at:
            return v, ids
    raise AssertionError("no token")
