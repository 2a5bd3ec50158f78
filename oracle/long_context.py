"""Plain reference of the operators for long contexts, in 64 bits: the 4-bit
format of a cache's rows, the digests of its blocks, their scores and the
selection among them.  Shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------------------
# 4 bits
# ---------------------------------------------------------------------------
def block_scale(m):
    """The scale of a block whose element of the largest magnitude is m: -m / 8
    with eight significant bits (to even), on fp16's grid, at most 8160, 0 without a sign."""
    d = -float(m) / 8.0
    if d == 0.0:
        return 0.0
    mant, ex = math.frexp(abs(d))                      # mant in [1/2, 1)
    r = math.ldexp(_even(mant * 256.0), ex - 8)        # eight bits
    if r < 2.0 ** -14:                                 # fp16's subnormal grid
        r = _even(r * 2.0 ** 24) * 2.0 ** -24
    return math.copysign(min(r, 8160.0), d) if r != 0.0 else 0.0


def _even(x):
    """The nearest whole number, ties to even."""
    f = math.floor(x)
    r = x - f
    return f + (1 if r > 0.5 or (r == 0.5 and f % 2 == 1) else 0)


def quantise(x):
    """[..., hd] fp16 -> q [..., hd] whole numbers of [-8, 7] and scales [..., hd / 32]."""
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, 32)
    q, s = np.zeros(flat.shape, np.int64), np.zeros(flat.shape[0])
    for i, b in enumerate(flat):
        if not np.isfinite(b).all():
            s[i] = math.nan
            continue
        s[i] = block_scale(b[int(np.argmax(np.abs(b)))])  # (the first of several)
        if s[i] != 0.0:
            q[i] = [min(7, max(-8, _even(v / s[i]))) for v in b]
    return q.reshape(x.shape), s.reshape(x.shape[:-1] + (-1,))


def pack(q, scales):
    """Codes uint8 [..., hd / 32, 16] and scales fp16 [..., hd / 32] of a cache's planes."""
    u = (np.asarray(q) + 8).astype(np.uint8).reshape(q.shape[:-1] + (-1, 32))
    return u[..., :16] | (u[..., 16:] << 4), np.asarray(scales).astype(np.float16)


def values(codes, scales):
    """[..., hd] in 64 bits of what codes and scales stand for."""
    codes = np.asarray(codes)
    u = np.concatenate([codes & 15, codes >> 4], -1).astype(np.float64) - 8.0
    with np.errstate(invalid="ignore"):
        v = u * np.asarray(scales, np.float64)[..., None]
    return v.reshape(v.shape[:-2] + (-1,))


# ---------------------------------------------------------------------------
# blocks
# ---------------------------------------------------------------------------
def digest(k):
    """[2][hd]: the least and the largest value of every channel of keys [n][hd]."""
    k = np.asarray(k, np.float64)
    return np.stack([k.min(0), k.max(0)])  # (a NaN spreads)


def score(q, d):
    """q [heads][hd] of one kv head, a block's digest [2][hd]: the largest bound of a
    head's logits, and the sum of magnitudes behind it."""
    q, d = np.asarray(q, np.float64), np.asarray(d, np.float64)
    with np.errstate(invalid="ignore"):
        x = np.maximum(q * d[0], q * d[1])
    return x.sum(-1).max(), np.abs(x).sum(-1).max()


def select(scores, nb, keep, first, last):
    """Ascending ids of nb blocks: the first, the last, and the largest-scored of the
    others (the lowest of equal ones; NaN as infinity)."""
    if nb <= keep:
        return list(range(nb))
    forced = [j for j in range(nb) if j < first or j >= nb - last]
    rest = [j for j in range(nb) if first <= j < nb - last]
    value = lambda j: math.inf if math.isnan(scores[j]) else float(scores[j])  # noqa: E731
    rest.sort(key=lambda j: (-value(j), j))
    return sorted(forced + rest[:keep - len(forced)])
