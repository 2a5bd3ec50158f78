"""oracle/long_context.py pinned by hand, and by properties of its definitions."""
import math

import numpy as np

from oracle import long_context as lc


def test_scales_have_eight_bits_and_are_fp16s():
    assert lc.block_scale(-8.0) == 1.0 and lc.block_scale(8.0) == -1.0 and lc.block_scale(0.0) == 0.0
    assert lc.block_scale(-8.0 * 255 / 256) == 255 / 256
    assert lc.block_scale(-8.0 * 511 / 512) == 1.0 and lc.block_scale(-8.0 * 509 / 512) == 254 / 256  # ties to even
    assert lc.block_scale(65504.0) == -8160.0
    assert lc.block_scale(-2.0 ** -21) == 2.0 ** -24 and lc.block_scale(-2.0 ** -22) == 0.0  # a tie below the smallest
    g = np.random.default_rng(0)
    for m in np.concatenate([g.standard_normal(500), np.exp2(g.uniform(-24, 15.9, 500))]).astype(np.float16):
        s = lc.block_scale(m)
        assert s == np.float64(np.float16(s)) and s == np.float64(np.float32(s))
        mant = math.frexp(s)[0] * 256
        assert mant == int(mant)
        q = np.arange(-8, 8) * s
        assert np.array_equal(q, q.astype(np.float16).astype(np.float64))  # every value is fp16's
        if abs(m) >= 2.0 ** -10:
            assert abs(abs(s) * 8 / abs(float(m)) - 1) <= 2.0 ** -8


def test_codes():
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 5, 64)).astype(np.float16)
    q, s = lc.quantise(x)
    assert q.min() >= -8 and q.max() <= 7
    codes, sc = lc.pack(q, s)
    v = lc.values(codes, sc)
    assert np.array_equal(v, q.reshape(3, 5, 2, 32).astype(np.float64).reshape(3, 5, 64) * np.repeat(s, 32, -1))
    # half a step, but for what the clamp at 7 cuts off: up to a step where the largest has the other sign
    err = np.abs(v - x).reshape(3, 5, 2, 32).max(-1)
    assert (err <= np.abs(s) * 1.04).all() and np.median(err / np.abs(s)) < 0.6
    assert codes.shape == (3, 5, 2, 16)
    assert codes[1, 2, 1, 3] == (q[1, 2, 32 + 3] + 8) | (q[1, 2, 32 + 19] + 8) << 4
    x[0, 0, 3], x[1, 1, 40] = np.inf, np.nan
    q, s = lc.quantise(x)
    assert np.isnan(s[0, 0, 0]) and np.isnan(s[1, 1, 1]) and np.isfinite(s[0, 0, 1]) and (q[0, 0, :32] == 0).all()
    # the first of several largest
    t = np.zeros(32, np.float16)
    t[4], t[9] = 2, -2
    assert lc.quantise(t)[1][0] == -0.25 and lc.quantise(-t)[1][0] == 0.25


def test_scores_bound_every_key_of_a_block():
    g = np.random.default_rng(2)
    k, q = g.standard_normal((16, 64)), g.standard_normal((4, 64))
    d = lc.digest(k)
    top, mag = lc.score(q, d)
    assert top >= (q @ k.T).max() and mag >= abs(top)
    assert lc.score(q, lc.digest(k[3:4]))[0] == (q @ k[3]).max() or math.isclose(
        lc.score(q, lc.digest(k[3:4]))[0], (q @ k[3]).max())


def test_selection():
    x = [5.0, 1.0, 7.0, 7.0, float("nan"), -1.0, 7.0, 0.0]
    assert lc.select(x, 8, 4, 1, 1) == [0, 2, 4, 7]
    assert lc.select(x, 8, 5, 1, 1) == [0, 2, 3, 4, 7]
    assert lc.select(x, 8, 3, 0, 0) == [2, 3, 4]
    assert lc.select(x, 5, 5, 1, 1) == [0, 1, 2, 3, 4] and lc.select(x, 0, 3, 1, 1) == []
    assert lc.select(x, 8, 2, 2, 0) == [0, 1]
