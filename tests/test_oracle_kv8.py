"""Pins of the paged 8-bit cache's oracle: the exponent by its definition, the rounding by a
search over the grid, attention by closed forms, eviction by enumeration."""
import math

import numpy as np
import pytest

from oracle import kv8
from oracle.formats import e4m3_decode

GRID = np.sort(np.unique(e4m3_decode(np.arange(127))))  # the 127 finite magnitudes


def _pool(P, H, page, d, seed=0):
    r = np.random.default_rng(seed)
    c = {x: r.integers(0, 127, (P, H, page, d)).astype(np.uint8) for x in "kv"}
    return {**c, **{x + "s": r.integers(118, 124, (P, H)).astype(np.uint8) for x in "kv"}}


@pytest.mark.parametrize("x", [448.0, 448.0000001, 1.75, 1.7500001, 3.5 * 2.0 ** -120, 2.0 ** -133, 1e-30, 3e38])
def test_exponent_is_the_smallest(x):
    e = kv8.exponent(x)
    assert x <= 448.0 * 2.0 ** e or e > 127
    assert e == -127 or x > 448.0 * 2.0 ** (e - 1)


def test_append_rounds_to_the_nearest_code_and_again_when_the_exponent_rises():
    r = np.random.default_rng(1)
    pool = _pool(3, 2, 16, 8)
    x = r.normal(size=(10, 2, 8))
    kv8.append(pool, x, x * 3, [[2, 1]], [10], [0, 10])
    for h in range(2):
        e = int(pool["ks"][2, h]) - 127
        assert e == kv8.exponent(np.abs(x[:, h]).max())
        got = np.abs(np.ldexp(e4m3_decode(pool["k"][2, h, :10]), 0))
        want = np.abs(np.ldexp(x[:, h], -e))
        best = np.abs(want[..., None] - GRID).min(-1)
        assert np.array_equal(np.abs(want - got), best)
    was = np.ldexp(e4m3_decode(pool["k"][2, :, :10]), (pool["ks"][2].astype(int) - 127)[:, None, None])
    big = x[:7] * 64  # six tokens fill the page, one starts the next
    kv8.append(pool, big, big, [[2, 1]], [17], [0, 7])
    for h in range(2):
        e = int(pool["ks"][2, h]) - 127
        assert e == kv8.exponent(np.abs(big[:6, h]).max())
        again = np.abs(e4m3_decode(pool["k"][2, h, :10]))
        want = np.abs(np.ldexp(was[h], -e))
        assert np.array_equal(np.abs(want - again), np.abs(want[..., None] - GRID).min(-1))
        assert int(pool["ks"][1, h]) - 127 == kv8.exponent(np.abs(big[6:, h]).max())


def test_attention_closed_forms():
    pool = _pool(4, 1, 16, 4)
    table = [[3, 0, 1]]
    # zero queries: equal weights over the visible tokens
    q = np.zeros((3, 2, 4))
    r = kv8.attend(pool, q, table, [40], [0, 3], window=5, sinks=2)
    V = kv8.tokens(pool, "v", table[0], 40, 0)
    for i, p in enumerate((37, 38, 39)):
        see = [0, 1] + list(range(p - 4, p + 1))
        assert np.allclose(r["o"][i, 0], V[see].mean(0)) and math.isclose(r["lse"][i, 1], math.log(7))
    assert np.isclose(r["w"].sum(), 6)  # every row spends one
    # a token that outweighs the rest
    K = kv8.tokens(pool, "k", table[0], 40, 0)
    j = int(np.argmax(K[:, 0]))
    q[:] = 0
    q[2, 0, 0] = 1e6
    r = kv8.attend(pool, q, table, [40], [0, 3])
    top = np.flatnonzero(K[:, 0] == K[j, 0])
    assert np.allclose(r["o"][2, 0], V[top].mean(0))
    # more new tokens than the sequence holds: the first rows see nothing
    r = kv8.attend(pool, q, table, [1], [0, 3])
    assert np.all(r["o"][:2] == 0) and np.all(np.isneginf(r["lse"][:2])) and np.allclose(r["o"][2, 1], V[0])


def test_eviction_keeps_forced_tokens_and_the_largest_with_the_lowest_first():
    w = np.array([0, 5, 1, 5, 5, 2, 0, 0], dtype=np.float64)
    assert kv8.keep_set(w, 8, 4, 1, 1).tolist() == [0, 1, 3, 7]
    assert kv8.keep_set(w, 8, 2, 1, 1).tolist() == [0, 7]
    assert kv8.keep_set(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert kv8.keep_set(w, 8, 3, 0, 0).tolist() == [1, 3, 4]
    pool, dst = _pool(4, 2, 16, 4), _pool(2, 2, 16, 4, seed=9)
    r = np.random.default_rng(2)
    ww, dw = r.random((1, 2, 48)), np.ones((1, 2, 32))
    lens, kept = kv8.evict(pool, [[3, 0, 1]], [45], ww, dst, [[1, 0]], dw, 20, 2, 3)
    assert lens.tolist() == [20]
    for h in range(2):
        ids = kept[0, h]
        assert np.all(np.diff(ids) > 0) and ids[:2].tolist() == [0, 1] and ids[-3:].tolist() == [42, 43, 44]
        assert ww[0, h, ids[2:-3]].min() >= np.delete(ww[0, h, 2:42], ids[2:-3] - 2).max()
        old = kv8.tokens(pool, "v", [3, 0, 1], 45, h)[ids]
        new = kv8.tokens(dst, "v", [1, 0], 20, h)
        # rounding again costs at most half a step of the smallest e4m3 spacing at the page's exponent
        e = dst["vs"][[1] * 16 + [0] * 4, h].astype(int) - 127
        assert np.all(np.abs(old - new) <= np.ldexp(1.0, -10 + e)[:, None] + np.abs(old) * 2.0 ** -4)
        assert np.array_equal(dw[0, h, :20], ww[0, h, ids]) and not dw[0, h, 20:].any()


@pytest.mark.parametrize("number", [-1, 4, 2 ** 31 - 1])
def test_tokens_of_pages_outside_the_pool_are_not_visible(number):
    pool = _pool(4, 1, 16, 4)
    q = np.random.default_rng(3).normal(size=(3, 2, 4))
    r = kv8.attend(pool, q, [[3, number, 1]], [40], [0, 3])
    short = dict(pool)  # the same tokens without the page, as a sequence of 24
    for i, p in enumerate((37, 38, 39)):
        one = kv8.attend(short, q[i:i + 1], [[3, 1]], [p - 15], [0, 1])
        assert np.allclose(r["o"][i], one["o"][0]) and np.allclose(r["lse"][i], one["lse"][0])
    assert not r["w"][0, 0, 16:32].any() and np.isclose(r["w"].sum(), 6)
    r = kv8.attend(pool, q, [[number, number, number]], [40], [0, 3])
    assert np.all(r["o"] == 0) and np.all(np.isneginf(r["lse"])) and not r["w"].any()
