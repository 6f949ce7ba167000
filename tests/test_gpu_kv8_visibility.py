"""The paged 8-bit cache's attention and the pages that its rows do not see: entries of pages that a window
has left behind hold anything, and pages outside the pool count as not visible -- in the outputs and in the
weight sums, whatever number of rows picks the kernel.  Bounds as in test_gpu_kv8.py."""
import numpy as np
import pytest
import torch

import mixed_precision_bit_quant_b200 as mq
from oracle import kv8
from test_gpu_kv8 import DT, _check, _fill, _i32, _np, _pool, _tables

pytestmark = pytest.mark.gpu


def _call(cache, table, lens, news, Hq, w0, seed=1, dtype="bf16", **kw):
    cu = np.concatenate([[0], np.cumsum(news)])
    q = torch.randn((int(cu[-1]), Hq, cache.d), generator=torch.Generator().manual_seed(seed)).to(DT[dtype])
    w = torch.from_numpy(w0).float().cuda()
    o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news), weights=w,
                              want_lse=True, **kw)
    return q.double().numpy(), cu, o, lse, w


def _sums(B, Hkv, cols, seed):
    return np.random.default_rng(seed).random((B, Hkv, cols)).astype(np.float32).astype(np.float64)


# ------------------------------------------------- pages that a window has left behind
def _freed(table, lens, news, page, window, sinks, entry):
    """The table with `entry` in place of every page that no new token sees, and the tokens of those pages."""
    t, gone = table.copy(), []
    for b, (n, k) in enumerate(zip(lens, news)):
        for col in range(-(-n // page)):
            lo, hi = col * page, min(n, (col + 1) * page)
            if lo >= sinks and hi - 1 <= n - k - window:
                t[b, col] = entry
                gone.append((b, lo, hi))
    return t, gone


@pytest.mark.parametrize("page,d,lens,news,window,sinks", [
    (16, 64, [700, 517], [130, 70], 100, 5),     # a tile of 128 tokens holds pages that are seen and pages that are not
    (32, 128, [1000, 400], [65, 129], 40, 33),
    (64, 64, [900], [200], 150, 0),
    (16, 128, [3000], [1000], 17, 1),
    (16, 64, [700, 517], [1, 1], 100, 5),        # few rows: one cluster a unit
    (16, 64, [13001, 700], [3, 1], 300, 20),     # and shares of all tiles
])
@pytest.mark.parametrize("entry", ["pool", -1, 2 ** 31 - 1])
def test_entries_of_pages_left_behind_hold_anything(page, d, lens, news, window, sinks, entry):
    """A page of the pool whose codes are NaN and whose exponents are the largest stands in their place (a page that
    another sequence may be writing, or that nobody ever wrote), or no page at all."""
    B, Hq, Hkv = len(lens), 8, 2
    cols = -(-max(lens) // page) + 1
    table, P = _tables(lens, page, cols, 3)
    cache = _pool(P, Hkv, page, d, 3)
    _fill(cache, table, lens, 3)
    spare = sorted(set(range(P)) - set(table.reshape(-1).tolist()))[0]
    cache.k[spare], cache.v[spare] = 0x7F, 0xFF
    cache.ks[spare], cache.vs[spare] = 255, 255
    t, gone = _freed(table, lens, news, page, window, sinks, spare if entry == "pool" else entry)
    assert gone
    w0 = _sums(B, Hkv, cols * page, 4)
    q, cu, o, lse, w = _call(cache, t, lens, news, Hq, w0, window=window, sinks=sinks)
    ref = kv8.attend(_np(cache), q, table, lens, cu, window, sinks)
    _check(o, lse, w, w0, ref, d, max(lens), "bf16")
    got = w.cpu().numpy()
    for b, lo, hi in gone:  # not even rounded
        assert np.array_equal(got[b, :, lo:hi], w0[b, :, lo:hi].astype(np.float32))


# ------------------------------------------------- pages outside the pool
@pytest.mark.parametrize("page,d,lens,news,bad", [
    (16, 64, [1, 40, 20], [1, 1, 1], {0: [0], 1: [1]}),              # a padded slot; one page of three; a cluster a unit
    (16, 64, [16, 33], [2, 3], {0: [0], 1: [0, 1, 2]}),
    (64, 128, [7001, 64, 513], [1, 1, 1], {0: [3, 50], 1: [0]}),     # shares of all tiles, joined afterwards
    (32, 64, [6400, 32], [3, 2], {0: list(range(200)), 1: [0]}),     # nothing is left of either
    (64, 64, [300, 128, 90], [80, 128, 20], {0: [1], 1: [0, 1]}),    # many rows
    (16, 128, [1000, 16], [40, 16], {0: [0, 1, 2, 30, 62], 1: [0]}),
    (128, 64, [300], [300], {0: [0, 1, 2]}),
])
@pytest.mark.parametrize("number", [-1, 2 ** 31 - 1])
def test_pages_outside_the_pool_give_no_weight(page, d, lens, news, bad, number):
    B, Hq, Hkv = len(lens), 8, 2
    cols = -(-max(lens) // page)
    table, P = _tables(lens, page, cols, 5)
    cache = _pool(P, Hkv, page, d, 5)
    _fill(cache, table, lens, 5)
    for b, c in bad.items():
        table[b, c] = number
    w0 = _sums(B, Hkv, cols * page, 6)
    q, cu, o, lse, w = _call(cache, table, lens, news, Hq, w0)
    assert mq.device_status() == (1, 1 << 16)
    ref = kv8.attend(_np(cache), q, table, lens, cu)
    _check(o, lse, w, w0, ref, d, max(lens), "bf16")
    got = w.cpu().numpy()
    for b, c in bad.items():
        for col in c:
            lo, hi = col * page, min(lens[b], (col + 1) * page)
            assert np.array_equal(got[b, :, lo:hi], w0[b, :, lo:hi].astype(np.float32))
