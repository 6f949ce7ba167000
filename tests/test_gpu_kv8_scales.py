"""The paged 8-bit cache's attention where pages' scales lie far apart: a row's result is as good as the pages that
it sees allow, whatever other pages its tile holds.

Bounds, per element, on top of test_gpu_kv8.py's (d 2^-23 s on a logit, 2^-11 on a probability, half a step of the
output).  P enters the products as FP16, whose subnormals are off by 2^-25 at most:

* taken by up to 64 rows, and by more where scales lie far apart: P carries its page's V scale, and the row's
  largest product u = max p 2^e enters at 2^11 or above: 2^-36 u a token;
* more than 64 rows and V scales up to 2^12 apart: the largest p enters at 2^9 or above: 2^-34 max p a token, times
  the token's 2^e.

Each acts on codes up to 448.  A logit's own sums are taken relative to s, the row's largest scale * sum |q k|."""
import numpy as np
import pytest
import torch

import mixed_precision_bit_quant_b200 as mq
from oracle import kv8
from oracle.formats import e4m3_encode
from test_gpu_kv8 import DT, _i32, _np, _pool

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
NEAR = 12  # V scales this many binades apart stay with the many-rows kernel


def _reference(pool, q, table, lens, cu, window, sinks, near):
    """o, lse, w and their bounds (without the output's own rounding)."""
    n, Hq, d = q.shape
    Hkv, page = pool["k"].shape[1:3]
    B, G = len(lens), Hq // Hkv
    o, ob, lse, lb = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    w, wb = np.zeros((B, Hkv, max(lens))), np.zeros((B, Hkv, max(lens)))
    for b in range(B):
        L, k = lens[b], cu[b + 1] - cu[b]
        at = table[b][np.arange(L) // page]
        for h in range(Hkv):
            K, V = kv8.tokens(pool, "k", table[b], L, h), kv8.tokens(pool, "v", table[b], L, h)
            e2 = np.ldexp(1.0, pool["vs"][at, h].astype(int) - 127)
            for i in range(k):
                see = kv8.visible(L - k + i, L, window, sinks)
                if not see.any():
                    continue
                Ks, Vs, es = K[see], V[see], e2[see]
                for j in range(h * G, (h + 1) * G):
                    r = cu[b] + i
                    x = Ks @ q[r, j] / np.sqrt(d)
                    m = x.max()
                    p = np.exp(x - m)
                    lse[r, j] = m + np.log(p.sum())
                    p /= p.sum()
                    delta = (d + 2) * 2.0 ** -23 * (np.abs(Ks) @ np.abs(q[r, j])).max() / np.sqrt(d) + 2.0 ** -22 * abs(lse[r, j])
                    rel = 2 * delta + 2.0 ** -21
                    T = see.sum()
                    small = 2.0 ** -36 * (p * es).max() * T + (2.0 ** -34 * p.max() * es.sum() if near else 0.0)
                    o[r, j] = p @ Vs
                    ob[r, j] = (2.0 ** -11 + rel + T * 2.0 ** -23) * (p @ np.abs(Vs)) + 448 * small
                    lb[r, j] = delta + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r, j])
                    w[b, h, :L][see] += p
                    # under the smallest normal number a weight may count as nothing
                    wb[b, h, :L][see] += (rel + 2.0 ** -21) * p + 2.0 ** -125
    return o, ob, lse, lb, w, wb


def _run(Hq, Hkv, d, page, lens, news, ke, ve, window=0, sinks=0, dtype="bf16", seed=0, light=0.0, weights=True, zero=()):
    """ke, ve: exponents (plus 127) of a sequence's pages in order, repeated; light: the logits (natural) of the pages
    whose V is not of the smallest scale, about; zero: pages of zero codes.  K's pages of far larger scale have
    their values in one channel, where the queries are 0: logits of 2^20 and more would mean nothing in FP32."""
    B, cols = len(lens), -(-max(lens) // page)
    table = np.random.default_rng(seed).permutation(B * cols).reshape(B, cols)
    cache = _pool(B * cols, Hkv, page, d, seed)
    r = np.random.default_rng(seed + 1)
    pool = _np(cache)
    for b, n in enumerate(lens):
        for c in range(-(-n // page)):
            m, pg = min(page, n - c * page), table[b, c]
            for f, e in (("k", ke), ("v", ve)):
                pool[f][pg, :, :m] = e4m3_encode(r.normal(size=(Hkv, m, d)) * 60)
                pool[f + "s"][pg] = e[c % len(e)]
            if ke[c % len(ke)] > min(ke) + 12:
                pool["k"][pg, ..., 1:] &= 0x80
            if light and ve[c % len(ve)] > min(ve):
                val = light / np.sqrt(d) * (1 + 0.01 * r.normal(size=(Hkv, m, d)))
                pool["k"][pg, :, :m] = e4m3_encode(np.ldexp(val, 127 - ke[c % len(ke)]))
            if c in zero:
                pool["k"][pg], pool["v"][pg] = 0, 0
    for f in pool:
        getattr(cache, f).copy_(torch.from_numpy(pool[f]))
    cu = [0]
    for x in news:
        cu.append(cu[-1] + x)
    q = torch.randn((cu[-1], Hq, d), generator=torch.Generator().manual_seed(seed + 2))
    q = (1 + 0.01 * q if light else q).to(DT[dtype])
    if max(ke) > min(ke) + 12:
        q[..., 0] = 0
    w = torch.zeros((B, Hkv, cols * page), device="cuda") if weights else None
    o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news), window=window,
                              sinks=sinks, weights=w, want_lse=True)
    assert mq.device_status() == (0, 0)
    live = [x for x in ve if x > 0] or [0]
    many = max(news) * (Hq // Hkv) > 64
    # (an exponent of -127 marks values below 2^-118, which count as zero beside pages of ordinary scale)
    ro, ob, rl, lb, rw, wb = _reference(pool, q.double().numpy(), table, lens, cu, window, sinks,
                                        many and max(live) - min(live) <= NEAR)
    go, gl = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(go - ro) <= HALF[dtype] * np.abs(ro) + 1.01 * ob + 2.0 ** -110)
    assert not bad.any(), (bad.mean(), np.argwhere(bad)[:3], go[bad][:3], ro[bad][:3])
    bad = ~((np.abs(gl - rl) <= lb) | (np.isneginf(gl) & np.isneginf(rl)))
    assert not bad.any(), (bad.mean(), gl[bad][:3], rl[bad][:3])
    if weights:
        bad = ~(np.abs(w.cpu().numpy()[..., :max(lens)] - rw) <= wb + 2.0 ** -22 * rw)
        assert not bad.any(), (bad.mean(), np.argwhere(bad)[:3])


ROWS = [  # Hq, Hkv, d, page, lens, news: few rows, several tiles of them, many
    (4, 1, 64, 16, [192], [1]), (4, 1, 128, 16, [190], [16]), (8, 2, 64, 32, [300, 100], [7, 5]),
    (4, 1, 64, 16, [192], [192]), (4, 1, 128, 16, [187], [187]), (6, 2, 64, 16, [400, 130], [390, 130]),
    (4, 1, 64, 16, [3000], [1]), (8, 2, 128, 16, [2500, 1900], [5, 1]), (4, 1, 128, 64, [700], [300])]
GAPS = [5, 12, 13, 21, 22, 25, 31, 40, 90]


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,news", ROWS)
@pytest.mark.parametrize("gap", GAPS)
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_rows_that_see_only_pages_of_small_scale(Hq, Hkv, d, page, lens, news, gap, which):
    """Non-zero pages 2^gap apart: causal rows before the first large page, and rows whose window lies between them."""
    n = -(-max(lens) // page)
    s, g = 118, 118 + gap
    for order, window, sinks in (([s] * (n // 2) + [g] * n, 0, 0), ([g] + [s] * (n - 1), 20, 0), ([s, g, s], 9, 0),
                                 ([g, s, s, s], 24, 1)):
        flat = [119] * len(order)
        _run(Hq, Hkv, d, page, lens, news, order if which != "v" else flat, order if which != "k" else flat,
             window=window, sinks=sinks, seed=gap)


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,news", ROWS)
@pytest.mark.parametrize("gap", [8, 12, 13, 20, 30, 40, 60])
def test_small_weights_on_pages_of_large_scale(Hq, Hkv, d, page, lens, news, gap):
    """The V of some pages is 2^gap larger and their weights 2^-gap smaller: both count in the output."""
    for ve in ([118, 118 + gap], [118 + gap, 118, 118]):
        _run(Hq, Hkv, d, page, lens, news, [121], ve, light=-gap * np.log(2.0), seed=gap)


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,news", [
    (4, 1, 64, 16, [6500], [1]), (8, 1, 128, 16, [6500], [3]),      # shares of all tiles, joined afterwards
    (16, 8, 64, 64, [600, 600], [600, 600])])                       # as many tiles of rows as SMs: no runs to join
@pytest.mark.parametrize("gap", [13, 40])
def test_long_calls_with_pages_of_far_scales(Hq, Hkv, d, page, lens, news, gap):
    s, g = 118, 118 + gap
    _run(Hq, Hkv, d, page, lens, news, [119], [s, s, s, g], seed=1)
    _run(Hq, Hkv, d, page, lens, news, [s, s, s, g, s], [s, g, s, s], window=40, sinks=3, seed=2)
    _run(Hq, Hkv, d, page, lens, news, [121], [s, g, s], light=-gap * np.log(2.0), seed=3)


@pytest.mark.parametrize("news", [[1], [16], [180]])
@pytest.mark.parametrize("small", [0, 1, 2])
def test_the_smallest_scales(news, small):
    """Pages of zeros and of values near the smallest beside ordinary ones, and a cache of nothing else."""
    _run(4, 1, 64, 16, [190], news, [118, small, 119], [small, 119, 118], seed=3, zero=(0, 4))
    _run(4, 1, 64, 16, [190], news, [small, 118], [119, small, 118], window=17, seed=4, zero=(1, 5))
    _run(4, 1, 64, 16, [190], news, [small], [small], seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_repeats_are_equal(dtype):
    """The same call again gives the same bits, runs that are joined and pages of far scales included."""
    B, Hq, Hkv, d, page, lens = 2, 8, 2, 64, 16, [900, 700]
    cols = 57
    table = np.random.default_rng(0).permutation(B * cols).reshape(B, cols)
    cache = _pool(B * cols, Hkv, page, d, 0, nan=False)
    q = torch.randn((400, Hq, d), generator=torch.Generator().manual_seed(1)).to(DT[dtype]).cuda()
    for far in (False, True):
        if far:
            cache.vs[::3] = 90
        for cu in ([0, 200, 400], [0, 1, 4]):
            runs = []
            for _ in range(4):
                w = torch.zeros((B, Hkv, cols * page), device="cuda")
                o, lse = mq.kv8_attention(q[:cu[-1]], cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(cu[1], cu[2] - cu[1]),
                                          weights=w, want_lse=True)
                runs.append((o, lse, w))
            assert mq.device_status() == (0, 0)
            for r in runs[1:]:
                assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_a_captured_chunk_follows_the_scales_and_two_streams_do_not_meet():
    """Whether scales lie far apart is decided when a call runs: one capture, replayed with other scales; and the
    calls of two streams at once, each with its own workspace, as those alone."""
    Hq, Hkv, d, page, L, n = 8, 2, 128, 16, 700, 150
    cols = -(-L // page)
    table = np.random.default_rng(0).permutation(cols)[None]
    cache = _pool(cols, Hkv, page, d, 0, nan=False)
    near = cache.vs.clone()
    far = near.clone()
    far[torch.from_numpy(table[0, 1::3]).cuda()] = 60
    q = torch.randn((n, Hq, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    t, ln, cu = _i32(table), _i32([L]), _i32([0, n])
    size = mq.kv8_attention_workspace(q, cache, t, ln, cu=cu, weights=torch.zeros((1, Hkv, cols * page), device="cuda"))

    def make():
        return (torch.zeros((1, Hkv, cols * page), device="cuda"), torch.zeros_like(q), torch.zeros((n, Hq), device="cuda"),
                torch.empty(size, dtype=torch.uint8, device="cuda"))

    def call(w, o, lse, ws):
        w.zero_()
        mq.kv8_attention(q, cache, t, ln, cu=cu, weights=w, o=o, lse=lse, ws=ws)
    alone = []
    for s in (near, far):
        cache.vs.copy_(s)
        alone.append(make())
        call(*alone[-1])
    torch.cuda.synchronize()
    assert not torch.equal(alone[0][1], alone[1][1])
    streams, got = [torch.cuda.Stream() for _ in range(2)], [make(), make()]
    for st, x in zip(streams, got):
        with torch.cuda.stream(st):
            call(*x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*got[0])
    for i in (0, 1, 0, 1):
        cache.vs.copy_((near, far)[i])
        torch.cuda.synchronize()
        for x in got[0]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[0][:3], alone[i][:3]))
        for _ in range(5):
            for st, x in zip(streams, got):
                with torch.cuda.stream(st):
                    call(*x)
        torch.cuda.synchronize()
        for x in got:
            assert all(torch.equal(a, b) for a, b in zip(x[:3], alone[i][:3]))
    assert mq.device_status() == (0, 0)
