"""Oracle: the paged 8-bit KV cache -- append, attention, eviction (FP64).

TEST INFRASTRUCTURE (see ``oracle/formats.py``): only tests and the smoke check
use this module.

What it follows.  HyQuant: Hybrid-Precision Quantization for LLM Attention
(abstract, decode stage) decodes from a compressed cache and singles out sink
tokens, the local window and the tokens that many queries attend to.  The page
gives no formats or interfaces; the serving form is this library's:

* a pool of pages of ``page`` tokens, e4m3 codes, one exponent e per page, kv
  head and operand (stored as e + 127): value = code * 2^e;
* append: e is the smallest integer >= -127 with amax <= 448 * 2^e over the
  page's new tokens, at least the page's old e if it holds older tokens of the
  sequence, whose codes are then rounded again;
* attention: the query at position p sees t <= p and, under a window W,
  only t > p - W or t < sinks; exact softmax; a row that sees nothing gives 0 and -inf; a token
  whose page is outside the pool counts as not visible;
* eviction: the first ``sinks``, the last ``recent`` and the tokens with the
  largest weights (ties: the lower position) stay, in their order.

The pool is a dict of numpy arrays ``k, v [P, Hkv, page, d]`` and ``ks, vs
[P, Hkv]`` (uint8).  Parity pins: tests/test_oracle_kv8.py.
"""
from __future__ import annotations

import math

import numpy as np

from .formats import e4m3_decode, e4m3_encode


def exponent(amax: float) -> int:
    """Smallest integer e >= -127 with amax <= 448 * 2^e."""
    if amax <= 0:
        return -127
    m, x = math.frexp(float(amax))  # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    return max(-127, x - 9 + (1 if m > 0.875 else 0))


def append(pool, k, v, table, lens, cu):
    """Quantise packed rows k, v [n, Hkv, d] (float64) into ``pool`` (changed in place)."""
    page = pool["k"].shape[2]
    for b in range(len(lens)):
        q0, q1 = int(cu[b]), int(cu[b + 1])
        first = int(lens[b]) - (q1 - q0)
        pos = max(first, 0)
        while pos < lens[b]:
            col, lo = divmod(pos, page)
            hi = min(page, int(lens[b]) - col * page)
            pg = int(table[b][col])
            for codes, sc, x in ((pool["k"], pool["ks"], k), (pool["v"], pool["vs"], v)):
                new = x[q0 + pos - first:q0 + pos - first + hi - lo]
                for h in range(codes.shape[1]):
                    e = exponent(np.abs(new[:, h]).max())
                    if lo > 0:
                        old = int(sc[pg, h]) - 127
                        e = max(e, old)
                        codes[pg, h, :lo] = e4m3_encode(np.ldexp(e4m3_decode(codes[pg, h, :lo]), old - e))
                    codes[pg, h, lo:hi] = e4m3_encode(np.ldexp(new[:, h], -e))
                    sc[pg, h] = e + 127
            pos = col * page + hi


def tokens(pool, which, table_row, n, h):
    """[n, d] float64: the first n tokens of kv head h in K ("k") or V ("v")."""
    page, d = pool[which].shape[2:]
    out = np.empty((n, d))
    for col in range(-(-n // page)):
        pg, m = int(table_row[col]), min(page, n - col * page)
        if pg < 0 or pg >= pool[which].shape[0]:
            out[col * page:col * page + m] = np.nan
            continue
        out[col * page:col * page + m] = np.ldexp(e4m3_decode(pool[which][pg, h, :m]),
                                                  int(pool[which + "s"][pg, h]) - 127)
    return out


def visible(p: int, n: int, window: int, sinks: int) -> np.ndarray:
    t = np.arange(n)
    see = t <= p
    if window > 0:
        see &= (t > p - window) | (t < sinks)
    return see


def attend(pool, q, table, lens, cu, window=0, sinks=0, scale=0.0):
    """Packed queries q [n, Hq, d] (float64) -> dict: o, lse, the weight each token received
    w [B, Hkv, max len], and what error bounds are made of: a = sum p |v|, and s = the largest
    scale * sum |q_c k_c| of a row.  Rows of no sequence stay NaN."""
    n, Hq, d = q.shape
    Hkv = pool["k"].shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    o, a = np.full((n, Hq, d), np.nan), np.full((n, Hq, d), np.nan)
    lse, smax = np.full((n, Hq), np.nan), np.zeros((n, Hq))
    w = np.zeros((len(lens), Hkv, max(1, int(max(lens)))))
    for b in range(len(lens)):
        q0, q1, L = int(cu[b]), int(cu[b + 1]), int(lens[b])
        for h in range(Hkv if q1 > q0 else 0):
            K, V = tokens(pool, "k", table[b], L, h), tokens(pool, "v", table[b], L, h)
            pages = np.asarray(table[b])[np.arange(L) // pool["k"].shape[2]]
            held = (pages >= 0) & (pages < pool["k"].shape[0])
            for r in range(q0, q1):
                see = visible(L - (q1 - q0) + r - q0, L, window, sinks) & held
                for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    if not see.any():
                        o[r, j], a[r, j], lse[r, j] = 0.0, 0.0, -math.inf
                        continue
                    Ks, Vs = K[see], V[see]
                    s = Ks @ q[r, j] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    lse[r, j] = m + math.log(p.sum())
                    p /= p.sum()
                    o[r, j], a[r, j] = p @ Vs, p @ np.abs(Vs)
                    smax[r, j] = (np.abs(Ks) @ np.abs(q[r, j])).max() * scale
                    w[b, h, :L][see] += p
    return dict(o=o, lse=lse, w=w, a=a, s=smax)


def keep_set(w, n: int, keep: int, sinks: int, recent: int) -> np.ndarray:
    """The positions that stay of n tokens with weights w[:n]."""
    if n <= keep:
        return np.arange(n)
    free = sorted(range(sinks, n - recent), key=lambda t: (-float(w[t]), t))
    stay = list(range(sinks)) + free[:keep - sinks - recent] + list(range(n - recent, n))
    return np.array(sorted(stay), dtype=np.int64)


def evict(pool, table, lens, w, dst, dst_table, dst_w, keep, sinks, recent):
    """Fills ``dst`` and dst_w in place; returns (dst_lens, kept)."""
    B, Hkv = w.shape[:2]
    page = pool["k"].shape[2]
    kept = np.full((B, Hkv, keep), -1, dtype=np.int32)
    out = np.array([min(int(n), keep) for n in lens], dtype=np.int32)
    dst_w[:] = 0
    for b in range(B):
        for h in range(Hkv):
            ids = keep_set(w[b, h], int(lens[b]), keep, sinks, recent)
            kept[b, h, :len(ids)] = ids
            dst_w[b, h, :len(ids)] = w[b, h, ids]
            for j in range(-(-len(ids) // page)):
                part = ids[j * page:(j + 1) * page]
                src = np.array([int(table[b][t // page]) for t in part])
                dp = int(dst_table[b][j])
                for c, s in (("k", "ks"), ("v", "vs")):
                    e = pool[s][src, h].astype(np.int64)
                    codes = pool[c][src, h, part % page]
                    val = np.ldexp(e4m3_decode(codes), (e - e.max())[:, None])
                    dst[c][dp, h, :len(part)] = e4m3_encode(val)
                    dst[s][dp, h] = e.max()
    return out, kept
