"""GPU parity of the paged 8-bit cache (thrift_kv8_append, thrift_kv8_attn,
thrift_kv8_evict) and its FP64 oracle (oracle/kv8.py).

Codes, exponents, kept positions and lengths are compared bit for bit.  The
attention's bounds are derived here, per element, before any run:

* a product of d terms in FP32 is off by at most d 2^-23 sum |q_c k_c| (each step may
  truncate), so a logit by delta = d 2^-23 s + 2^-22 |logit| (s from the oracle; the second
  term is the scaling and the subtraction of the maximum), a probability relatively by
  2 delta + 2^-21 (its own logit, the sum's, the exponential);
* P is rounded to FP16: 2^-11 relative; the PV sum in FP32 over T terms adds T 2^-23;
  together they act on a = sum p |v|;
* the output's rounding is half a step: 2^-8 (BF16), 2^-11 (FP16) of the value.
"""
import numpy as np
import pytest
import torch

import mixed_precision_bit_quant_b200 as mq
from oracle import kv8
from oracle.formats import e4m3_encode

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _pool(P, Hkv, page, d, seed, nan=True):
    """A pool whose every slot holds garbage (NaN codes among it) and scales of several binades."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randint(0, 256, (P, Hkv, page, d), generator=g, dtype=torch.uint8) for _ in "kv")
    if not nan:
        for c in (k, v):
            c[(c & 127) == 127] = 1
    ks, vs = (torch.randint(116, 124, (P, Hkv), generator=g, dtype=torch.uint8) for _ in "kv")
    return mq.Kv8Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda())


def _np(cache):
    return {f: getattr(cache, f).cpu().numpy() for f in ("k", "v", "ks", "vs")}


def _fill(cache, table, lens, seed, spread=1.0):
    """Real codes for the tokens of the sequences (normal values at each page's scale); the rest stays garbage."""
    r = np.random.default_rng(seed)
    page, d = cache.page, cache.d
    for c in (cache.k, cache.v):
        h = c.cpu().numpy()
        for b, n in enumerate(lens):
            for col in range(-(-n // page)):
                m = min(page, n - col * page)
                h[table[b][col], :, :m] = e4m3_encode(r.normal(size=(cache.Hkv, m, d)) * 60 * spread)
        c.copy_(torch.from_numpy(h))


def _tables(lens, page, cols, seed, spare=3):
    need = [-(-n // page) for n in lens]
    perm = np.random.default_rng(seed).permutation(sum(need) + spare)
    table = np.full((len(lens), cols), 2 ** 31 - 1, dtype=np.int64)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, sum(need) + spare


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _check(got_o, got_lse, got_w, w0, ref, d, T, dtype, rows=None):
    hs = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype]
    delta = d * 2.0 ** -23 * ref["s"] + 2.0 ** -22 * np.abs(np.nan_to_num(ref["lse"], neginf=0.0)) + 2.0 ** -22 * ref["s"]
    rel = 2 * delta + 2.0 ** -21
    live = ~np.isnan(ref["lse"])
    o, lse = got_o.float().cpu().numpy().astype(np.float64), got_lse.cpu().numpy().astype(np.float64)
    bound = hs * np.abs(ref["o"]) + (2.0 ** -11 + rel + T * 2.0 ** -23)[..., None] * ref["a"] * 1.01 + 2.0 ** -24
    bad = np.abs(o - ref["o"]) > bound
    assert not bad[live].any(), (np.abs(o - ref["o"])[live].max(), bad[live].mean())
    fin = live & np.isfinite(ref["lse"])
    assert np.array_equal(np.isneginf(lse[live]), np.isneginf(ref["lse"][live]))
    assert (np.abs(lse[fin] - ref["lse"][fin]) <= (delta + 2.0 ** -20)[fin] + 2.0 ** -22 * np.abs(ref["lse"][fin])).all()
    if got_w is not None:
        w = got_w.cpu().numpy().astype(np.float64)
        want = w0.copy()
        want[..., :ref["w"].shape[-1]] += ref["w"]
        tol = (rel[live].max() if live.any() else 0.0) * ref["w"] + 2.0 ** -21 * ref["w"] + 2.0 ** -23 * np.abs(
            want[..., :ref["w"].shape[-1]])
        assert (np.abs(w - want)[..., :ref["w"].shape[-1]] <= tol).all()
        assert np.array_equal(w[..., ref["w"].shape[-1]:], want[..., ref["w"].shape[-1]:])
    assert mq.device_status() == (0, 0)


def _attend(Hq, Hkv, d, page, lens, news, dtype="bf16", window=0, sinks=0, weights=False, seed=0, gap=0, cols=None,
            max_len=None, q_scale=1.0, spread=1.0, pool_scale=None):
    B = len(lens)
    cols = cols or -(-max(lens + [1]) // page) + 1
    table, P = _tables(lens, page, cols, seed)
    cache = _pool(P, Hkv, page, d, seed)
    _fill(cache, table, lens, seed, spread)
    cu = [gap]
    for n in news:
        cu.append(cu[-1] + n)
    n = cu[-1] + 2 * gap
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((n, Hq, d), generator=g) * q_scale).to(DT[dtype])
    w = torch.rand((B, Hkv, cols * page), generator=g).cuda() if weights else None
    w0 = None if w is None else w.cpu().numpy().astype(np.float64)
    o = torch.full((n, Hq, d), 7.0, dtype=DT[dtype], device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news), max_len=max_len,
                     window=window, sinks=sinks, weights=w, o=o, lse=lse)
    ref = kv8.attend(_np(cache), q.double().numpy(), table, lens, cu, window, sinks)
    _check(o, lse, w, w0, ref, d, max(lens + [1]), dtype)
    idle = np.isnan(ref["lse"])
    assert (o.cpu()[torch.from_numpy(idle)] == 7).all() and (lse.cpu()[torch.from_numpy(idle)] == 7).all()


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("Hq,Hkv,d,page,lens,news", [
    (1, 1, 64, 16, [1], [1]),                       # one token
    (4, 4, 128, 16, [0, 1, 15, 16, 17], [1, 1, 1, 1, 1]),   # an empty sequence (its row sees nothing), page edges
    (8, 2, 128, 64, [63, 64, 65, 129, 517], [1] * 5),
    (6, 2, 64, 32, [100, 31, 33], [1, 0, 1]),       # a sequence with nothing new
    (16, 1, 128, 128, [700, 128], [1, 1]),          # 16 heads a group
    (10, 2, 64, 16, [300], [3]),                    # groups of 5, 15 rows
    (7, 1, 128, 64, [130, 40], [2, 5]),             # 35 rows: several tiles of rows
    (8, 8, 64, 16, [40, 3], [40, 5]),               # a whole prompt; more new tokens than the length holds
    (3, 1, 128, 32, [257], [129]),
    (12, 12, 64, 64, [197, 197], [197, 197]),       # the vit sizes, causal
    (4, 2, 128, 64, [1000, 2049], [150, 70]),
    (32, 8, 128, 64, [4097], [1]),                  # many runs
    # sequences too long for a cluster: shares of all tiles, units cut at any place
    (6, 2, 64, 32, [7001, 0, 513], [1, 1, 1]),
    (16, 1, 128, 128, [6400], [1]),
    (7, 1, 128, 64, [6300, 40, 16], [2, 5, 0]),
    (20, 2, 64, 16, [6401, 900], [3, 4]),
])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention(Hq, Hkv, d, page, lens, news, dtype):
    _attend(Hq, Hkv, d, page, lens, news, dtype, seed=len(lens) * 7 + d)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 16), (33, 4), (64, 0), (100, 17), (300, 64),
                                          (10 ** 6, 3), (2 ** 31 - 1, 2 ** 31 - 1), (40, 10 ** 6)])
@pytest.mark.parametrize("lens,news", [([1, 40, 517], [1, 1, 1]), ([13001, 700], [1, 1]), ([300, 129], [140, 33]), ([64, 20], [64, 27])])
def test_window_and_sinks(window, sinks, lens, news):
    _attend(8, 4, 64, 16, lens, news, window=window, sinks=sinks, weights=True, seed=window % 97 + sinks % 89)


@pytest.mark.parametrize("Hq,Hkv,d,page,lens,news", [
    (4, 4, 64, 16, [1, 0, 77], [1, 1, 1]), (8, 1, 128, 64, [1500, 3], [1, 1]), (12, 2, 128, 32, [200, 150], [20, 3]),
    (16, 1, 64, 128, [400], [130]), (6, 6, 128, 16, [513, 511], [512, 511]),
    (6, 2, 64, 32, [7001, 513], [1, 1]), (14, 2, 128, 64, [6300, 40], [2, 5])])
def test_weight_sums(Hq, Hkv, d, page, lens, news):
    _attend(Hq, Hkv, d, page, lens, news, weights=True, seed=d + page)


def test_rows_of_no_sequence_are_left_alone():
    _attend(4, 2, 64, 16, [40, 70], [3, 20], gap=5, seed=3)
    _attend(4, 2, 128, 16, [40, 700], [0, 1], gap=2, seed=4)


@pytest.mark.parametrize("q_scale,spread", [(2.0 ** -30, 1.0), (2.0 ** 20, 2.0 ** -8), (24.0, 1.0), (0.0, 1.0)])
def test_query_magnitudes(q_scale, spread):
    """Tiny and large queries (bfloat16 keeps their range), a peaked softmax, zero queries."""
    _attend(8, 2, 128, 64, [300, 77], [1, 9], q_scale=q_scale, spread=spread, seed=11)


def test_page_scales_far_apart():
    """V pages 2^12 apart in scale, and a zero page: the products keep what counts."""
    lens, page = [96], 16
    table, P = _tables(lens, page, 6, 0)
    cache = _pool(P, 1, page, 64, 0)
    _fill(cache, table, lens, 1)
    e = [121, 109, 121, 1, 115, 109]
    for i, x in enumerate(e):
        cache.vs[int(table[0, i]), 0] = x
    cache.k[int(table[0, 3])] = 0
    cache.v[int(table[0, 3])] = 0
    cache.ks[int(table[0, 3]), 0] = 0
    for news in ([1], [96]):
        q = torch.randn((news[0], 4, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
        o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32([0, news[0]]), want_lse=True)
        ref = kv8.attend(_np(cache), q.double().numpy(), table, lens, [0, news[0]])
        _check(o, lse, None, None, ref, 64, 96, "bf16")


def test_strided_queries_and_a_given_scale():
    lens, page = [70, 33], 32
    table, P = _tables(lens, page, 3, 5)
    cache = _pool(P, 2, page, 64, 5)
    _fill(cache, table, lens, 5)
    fused = torch.randn((6, 12, 64), generator=torch.Generator().manual_seed(2)).to(torch.float16).cuda()
    q = fused[:, 2:10]
    o, lse = mq.kv8_attention(q, cache, _i32(table), _i32(lens), cu=_i32([0, 4, 6]), max_q=4, softmax_scale=0.03,
                              want_lse=True)
    ref = kv8.attend(_np(cache), q.double().cpu().numpy(), table, lens, [0, 4, 6], scale=np.float32(0.03))
    _check(o, lse, None, None, ref, 64, 70, "fp16")


def test_long_offsets():
    """Pages past 2^32 bytes of a pool, and a length of 131072 + 7 under a window and without one."""
    page, d, Hkv = 128, 128, 2
    P = 2 ** 32 // (Hkv * page * d) + 1040
    k = torch.zeros((P, Hkv, page, d), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    s = torch.full((P, Hkv), 121, dtype=torch.uint8, device="cuda")
    cache = mq.Kv8Cache(k, v, s, s.clone())
    n = 131072 + 7
    cols = -(-n // page)
    table = np.arange(P - cols, P)[::-1].copy()[None]
    g = torch.Generator(device="cuda").manual_seed(3)
    for c in (k, v):
        c[P - cols:] = (torch.randn((cols, Hkv, page, d), generator=g, device="cuda") * 60).to(
            torch.float8_e4m3fn).view(torch.uint8)
    q = torch.randn((1, 8, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    pool = _np(mq.Kv8Cache(k[P - cols:], v[P - cols:], s[P - cols:], s[P - cols:]))
    for window, sinks in ((0, 0), (700, 5)):
        o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32([n]), window=window, sinks=sinks, want_lse=True)
        ref = kv8.attend(pool, q.double().numpy(), table - (P - cols), [n], [0, 1], window, sinks)
        _check(o, lse, None, None, ref, d, n, "bf16")


# ---------------------------------------------------------------- what the host cannot check
def test_bad_lengths_ranges_and_pages_are_reported():
    lens, page = [40, 50, 60, 33], 16
    table, P = _tables(lens, page, 4, 8)
    cache = _pool(P, 2, page, 64, 8)
    _fill(cache, table, lens, 8)
    q = torch.randn((4, 4, 64), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    w = torch.zeros((4, 2, 64), device="cuda")

    def call(table=table, lens=lens, cu=(0, 1, 2, 3, 4), **kw):
        o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=1, want_lse=True,
                                  weights=w, **kw)
        st, word = mq.device_status()
        assert st == 1 and word == 1 << 16, (st, hex(word))
        assert mq.device_status() == (0, 0)
        return o.float().cpu().numpy(), lse.cpu().numpy()
    ref = kv8.attend(_np(cache), q.double().numpy(), table, lens, [0, 1, 2, 3, 4])
    for bad in (-1, 65, 2 ** 31 - 1, -2 ** 31):
        o, lse = call(lens=[40, bad, 60, 33])  # that sequence counts as empty
        assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
        assert np.allclose(lse[[0, 2, 3]], ref["lse"][[0, 2, 3]], atol=1e-4)
    call(max_len=59)  # sequence 2 is longer than promised
    for pg in (-1, P, 2 ** 31 - 1):
        t = table.copy()
        t[2, 1] = pg  # tokens 16..31 of sequence 2 are not visible then
        o, lse = call(table=t)
        K = kv8.tokens(_np(cache), "k", table[2], 60, 0)
        s = np.delete(K, range(16, 32), 0) @ q[2, 0].double().numpy() / 8
        assert np.isclose(lse[2, 0], np.log(np.exp(s).sum()), atol=1e-4)
    for cu in ((0, 1, 0, 3, 4), (-1, 1, 2, 3, 4), (0, 1, 2, 3, 5), (0, 2, 3, 3, 4)):
        o, lse = call(cu=cu)
    k = torch.randn((4, 2, 64)).to(torch.bfloat16).cuda()
    before = _np(cache)
    t = table.copy()
    t[:, :] = np.array([[-1], [P], [2 ** 30], [-2 ** 31]])
    mq.kv8_append(cache, k, k, _i32(t), _i32(lens))
    assert mq.device_status() == (1, 1 << 16)
    mq.kv8_append(cache, k, k, _i32(table), _i32([-1, 65, 2 ** 31 - 1, 0]))  # nothing is written (0: no room)
    assert mq.device_status() == (1, 1 << 16)
    assert all(np.array_equal(before[f], x) for f, x in _np(cache).items())


def test_a_workspace_that_is_too_small_is_refused():
    cache = _pool(40, 2, 64, 128, 0)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    table, lens = _i32(np.arange(32)[None].repeat(8, 1)), _i32([2000])  # max_len 16384: more than a cluster takes
    need = mq.kv8_attention_workspace(q, cache, table, lens)
    assert need > 0
    with pytest.raises(ValueError, match="ws"):
        mq.kv8_attention(q, cache, table, lens, ws=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- append
def _append_case(Hkv, d, page, steps, dtype, seed, spread):
    """Several appends into the same sequences against the oracle's; values grow so that exponents rise."""
    B = len(steps[0])
    total = [sum(s[b] for s in steps) for b in range(B)]
    table, P = _tables(total, page, -(-max(total) // page), seed)
    cache = _pool(P, Hkv, page, d, seed)
    pool = _np(cache)
    lens = [0] * B
    g = torch.Generator().manual_seed(seed)
    for i, news in enumerate(steps):
        lens = [a + b for a, b in zip(lens, news)]
        cu = np.concatenate([[0], np.cumsum(news)])
        x = torch.randn((int(cu[-1]) + 1, Hkv, 2, d), generator=g) * spread ** i
        x *= torch.exp2(torch.randint(-3, 3, x.shape[:1], generator=g).float())[:, None, None, None]
        x = x.to(DT[dtype])
        k, v = x[:, :, 0].contiguous(), x[:, :, 1].contiguous()
        fused = torch.cat([k, v], 1).cuda()  # strided rows, as in a fused projection
        mq.kv8_append(cache, fused[:, :Hkv], fused[:, Hkv:], _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news))
        kv8.append(pool, k.double().numpy(), v.double().numpy(), table, lens, cu)
        got = _np(cache)
        for f in ("ks", "vs", "k", "v"):
            assert np.array_equal(got[f], pool[f]), (f, i)
    assert mq.device_status() == (0, 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hkv,d,page,steps", [
    (2, 64, 16, [[1, 0], [1, 1], [14, 3], [1, 12], [1, 1], [40, 33]]),
    (1, 128, 64, [[100], [1], [1], [63], [200]]),
    (3, 128, 128, [[5, 128, 129], [1, 1, 1], [300, 0, 127]]),
    (8, 64, 32, [[31, 1, 33, 2], [1, 1, 1, 1], [1, 1, 1, 1]]),
])
@pytest.mark.parametrize("spread", [1.0, 4.0, 0.25])
def test_append(Hkv, d, page, steps, dtype, spread):
    _append_case(Hkv, d, page, steps, dtype, Hkv * page + len(steps), spread)


def test_append_every_bf16_value():
    """All finite BF16 values, a binade a page, by themselves and beside a larger value: subnormals, the largest."""
    page, d = 64, 64
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    x = (bits << 16).view(torch.float32)
    x = torch.stack([x, -x], 1).reshape(-1)
    x = torch.cat([x, torch.zeros(-x.numel() % (page * d))]).view(-1, 1, d).to(torch.bfloat16)
    n = x.shape[0]
    pages = n // page
    for flip in (False, True):
        v = x.flip(0).contiguous() if flip else x
        cache = _pool(pages, 1, page, d, 1)
        pool = _np(cache)
        table = np.arange(pages)[None]
        mq.kv8_append(cache, x.cuda(), v.cuda(), _i32(table), _i32([n]), cu=_i32([0, n]))
        kv8.append(pool, x.double().numpy(), v.double().numpy(), table, [n], [0, n])
        got = _np(cache)
        for f in ("ks", "vs", "k", "v"):
            assert np.array_equal(got[f], pool[f]), f


# ---------------------------------------------------------------- eviction
def _evict_case(Hkv, d, page, lens, keep, sinks, recent, w=None, seed=0, same_pool=False):
    B = len(lens)
    cols = -(-max(lens + [1]) // page)
    table, P = _tables(lens, page, cols, seed)
    dcols = -(-min(keep, cols * page) // page) + 1
    extra = B * dcols if same_pool else 0
    cache = _pool(P + extra, Hkv, page, d, seed, nan=False)
    dst = cache if same_pool else _pool(B * dcols, Hkv, page, d, seed + 1)
    base = P if same_pool else 0
    dtable = base + np.random.default_rng(seed).permutation(B * dcols).reshape(B, dcols)
    g = torch.Generator().manual_seed(seed)
    if w is None:
        w = torch.rand((B, Hkv, cols * page + 3), generator=g)
    dw = torch.rand((B, Hkv, dcols * page + 1), generator=g)
    pool, dpool, dwn = _np(cache), _np(dst), dw.numpy().copy()
    if same_pool:
        dpool = {f: x.copy() for f, x in pool.items()}
    dwd = dw.cuda()
    got_lens, kept = mq.kv8_evict(cache, _i32(table), _i32(lens), w.cuda(), dst, _i32(dtable), dwd, keep, sinks, recent)
    want_lens, want_kept = kv8.evict(pool, table, lens, w.numpy(), dpool, dtable, dwn, keep, sinks, recent)
    assert mq.device_status() == (0, 0)
    assert np.array_equal(got_lens.cpu().numpy(), want_lens)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(dwd.cpu().numpy(), dwn)
    got = _np(dst)
    for f in ("ks", "vs", "k", "v"):
        assert np.array_equal(got[f], dpool[f]), f


@pytest.mark.parametrize("Hkv,d,page,lens,keep,sinks,recent", [
    (2, 64, 16, [0, 1, 5, 100, 37], 20, 2, 3), (1, 128, 64, [4099], 1024, 4, 128), (8, 128, 128, [300, 299], 299, 0, 0),
    (3, 64, 32, [700, 31], 1, 0, 1), (1, 64, 16, [2000], 7, 0, 0), (2, 128, 16, [50], 64, 4, 4),
    (1, 128, 16, [333], 20, 20, 0), (1, 128, 16, [333], 20, 0, 20), (1, 64, 16, [333], 20, 8, 12),
    (1, 64, 64, [40000], 9000, 3, 77), (2, 64, 64, [20001, 0, 300, 8193], 3001, 3, 77), (1, 64, 128, [9000], 4000, 4000, 0),
    (1, 64, 128, [8193, 50], 1, 0, 0), (1, 64, 64, [33000, 100, 0], 12001, 12000, 1)])
def test_evict(Hkv, d, page, lens, keep, sinks, recent):
    _evict_case(Hkv, d, page, lens, keep, sinks, recent, seed=keep)
    _evict_case(Hkv, d, page, lens, keep, sinks, recent, seed=keep + 1, same_pool=True)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "inf", "close", "tiny"])
def test_evict_ties_and_odd_weights(kind):
    n = 2500
    g = torch.Generator().manual_seed(5)
    w = {"equal": torch.ones((1, 2, n)), "few": torch.randint(0, 3, (1, 2, n), generator=g).float(),
         "signs": torch.randint(-2, 3, (1, 2, n), generator=g).float() * 0.5,
         "inf": torch.where(torch.rand((1, 2, n), generator=g) < 0.3, torch.inf, -torch.inf),
         "close": 1 + torch.randint(0, 500, (1, 2, n), generator=g).float() * 2.0 ** -23,
         "tiny": torch.randint(0, 900, (1, 2, n), generator=g).float() * 2.0 ** -149}[kind]
    if kind == "signs":
        w[w == 0] = torch.where(torch.rand(int((w == 0).sum()), generator=g) < 0.5, 0.0, -0.0)  # -0 equals 0
    _evict_case(2, 64, 32, [n - 37], 1000, 3, 50, w=torch.nn.functional.pad(w, (0, 12)), seed=2)


@pytest.mark.parametrize("n", [20000, 33100])
@pytest.mark.parametrize("kind", ["equal", "few", "close"])
def test_evict_ties_of_long_sequences(kind, n):
    """The kept ones of equal weights are the first, wherever in a sequence that several CTAs share they lie."""
    g = torch.Generator().manual_seed(6)
    w = {"equal": torch.ones((1, 2, n)), "few": torch.randint(0, 3, (1, 2, n), generator=g).float(),
         "close": 1 + torch.randint(0, 500, (1, 2, n), generator=g).float() * 2.0 ** -23}[kind]
    _evict_case(2, 64, 128, [n - 37], 9001, 3, 50, w=torch.nn.functional.pad(w, (0, -n % 128)), seed=2)


def test_evict_bad_pages_are_reported():
    cache, dst = _pool(8, 2, 16, 64, 0, nan=False), _pool(4, 2, 16, 64, 1)
    w, dw = torch.rand((2, 2, 64), device="cuda"), torch.zeros((2, 2, 32), device="cuda")
    before = _np(dst)
    lens, kept = mq.kv8_evict(cache, _i32([[0, 1, 9, 2], [3, 4, 5, 6]]), _i32([64, 65]), w, dst, _i32([[0, 1], [7, -1]]),
                              dw, 32, 2, 30)
    assert mq.device_status() == (1, 1 << 16)
    got = _np(dst)
    assert lens.tolist() == [32, 0] and (kept[1] == -1).all()
    ids = kept[0, 0].tolist()
    for r, t in enumerate(ids):  # tokens of the bad page come as zeros
        if t // 16 == 2:
            assert (got["k"][r // 16, 0, r % 16] == 0).all()
    assert all(np.array_equal(got[f][2:], before[f][2:]) for f in got)


# ---------------------------------------------------------------- as a server uses them
@pytest.mark.parametrize("Hq,Hkv,d,page,dtype", [(8, 2, 128, 64, "bf16"), (4, 4, 64, 16, "fp16")])
def test_a_serving_loop(Hq, Hkv, d, page, dtype):
    """Prompts, generated tokens, verification of several tokens, eviction, more tokens: each step against the
    oracle on the library's own state."""
    B, cap = 3, 8
    cache = mq.kv8_alloc(2 * B * cap, Hkv, page, d, "cuda")
    cache.k.fill_(0x7F), cache.v.fill_(0xFF), cache.ks.fill_(200), cache.vs.fill_(200)
    perm = np.random.default_rng(1).permutation(2 * B * cap).reshape(2, B, cap)
    table, lens = perm[0], np.zeros(B, dtype=np.int64)
    w = torch.zeros((B, Hkv, cap * page), device="cuda")
    g = torch.Generator().manual_seed(2)
    for step, news in enumerate([[37, 100, 1], [1, 1, 1], [1, 1, 1], [4, 4, 2], "evict", [1, 1, 1], [3, 1, 17]]):
        if news == "evict":
            dw = torch.zeros_like(w)
            pool = _np(cache)
            dpool, dwn = {f: x.copy() for f, x in pool.items()}, dw.cpu().numpy()
            got, kept = mq.kv8_evict(cache, _i32(table), _i32(lens), w, cache, _i32(perm[1]), dw, 40, 2, 16)
            want, want_kept = kv8.evict(pool, table, lens, w.cpu().numpy(), dpool, perm[1], dwn, 40, 2, 16)
            assert np.array_equal(kept.cpu().numpy(), want_kept) and np.array_equal(got.cpu().numpy(), want)
            assert all(np.array_equal(x, dpool[f]) for f, x in _np(cache).items())
            assert np.array_equal(dw.cpu().numpy(), dwn)
            table, lens, w = perm[1], want.astype(np.int64), dw
            continue
        cu = np.concatenate([[0], np.cumsum(news)])
        lens = lens + np.array(news)
        qkv = torch.randn((int(cu[-1]), Hq + 2 * Hkv, d), generator=g).to(DT[dtype]).cuda()
        pool = _np(cache)
        one = cu if max(news) > 1 else None
        args = dict(cu=None if one is None else _i32(cu), max_q=None if one is None else max(news))
        mq.kv8_append(cache, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], _i32(table), _i32(lens), **args)
        x = qkv.double().cpu().numpy()
        kv8.append(pool, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], table, lens, cu)
        assert all(np.array_equal(y, pool[f]) for f, y in _np(cache).items()), step
        w0 = w.cpu().numpy().astype(np.float64)
        win = dict(window=24, sinks=2) if step % 2 else {}
        o, lse = mq.kv8_attention(qkv[:, :Hq], cache, _i32(table), _i32(lens), weights=w, want_lse=True, **args, **win)
        ref = kv8.attend(pool, x[:, :Hq], table, lens, cu, **win)
        _check(o, lse, w, w0, ref, d, int(lens.max()), dtype)


def test_sequences_that_share_pages():
    """A common prefix of full pages in two sequences; the sums stay each sequence's own, and repeats are equal."""
    page, Hkv, d = 16, 2, 64
    table = np.array([[0, 1, 2, 9], [0, 1, 5, 6]])
    lens = [45, 64]
    cache = _pool(10, Hkv, page, d, 0, nan=False)
    q = torch.randn((2, 4, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    runs = []
    for _ in range(3):
        w = torch.zeros((2, Hkv, 64), device="cuda")
        o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), weights=w, want_lse=True)
        runs.append((o, lse, w))
    ref = kv8.attend(_np(cache), q.double().numpy(), table, lens, [0, 1, 2])
    _check(*runs[0], np.zeros((2, Hkv, 64)), ref, d, 64, "bf16")
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_captured_calls_read_lengths_when_they_run():
    """One capture of append, attention and eviction, replayed as the sequences grow."""
    B, Hq, Hkv, d, page, cap = 3, 8, 2, 128, 32, 24
    cache, dst = mq.kv8_alloc(B * cap, Hkv, page, d, "cuda"), mq.kv8_alloc(B * 2, Hkv, page, d, "cuda")
    for c in (cache, dst):
        c.k.fill_(1), c.v.fill_(2), c.ks.fill_(120), c.vs.fill_(120)
    table = np.random.default_rng(0).permutation(B * cap).reshape(B, cap)
    t, lens = _i32(table), torch.zeros(B, dtype=torch.int32, device="cuda")
    dt = _i32(np.arange(B * 2).reshape(B, 2))
    qkv = torch.zeros((B, Hq + 2 * Hkv, d), dtype=torch.bfloat16, device="cuda")
    w, dw = torch.zeros((B, Hkv, cap * page), device="cuda"), torch.zeros((B, Hkv, 64), device="cuda")
    o = torch.zeros((B, Hq, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((B, Hq), device="cuda")
    dl, kept = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros((B, Hkv, 48), dtype=torch.int32, device="cuda")
    ws = torch.empty(mq.kv8_attention_workspace(qkv[:, :Hq], cache, t, lens, weights=w), dtype=torch.uint8, device="cuda")

    def calls():
        mq.kv8_append(cache, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], t, lens)
        mq.kv8_attention(qkv[:, :Hq], cache, t, lens, weights=w, o=o, lse=lse, ws=ws)
        mq.kv8_evict(cache, t, lens, w, dst, dt, dw, 48, 2, 20, dst_lens=dl, kept=kept)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    w.zero_()
    g = torch.Generator().manual_seed(0)
    for step, n in enumerate([(1, 30, 700), (2, 31, 701), (3, 32, 702), (4, 33, 703)]):
        lens.copy_(_i32(n))
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        pool, w0 = _np(cache), w.cpu().numpy().astype(np.float64)
        graph.replay()
        torch.cuda.synchronize()
        x = qkv.double().cpu().numpy()
        kv8.append(pool, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], table, n, np.arange(B + 1))
        assert all(np.array_equal(y, pool[f]) for f, y in _np(cache).items())
        ref = kv8.attend(pool, x[:, :Hq], table, n, np.arange(B + 1))
        _check(o, lse, w, w0, ref, d, max(n), "bf16")
        want = [kv8.keep_set(w[b, h].cpu().numpy(), n[b], 48, 2, 20) for b in range(B) for h in range(Hkv)]
        assert all(kept.view(-1, 48)[i, :len(x)].tolist() == x.tolist() for i, x in enumerate(want))
        assert dl.tolist() == [min(x, 48) for x in n]


def test_a_captured_chunk_reads_lengths_when_it_runs():
    """Chunks of several tokens under a window, with sums, captured once: the tile kernels."""
    B, Hq, Hkv, d, page, cap, n = 2, 16, 2, 64, 32, 16, 60
    cache = mq.kv8_alloc(B * cap, Hkv, page, d, "cuda")
    table = np.random.default_rng(0).permutation(B * cap).reshape(B, cap)
    _fill(cache, table, [cap * page] * B, 3)
    cache.ks.fill_(121), cache.vs.fill_(120)
    t, lens, cu = _i32(table), _i32([40, 20]), _i32([0, 40, 60])
    q = torch.zeros((n, Hq, d), dtype=torch.float16, device="cuda")
    w = torch.zeros((B, Hkv, cap * page), device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros((n, Hq), device="cuda")
    ws = torch.empty(mq.kv8_attention_workspace(q, cache, t, lens, cu=cu, max_q=50, window=100, sinks=3, weights=w),
                     dtype=torch.uint8, device="cuda")

    def call():
        mq.kv8_attention(q, cache, t, lens, cu=cu, max_q=50, window=100, sinks=3, weights=w, o=o, lse=lse, ws=ws)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g = torch.Generator().manual_seed(0)
    for ln, c in (([40, 20], [0, 40, 60]), ([500, 300], [0, 50, 60]), ([333, 512], [0, 12, 60])):
        lens.copy_(_i32(ln)), cu.copy_(_i32(c)), q.copy_(torch.randn(q.shape, generator=g)), w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        ref = kv8.attend(_np(cache), q.double().cpu().numpy(), table, ln, c, 100, 3)
        _check(o, lse, w, np.zeros(w.shape), ref, d, max(ln), "fp16")


def test_calls_on_two_streams_at_once():
    """Two streams, each with its own workspace, against the same calls one after the other."""
    page, Hkv, Hq, d = 64, 8, 32, 128
    lens = [9000, 7001]
    table, P = _tables(lens, page, 150, 1)
    cache = _pool(P, Hkv, page, d, 1, nan=False)
    qs = [torch.randn((2, Hq, d), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in (1, 2)]
    t, ln = _i32(table), _i32(lens)
    alone = [mq.kv8_attention(q, cache, t, ln, want_lse=True) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(20):
        got = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(mq.kv8_attention(q, cache, t, ln, want_lse=True))
        torch.cuda.synchronize()
        for (o, l), (o1, l1) in zip(got, alone):
            assert torch.equal(o, o1) and torch.equal(l, l1)
