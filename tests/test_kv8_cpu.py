"""The paged 8-bit cache's entry points refuse bad arguments on the host (no kernel is launched)."""
import ctypes

import pytest
import torch

import mixed_precision_bit_quant_b200 as mq
from mixed_precision_bit_quant_b200 import _lib

OK, INVALID, UNSUPPORTED = _lib.THRIFT_OK, _lib.THRIFT_ERR_INVALID, _lib.THRIFT_ERR_UNSUPPORTED


def _shape(**kw):
    a = dict(B=2, Hq=8, Hkv=2, d=128, page=64, table_cols=4, n=2, max_q=1, max_len=200, dtype=0)
    a.update(kw)
    return _lib.Kv8Shape(**a)


def _cache(num_pages=8, **kw):
    a = dict(k=16, v=16, ks=16, vs=16)
    a.update(kw)
    return _lib.Kv8CacheStruct(a["k"], a["v"], a["ks"], a["vs"], num_pages)


def _attn(shape=None, mask=(0, 0, 0.0), cache=None, q=16, qs=1024, table=16, lens=16, cu=None, o=16, lse=None, w=None,
          w_cols=0, ws=16, ws_bytes=1 << 40):
    s, m, c = shape or _shape(), _lib.Kv8Mask(*mask), cache or _cache()
    return mq.lib().thrift_kv8_attn(ctypes.byref(s), ctypes.byref(m), ctypes.byref(c), q, qs, table, lens, cu, o, lse,
                                    w, w_cols, ws, ws_bytes, None)


def _append(shape=None, cache=None, k=16, ks=256, v=16, vs=256, table=16, lens=16, cu=None):
    s, c = shape or _shape(), cache or _cache()
    return mq.lib().thrift_kv8_append(ctypes.byref(s), ctypes.byref(c), k, ks, v, vs, table, lens, cu, None)


def _evict(shape=None, cache=None, table=16, lens=16, w=16, w_cols=256, keep=64, sinks=4, recent=8, dst=None,
           dst_table=16, dst_cols=1, dst_lens=1 << 20, dst_w=1 << 21, dst_w_cols=64, kept=1 << 22):
    s, c, e = shape or _shape(), cache or _cache(), dst or _cache()
    return mq.lib().thrift_kv8_evict(ctypes.byref(s), ctypes.byref(c), table, lens, w, w_cols, keep, sinks, recent,
                                     ctypes.byref(e), dst_table, dst_cols, dst_lens, dst_w, dst_w_cols, kept, None)


def test_cache_bytes():
    f = mq.lib().thrift_kv8_cache_bytes
    assert [f(10, 8, 64, 128, i) for i in range(5)] == [10 * 8 * 64 * 128] * 2 + [80, 80, 0]
    assert f(1 << 20, 8, 128, 128, 0) == (1 << 20) * 8 * 128 * 128  # past 32 bits
    for bad in ((0, 8, 64, 128), (10, 0, 64, 128), (10, 8, 48, 128), (10, 8, 64, 96), ((1 << 30) + 1, 8, 64, 128)):
        assert f(*bad, 0) == 0


SHAPES = [(dict(B=0), INVALID), (dict(table_cols=0), INVALID), (dict(n=-1), INVALID), (dict(max_len=0), INVALID),
          (dict(max_len=257), INVALID), (dict(max_q=3), INVALID), (dict(max_q=0), INVALID), (dict(dtype=2), INVALID), (dict(d=96), UNSUPPORTED),
          (dict(page=48), UNSUPPORTED), (dict(page=8, max_len=8), UNSUPPORTED), (dict(Hkv=0), INVALID),
          (dict(B=32768, Hkv=2, n=32768), UNSUPPORTED), (dict(table_cols=(1 << 18) + 1), UNSUPPORTED)]


@pytest.mark.parametrize("bad,want", SHAPES)
def test_bad_shapes(bad, want):
    s = _shape(**bad)
    assert _append(s) == want and _evict(s) == want
    assert _attn(s) == want
    assert mq.lib().thrift_kv8_attn_workspace_bytes(ctypes.byref(s), ctypes.byref(_lib.Kv8Mask(0, 0, 0.0)), 1) == 0


def test_bad_heads_and_rows_of_attention():
    assert _attn(_shape(Hq=3)) == INVALID
    assert _attn(_shape(Hq=0)) == INVALID
    assert _attn(_shape(n=3)) == INVALID  # no cu: one token per sequence
    assert _append(_shape(n=3)) == INVALID
    assert _attn(_shape(B=1, n=1 << 28, max_q=1), cu=16) == UNSUPPORTED  # n * Hq
    assert _attn(_shape(B=1, n=1 << 24, max_q=1 << 24), cu=16) == UNSUPPORTED  # rows of a sequence
    assert _attn(_shape(n=0, max_q=0), q=None, o=None, cu=16) == OK  # nothing to do
    assert _append(_shape(n=0, max_q=0), k=None, v=None, cu=16) == OK


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=24), dict(o=None), dict(table=None), dict(table=18), dict(lens=None),
                                dict(lens=17), dict(cu=18), dict(lse=18), dict(qs=1020), dict(qs=512), dict(ws=None),
                                dict(ws_bytes=16), dict(ws=24), dict(w=16, w_cols=199), dict(w=20, w_cols=200),
                                dict(mask=(-1, 0, 0.0)), dict(mask=(0, -1, 0.0)), dict(mask=(0, 0, -1.0)),
                                dict(mask=(0, 0, float("inf"))), dict(mask=(0, 0, float("nan"))),
                                dict(cache=_cache(0)), dict(cache=_cache(k=None)), dict(cache=_cache(v=24)),
                                dict(cache=_cache(ks=None)), dict(cache=_cache((1 << 30) + 1))])
def test_bad_attention_arguments(kw):
    # (long enough that the call needs a workspace)
    assert _attn(_shape(max_len=65536, table_cols=1024) if "w" not in kw else None, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k=None), dict(k=24), dict(v=8), dict(ks=248), dict(ks=260), dict(vs=100),
                                dict(table=None), dict(lens=2), dict(cu=2), dict(cache=_cache(0))])
def test_bad_append_arguments(kw):
    assert _append(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(w=None), dict(w=20), dict(w_cols=199), dict(keep=0), dict(sinks=-1), dict(recent=-1),
                                dict(sinks=60, recent=5), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
                                dict(dst=_cache(0)), dict(dst=_cache(v=24)), dict(dst_table=None), dict(dst_cols=0),
                                dict(keep=65, dst_cols=1), dict(dst_w_cols=63), dict(dst_w=None), dict(dst_lens=None),
                                dict(kept=None), dict(kept=18), dict(dst_w=(1 << 21) + 8),
                                # outputs over inputs that other CTAs still read
                                dict(dst_lens=16), dict(dst_lens=20), dict(lens=1 << 20, dst_lens=(1 << 20) - 4),
                                dict(dst_w=16), dict(dst_w=16 + 4 * 256), dict(w=1 << 21, dst_w=(1 << 21) - 64)])
def test_bad_evict_arguments(kw):
    assert _evict(**kw) == INVALID


def test_workspace_covers_both_parts():
    f = mq.lib().thrift_kv8_attn_workspace_bytes
    s, m = _shape(max_len=256), _lib.Kv8Mask(0, 0, 0.0)
    without, with_w = f(ctypes.byref(s), ctypes.byref(m), 0), f(ctypes.byref(s), ctypes.byref(m), 1)
    assert with_w > without
    assert f(ctypes.byref(s), None, 0) == 0 and f(None, ctypes.byref(m), 0) == 0


# --------------------------------------------------------------------------- the binding
@pytest.fixture
def any_device(monkeypatch):
    monkeypatch.setattr(_lib, "_on_device", lambda t, name, device=None: None)
    monkeypatch.setattr(_lib, "_kv8_call", lambda fn, what, device, *args: None)


def _args(B=2, Hq=4, Hkv=2, d=64, page=16, cols=3):
    c = mq.Kv8Cache(*(torch.zeros(s, dtype=torch.uint8) for s in ((8, Hkv, page, d),) * 2 + ((8, Hkv),) * 2))
    return dict(q=torch.zeros((B, Hq, d), dtype=torch.bfloat16), cache=c,
                table=torch.zeros((B, cols), dtype=torch.int32), lens=torch.ones(B, dtype=torch.int32))


def test_host_tensors_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        mq.kv8_alloc(4, 2, 16, 64, "cpu")


def test_binding_accepts_documented_calls(any_device):
    a = _args()
    o, lse = mq.kv8_attention(**a)
    assert o.shape == a["q"].shape and o.dtype == torch.bfloat16 and lse is None
    _, lse = mq.kv8_attention(**a, want_lse=True, weights=torch.zeros((2, 2, 48)))
    assert lse.shape == (2, 4)
    a["q"] = torch.zeros((5, 3, 4, 64), dtype=torch.float16)[:, 1]  # tokens strided, as in a fused projection
    mq.kv8_attention(**a, cu=torch.tensor([0, 2, 5], dtype=torch.int32))
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    assert mq.kv8_append(a["cache"], k, k, a["table"], a["lens"]) is None
    w = torch.zeros((2, 2, 48))
    lens, kept = mq.kv8_evict(a["cache"], a["table"], a["lens"], w, a["cache"], a["table"], torch.zeros((2, 2, 16)), 16)
    assert lens.shape == (2,) and kept.shape == (2, 2, 16)


@pytest.mark.parametrize("bad,match", [
    (dict(q=torch.zeros((2, 4, 64))), "dtype"), (dict(q=torch.zeros((2, 256), dtype=torch.bfloat16)), "tensor"),
    (dict(q=torch.zeros((2, 4, 128), dtype=torch.bfloat16)), "shape"),
    (dict(q=torch.zeros((2, 64, 4), dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(q=torch.zeros((2, 4, 68), dtype=torch.bfloat16)[..., :64]), "contiguous"),
    (dict(q=torch.zeros((3, 4, 64), dtype=torch.bfloat16)), "without cu"),
    (dict(table=torch.zeros((2, 3), dtype=torch.int64)), "table"),
    (dict(table=torch.zeros((2, 6), dtype=torch.int32)[:, ::2]), "table"),
    (dict(table=torch.zeros(6, dtype=torch.int32)), "table"),
    (dict(lens=torch.ones(3, dtype=torch.int32)), "lens"),
    (dict(cu=torch.zeros(2, dtype=torch.int32)), "cu"),
    (dict(weights=torch.zeros((2, 4, 48))), "weights"), (dict(weights=torch.zeros((2, 2, 48)).half()), "weights"),
    (dict(o=torch.zeros((2, 4, 64))), "o"), (dict(lse=torch.zeros((4, 2))), "lse"),
])
def test_binding_refuses(any_device, bad, match):
    with pytest.raises(ValueError, match=match):
        mq.kv8_attention(**{**_args(), **bad})


def test_binding_refuses_append_and_evict(any_device):
    a = _args()
    c, t, n = a["cache"], a["table"], a["lens"]
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    for kk, vv, m in ((k, k.half(), "v"), (k, k[:1], "v"), (k[:, :1], k, "k"), (k.float(), k, "k")):
        with pytest.raises(ValueError, match=m):
            mq.kv8_append(c, kk, vv, t, n)
    with pytest.raises(TypeError):
        mq.kv8_append({}, k, k, t, n)
    with pytest.raises(TypeError):
        mq.kv8_attention(a["q"], {"k": 1}, t, n)
    w, dw = torch.zeros((2, 2, 48)), torch.zeros((2, 2, 16))
    with pytest.raises(ValueError, match="overlap"):
        mq.kv8_evict(c, t, n, w, c, t, w, 16)
    with pytest.raises(ValueError, match="dst_lens"):
        mq.kv8_evict(c, t, n, w, c, t, dw, 16, dst_lens=n)
    with pytest.raises(ValueError, match="dst"):
        mq.kv8_evict(c, t, n, w, _args(page=32)["cache"], t, dw, 16)
    with pytest.raises(ValueError, match="kept"):
        mq.kv8_evict(c, t, n, w, c, t, dw, 16, kept=torch.zeros((2, 2, 15), dtype=torch.int32))


def test_a_call_follows_its_tensors_device(monkeypatch):
    """Where the cache lives on another device than the current one, the call runs with that device current and
    on that device's stream."""
    seen = []

    class Guard:
        def __init__(self, d): self.d = d
        def __enter__(self): seen.append(("in", self.d))
        def __exit__(self, *a): seen.append(("out", self.d))

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(_lib, "_raw_stream", lambda index: 100 + index)
    _lib._kv8_call(lambda *a: seen.append(a) or 0, "x", torch.device("cuda", 1), 7)
    assert seen == [("in", 1), (7, 101), ("out", 1)]
    seen.clear()
    _lib._kv8_call(lambda *a: seen.append(a) or 0, "x", torch.device("cuda", 0), 7)
    assert seen == [(7, 100)]
    with pytest.raises(mq.ThriftError, match="THRIFT_ERR_INVALID"):
        _lib._kv8_call(lambda *a: 1, "x", torch.device("cuda", 0))


def test_workspace_of_a_window_does_not_grow_with_the_text():
    """The logits kept for the weight sums are the visible tokens', for every number of rows."""
    f = mq.lib().thrift_kv8_attn_workspace_bytes
    for max_q, Hq in ((1, 8), (1, 64), (4, 64), (8, 64), (40, 64)):
        sizes = []
        for n in (16384, 131072, 1 << 20):
            s = _shape(B=8, Hq=Hq, Hkv=8, n=8 * max_q, max_q=max_q, max_len=n, table_cols=n // 64)
            sizes.append(f(ctypes.byref(s), ctypes.byref(_lib.Kv8Mask(4096, 4, 0.0)), 1))
            # without a window: a logit of every token, at least
            if max_q * (Hq // 8) <= 64:
                assert f(ctypes.byref(s), ctypes.byref(_lib.Kv8Mask(0, 0, 0.0)), 1) >= 4 * 8 * 8 * max_q * (Hq // 8) * n
        assert sizes[0] == sizes[1] == sizes[2]
        if max_q * (Hq // 8) <= 64:
            rows = -(-max_q * (Hq // 8) // 16) * 16
            assert sizes[0] <= 4 * 8 * 8 * rows * (4096 + 200) + (96 << 20)
