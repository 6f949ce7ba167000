"""The paged 8-bit cache's attention: batches of more sequences than a CTA has threads, and windows far into long
texts with weight sums.  Bounds as in test_gpu_kv8.py."""
import numpy as np
import pytest
import torch

import mixed_precision_bit_quant_b200 as mq
from oracle import kv8
from test_gpu_kv8 import _attend, _check, _i32, _np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [128, 129, 256, 300, 500])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (24, 3)])
def test_batches_of_many_sequences(B, weights, window, sinks):
    """Shares that start in every part of the list of sequences; empty sequences and ones with nothing new among them."""
    r = np.random.default_rng(B)
    lens = [int(x) for x in r.integers(0, 90, B)]
    lens[0], lens[130 % B], lens[B - 1] = 400, 300, 500
    news = [int(x) for x in r.integers(0, 3, B)]
    news[0] = news[B - 1] = 2
    _attend(2, 1, 64, 16, lens, news, window=window, sinks=sinks, weights=weights, seed=B, cols=32)
    _attend(10, 1, 64, 16, [int(x) for x in r.permutation(lens)], news, window=window, sinks=sinks, weights=weights, seed=B,
            cols=32)


def test_batches_where_all_the_work_is_in_one_sequence():
    for at in (0, 127, 128, 200, 299):
        lens = [0] * 300
        lens[at] = 700
        _attend(2, 1, 64, 16, lens, [1] * 300, weights=True, seed=at, cols=45)


@pytest.mark.parametrize("Hq,Hkv,d,news,window,sinks", [
    (8, 2, 64, [1, 1], 300, 5), (8, 2, 128, [4, 1], 1000, 0), (16, 1, 64, [4, 2], 17, 40), (2, 1, 64, [1, 0], 4096, 4),
    (8, 1, 64, [1, 1], 1, 0)])
def test_weight_sums_of_a_window_far_into_a_text(Hq, Hkv, d, news, window, sinks):
    """The logits that the sums are made of are kept for the visible tokens only."""
    page, lens = 128, [70007, 4097]
    cols = -(-max(lens) // page)
    g = torch.Generator(device="cuda").manual_seed(3)
    P = 2 * cols
    codes = [(torch.randn((P, Hkv, page, d), generator=g, device="cuda") * 60).to(torch.float8_e4m3fn).view(torch.uint8)
             for _ in "kv"]
    s = torch.full((P, Hkv), 121, dtype=torch.uint8, device="cuda")
    cache = mq.Kv8Cache(codes[0], codes[1], s, s.clone())
    table = np.random.default_rng(1).permutation(P).reshape(2, cols)
    cu = np.concatenate([[0], np.cumsum(news)])
    q = torch.randn((int(cu[-1]), Hq, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    w = torch.rand((2, Hkv, cols * page), generator=g, device="cuda")
    w0 = w.cpu().numpy()
    ws = torch.empty(mq.kv8_attention_workspace(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news),
                                                window=window, sinks=sinks, weights=w) + 256, dtype=torch.uint8, device="cuda")
    ws[-256:] = 77
    o, lse = mq.kv8_attention(q.cuda(), cache, _i32(table), _i32(lens), cu=_i32(cu), max_q=max(news), window=window,
                              sinks=sinks, weights=w, want_lse=True, ws=ws)
    ref = kv8.attend(_np(cache), q.double().numpy(), table, lens, cu, window, sinks)
    _check(o, lse, w, w0.astype(np.float64), ref, d, window + sinks + 8, "bf16")
    assert (ws[-256:] == 77).all()
    got = w.cpu().numpy()
    for b, n in enumerate(lens):  # tokens that no row sees keep their sums to the bit
        lo, hi = min(sinks, n), max(n - news[b] - window + 1, 0)
        assert np.array_equal(got[b, :, lo:hi], w0[b, :, lo:hi]) and np.array_equal(got[b, :, n:], w0[b, :, n:])
