"""The paged 8-bit KV cache: what is measured, and its plain forms.

Three operators that a serving loop runs one after the other on the same cache
(pages of `page` tokens, e4m3 codes, one power-of-two scale per page and kv head):

  append   new tokens' K and V are quantised into their sequences' pages
  attend   attention of the new tokens' queries over the cache: causal, with an
           optional sliding window and first tokens that stay visible (sinks);
           optionally the attention weight that each cached token received is
           added to a running sum
  evict    the tokens with the largest sums (plus sinks and the most recent
           ones) are moved, in order, to fewer pages

With `own` false, `run` computes them with elementary torch operations; with
`own` true it calls the package.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------- cases
def _attend(name, B, Hq, Hkv, d, page, L, nq, ragged, dtype="bf16", window=0, sinks=0, weights=False):
    """L: the longest sequence with its new tokens; nq: the most new tokens of a sequence; ragged: whether
    lengths differ (lens and new tokens spread below L and nq)."""
    return dict(name=name, op="attend", B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, L=L, nq=nq, ragged=ragged,
                dtype=dtype, window=window, sinks=sinks, weights=weights)


def listed():
    return [
        # one generated token per sequence enters the cache of a serving batch
        dict(name="append_b32_1", op="append", B=32, Hkv=8, d=128, page=64, L=2048, nq=1, ragged=True, dtype="bf16"),
        # four prompts of the llm8k length enter the cache
        dict(name="append_b4_8192", op="append", B=4, Hkv=8, d=128, page=64, L=8192, nq=8192, ragged=False,
             dtype="bf16"),
        # the smallest call: one sequence, a short context of odd length, one query head per kv head
        _attend("decode_b1_517", 1, 12, 12, 64, 16, 517, 1, False),
        # the decode step of the repository's own benchmark: 8 sequences of 32768 tokens
        _attend("decode_b8_32768", 8, 32, 8, 128, 64, 32768, 1, False),
        # a batch of mixed lengths that also keeps the sums for eviction
        _attend("decode_w_b32_8191", 32, 32, 8, 128, 64, 8191, 1, True, weights=True),
        # streaming generation far into a text: a window and four sinks
        _attend("decode_win_b4_131072", 4, 32, 8, 128, 128, 131072, 1, True, dtype="fp16", window=4096, sinks=4),
        # four drafted tokens per sequence are verified in one call, eight query heads per kv head
        _attend("verify_b8_q4_16384", 8, 64, 8, 128, 32, 16384, 4, True),
        # prompts of mixed lengths under a window, heads of 64
        _attend("prompt_win_b4_4096", 4, 12, 12, 64, 16, 4096, 4096, True, window=1024, sinks=4),
        # a chunk of a long prompt that also keeps the sums
        _attend("chunk_w_b2_4096", 2, 32, 8, 128, 64, 4096, 1024, True, weights=True),
        # a large chunk at the end of a long prompt
        _attend("chunk_b1_16389", 1, 32, 8, 128, 64, 16389, 4096, False),
        # one sequence's cache is cut to a quarter
        dict(name="evict_b1_4099", op="evict", B=1, Hkv=8, d=128, page=64, L=4099, ragged=False, keep=1024, sinks=4,
             recent=128),
        # eight long sequences' caches are cut to a quarter
        dict(name="evict_b8_32768", op="evict", B=8, Hkv=8, d=128, page=64, L=32768, ragged=True, keep=8192, sinks=4,
             recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict"])
    Hkv, d, page = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    B, ragged, dtype = _log(rng, 1, 48), rng.random() < 0.7, rng.choice(["bf16", "bf16", "fp16"])
    if op == "append":
        L = _log(rng, 1, 32768)
        nq = 1 if rng.random() < 0.4 else _log(rng, 1, L)
        B = max(1, min(B, 2 ** 21 // (L * Hkv)))
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, L=L, nq=nq, ragged=ragged, dtype=dtype)
    if op == "evict":
        L = _log(rng, 16, 32768)
        B = max(1, min(B, 2 ** 21 // (L * Hkv)))
        keep = max(8, _log(rng, max(1, L // 16), L))
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, L=L, ragged=ragged, keep=keep, sinks=rng.randint(0, 4),
                    recent=rng.randint(0, keep - 4))
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    kind = rng.choice(["one", "few", "many"])
    window, sinks = (_log(rng, 16, 8192), rng.choice([0, 1, 4, 64])) if rng.random() < 0.4 else (0, 0)
    L = _log(rng, 1, 65536 if kind == "one" else 16384)
    nq = 1 if kind == "one" else min(L, _log(rng, 2, 8) if kind == "few" else _log(rng, 9, 2048))
    nq = max(1, min(nq, 2 ** 30 // (L * Hkv * G)))
    B = max(1, min(B, 2 ** 21 // (L * Hkv), 2 ** 30 // (L * nq * Hkv * G)))
    case = _attend("", B, Hkv * G, Hkv, d, page, L, nq, ragged, dtype, window, sinks, rng.random() < 0.3)
    del case["name"]
    return case


def _sizes(case):
    """(lens, news) of the sequences, fixed by the case: the lengths with the new tokens, and the new tokens."""
    B, L, nq = case["B"], case["L"], case.get("nq", 0)
    r = random.Random(L * 131 + B)
    lens = [L] + [r.randint(max(1, L // 4), L) if case["ragged"] else L for _ in range(B - 1)]
    news = [min(n, nq if not case["ragged"] or i == 0 else r.randint(max(1, nq // 4), max(1, nq)))
            for i, n in enumerate(lens)]
    return lens, news


# --------------------------------------------------------------------------- inputs
def _pool(g, P, Hkv, page, d, dev):
    """Pages of codes as appended text leaves them: normal values around channel offsets, the largest of a page
    near the end of the e4m3 range; scales of a few binades. Slots past a sequence's end hold older tokens."""
    codes, scales = [], []
    for _ in range(2):
        c = torch.empty((P, Hkv, page, d), dtype=torch.uint8, device=dev)
        off = torch.randn((Hkv, 1, d), generator=g, device=dev) * 40
        step = max(1, (1 << 26) // (Hkv * page * d))
        for p in range(0, P, step):
            x = torch.randn((min(step, P - p), Hkv, page, d), generator=g, device=dev) * 70 + off
            c[p:p + step] = x.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        codes.append(c)
        scales.append(torch.randint(127 - 8, 127 - 5, (P, Hkv), generator=g, device=dev, dtype=torch.uint8))
    return [codes[0], codes[1], scales[0], scales[1]]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    lens, news = _sizes(case)
    npg = [-(-n // page) for n in lens]
    cols = max(npg)
    win, sinks = case.get("window", 0), case.get("sinks", 0)
    rows = []  # which pages of each sequence are held: under a window the pages that nothing can see have been freed
    for n, q, k in zip(lens, news, npg):
        lo = max(0, n - q - win + 1) // page if case["op"] == "attend" and win else 0
        rows.append([j for j in range(k) if j >= lo or j * page < sinks])
    P = sum(len(r) for r in rows) + 1
    perm = torch.randperm(P, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = 0
    for b, r in enumerate(rows):
        table[b, r] = perm[at:at + len(r)]
        at += len(r)
    s = {"case": case, "table": table.to(dev), "lens": torch.tensor(lens, dtype=torch.int32, device=dev),
         "cu": None, "max_len": max(lens), "max_q": max(news) if news else 0}
    s["k"], s["v"], s["ks"], s["vs"] = _pool(g, P, Hkv, page, d, dev)
    if case["op"] != "evict":
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        s["n"] = cu[-1]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case.get("nq") == 1:
            s["cu"] = None  # one token per sequence
    dt = _DT.get(case.get("dtype"))
    if case["op"] == "append":
        off = torch.randn((1, Hkv, d), generator=g, device=dev)
        s["xk"] = (torch.randn((s["n"], Hkv, d), generator=g, device=dev) + off).to(dt)
        s["xv"] = torch.randn((s["n"], Hkv, d), generator=g, device=dev).to(dt)
    elif case["op"] == "attend":
        s["q"] = torch.randn((s["n"], case["Hq"], d), generator=g, device=dev).to(dt)
        s["w"] = torch.zeros((B, Hkv, cols * page), device=dev) if case["weights"] else None
    else:
        # sums after some thousand steps: a few tokens with much weight, most with little
        s["w"] = torch.randn((B, Hkv, cols * page), generator=g, device=dev).mul_(1.5).exp_()
        dcols = -(-case["keep"] // page)
        DP = B * dcols
        s["dtable"] = torch.randperm(DP, generator=g, device=dev).to(torch.int32).view(B, dcols)
        s["dk"] = torch.zeros((DP, Hkv, page, d), dtype=torch.uint8, device=dev)
        s["dv"] = torch.zeros_like(s["dk"])
        s["dks"] = torch.zeros((DP, Hkv), dtype=torch.uint8, device=dev)
        s["dvs"] = torch.zeros_like(s["dks"])
        s["dw"] = torch.zeros((B, Hkv, dcols * page), device=dev)
    if own:
        import mixed_precision_bit_quant_b200 as mq
        s["mq"] = mq
        s["cache"] = mq.Kv8Cache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] == "evict":
            s["dst"] = mq.Kv8Cache(s["dk"], s["dv"], s["dks"], s["dvs"])
    return s


# --------------------------------------------------------------------------- the calls
def run(s):
    c = s["case"]
    if c["op"] == "append":
        if own:
            s["mq"].kv8_append(s["cache"], s["xk"], s["xv"], s["table"], s["lens"], cu=s["cu"], max_q=s["max_q"])
        else:
            _plain_append(s)
        return _cache_values(s, "")
    if c["op"] == "attend":
        if own:
            o, lse = s["mq"].kv8_attention(s["q"], s["cache"], s["table"], s["lens"], cu=s["cu"], max_q=s["max_q"],
                                           max_len=s["max_len"], window=c["window"], sinks=c["sinks"],
                                           weights=s["w"], want_lse=True)
        else:
            o, lse = _plain_attend(s)
        return {"o": o, "lse": lse, "w": s["w"]}
    if own:
        lens, kept = s["mq"].kv8_evict(s["cache"], s["table"], s["lens"], s["w"], s["dst"], s["dtable"], s["dw"],
                                       keep=c["keep"], sinks=c["sinks"], recent=c["recent"], max_len=s["max_len"])
    else:
        lens, kept = _plain_evict(s)
    return {"lens": lens, "kept": kept, "w": s["dw"], **_cache_values(s, "d")}


def _cache_values(s, p):
    """The state's own pages: codes as the e4m3 values that they are, scales as their exponents' codes."""
    return {"k": s[p + "k"].view(torch.float8_e4m3fn), "v": s[p + "v"].view(torch.float8_e4m3fn),
            "ks": s[p + "ks"], "vs": s[p + "vs"]}


# --------------------------------------------------------------------------- plain forms
def _rows(s, n):
    """Of each packed new token: its sequence and its place among the sequence's new tokens; and each sequence's
    number of new tokens."""
    B = s["lens"].shape[0]
    cu = s["cu"] if s["cu"] is not None else torch.arange(B + 1, device=s["lens"].device, dtype=torch.int32)
    j = torch.arange(n, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), j, right=True)
    return b, j - cu[b], cu[1:] - cu[:-1], cu


def _pow2(e):
    """2^e in 32 bits, exactly, for whole e in [-127, 127] (clamped to it)."""
    e = e.int().clamp(-127, 127)
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).int().view(torch.float32)


def _need(amax):
    """The smallest e with amax <= 448 * 2^e, at least -127."""
    m, x = torch.frexp(amax)
    return torch.where(amax > 0, x - 9 + (m > 0.875).int(), torch.full_like(x, -127)).clamp_(min=-127)


def _plain_append(s):
    page = s["case"]["page"]
    b, i, new, _ = _rows(s, s["n"])
    start = s["lens"] - new
    pos = start[b] + i
    pg = s["table"][b, (pos // page).long()].long()
    slot = (pos % page).long()
    first_col = (start // page).clamp(max=s["table"].shape[1] - 1).long()
    pg0 = s["table"].gather(1, first_col[:, None])[:, 0].long()
    old = (start % page) * (new > 0)  # tokens that the first page already holds
    for x, c, sc in ((s["xk"], s["k"], s["ks"]), (s["xv"], s["v"], s["vs"])):
        x = x.float()
        am = torch.zeros(sc.shape, device=sc.device).index_reduce_(0, pg, x.abs().amax(-1), "amax")
        e = _need(am)
        e_old = sc[pg0].int() - 127
        e0 = torch.where(old[:, None] > 0, torch.maximum(e[pg0], e_old), e[pg0])
        head = c[pg0]
        re = head.view(torch.float8_e4m3fn).float() * _pow2(e_old - e0)[:, :, None, None]
        keep = torch.arange(page, device=c.device)[None, :] < old[:, None]
        c[pg0] = torch.where(keep[:, None, :, None], re.to(torch.float8_e4m3fn).view(torch.uint8), head)
        e[pg0] = e0
        sc[pg] = (e[pg] + 127).to(torch.uint8)
        c[pg, :, slot] = (x * _pow2(-e[pg])[:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _dense(codes, scales, table):
    """[B, Hkv, T, d] in 32 bits: the values of each sequence's pages in order."""
    t = table.long().clamp(min=0)
    x = codes[t].view(torch.float8_e4m3fn).float().mul_(_pow2(scales[t].int() - 127)[..., None, None])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, d, win, sinks = c["B"], c["Hq"], c["Hkv"], c["d"], c["window"], c["sinks"]
    G, M = Hq // Hkv, s["max_q"]
    b, i, new, cu = _rows(s, s["n"])
    k, v = _dense(s["k"], s["ks"], s["table"]), _dense(s["v"], s["vs"], s["table"])
    T = k.shape[2]
    mi = torch.arange(M, device=k.device)
    q = s["q"][(cu[:-1, None] + mi).clamp(max=s["n"] - 1).long()].float()  # [B, M, Hq, d]
    q = q.view(B, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(B, Hkv, G, M, T)
    pos = (s["lens"] - new)[:, None] + mi
    t = torch.arange(T, device=k.device)
    see = (t <= pos[..., None]) & (mi < new[:, None])[..., None]
    if win:
        see &= (t > pos[..., None] - win) | (t < sinks)
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    x.div_(l.clamp(min=torch.finfo(torch.float32).tiny))
    if s["w"] is not None:
        s["w"] += x.sum((2, 3))
    o = torch.matmul(x.view(B, Hkv, G * M, T), v)
    o = o.view(B, Hkv, G, M, d).permute(0, 3, 1, 2, 4).reshape(B, M, Hq, d)
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2).reshape(B, M, Hq)
    return o[b, i].to(s["q"].dtype), lse[b, i]


def _plain_evict(s):
    c = s["case"]
    page, keep, sinks, recent, L = c["page"], c["keep"], c["sinks"], c["recent"], s["max_len"]
    lens = s["lens"]
    dev = lens.device
    T = s["table"].shape[1] * page
    t = torch.arange(T, device=dev)
    m = lens.clamp(max=keep)
    n = lens[:, None]
    force = (t < sinks) | (t >= n - recent)
    key = s["w"].masked_fill(force[:, None], math.inf).masked_fill((t >= n)[:, None], -math.inf)
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., :keep]
    rank = torch.arange(order.shape[-1], device=dev)
    ok = (rank < m[:, None])[:, None].expand(order.shape)
    idx = torch.where(ok, order, T).sort(-1).values  # the kept tokens, in their order
    at = idx.clamp(max=T - 1)
    kept = torch.full((*idx.shape[:2], keep), -1, dtype=torch.int32, device=dev)
    kept[..., :idx.shape[-1]] = torch.where(ok, idx, -1)
    s["dw"].zero_()
    s["dw"][..., :idx.shape[-1]] = torch.where(ok, s["w"].gather(2, at), 0)
    B, Hkv, R = idx.shape
    R2 = -(-R // page) * page
    pad = torch.nn.functional.pad(at, (0, R2 - R)), torch.nn.functional.pad(ok, (0, R2 - R))
    src = s["table"].gather(1, (pad[0] // page).view(B, -1)).view(B, Hkv, R2).long().clamp(min=0)
    h = torch.arange(Hkv, device=dev)[None, :, None]
    dpg = s["dtable"][:, :R2 // page].long()
    for codes, sc, dc, dsc in ((s["k"], s["ks"], s["dk"], s["dks"]), (s["v"], s["vs"], s["dv"], s["dvs"])):
        e = torch.where(pad[1], sc[src, h].int(), -1).view(B, Hkv, -1, page)
        top = e.amax(-1)
        x = codes[src, h, pad[0] % page].view(torch.float8_e4m3fn).float().view(B, Hkv, -1, page, codes.shape[-1])
        y = (x * _pow2(e - top[..., None])[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        was = dc[dpg].transpose(1, 2)
        dc[dpg] = torch.where(pad[1].view(B, Hkv, -1, page, 1), y, was).transpose(1, 2)
        dsc[dpg] = torch.where(top >= 0, top, dsc[dpg].transpose(1, 2).int()).to(torch.uint8).transpose(1, 2)
    return m, kept


# --------------------------------------------------------------------------- what a pass cannot do without
def _pairs(case):
    """Of the attention: (query, token) pairs that are visible, and the tokens that some query sees, over the batch."""
    pairs = tokens = 0
    win, sinks = case["window"], case["sinks"]
    for n, q in zip(*_sizes(case)):
        first = n - q  # position of the first new token
        if not win:
            pairs += q * (first + n + 1) // 2
            tokens += n
            continue
        for p in range(first, n):
            lo = max(0, p - win + 1)
            pairs += p + 1 - lo + min(sinks, lo)
        lo = max(0, first - win + 1)
        tokens += n - lo + min(sinks, lo)
    return pairs, tokens


def work(case):
    Hkv, d, page = case["Hkv"], case["d"], case["page"]
    lens, news = _sizes(case)
    if case["op"] == "append":
        n = sum(news)
        pages = sum(-(-a // page) - (a - q) // page for a, q in zip(lens, news))
        return {"bytes": 2.0 * n * Hkv * d * (2 + 1) + 2.0 * pages * Hkv + 4.0 * pages, "flops": 4.0 * n * Hkv * d}
    if case["op"] == "evict":
        m = [min(a, case["keep"]) for a in lens]
        return {"bytes": Hkv * (4.0 * sum(lens) + sum(m) * (4 * d + 8)), "flops": 1.0 * Hkv * sum(lens)}
    pairs, tokens = _pairs(case)
    n, Hq = sum(news), case["Hq"]
    b = 2.0 * tokens * Hkv * d + 2.0 * tokens // page * Hkv + 4.0 * n * Hq * d + 4.0 * n * Hq
    if case["weights"]:
        b += 8.0 * sum(lens) * Hkv
    return {"bytes": b, "flops": 4.0 * d * Hq * pairs}


# --------------------------------------------------------------------------- 64 bits
def _two(e):
    """2^e in 64 bits, exactly, for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _value(codes, scales):
    """What codes [.., page, d] and scale codes [..] stand for, in 64 bits."""
    c = codes.to(torch.int64)
    ex, man = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(ex > 0, (1 + man / 8) * _two(ex.double() - 7), man * 2.0 ** -9)
    val = torch.where(c >= 128, -mag, mag)
    return val if scales is None else val * _two(scales.double() - 127)[..., None, None]


def _round(x):
    """To the nearest e4m3 value, ties to the even one (|x| <= 448), in 64 bits."""
    step = _two(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -20))).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](s)


def _least(a):
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(a > 448 * _two(e), e + 1, e)
    e = torch.where(a <= 448 * _two(e - 1), e - 1, e)
    return torch.where(a > 0, e, torch.full_like(e, -127.0)).clamp(min=-127)


def _exact_append(s):
    page, lens, news = s["case"]["page"], *_sizes(s["case"])
    table = s["table"].tolist()
    out = {}
    for name, x in (("k", s["xk"].double()), ("v", s["xv"].double())):
        val, sc = _value(s[name], None).float(), s[name + "s"].double() - 127
        at = 0
        for b, (n, q) in enumerate(zip(lens, news)):
            pos = n - q
            while pos < n:
                j, lo = pos // page, pos % page
                hi = min(page, n - j * page)
                pg, new = table[b][j], x[at:at + hi - lo]  # [tokens, Hkv, d]
                e = _least(new.abs().amax((0, 2)))
                if lo:
                    e = torch.maximum(e, sc[pg])
                    val[pg, :, :lo] = _round(val[pg, :, :lo].double() * _two(sc[pg] - e)[:, None, None]).float()
                val[pg, :, lo:hi] = _round(new / _two(e)[None, :, None]).transpose(0, 1).float()
                sc[pg] = e
                at, pos = at + hi - lo, j * page + hi
        out[name], out[name + "s"] = val, sc + 127
    return out


def _exact_attend(s):
    c = s["case"]
    lens, news = _sizes(c)
    G, win, sinks, page = c["Hq"] // c["Hkv"], c["window"], c["sinks"], c["page"]
    if sum(n * q for n, q in zip(lens, news)) * c["Hq"] > 2 ** 32:
        return None
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(o.shape[:2], dtype=torch.float64, device=o.device)
    w = None if s["w"] is None else s["w"].double()
    at = 0
    for b, (n, q) in enumerate(zip(lens, news)):
        first = n - q
        t = torch.arange(n, device=o.device)
        if win:
            t = t[(t < sinks) | (t > first - win)]
        pg, sl = s["table"][b].long()[t // page], t % page
        pos = torch.arange(first, n, device=o.device)[:, None]
        hide = t > pos
        if win:
            hide |= (t <= pos - win) & (t >= sinks)
        for h in range(c["Hkv"]):
            k = _value(s["k"][pg, h, sl][:, None], s["ks"][pg, h])[:, 0]
            v = _value(s["v"][pg, h, sl][:, None], s["vs"][pg, h])[:, 0]
            for g in range(h * G, (h + 1) * G):
                x = s["q"][at:at + q, g].double() @ k.T / math.sqrt(c["d"])
                x[hide] = -math.inf
                z = torch.logsumexp(x, 1)
                p = torch.exp(x - z[:, None])
                o[at:at + q, g], lse[at:at + q, g] = p @ v, z
                if w is not None:
                    w[b, h, t] += p.sum(0)
        at += q
    return {"o": o, "lse": lse, "w": w}


def _exact_evict(s):
    c = s["case"]
    page, keep = c["page"], c["keep"]
    lens, _ = _sizes(c)
    dw = torch.zeros(s["dw"].shape, dtype=torch.float64, device=s["dw"].device)
    kept = torch.full((c["B"], c["Hkv"], keep), -1, dtype=torch.int64)
    out = {}
    for name in ("k", "v"):
        out[name] = torch.zeros(s["dk"].shape, device=s["dk"].device)
        out[name + "s"] = torch.zeros(s["dks"].shape, dtype=torch.int64, device=s["dk"].device)
    table, dtable = s["table"].tolist(), s["dtable"].tolist()
    for b, n in enumerate(lens):
        m, pgs = min(n, keep), torch.tensor(table[b], device=dw.device)
        for h in range(c["Hkv"]):
            w = s["w"][b, h, :n].double().cpu().numpy()
            lo, hi = min(c["sinks"], n), max(n - c["recent"], 0)
            free = list(range(lo, max(lo, hi)))
            must = n - len(free)
            free.sort(key=lambda t: (-w[t], t))
            drop = set(free[max(0, m - must):])
            ids = [t for t in range(n) if t not in drop]
            kept[b, h, :m] = torch.tensor(ids)
            ids = torch.tensor(ids, device=dw.device)
            dw[b, h, :m] = s["w"][b, h, ids].double()
            pg, sl = pgs[ids // page], ids % page
            for name in ("k", "v"):
                fill = -m % page
                sc = torch.nn.functional.pad(s[name + "s"][pg, h].double(), (0, fill), value=-1).view(-1, page)
                val = torch.nn.functional.pad(_value(s[name][pg, h, sl], None), (0, 0, 0, fill)).view(*sc.shape, -1)
                top = sc.amax(1)
                y = _round(val * _two((sc - top[:, None]).clamp(min=-300))[..., None]).float()
                to = torch.tensor(dtable[b][:top.shape[0]], device=dw.device)
                out[name][to, h] = y
                out[name + "s"][to, h] = top.long()
    return {"lens": torch.tensor([min(n, keep) for n in lens]), "kept": kept, "w": dw, **out}
