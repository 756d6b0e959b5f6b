"""Timed cases of the 4-bit cache: writing it, reading it back, and attention over it.

Each case is one call (writing: the call and the read-back of what it wrote) as a
serving loop makes it.  With `own` false, `run` computes the operator in a plain
form (torch products, sums, exp, comparisons and indexing, in 32 bits); with
`own` true it calls the library.  `exact` evaluates the definitions in 64 bits.

The cache holds, per page, head and block of 16 tokens: K codes, K metadata, V
codes, V metadata, as 32-bit words.  A code word has 8 codes (lowest bits first,
each q + 8) of channels 8w .. 8w+7 of one token; a metadata word has the bf16
scale (low half) and bias of one group of channels.
  K codes  [token][word]: word w at 2 (w % 4) + w / 4 for heads of 64, else at
           16 (w / 16) + 4 (w % 4) + (w % 16) / 4
  V codes  [word][token]: token t at 4 (t / 2 % 4) + t % 2 + 2 (t / 8)
  metadata [token][group]
"""
import math

import numpy as np
import torch

own = False

LIMIT = 32768.0      # larger magnitudes are stored as this
TINY = 2.0 ** -100   # smaller scales are stored as 0


def listed():
    return [
        # one stream's new token into its cache: the smallest call of a decode step
        dict(name="append step b1", op="append", B=1, L=1, past=1000, ragged=False, HK=8, D=128, gs=64, page=64, dtype="bf16"),
        # a full continuous batch, one token each, large heads
        dict(name="append step b256", op="append", B=256, L=1, past=300, ragged=True, HK=4, D=256, gs=128, page=16, dtype="fp16"),
        # a long prompt's keys and values
        dict(name="append prompt 8192", op="append", B=1, L=8192, past=0, ragged=False, HK=8, D=128, gs=64, page=64, dtype="bf16"),
        # cached prefixes of odd lengths taken out in fp32
        dict(name="load ragged D64 fp32", op="load", B=3, L=1111, past=0, ragged=True, HK=12, D=64, gs=64, page=32, dtype="fp32"),
        # a batch of cached contexts taken out in bf16
        dict(name="load 16x4096", op="load", B=16, L=4096, past=0, ragged=False, HK=8, D=128, gs=64, page=64, dtype="bf16"),
        # one stream, one token, an ordinary context: what a single user waits for
        dict(name="attend b1 4k", op="attend", B=1, L=1, past=4095, ragged=False, HQ=32, HK=8, D=128, gs=64, page=64, window=0, dtype="bf16"),
        # one stream, one token, a very long context, large heads
        dict(name="attend b1 200k", op="attend", B=1, L=1, past=200000, ragged=False, HQ=24, HK=4, D=256, gs=128, page=128, window=0, dtype="bf16"),
        # a full continuous batch: the cache's traffic
        dict(name="attend b64 8k", op="attend", B=64, L=1, past=8000, ragged=True, HQ=40, HK=8, D=128, gs=64, page=64, window=0, dtype="bf16"),
        # verifier windows of a few tokens, small heads, fp32 activations, a sliding window
        dict(name="attend windows fp32", op="attend", B=7, L=5, past=1500, ragged=True, HQ=12, HK=12, D=64, gs=64, page=16, window=700, dtype="fp32"),
        # one long prompt
        dict(name="attend prompt 8192", op="attend", B=1, L=8192, past=0, ragged=False, HQ=32, HK=8, D=128, gs=64, page=64, window=0, dtype="bf16"),
        # the next piece of a prompt whose first part is cached, large heads
        dict(name="attend piece 1000 over 15k", op="attend", B=1, L=1000, past=15000, ragged=False, HQ=24, HK=4, D=256, gs=64, page=64, window=0, dtype="fp16"),
        # several short prompts of odd lengths, small heads, a sliding window
        dict(name="attend ragged prompts", op="attend", B=6, L=650, past=200, ragged=True, HQ=16, HK=4, D=64, gs=64, page=32, window=512, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    D = rng.choice([64, 128, 128, 256])
    gs = 64 if D == 64 else rng.choice([64, 64, 128])
    HK = rng.choice([1, 2, 4, 8, 8, 12])
    page = rng.choice([16, 32, 64, 64, 128])
    x = rng.random()
    if x < 0.3:
        T = _log_int(rng, 1, 8192 * 1024 // (HK * D))     # tokens in all
        op = rng.choice(["append", "append", "load"])
        one = op == "append" and rng.random() < 0.4
        B = min(T, 512) if one else _log_int(rng, 1, min(T, 32))
        return dict(op=op, B=B, L=1 if one else max(1, T // B), past=_log_int(rng, 1, 2000) if op == "append" else 0,
                    ragged=rng.random() < 0.6, HK=HK, D=D, gs=gs, page=page, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    r = rng.choice([1, 2, 4, 5, 6, 8, 16])
    window = rng.choice([0, 0, 0, _log_int(rng, 16, 4096)])
    if x < 0.7:      # decode: one token or a window
        B = _log_int(rng, 1, 128)
        L = rng.choice([1, 1, 1, 1, 2, 3, 4, 8])
        past = _log_int(rng, 1, min(200000, 64 * 8000 * 1024 // (HK * D * B)))
        return dict(op="attend", B=B, L=L, past=past, ragged=rng.random() < 0.7, HQ=HK * r, HK=HK, D=D, gs=gs, page=page,
                    window=window, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    B = _log_int(rng, 1, 8)
    L = _log_int(rng, 20, 8192 // B)
    past = rng.choice([0, _log_int(rng, 1, 16000)])
    while B * L * (past + L / 2) * HK * r * D > 8192 * 4096 * 32 * 128:
        r, past, L = max(1, r // 2), past // 2, L if r > 1 else L // 2 + 1
    return dict(op="attend", B=B, L=L, past=past, ragged=rng.random() < 0.7, HQ=HK * r, HK=HK, D=D, gs=gs, page=page,
                window=window, dtype=rng.choice(["bf16", "bf16", "fp16"]))


_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lengths(case):
    """New and cached tokens of each sequence, the same for every seed: L and past each, or (ragged) L (if it is
    more than one) and past times about 1/4 to 7/4."""
    B, L, past = case["B"], case["L"], case["past"]
    if not case["ragged"]:
        return [L] * B, [past] * B
    f = [0.25 + 1.5 * ((i * 0.6180339887 + 0.37) % 1.0) for i in range(B)]
    new = [L if L == 1 else max(1, int(L * f[(i * 7 + 3) % B])) for i in range(B)]
    return new, [int(past * f[i]) for i in range(B)]


def _word_places(D):
    """Within a block: where word w of token t's K and V codes is, int64 [16, D/8] each, and the blocks' words."""
    w, t = torch.arange(D // 8), torch.arange(16)[:, None]
    pos = 2 * (w % 4) + w // 4 if D == 64 else 16 * (w // 16) + 4 * (w % 4) + (w % 16) // 4
    return t * (D // 8) + pos, w * 16 + (4 * (t // 2 % 4) + t % 2 + 2 * (t // 8))


def _quantise(x, gs):
    """x fp32 [..., D] -> code words int32 [..., D/8] and metadata words int32 [..., D/gs]."""
    dev = x.device
    g = x.clamp(-LIMIT, LIMIT).unflatten(-1, (-1, gs))
    lo, hi = g.amin(-1), g.amax(-1)
    b = (lo + 8.0 * ((hi - lo) * torch.tensor(1 / 15, dtype=torch.float32, device=dev))).bfloat16()
    s = torch.maximum((hi - b.float()) * torch.tensor(1 / 7, dtype=torch.float32, device=dev), (b.float() - lo) * 0.125).bfloat16()
    s = torch.where(s < TINY, 0.0, s)
    inv = torch.where(s > 0, torch.ones_like(lo) / s.float(), 0.0)
    q = torch.round((g - b.float()[..., None]) * inv[..., None]).nan_to_num(0.0).clamp(-8, 7)
    u = (q.to(torch.int64) + 8).flatten(-2).unflatten(-1, (-1, 8))
    words = (u << (4 * torch.arange(8, device=dev))).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return words, torch.stack([s, b], -1).view(torch.int32)[..., 0]


def _pages(table, pos, seq, page):
    """Page and block of each position and its place in the block."""
    return table.long()[seq, pos // page], pos % page // 16, pos % 16


def _put(cache, case, table, pos, seq, k, v):
    """k, v [T, HK, D] quantised into the pages of positions `pos` of sequences `seq`."""
    D, gs, HK = case["D"], case["gs"], case["HK"]
    W, G = D // 8, D // gs
    words = cache.view(torch.int32)
    pg, blk, t = _pages(table, pos, seq, case["page"])
    base = (((pg[:, None] * HK + torch.arange(HK, device=pos.device)) * (case["page"] // 16) + blk[:, None]) * words.shape[-1])[..., None]
    flat = words.view(-1)
    pk, pv = (p.to(pos.device)[t][:, None] for p in _word_places(D))
    meta = (t[:, None] * G + torch.arange(G, device=pos.device))[:, None]
    for x, p, at in ((k, pk, 0), (v, pv, 16 * (W + G))):
        codes, m = _quantise(x.float(), gs)
        flat[base + at + p] = codes
        flat[base + at + 16 * W + meta] = m


def _get(cache, case, table, pos, seq):
    """k, v fp32 [T, HK, D] of positions `pos` of sequences `seq`."""
    D, gs, HK = case["D"], case["gs"], case["HK"]
    W, G = D // 8, D // gs
    words = cache.view(torch.int32)
    pg, blk, t = _pages(table, pos, seq, case["page"])
    base = (((pg[:, None] * HK + torch.arange(HK, device=pos.device)) * (case["page"] // 16) + blk[:, None]) * words.shape[-1])[..., None]
    flat = words.view(-1)
    pk, pv = (p.to(pos.device)[t][:, None] for p in _word_places(D))
    meta = (t[:, None] * G + torch.arange(G, device=pos.device))[:, None]
    out = []
    for p, at in ((pk, 0), (pv, 16 * (W + G))):
        q = ((flat[base + at + p][..., None] >> (4 * torch.arange(8, device=pos.device, dtype=torch.int32))) & 15) - 8
        m = flat[base + at + 16 * W + meta][..., None].view(torch.bfloat16).float()   # scale, bias
        out.append((q.float().flatten(-2).unflatten(-1, (G, gs)) * m[..., :1] + m[..., 1:]).flatten(-2))
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1_000_003 + 29)
    dt, D, HK, page = _DT[case["dtype"]], case["D"], case["HK"], case["page"]

    def randn(*shape):
        return torch.randn(shape, device=dev, generator=g)

    new, past = _lengths(case)
    B, T = case["B"], sum(new)
    lengths = [n + p for n, p in zip(new, past)]
    per = [-(-n // page) for n in lengths]
    # pages in any order; what nothing has written yet holds anything
    n_pages, width = sum(per) + 3, max(per) + 1
    order = torch.randperm(n_pages, device=dev, generator=g).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    first = 0
    for b, n in enumerate(per):
        table[b, :n] = order[first:first + n]
        first += n
    block = 16 * (D + 8 * (D // case["gs"]))
    cache = torch.randint(-2 ** 31, 2 ** 31 - 1, (n_pages, HK, page // 16, block // 4), dtype=torch.int32, device=dev, generator=g).view(torch.uint8)

    # keys: a mean per channel and a few large channels; values without
    mean = 0.5 * randn(HK, D)
    size = torch.where(torch.rand(HK, D, device=dev, generator=g) < 0.03, 4.0, 1.0)

    def key(n):
        return (randn(n, HK, D) + mean) * size

    have = lengths if case["op"] != "append" else past
    for b, n in enumerate(have):
        for a in range(0, n, 32768):
            pos = torch.arange(a, min(n, a + 32768), device=dev)
            _put(cache, case, table, pos, torch.full_like(pos, b), key(len(pos)), randn(len(pos), HK, D))

    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s = dict(op=case["op"], case=case, cache=cache, table=table, new=new, past=past, T=T,
             lengths=torch.tensor(lengths, dtype=torch.int32, device=dev), cu_seqlens=torch.from_numpy(starts).to(dev),
             pos=torch.cat([torch.arange(p, p + n, device=dev) for n, p in zip(new, past)]),
             seq=torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(new, device=dev)),
             max_q=max(new), max_len=max(lengths), dtype=dt)
    # k and v (or q) as columns of one projection's rows
    if case["op"] == "append":
        row = torch.cat([key(T).view(T, HK * D), randn(T, HK * D)], 1).to(dt)
        s["k"], s["v"] = row[:, :HK * D].view(T, HK, D), row[:, HK * D:].view(T, HK, D)
    elif case["op"] == "attend":
        HQ = case["HQ"]
        row = randn(T, (HQ + 2 * HK) * D).to(dt)
        s["q"] = row[:, :HQ * D].view(T, HQ, D)
        s["scale"] = D ** -0.5
    return s


def _plain_attend(s):
    case, q = s["case"], s["q"].float()
    HQ, HK, D, window = case["HQ"], case["HK"], case["D"], case["window"]
    r, dev = HQ // HK, q.device
    o = torch.empty(s["T"], HQ, D, device=dev)
    lse = torch.empty(s["T"], HQ, device=dev)
    t0 = 0
    for b, (n, p) in enumerate(zip(s["new"], s["past"])):
        first = 0 if window == 0 else max(0, p + 1 - window)
        pos = torch.arange(first, p + n, device=dev)
        k, v = (x.transpose(0, 1) for x in _get(s["cache"], case, s["table"], pos, torch.full_like(pos, b)))   # [HK, len, D]
        step = max(1, (1 << 29) // (HQ * len(pos)))
        for a in range(0, n, step):
            e = min(n, a + step)
            at = torch.arange(p + a, p + e, device=dev)[:, None]
            seen = pos[None] <= at
            if window:
                seen &= pos[None] > at - window
            qb = q[t0 + a:t0 + e].unflatten(1, (HK, r)).permute(1, 2, 0, 3).flatten(1, 2)        # [HK, r * rows, D]
            x = (qb @ k.transpose(1, 2) * s["scale"]).unflatten(1, (r, e - a)).masked_fill_(~seen, -math.inf)
            m = x.amax(-1, keepdim=True)
            x = torch.exp(x - m)
            l = x.sum(-1, keepdim=True)
            y = (x.flatten(1, 2) @ v).unflatten(1, (r, e - a)) / l
            o[t0 + a:t0 + e] = y.permute(2, 0, 1, 3).flatten(1, 2)
            lse[t0 + a:t0 + e] = (m + torch.log(l))[..., 0].permute(2, 0, 1).flatten(1, 2)
        t0 += n
    return {"o": o.to(s["dtype"]), "lse": lse}


def run(s):
    case = s["case"]
    if own:
        from bit_affine_quantized_g128_gb300 import q1
        kw = dict(cu_seqlens=s["cu_seqlens"])
        if s["op"] == "attend":
            o, lse = q1.kv_attention(s["q"], s["cache"], s["table"], s["lengths"], max_q=s["max_q"], max_len=s["max_len"],
                                     scale=s["scale"], window=case["window"], return_lse=True, **kw)
            return {"o": o, "lse": lse}
        if s["op"] == "append":
            q1.kv_store(s["cache"], s["k"], s["v"], s["table"], s["lengths"], **kw)
        k, v = q1.kv_load(s["cache"], s["table"], s["lengths"], s["T"], dtype=s["dtype"], **kw)
        return {"k": k, "v": v}
    if s["op"] == "attend":
        return _plain_attend(s)
    if s["op"] == "append":
        _put(s["cache"], case, s["table"], s["pos"], s["seq"], s["k"], s["v"])
    k, v = _get(s["cache"], case, s["table"], s["pos"], s["seq"])
    return {"k": k.to(s["dtype"]), "v": v.to(s["dtype"])}


def work(case):
    new, past = _lengths(case)
    es = 4 if case["dtype"] == "fp32" else 2
    D, HK, T = case["D"], case["HK"], sum(new)
    cached = HK * (D + 8 * (D // case["gs"]))     # bytes of a token's K and V in the cache
    if case["op"] != "attend":
        dense = T * HK * D * 2 * es
        return {"bytes": T * cached + dense * (2 if case["op"] == "append" else 1), "flops": T * HK * D * 2 * (8 if case["op"] == "append" else 2)}
    HQ, window = case["HQ"], case["window"]
    tokens = pairs = 0
    for n, p in zip(new, past):
        w = window if window else p + n
        tokens += min(p + n, n + w - 1)
        full = max(0, p + n - max(p, w))            # rows with w tokens in sight, the others see 1, 2, .. more than before
        pairs += full * w + (n - full) * p + (n - full) * (n - full + 1) // 2
    return {"bytes": tokens * cached + T * HQ * (2 * D * es + 4), "flops": 4 * D * HQ * pairs}


def _exact_codes(x, gs):
    """The definition on the host, [..., D]: codes q and the scales and biases of their groups, the roundings to
    fp32 and bf16 that it names done one by one."""
    f = np.float32

    def bf16(a):
        u = a.astype(f).view(np.uint32).astype(np.uint64)
        return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(f)

    g = np.clip(x.astype(f), f(-LIMIT), f(LIMIT)).reshape(*x.shape[:-1], -1, gs)
    lo, hi = g.min(-1), g.max(-1)
    b = bf16(lo + f(8) * ((hi - lo) * f(1 / 15)))
    s = bf16(np.maximum((hi - b) * f(1 / 7), (b - lo) * f(0.125)))
    s[s < TINY] = 0
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, f(1) / s, f(0)).astype(f)
    q = np.clip(np.rint((g - b[..., None]) * inv[..., None]), -8, 7)
    return (q.astype(np.float64) * s[..., None].astype(np.float64) + b[..., None].astype(np.float64)).reshape(x.shape)


def _exact_cached(s, b, first, last):
    """K and V of positions first .. last-1 of sequence b in float64 [HK, n, D], nibble by nibble."""
    case = s["case"]
    D, gs, HK, page = case["D"], case["gs"], case["HK"], case["page"]
    G = D // gs
    kat, vat = np.zeros((16, D), np.int64), np.zeros((16, D), np.int64)   # byte of each code; the shift is 4 (c % 2)
    for t in range(16):
        place = [0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15][t]
        for c in range(D):
            w, j = c // 8, c % 32 // 8                    # j: the lane quarter of a group of 32 channels
            half, sub = c // 128, c % 128 // 32
            kat[t, c] = 4 * (t * (D // 8) + half * 16 + j * min(4, D // 32) + sub) + c % 8 // 2
            vat[t, c] = 8 * D + 64 * G + 4 * (16 * w + place) + c % 8 // 2
    pos = np.arange(first, last)
    table = s["table"][b].cpu().numpy()
    dev = s["cache"].device
    pg = torch.from_numpy(table[pos // page].astype(np.int64)).to(dev)
    rec = s["cache"][pg, :, torch.from_numpy(pos % page // 16).to(dev)]                # [n, HK, bytes]
    t = torch.from_numpy(pos % 16).to(dev)
    shift = (4 * (torch.arange(D, device=dev) % 2)).to(torch.uint8)
    out = []
    for at, meta in ((kat, 8 * D), (vat, 16 * D + 64 * G)):
        idx = torch.from_numpy(at).to(dev)[t][:, None].expand(-1, HK, -1)
        code = ((rec.gather(2, idx) >> shift) & 15).double() - 8
        mi = (meta + 4 * (t[:, None] * G + torch.arange(D, device=dev) // gs))[:, None].expand(-1, HK, -1)

        def half(o):
            bits = rec.gather(2, mi + o).int() + 256 * rec.gather(2, mi + o + 1).int()
            return (bits << 16).view(torch.float32).double()

        out.append((code * half(0) + half(2)).transpose(0, 1))
    return out


def exact(case, seed):
    if work(case)["flops"] > 1.2e12 or work(case)["bytes"] > 2e9:
        return None   # over 20 seconds
    s = prepare(case, seed)
    if case["op"] == "append":
        k, v = (torch.from_numpy(_exact_codes(s[n].float().cpu().numpy(), case["gs"])) for n in ("k", "v"))
        return {"k": k, "v": v}
    if case["op"] == "load":
        parts = [_exact_cached(s, b, p, p + n) for b, (n, p) in enumerate(zip(s["new"], s["past"]))]
        return {n: torch.cat([x[i].transpose(0, 1) for x in parts]) for i, n in enumerate(("k", "v"))}
    HQ, HK, D, window = case["HQ"], case["HK"], case["D"], case["window"]
    q = s["q"].double()
    o = torch.zeros(s["T"], HQ, D, dtype=torch.float64, device=q.device)
    lse = torch.zeros(s["T"], HQ, dtype=torch.float64, device=q.device)
    t0 = 0
    for b, (n, p) in enumerate(zip(s["new"], s["past"])):
        for a in range(0, n, 512):      # rows a .. e-1 and the tokens that any of them sees
            e = min(n, a + 512)
            first = max(0, p + a + 1 - window) if window else 0
            k, v = _exact_cached(s, b, first, p + e)
            row = torch.arange(p + a, p + e, device=q.device)[:, None]
            col = torch.arange(first, p + e, device=q.device)[None]
            hidden = (col > row) | ((col <= row - window) if window else torch.zeros_like(col > row))
            for h in range(HQ):
                x = (q[t0 + a:t0 + e, h] @ k[h // (HQ // HK)].T) * s["scale"]
                x[hidden] = -math.inf
                z = torch.logsumexp(x, 1)
                lse[t0 + a:t0 + e, h] = z
                o[t0 + a:t0 + e, h] = torch.exp(x - z[:, None]) @ v[h // (HQ // HK)]
        t0 += n
    return {"o": o, "lse": lse}
