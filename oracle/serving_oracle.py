"""Plain CPU implementations, in float64, of the serving operators: the gated
delta rule and the sampler.  They follow the definitions one token (one row) at
a time and share no code with the library.
"""
import numpy as np


def gated_delta(q, k, v, g, beta, state, starts, scale, l2norm, slots=None, fresh=None):
    """o [T, HV, DV], the updated state pool, and per sequence and head the largest
    column norms [DV] and Frobenius norm that its state had (bounds on what
    rounding can move)."""
    q, k, v, g, beta = (np.asarray(x, np.float64) for x in (q, k, v, g, beta))
    state = np.array(state, np.float64)
    T, HK, DK = q.shape
    HV, DV = v.shape[1:]
    o = np.zeros((T, HV, DV))
    B = len(starts) - 1
    colmax = np.zeros((B, HV, DV))
    if l2norm:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    q, k = np.repeat(q, HV // HK, 1), np.repeat(k, HV // HK, 1)
    for b in range(B):
        slot = b if slots is None else int(slots[b])
        have = 0 <= slot < state.shape[0]
        S = state[slot].copy() if have and not (fresh is not None and fresh[b]) else np.zeros((HV, DK, DV))
        colmax[b] = np.sqrt((S * S).sum(1))
        for t in range(starts[b], starts[b + 1]):
            S = S * np.exp(g[t])[:, None, None]
            d = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
            S = S + k[t][:, :, None] * d[:, None, :]
            o[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
            colmax[b] = np.maximum(colmax[b], np.sqrt((S * S).sum(1)))
        if have:
            state[slot] = S
    return o, state, colmax


def delta_sizes(k, v, g, beta, state, starts, l2norm, slots=None, fresh=None):
    """What rounding at a token can be relative to, per value column: the largest norm
    that the column's state or a token's write had, decayed by the gates since (a
    correction that erases does not make it smaller).  [T, HV, DV], and what it
    is after the last token, [B, HV, DV]."""
    k, v, g, beta, state = (np.asarray(x, np.float64) for x in (k, v, g, beta, state))
    T, HK, DK = k.shape
    HV, DV = v.shape[1:]
    if l2norm:
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    k = np.repeat(k, HV // HK, 1)
    sizes, last = np.zeros((T, HV, DV)), np.zeros((len(starts) - 1, HV, DV))
    for b in range(len(starts) - 1):
        slot = b if slots is None else int(slots[b])
        have = 0 <= slot < state.shape[0]
        S = state[slot].copy() if have and not (fresh is not None and fresh[b]) else np.zeros((HV, DK, DV))
        z = np.sqrt((S * S).sum(1))
        for t in range(starts[b], starts[b + 1]):
            a = np.exp(g[t])[:, None]
            S = S * a[:, :, None]
            S = S + k[t][:, :, None] * (beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t])))[:, None, :]
            write = beta[t][:, None] * np.linalg.norm(k[t], axis=-1)[:, None] * np.abs(v[t])
            z = np.maximum(np.maximum(a * z, write), np.sqrt((S * S).sum(1)))
            sizes[t] = z
        last[b] = z
    return sizes, last


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, prob) of one row."""
    x = np.asarray(logits, np.float64).copy()
    x[np.isnan(x)] = -np.inf
    m = x.max()
    if m == -np.inf:
        return -1, 0.0
    if not temperature > 0:
        return int(np.argmax(x)), 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(x == m, 1.0, 0.0) if m == np.inf else np.exp((x - m) / temperature)
    w[np.isnan(w)] = 0.0
    order = np.argsort(-x, kind="stable")
    order = order[w[order] > 0]
    if 0 < top_k < len(x):
        order = order[:top_k]
    if top_p < 1:
        c = np.cumsum(w[order])
        before = np.concatenate([[0.0], c[:-1]])
        keep = before < top_p * c[-1]
        keep[0] = True
        order = order[keep]
    if min_p > 0:
        order = order[w[order] >= min(min_p, 1.0)]
    ids = np.sort(order)
    c = np.cumsum(w[ids])
    at = 0 if not u > 0 else min(int((c <= u * c[-1]).sum()), len(ids) - 1)
    return int(ids[at]), float(w[ids[at]] / c[-1])


# ---- the 4-bit cache
def _bf16(x):
    """fp32 rounded to the nearest bf16 (ties to even), as fp32."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def kv_quantise(x, gs):
    """q int [..., D], scale and bias fp32 [..., D/gs] of rows x fp32 [..., D]: one fp32 rounding per operation."""
    f = np.float32
    x = np.asarray(x, f)
    g = np.clip(x, f(-32768), f(32768)).reshape(*x.shape[:-1], x.shape[-1] // gs, gs)
    bad = np.isnan(g).any(-1)
    g = np.where(bad[..., None], f(0), g)
    lo, hi = g.min(-1), g.max(-1)
    bias = _bf16(lo + f(8) * ((hi - lo) * f(1 / 15)))
    scale = _bf16(np.maximum((hi - bias) * f(1 / 7), (bias - lo) * f(0.125)))
    scale = np.where(scale < 2.0 ** -100, f(0), scale)
    inv = np.where(scale > 0, f(1) / np.where(scale > 0, scale, f(1)), f(0)).astype(f)
    q = np.clip(np.rint((g - bias[..., None]) * inv[..., None]), -8, 7).astype(np.int64).reshape(x.shape)
    nan = np.array(0x7FC00000, np.uint32).view(f)
    return q, np.where(bad, nan, scale).astype(f), np.where(bad, nan, bias).astype(f)


def kv_values(q, scale, bias):
    """The cached values in fp32: q scale + bias, rounded once."""
    gs = q.shape[-1] // scale.shape[-1]
    s, b = (np.repeat(np.asarray(a, np.float64), gs, -1) for a in (scale, bias))
    return (q * s + b).astype(np.float32)


def kv_block(kq, ks, kb, vq, vs, vb):
    """The bytes of a block: codes int [16, D] and fp32 (bf16 values) metadata [16, G] of 16 tokens of one head."""
    D = kq.shape[1]
    out = []
    for q, s, b, v in ((kq, ks, kb, False), (vq, vs, vb, True)):
        words = np.zeros(2 * D, np.uint32)
        for t in range(16):
            for w in range(D // 8):
                word = 0
                for i in range(8):
                    word |= (int(q[t, 8 * w + i]) + 8) << (4 * i)
                if v:
                    at = 16 * w + 4 * (t // 2 % 4) + t % 2 + 2 * (t // 8)
                elif D == 64:
                    at = t * 8 + 2 * (w % 4) + w // 4
                else:
                    at = t * (D // 8) + 16 * (w // 16) + 4 * (w % 4) + w % 16 // 4
                words[at] = word
        meta = (s.astype(np.float32).view(np.uint32) >> 16) | (b.astype(np.float32).view(np.uint32) & 0xFFFF0000)
        out += [words, meta.astype(np.uint32).reshape(-1)]
    return np.concatenate(out).view(np.uint8)


def kv_attention(q, k, v, pos, scale, causal=True, window=0, there=None):
    """o, lse, and what rounding errors of o are relative to, of rows q [n, HQ, D] at positions pos [n] over k, v [len,
    HK, D] (float64).  `there` [len]: tokens that have a page.  Returns o, lse [n, HQ], sum p |v| [n, HQ, D] and the
    largest scale sum_d |q_d k_d| of a row [n, HQ]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, HQ, D = q.shape
    L, HK = k.shape[:2]
    o, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, big = np.full((n, HQ), -np.inf), np.zeros((n, HQ))
    j = np.arange(L)
    for i in range(n):
        see = (j <= pos[i]) if causal else np.full(L, pos[i] >= 0)
        if window:
            see &= j > pos[i] - window
        if there is not None:
            see &= there
        if not see.any():
            continue
        for h in range(HQ):
            kk, vv = k[see, h // (HQ // HK)], v[see, h // (HQ // HK)]
            x = scale * (kk @ q[i, h])
            m = x.max()
            p = np.exp(x - m)
            s = p.sum()
            o[i, h], size[i, h] = p @ vv / s, p @ np.abs(vv) / s
            lse[i, h] = m + np.log(s)
            big[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return o, lse, size, big
