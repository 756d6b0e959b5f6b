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
