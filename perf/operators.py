"""Timed cases of the serving operators: the gated delta rule and the sampler.

Each case is one call as a serving loop makes it.  With `own` false, `run`
computes the operator in a plain form (torch products, sums, exp, comparisons,
sorting and indexing, in 32 or 64 bits); with `own` true it calls the
library.  `exact` evaluates the definitions in 64 bits, token by token (delta
rule) or row by row (sampler).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6     # added to a key's or query's sum of squares before its root
CHUNK = 64     # tokens per chunk of the plain delta rule


def listed():
    return [
        # one stream decoding one token: what a single user waits for
        dict(name="delta step b1", op="delta", B=1, L=1, ragged=False, HK=16, HV=32, DK=128, DV=128, dtype="bf16", fresh=False),
        # a full continuous batch, one token each: state traffic
        dict(name="delta step b64", op="delta", B=64, L=1, ragged=False, HK=16, HV=32, DK=128, DV=128, dtype="bf16", fresh=False),
        # verifier windows: a few tokens for each of a few streams, fp16
        dict(name="delta window 8x8", op="delta", B=8, L=8, ragged=False, HK=16, HV=48, DK=128, DV=128, dtype="fp16", fresh=False),
        # small heads, fp32 activations, windows of odd lengths
        dict(name="delta ragged fp32", op="delta", B=7, L=29, ragged=True, HK=6, HV=12, DK=64, DV=64, dtype="fp32", fresh=False),
        # a prompt chunk that goes on from cached states, several short ragged prompts
        dict(name="delta ragged prompts", op="delta", B=5, L=777, ragged=True, HK=8, HV=16, DK=128, DV=64, dtype="fp16", fresh=False),
        # one long prompt
        dict(name="delta prompt 8192", op="delta", B=1, L=8192, ragged=False, HK=16, HV=32, DK=128, DV=128, dtype="bf16", fresh=True),
        # a batch of prompts of different lengths
        dict(name="delta prompts 8x2048", op="delta", B=8, L=2048, ragged=True, HK=16, HV=32, DK=128, DV=128, dtype="bf16", fresh=True),
        # one row from the tied head, the usual three truncations
        dict(name="sample b1", op="sample", B=1, V=152064, dtype="bf16", mode="all"),
        # a small batch of requests with settings of their own, fp32 logits
        dict(name="sample b9 fp32", op="sample", B=9, V=152064, dtype="fp32", mode="mixed"),
        # a full batch, temperature only: every token can be drawn
        dict(name="sample b64", op="sample", B=64, V=152064, dtype="bf16", mode="temperature"),
        # a large batch over a smaller vocabulary of odd size, nucleus only
        dict(name="sample b301 v32003", op="sample", B=301, V=32003, dtype="fp16", mode="top_p"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        V = rng.choice([_log_int(rng, 1000, 152064), 152064, 32003])
        B = _log_int(rng, 1, max(1, min(512, 9_700_000 // V)))
        return dict(op="sample", B=B, V=V, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    mode=rng.choice(["all", "mixed", "temperature", "top_p", "top_k", "greedy"]))
    HK = rng.choice([4, 6, 8, 16])
    HV = HK * rng.choice([1, 2, 3])
    DK, DV = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64), (64, 128)])
    if rng.random() < 0.5:      # decode: one token or a window
        B, L = _log_int(rng, 1, 56), rng.choice([1, 1, 1, 2, 3, 5, 8, 13, 29])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        ragged = L > 1 and rng.random() < 0.5
        return dict(op="delta", B=B, L=L, ragged=ragged, HK=HK, HV=HV, DK=DK, DV=DV, dtype=dtype, fresh=False)
    B = _log_int(rng, 1, 12)
    L = _log_int(rng, 17, 8192 if B == 1 else 8192 // B)
    return dict(op="delta", B=B, L=L, ragged=B > 1 and rng.random() < 0.7, HK=HK, HV=HV, DK=DK, DV=DV,
                dtype=rng.choice(["bf16", "bf16", "fp16"]), fresh=rng.random() < 0.5)


_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _lengths(case):
    """The sequences' lengths: L each, or (ragged) B lengths from about L/4 to 7L/4, the same for every seed."""
    B, L = case["B"], case["L"]
    if not case["ragged"]:
        return [L] * B
    return [max(1, int(L * (0.25 + 1.5 * ((i * 0.6180339887 + 0.37) % 1.0)))) for i in range(B)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1_000_003 + 17)
    dt = _DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, device=dev, generator=g)

    def rand(*shape):
        return torch.rand(shape, device=dev, generator=g)

    if case["op"] == "sample":
        B, V, mode = case["B"], case["V"], case["mode"]
        # a wide body and a few likely tokens, as a language model's logits have
        logits = 2.0 * randn(B, V) - 1.0
        top = torch.randint(0, V, (B, 24), device=dev, generator=g)
        logits.scatter_add_(1, top, 4.0 + 5.0 * rand(B, 24))
        s = dict(op="sample", logits=logits.to(dt), u=rand(B), temperature=None, top_k=None, top_p=None, min_p=None)
        if mode in ("all", "temperature", "top_k", "top_p"):
            s["temperature"] = 0.5 + rand(B)
        if mode in ("all", "top_k"):
            s["top_k"] = torch.randint(1, 100, (B,), device=dev, generator=g, dtype=torch.int32)
        if mode in ("all", "top_p"):
            s["top_p"] = 0.8 + 0.19 * rand(B)
        if mode == "all":
            s["min_p"] = 0.1 * rand(B)
        if mode == "greedy":
            s["temperature"] = torch.zeros(B, device=dev)
        if mode == "mixed":  # each row switches some of the settings off
            row = torch.arange(B, device=dev)
            s["temperature"] = torch.where(row % 5 == 4, 0.0, 0.3 + 1.5 * rand(B))
            s["top_k"] = torch.where(row % 3 == 0, 0, torch.randint(1, 2000, (B,), device=dev, generator=g)).to(torch.int32)
            s["top_p"] = torch.where(row % 2 == 0, 1.0, 0.5 + 0.5 * rand(B))
            s["min_p"] = torch.where(row % 4 == 1, 0.05 * rand(B), 0.0)
        return s

    lengths = _lengths(case)
    B, T = case["B"], sum(lengths)
    HK, HV, DK, DV = case["HK"], case["HV"], case["DK"], case["DV"]
    # q, k and v as columns of one projection's rows
    row = randn(T, 2 * HK * DK + HV * DV).to(dt)
    q = row[:, :HK * DK].view(T, HK, DK)
    k = row[:, HK * DK:2 * HK * DK].view(T, HK, DK)
    v = row[:, 2 * HK * DK:].view(T, HV, DV)
    # decay: -a softplus(x), a in [1, 16], most steps between 0.001 and 0.1
    a = 1.0 + 15.0 * rand(HV)
    step = torch.exp(math.log(0.001) + rand(T, HV) * (math.log(0.1) - math.log(0.001)))
    decay = -a * step
    beta = torch.sigmoid(randn(T, HV))
    state = 0.3 * randn(B, HV, DK, DV)
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return dict(op="delta", q=q, k=k, v=v, g=decay, beta=beta, state=state, lengths=lengths, max_len=max(lengths),
                cu_seqlens=torch.from_numpy(starts).to(dev),
                slots=torch.randperm(B, device=dev, generator=g).to(torch.int32),
                fresh=torch.ones(B, dtype=torch.int32, device=dev) if case["fresh"] else None, scale=DK ** -0.5)


def _plain_sample(s):
    z = s["logits"].double()
    B, V = z.shape
    dev = z.device
    temp = s["temperature"].double() if s["temperature"] is not None else torch.ones(B, dtype=torch.float64, device=dev)
    greedy = temp <= 0
    w = torch.exp((z - z.amax(1, keepdim=True)) / torch.where(greedy, 1.0, temp)[:, None])
    z, order = torch.sort(z, dim=1, descending=True, stable=True)   # equal logits: lowest index first
    w = w.gather(1, order)
    rank = torch.arange(V, device=dev)[None]
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["top_k"] is not None:
        k = torch.where(s["top_k"] <= 0, V, s["top_k"]).long()
        keep &= rank < k[:, None]
    if s["top_p"] is not None:
        wk = torch.where(keep, w, 0.0)
        before = torch.cumsum(wk, 1) - wk
        p = s["top_p"].double()[:, None]
        keep &= (before < p * wk.sum(1, keepdim=True)) | (rank == 0) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double().clamp(max=1.0)[:, None]
    keep &= ~greedy[:, None] | (rank == 0)
    # draw over the kept tokens in the order of their indices
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    c = torch.cumsum(kept, 1)
    total = c[:, -1:]
    token = (c <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=V - 1)
    prob = kept.gather(1, token) / total
    return {"token": token[:, 0].to(torch.int32), "prob": prob[:, 0].float()}


def _plain_delta(s):
    dev = s["q"].device
    T, HK, DK = s["q"].shape
    HV, DV = s["v"].shape[1:]
    B, r = len(s["lengths"]), HV // HK
    C = min(CHUNK, s["max_len"])
    N = -(-s["max_len"] // C)
    # sequences padded to N chunks; a padded token has g = beta = 0 and changes nothing
    pos = torch.arange(N * C, device=dev)[None]
    cu = s["cu_seqlens"].long()
    valid = pos < (cu[1:] - cu[:-1])[:, None]
    idx = torch.where(valid, cu[:-1, None] + pos, 0)

    def chunks(x):   # [T, H, ...] -> [B, H, N, C, ...], padding zero
        y = torch.where(valid.view(B, N * C, *[1] * (x.dim() - 1)), x[idx].float(), 0.0)
        return y.view(B, N, C, *x.shape[1:]).movedim(3, 1)

    q, k, v, g, beta = (chunks(s[n]) for n in ("q", "k", "v", "g", "beta"))
    q = q / torch.sqrt((q * q).sum(-1, keepdim=True) + EPS) * s["scale"]
    k = k / torch.sqrt((k * k).sum(-1, keepdim=True) + EPS)
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    G = torch.cumsum(g.double(), -1)
    decay = torch.exp(torch.tril(G[..., :, None] - G[..., None, :])).float().tril()
    A = (beta[..., None] * decay * (k @ k.transpose(-1, -2))).tril(-1)
    inv = torch.zeros_like(A)
    for i in range(C):   # rows of (I + A)^-1 by forward substitution
        inv[..., i, :] = -(A[..., i:i + 1, :i] @ inv[..., :i, :])[..., 0, :]
        inv[..., i, i] += 1.0
    P = (q @ k.transpose(-1, -2)) * decay
    gam = torch.exp(G).float()[..., None]
    tail = torch.exp(G[..., -1:] - G).float()[..., None]
    slots = s["slots"].long()
    S = s["state"][slots]
    if s["fresh"] is not None:
        S = torch.where(s["fresh"].view(B, 1, 1, 1) != 0, 0.0, S)
    o = torch.empty(B, HV, N, C, DV, device=dev)
    for n in range(N):
        U = inv[:, :, n] @ (beta[:, :, n, :, None] * (v[:, :, n] - gam[:, :, n] * (k[:, :, n] @ S)))
        o[:, :, n] = gam[:, :, n] * (q[:, :, n] @ S) + P[:, :, n] @ U
        S = gam[:, :, n, -1:] * S + k[:, :, n].transpose(-1, -2) @ (tail[:, :, n] * U)
    s["state"][slots] = S
    out = o.movedim(1, 3).reshape(B, N * C, HV, DV)[valid]
    return {"o": out.to(s["q"].dtype), "state": s["state"]}


def run(s):
    if own:
        from bit_affine_quantized_g128_gb300 import q1
        if s["op"] == "sample":
            token, prob = q1.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                    top_p=s["top_p"], min_p=s["min_p"])
            return {"token": token, "prob": prob}
        o = q1.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], cu_seqlens=s["cu_seqlens"],
                           max_len=s["max_len"], slots=s["slots"], fresh=s["fresh"], scale=s["scale"], qk_l2norm=True)
        return {"o": o, "state": s["state"]}
    return _plain_sample(s) if s["op"] == "sample" else _plain_delta(s)


def work(case):
    es = 4 if case["dtype"] == "fp32" else 2
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        return {"bytes": B * V * es + B * 28, "flops": 4 * B * V}
    B, T = case["B"], sum(_lengths(case))
    HK, HV, DK, DV = case["HK"], case["HV"], case["DK"], case["DV"]
    state = B * HV * DK * DV * 4 * (1 if case["fresh"] else 2)
    # per token and value head: S^T k, k d^T and S^T q
    return {"bytes": T * (2 * HK * DK * es + 2 * HV * DV * es + 8 * HV) + state, "flops": T * HV * 6 * DK * DV}


def _exact_sample(s):
    logits = s["logits"].float().cpu().numpy().astype(np.float64)
    host = {n: (None if s[n] is None else s[n].cpu().numpy().astype(np.float64)) for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    B, V = logits.shape
    token, prob = np.zeros(B, np.int32), np.zeros(B, np.float64)
    for b in range(B):
        x, t = logits[b], 1.0 if host["temperature"] is None else host["temperature"][b]
        if t <= 0:
            token[b], prob[b] = int(np.argmax(x)), 1.0
            continue
        w = np.exp((x - x.max()) / t)
        order = np.argsort(-x, kind="stable")
        if host["top_k"] is not None and host["top_k"][b] > 0:
            order = order[:int(host["top_k"][b])]
        if host["top_p"] is not None and host["top_p"][b] < 1:
            c = np.cumsum(w[order])
            order = order[:1 + int(np.searchsorted(c, host["top_p"][b] * c[-1], side="left"))]
        if host["min_p"] is not None:
            order = order[w[order] >= min(1.0, host["min_p"][b])]
        ids = np.sort(order)
        c = np.cumsum(w[ids])
        at = min(int(np.searchsorted(c, host["u"][b] * c[-1], side="right")), len(ids) - 1)
        token[b], prob[b] = ids[at], w[ids[at]] / c[-1]
    return {"token": torch.from_numpy(token), "prob": torch.from_numpy(prob)}


def _exact_delta(s):
    """The recurrence itself, one token of every sequence at a time, in float64."""
    lengths, HV, HK = s["lengths"], s["v"].shape[1], s["q"].shape[1]
    start = s["cu_seqlens"].long()[:-1]
    n = torch.tensor(lengths, device=start.device)
    slots = s["slots"].long()
    S = s["state"].double()[slots]
    if s["fresh"] is not None:
        S = S * (s["fresh"] == 0).double().view(-1, 1, 1, 1)
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    q = q * torch.rsqrt(q.square().sum(-1, keepdim=True) + EPS) * s["scale"]
    k = k * torch.rsqrt(k.square().sum(-1, keepdim=True) + EPS)
    alpha, beta = torch.exp(s["g"].double()), s["beta"].double()
    o = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    for t in range(max(lengths)):
        live = torch.nonzero(t < n)[:, 0] if t >= min(lengths) else None
        at = start + t if live is None else start[live] + t
        St = S if live is None else S[live]
        kt = k[at].repeat_interleave(HV // HK, 1)
        qt = q[at].repeat_interleave(HV // HK, 1)
        St = St * alpha[at][..., None, None]
        d = beta[at][..., None] * (v[at] - torch.einsum("bhkv,bhk->bhv", St, kt))
        St = St + kt[..., :, None] * d[..., None, :]
        o[at] = torch.einsum("bhkv,bhk->bhv", St, qt)
        if live is None:
            S = St
        else:
            S[live] = St
    state = s["state"].double()
    state[slots] = S
    return {"o": o, "state": state}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "sample":
        return _exact_sample(s)
    if max(s["lengths"]) * case["B"] * case["HV"] * case["DK"] * case["DV"] > 3e10:
        return None   # over 20 seconds
    return _exact_delta(s)
