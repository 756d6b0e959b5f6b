"""q1_kv_store, q1_kv_load and q1_kv_attention against plain float64 implementations
(oracle/serving_oracle.py)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as O

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def q1():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    mod.load_library()
    return mod


def _rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def _rounded(x, dtype):
    """x as `dtype` holds it: the tensor, and its values in fp32."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(DTYPES[dtype])
    return t, t.float().numpy()


class Cache:
    """A cache of sequences with `lengths` tokens in pages of random order, and what it holds, by the oracle."""

    def __init__(self, q1, lengths, heads, D, gs=64, page=64, seed=0, spare=2, k=None, v=None, n_pages=None):
        rng = _rng(seed)
        self.lengths, self.heads, self.D, self.gs, self.page, self.B = list(lengths), heads, D, gs, page, len(lengths)
        per = [-(-max(n, 0) // page) for n in lengths]
        self.n_pages = n_pages or sum(per) + spare
        order = rng.permutation(self.n_pages)[:sum(per)] if n_pages is None else self.n_pages - 1 - np.arange(sum(per))
        self.table = np.full((self.B, max(per) + 1), -1, np.int32)
        at = 0
        for b, n in enumerate(per):
            self.table[b, :n] = order[at:at + n]
            at += n
        # a mean per channel and a few large channels in k
        mean, size = 0.5 * rng.standard_normal((heads, D)), np.where(rng.random((heads, D)) < 0.05, 4.0, 1.0)
        self.k = [(rng.standard_normal((n, heads, D)) + mean) * size for n in lengths] if k is None else k
        self.v = [rng.standard_normal((n, heads, D)) for n in lengths] if v is None else v
        self.kq = [O.kv_quantise(x, gs) for x in self.k]
        self.vq = [O.kv_quantise(x, gs) for x in self.v]
        self.kval = [O.kv_values(*x) for x in self.kq]
        self.vval = [O.kv_values(*x) for x in self.vq]

    def store(self, q1, noise=True):
        """The cache on the device, every token stored by one call (fp32 rows)."""
        c = q1.kv_cache(self.n_pages, self.heads, self.D, self.page, self.gs)
        if noise:
            c.copy_(torch.from_numpy(_rng(99).integers(0, 256, tuple(c.shape), dtype=np.uint8)))
        cu = np.concatenate([[0], np.cumsum(self.lengths)]).astype(np.int32)
        q1.kv_store(c, torch.from_numpy(np.concatenate(self.k).astype(np.float32)).cuda(),
                    torch.from_numpy(np.concatenate(self.v).astype(np.float32)).cuda(), self.d_table(), self.d_lengths(),
                    cu_seqlens=torch.from_numpy(cu).cuda())
        return c

    def d_table(self):
        return torch.from_numpy(self.table).cuda()

    def d_lengths(self):
        return torch.tensor(self.lengths, dtype=torch.int32).cuda()


# ---- the oracle's own pins (CPU)
def test_oracle_quantises_by_hand():
    # 0 .. 15: codes of step 1 about 8; the ends are met exactly
    x = np.arange(64, dtype=np.float32) % 16
    q, s, b = O.kv_quantise(x, 64)
    assert s == 1 and b == 8 and np.array_equal(q, np.arange(64) % 16 - 8)
    assert np.array_equal(O.kv_values(q, s, b), x)
    # a constant that bf16 holds: scale 0; one that it does not: the residue is the scale's
    q, s, b = O.kv_quantise(np.full(64, 2.5, np.float32), 64)
    assert s == 0 and b == 2.5 and (q == 0).all()
    q, s, b = O.kv_quantise(np.full(64, 5.03, np.float32), 64)
    assert b == 5.03125 and abs(O.kv_values(q, s, b)[0] - 5.03) < 2.0 ** -9 * 0.01
    # NaN, infinities
    x = np.linspace(-1, 1, 128, dtype=np.float32)
    x[3], x[100] = np.nan, np.inf
    q, s, b = O.kv_quantise(x, 64)
    assert np.isnan(s[0]) and np.isnan(b[0]) and O.kv_values(q, s, b)[100] == pytest.approx(32768, rel=2.0 ** -8)


def test_oracle_errors_are_half_a_step():
    x = _rng(1).standard_normal((50, 2, 128)).astype(np.float32)
    for gs in (64, 128):
        q, s, b = O.kv_quantise(x, gs)
        g = x.reshape(50, 2, -1, gs)
        step = (g.max(-1) - g.min(-1)) / 15
        # scale and bias are rounded to bf16: the step grows by up to 2^-7, codes at the ends are off by 2^-8 of 8 steps
        err = np.abs(O.kv_values(q, s, b) - x).reshape(g.shape).max(-1)
        assert (err <= step * (0.5 * (1 + 2.0 ** -6) + 8 * 2.0 ** -8)).all()


def test_oracle_attention_by_hand():
    # one key seen: its value; equal keys: the mean; nothing seen: 0 and -inf
    q, k = np.ones((3, 1, 64)), np.ones((4, 1, 64))
    v = np.arange(4.0)[:, None, None] * np.ones((4, 1, 64))
    o, lse, _, _ = O.kv_attention(q, k, v, [-1, 0, 3], 1 / 64)
    assert (o[0] == 0).all() and lse[0] == -np.inf and (o[1] == 0).all() and lse[1] == pytest.approx(1.0)
    assert np.allclose(o[2], 1.5) and lse[2] == pytest.approx(1 + np.log(4))
    o, _, _, _ = O.kv_attention(q[:1], k, v, [3], 1.0, window=2)
    assert np.allclose(o, 2.5)


# ---- writing and reading back
def _rows(q1, c, new, dtype, strided, seed):
    """New rows for the last `new` tokens of each sequence (more than there are tokens: those before the first are
    anything): tensors on the device, and their fp32 values per sequence."""
    rng = _rng(seed)
    T = sum(new)
    x = rng.standard_normal((T, 2 * c.heads * c.D)) * np.exp(rng.standard_normal((T, 1)))
    row, val = _rounded(x, dtype)
    if not strided:
        k, v = (row[:, i * c.heads * c.D:(i + 1) * c.heads * c.D].clone().cuda() for i in (0, 1))
    else:   # columns of one projection's rows
        row = row.cuda()
        k, v = row[:, :c.heads * c.D], row[:, c.heads * c.D:]
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    val = val.reshape(T, 2, c.heads, c.D)
    return k.view(T, c.heads, c.D), v.view(T, c.heads, c.D), cu, [val[cu[b]:cu[b + 1]] for b in range(len(new))]


def _expect_bytes(c, before, new, vals, missing=()):
    """`before` [pages, heads, blocks, bytes] with the rows of `vals` written, token by token."""
    want = before.copy()
    for b, n in enumerate(new):
        for i in range(n):
            p = c.lengths[b] - n + i
            if p < 0 or p // c.page >= c.table.shape[1]:
                continue
            pg = c.table[b, p // c.page]
            if not 0 <= pg < c.n_pages:
                continue
            for h in range(c.heads):
                cell = want[pg, h, p % c.page // 16]
                full = [np.zeros((16, c.D), np.int64), np.zeros((16, c.D // c.gs), np.float32), np.zeros((16, c.D // c.gs), np.float32)]
                mark = [np.zeros((16, c.D), np.int64) - 8, full[1], full[2]]
                new_k, new_v = (O.kv_quantise(vals[b][i, s, h], c.gs) for s in (0, 1))
                t = p % 16
                parts, owned = [], []
                for qn in (new_k, new_v):
                    q, s, o = (a.copy() for a in mark)
                    q[t], s[t], o[t] = qn
                    parts += [q, s, o]
                    q, s, o = (a.copy() for a in mark)
                    q[t], s[t], o[t] = 7, np.float32(np.array(0xFFFF0000, np.uint32).view(np.float32)), np.array(0xFFFF0000, np.uint32).view(np.float32)
                    owned += [q, s, o]
                data, own = O.kv_block(*parts), O.kv_block(*owned)
                cell[own != 0] = data[own != 0]
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,heads,page,dtype,strided", [
    (64, 64, 1, 16, "bf16", False), (64, 64, 3, 32, "fp32", True), (128, 64, 2, 64, "fp16", True),
    (128, 128, 3, 16, "bf16", True), (256, 64, 1, 128, "fp32", False), (256, 128, 2, 32, "bf16", True)])
def test_store_bytes(q1, D, gs, heads, page, dtype, strided):
    # ragged sequences, one without rows, one with more rows than tokens, a missing page: exactly the bytes of
    # the tokens stored change
    c = Cache(q1, [37, 5, 20, 3], heads, D, gs, page, seed=D + gs)
    c.table[2, 0] = c.n_pages if page < 32 else -7    # not there
    new = [37, 1, 20, 6] if page > 16 else [19, 0, 18, 6]
    before = _rng(5).integers(0, 256, (c.n_pages, heads, page // 16, 16 * (D + 8 * D // gs)), dtype=np.uint8)
    cache = torch.from_numpy(before).cuda()
    k, v, cu, vals = _rows(q1, c, new, dtype, strided, 7)
    q1.kv_store(cache, k, v, c.d_table(), c.d_lengths(), cu_seqlens=torch.from_numpy(cu).cuda())
    assert np.array_equal(cache.cpu().numpy(), _expect_bytes(c, before, new, vals))


@pytest.mark.gpu
def test_store_of_odd_groups(q1):
    rng = _rng(3)
    rows = [np.zeros(64), -np.zeros(64), np.full(64, 2.5), np.full(64, 5.03), np.full(64, -1e-30), np.full(64, 1e30),
            np.linspace(-1e-36, 1e-36, 64), np.linspace(100, 100.01, 64), rng.standard_normal(64) * 1e4, np.arange(64) / 2.0,
            np.where(np.arange(64) == 5, np.nan, 1.0), np.where(np.arange(64) == 9, np.inf, rng.standard_normal(64)),
            np.where(np.arange(64) == 63, -np.inf, 0.0), np.where(np.arange(64) % 2, 3.0e38, -3.0e38),
            np.where(np.arange(64) == 0, 1000.0, 1e-3 * rng.standard_normal(64)), np.full(64, np.nan)]
    x = np.stack(rows).astype(np.float32)[:, None]      # 16 tokens, one head
    c = Cache(q1, [16], 1, 64, 64, 16, k=[x], v=[x[::-1]])
    cache = c.store(q1, noise=False).cpu().numpy()
    want = O.kv_block(*(a[:, 0] for a in c.kq[0]), *(a[:, 0] for a in c.vq[0]))
    assert np.array_equal(cache[c.table[0, 0], 0, 0], want)
    k, v = q1.kv_load(torch.from_numpy(cache).cuda(), c.d_table(), c.d_lengths(), 16, dtype=torch.float32)
    assert np.array_equal(k[0].cpu().numpy(), c.kval[0], equal_nan=True)
    assert np.array_equal(v[0].cpu().numpy(), c.vval[0], equal_nan=True)


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,heads,page,dtype", [(64, 64, 3, 32, "fp32"), (128, 64, 2, 64, "bf16"), (128, 128, 1, 16, "fp16"),
                                                   (256, 64, 5, 16, "bf16"), (256, 128, 2, 128, "fp32")])
def test_load(q1, D, gs, heads, page, dtype):
    c = Cache(q1, [150, 33, 1, 64], heads, D, gs, page, seed=D)
    cache = c.store(q1)
    table = c.table.copy()
    table[1, 0] = -1                                      # tokens without a page are zeros
    new = [97, 33, 4, 0]                                  # the last ones; more than there are; none
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    k, v = q1.kv_load(cache, torch.from_numpy(table).cuda(), c.d_lengths(), sum(new), cu_seqlens=torch.from_numpy(cu).cuda(),
                      dtype=DTYPES[dtype])
    for got, val in ((k, c.kval), (v, c.vval)):
        for b, n in enumerate(new):
            want = np.zeros((n, heads, D), np.float32)
            for i in range(n):
                p = c.lengths[b] - n + i
                if p >= 0 and table[b, p // page] >= 0:
                    want[i] = val[b][p]
            assert torch.equal(got[cu[b]:cu[b + 1]].cpu(), torch.from_numpy(want).to(DTYPES[dtype])), b


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,dtype", [(64, 64, "bf16"), (128, 64, "fp32"), (128, 128, "fp16"), (256, 64, "fp32"), (256, 128, "bf16")])
def test_many_blocks(q1, D, gs, dtype):
    # enough blocks that a warp does a block's K and V: codes and values as the oracle's, whole blocks and cut ones
    c = Cache(q1, [1500, 205], 16, D, gs, 32, seed=D + gs)
    cache = c.store(q1)
    before = cache.clone()
    cu = torch.tensor([0, 1490, 1695], dtype=torch.int32).cuda()
    k, v = q1.kv_load(cache, c.d_table(), c.d_lengths(), 1695, cu_seqlens=cu, dtype=DTYPES[dtype])
    for got, vals in ((k, c.kval), (v, c.vval)):
        want, _ = _rounded(np.concatenate([vals[0][10:], vals[1]]), dtype)
        assert torch.equal(got.cpu(), want)
    q1.kv_store(cache, torch.from_numpy(np.concatenate([c.k[0][10:], c.k[1]]).astype(np.float32)).cuda(),
                torch.from_numpy(np.concatenate([c.v[0][10:], c.v[1]]).astype(np.float32)).cuda(), c.d_table(), c.d_lengths(), cu_seqlens=cu)
    assert torch.equal(cache, before)


@pytest.mark.gpu
def test_equal_lengths_without_offsets(q1):
    c = Cache(q1, [70, 70, 70], 2, 128, seed=4)
    cache = c.store(q1)
    k, v = q1.kv_load(cache, c.d_table(), c.d_lengths(), 7, dtype=torch.float32)
    assert k.shape == (3, 7, 2, 128) and np.array_equal(k.cpu().numpy(), np.stack([x[-7:] for x in c.kval]))
    again = q1.kv_cache(c.n_pages, 2, 128)
    whole = [torch.from_numpy(np.stack(x).astype(np.float32)).cuda() for x in (c.k, c.v)]
    q1.kv_store(again, *whole, c.d_table(), c.d_lengths())
    k2, v2 = q1.kv_load(again, c.d_table(), c.d_lengths(), 7, dtype=torch.float32)
    assert torch.equal(k, k2) and torch.equal(v, v2)
    q = torch.randn(3, 7, 4, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    o, lse = q1.kv_attention(q, cache, c.d_table(), c.d_lengths(), return_lse=True)
    cu = torch.tensor([0, 7, 14, 21], dtype=torch.int32).cuda()
    o2, lse2 = q1.kv_attention(q.flatten(0, 1), cache, c.d_table(), c.d_lengths(), cu_seqlens=cu, max_q=7, max_len=128, return_lse=True)
    assert o.shape == q.shape and lse.shape == (3, 7, 4) and torch.equal(o.flatten(0, 1), o2) and torch.equal(lse.flatten(0, 1), lse2)


@pytest.mark.gpu
def test_many_sequences(q1):
    # the search for a row's sequence: more of them than a warp looks at in one step, many without rows
    rng = _rng(8)
    lengths = [int(x) for x in rng.integers(0, 4, 2500)]
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    T = int(cu[-1])
    k = torch.from_numpy(rng.standard_normal((T, 1, 64)).astype(np.float32)).cuda()
    table = torch.arange(2500, dtype=torch.int32).view(-1, 1).cuda()
    cache = q1.kv_cache(2500, 1, 64, page_size=16)
    d_len, d_cu = torch.tensor(lengths, dtype=torch.int32).cuda(), torch.from_numpy(cu).cuda()
    q1.kv_store(cache, k, k, table, d_len, cu_seqlens=d_cu)
    got, _ = q1.kv_load(cache, table, d_len, T, cu_seqlens=d_cu, dtype=torch.float32)
    want = O.kv_values(*O.kv_quantise(k.cpu().numpy(), 64))
    assert np.array_equal(got.cpu().numpy(), want)
    # and one row at a time from the far end
    last, _ = q1.kv_load(cache, table[2400:], d_len[2400:], T - int(cu[2400]),
                         cu_seqlens=(d_cu[2400:] - d_cu[2400]).contiguous(), dtype=torch.float32)
    assert np.array_equal(last.cpu().numpy(), want[cu[2400]:])


# ---- attention
def check(q1, c, cache, new, HQ, dtype="bf16", causal=True, window=0, seed=11, scale=None, qsize=1.0, table=None, tiles=False, **kw):
    """One call against the oracle.  Per value, with p the softmax's weights (sum 1):
      the output's rounding          eps / 2 |o|, but no less than half a step of the type's subnormals, eps / 2 times its least
                                     normal value (2^-25 for fp16: below 2^-14 its steps stay 2^-24)
      P scale as fp16                2^-11 sum p |v - bias| <= 2^-11 (sum p |v| + |bias|): bf16 outputs; a sum of two, 2^-22, else
      a logit's fp32 rounding        (D / 8 + 16) 2^-24 scale sum |q k| of relative error of p, and 2^-21 from exp
    an error of p by a factor 1 + d moves o by at most 2 d sum p |v|.
    tiles: the form for many rows, whose V is rounded to fp16 as well: 2^-11 sum p |v| for P and for V, 2^-25 for values below
    fp16's normal ones and len 2^-32 max |v| for weights below them (2^-25 against a largest weight of at least 2^7); logits'
    code and bias parts are summed separately, both parts' sizes count, and sums of q enter with 2^-22."""
    rng = _rng(seed)
    D, HK, T = c.D, c.heads, sum(new)
    q, qv = _rounded(rng.standard_normal((T, HQ, D)) * qsize, dtype)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    tab = c.table if table is None else table
    # (the hint of a long context has few rows take the tiles' form, in parts)
    kw = {"max_q": max(new), "max_len": 1 << 20 if tiles else max(c.lengths), **kw}
    o, lse = q1.kv_attention(q.cuda(), cache, torch.from_numpy(tab).cuda(), c.d_lengths(), cu_seqlens=torch.from_numpy(cu).cuda(),
                             scale=scale, causal=causal, window=window, return_lse=True, **kw)
    assert o.dtype == DTYPES[dtype] and o.shape == (T, HQ, D) and lse.shape == (T, HQ)
    got, got_lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    scale = D ** -0.5 if scale is None else scale
    part = 2.0 ** -11 if dtype == "bf16" else 2.0 ** -22
    for b, n in enumerate(new):
        there = np.array([0 <= tab[b, p // c.page] < c.n_pages if p // c.page < tab.shape[1] else False for p in range(c.lengths[b])], bool)
        pos = np.arange(n) + c.lengths[b] - n
        rows = slice(cu[b], cu[b + 1])
        want, want_lse, size, big = O.kv_attention(qv[rows], c.kval[b], c.vval[b], pos, scale, causal, window, there)
        bias = np.repeat(np.abs(c.vq[b][2]).max(0).repeat(c.gs, -1), HQ // HK, 0) if c.lengths[b] else 0.0
        logit = (D / 8 + 16) * 2.0 ** -24 * big
        floor = 0.0
        if tiles and c.lengths[b]:
            kb = np.abs(c.kq[b][2]).max(0).repeat(c.gs, -1).repeat(HQ // HK, 0)
            sums = abs(scale) * (kb * np.abs(qv[rows])).sum(-1)
            logit = logit + ((D / 8 + 16) * 2.0 ** -24 * 2 + 2.0 ** -22) * sums
            part, bias = 2 * 2.0 ** -11, 0.0
            floor = 2.0 ** -25 + c.lengths[b] * 2.0 ** -32 * np.abs(c.vval[b]).max()
        info = torch.finfo(DTYPES[dtype])
        bound = info.eps / 2 * np.maximum(np.abs(want), info.tiny) + floor + part * (size + bias) + 2 * (2.0 ** -21 + logit)[..., None] * (size + bias)
        err = np.abs(got[rows] - want)
        assert (err <= bound).all(), (b, float((err / np.maximum(bound, 1e-300)).max()))
        empty = np.isneginf(want_lse)
        assert np.array_equal(np.isneginf(got_lse[rows]), empty) and (got[rows][empty] == 0).all()
        with np.errstate(invalid="ignore"):
            bad = np.abs(got_lse[rows] - want_lse) > 2.0 ** -21 + logit + 2.0 ** -23 * np.abs(want_lse)
        assert not bad[~empty].any(), b
    return o, lse


FEW = [  # D, gs, HK, HQ / HK, page, dtype, lengths, new, window
    (128, 64, 2, 4, 64, "bf16", [1, 16, 17, 300], [1, 1, 1, 1], 0),
    (128, 128, 1, 8, 16, "bf16", [129, 31], [1, 1], 0),
    (128, 64, 1, 5, 32, "fp16", [500, 77, 3], [3, 1, 2], 0),
    (128, 64, 3, 1, 64, "fp32", [65, 640], [2, 5], 100),
    (64, 64, 2, 1, 16, "bf16", [15, 47, 1000], [1, 2, 4], 0),
    (64, 64, 1, 16, 128, "fp16", [200, 129], [1, 1], 37),
    (64, 64, 12, 1, 16, "fp32", [333, 18], [5, 5], 16),
    (256, 64, 1, 6, 64, "bf16", [90, 700], [1, 1], 0),
    (256, 128, 2, 8, 128, "fp16", [257, 15], [1, 2], 0),
    (256, 64, 1, 3, 16, "fp32", [40, 333], [7, 2], 64),
    (256, 128, 1, 16, 32, "bf16", [130], [4], 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,HK,r,page,dtype,lengths,new,window", FEW)
def test_attention_of_few_rows(q1, D, gs, HK, r, page, dtype, lengths, new, window):
    c = Cache(q1, lengths, HK, D, gs, page, seed=sum(lengths))
    check(q1, c, c.store(q1), new, HK * r, dtype, window=window)


MANY = [  # D, gs, HK, HQ / HK, page, dtype, lengths, new, window
    (128, 64, 1, 4, 64, "bf16", [130], [130], 0),
    (128, 64, 2, 2, 32, "fp16", [300, 40], [300, 33], 0),
    (128, 128, 1, 5, 16, "bf16", [257, 600, 70], [100, 1, 70], 0),
    (64, 64, 2, 1, 16, "bf16", [520, 129], [300, 129], 0),
    (64, 64, 1, 8, 128, "fp16", [400, 33, 900], [17, 33, 90], 200),
    (256, 64, 1, 2, 64, "bf16", [200, 65], [200, 65], 0),
    (256, 128, 1, 6, 32, "fp16", [700, 64], [50, 64], 0),
    (256, 64, 2, 1, 16, "bf16", [333], [200], 64),
    (128, 64, 1, 1, 64, "bf16", [700], [513], 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,HK,r,page,dtype,lengths,new,window", MANY)
def test_attention_of_many_rows(q1, D, gs, HK, r, page, dtype, lengths, new, window):
    c = Cache(q1, lengths, HK, D, gs, page, seed=sum(lengths))
    check(q1, c, c.store(q1), new, HK * r, dtype, window=window, tiles=True)
    assert q1.device_errors() == 0


WHOLE = [  # the same, with enough heads that tiles are taken with their context in one part
    (128, 64, 32, 4, 64, "bf16", [260], [260], 0),
    (128, 64, 40, 2, 32, "fp16", [300, 140], [300, 33], 0),
    (128, 128, 16, 5, 16, "bf16", [257, 600, 70], [100, 1, 70], 0),
    (64, 64, 100, 1, 16, "bf16", [520, 129], [300, 129], 0),
    (64, 64, 24, 8, 128, "fp16", [800, 33, 900], [300, 33, 90], 300),
    (256, 64, 20, 2, 64, "bf16", [333, 65], [200, 65], 0),
    (256, 64, 30, 2, 64, "bf16", [400], [400], 0),
    (256, 128, 12, 6, 32, "fp16", [700, 64], [50, 64], 0),
    (128, 64, 24, 1, 64, "fp16", [900], [613], 33),
]


@pytest.mark.gpu
@pytest.mark.parametrize("D,gs,HK,r,page,dtype,lengths,new,window", WHOLE)
def test_attention_of_many_rows_and_heads(q1, D, gs, HK, r, page, dtype, lengths, new, window):
    c = Cache(q1, lengths, HK, D, gs, page, seed=sum(lengths))
    check(q1, c, c.store(q1), new, HK * r, dtype, window=window, tiles=True, max_len=max(lengths))
    assert q1.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_without_order(q1, dtype):
    c = Cache(q1, [90, 12], 2, 128, seed=5)
    check(q1, c, c.store(q1), [5, 12], 6, dtype, causal=False)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp32"), (256, "fp16")])
def test_long_contexts_are_split(q1, D, dtype):
    c = Cache(q1, [9000, 4001], 1, D, seed=6)
    cache = c.store(q1)
    check(q1, c, cache, [1, 2], 3, dtype)
    # hints that are too small, or none: the same rows, split another way
    for kw in (dict(max_q=1, max_len=1), dict(max_q=1, max_len=3000), dict(max_q=None, max_len=None), dict(max_len=1 << 30)):
        check(q1, c, cache, [1, 2], 3, dtype, **kw)
    check(q1, c, cache, [9, 1], 8, dtype, max_q=1)      # more row tiles than the hint foresees


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_long_sums_of_one_sign(q1, D):
    # V's codes of one sign (one channel of a group has the other) over a long context that the hint leaves to one CTA: hundreds
    # of blocks into one sum
    n = 30000
    rng = _rng(17)
    v = np.where(np.arange(D) % 64 == 5, -1.0, 1.0) * (1.0 + 0.05 * rng.random((n, 1, D)))
    c = Cache(q1, [n], 1, D, seed=18, k=[0.2 * rng.standard_normal((n, 1, D))], v=[v])
    check(q1, c, c.store(q1), [1], 2, "fp32", max_len=1)
    check(q1, c, c.store(q1), [5], 3, "fp32", max_len=1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rows_that_see_nothing(q1, dtype):
    # a sequence without tokens, more rows than tokens, a page that is not there (alone, and among others), a short table
    c = Cache(q1, [0, 3, 40, 100, 90], 2, 128, page=32, seed=7)
    cache = c.store(q1)
    table = c.table.copy()
    table[2, :2] = [-1, c.n_pages]
    table[3, 1] = 1 << 30
    check(q1, c, cache, [2, 5, 1, 2, 1], 4, dtype, table=table)
    check(q1, c, cache, [2, 5, 1, 2, 1], 4, dtype, table=np.ascontiguousarray(table[:, :2]))
    check(q1, c, cache, [2, 5, 1, 2, 1], 4, dtype, table=table, causal=False)
    # no row of a sequence, none at all
    check(q1, c, cache, [0, 0, 3, 0, 1], 4, dtype, table=table)
    none = torch.zeros(6, dtype=torch.int32).cuda()
    o, lse = q1.kv_attention(torch.zeros(0, 4, 128, device="cuda"), cache, c.d_table(), c.d_lengths(), cu_seqlens=none, return_lse=True)
    assert o.shape == (0, 4, 128) and lse.shape == (0, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_what_is_not_seen_may_hold_anything(q1, dtype):
    # NaN scales and biases behind the sequence's end, in front of the window, and in tokens that only later rows see
    c = Cache(q1, [100, 59], 1, 128, page=32, seed=8)
    nan = torch.full((1, 1, 128), float("nan"), device="cuda")
    for window, at in ((0, 99), (30, 99), (30, 69), (0, 58)):
        b = 0 if at != 58 else 1
        cache = torch.full((c.n_pages, 1, 2, 16 * (128 + 16)), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
        cu = torch.tensor([0, 100, 159], dtype=torch.int32).cuda()
        q1.kv_store(cache, torch.from_numpy(np.concatenate(c.k).astype(np.float32)).cuda(),
                    torch.from_numpy(np.concatenate(c.v).astype(np.float32)).cuda(), c.d_table(), c.d_lengths(), cu_seqlens=cu)
        lengths = torch.zeros(2, dtype=torch.int32)
        lengths[b] = at + 1
        cu = torch.tensor([0, 1 - b, 1], dtype=torch.int32).cuda()
        q1.kv_store(cache, nan, nan, c.d_table(), lengths.cuda(), cu_seqlens=cu)
        # four rows of each: the NaN token is seen by those at its position or behind (within the window)
        q, qv = _rounded(_rng(9).standard_normal((8, 2, 128)), dtype)
        o, lse = q1.kv_attention(q.cuda(), cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.tensor([0, 4, 8], dtype=torch.int32).cuda(),
                                 max_q=4, max_len=100, window=window, return_lse=True)
        for s in range(2):
            pos = np.arange(4) + c.lengths[s] - 4
            hit = (pos >= at) & ((pos < at + window) if window else True) if s == b else np.zeros(4, bool)
            want, _, size, _ = O.kv_attention(qv[4 * s:4 * s + 4], c.kval[s], c.vval[s], pos, 128 ** -0.5, True, window)
            got = o[4 * s:4 * s + 4].double().cpu().numpy()
            assert np.isnan(got[hit]).all() and np.isnan(lse[4 * s:4 * s + 4].cpu().numpy()[hit]).all()
            # the bound of check(), its logits' part at most 2^-16 here
            assert (np.abs(got - want)[~hit] <= (2.0 ** -8 * (size + 1))[~hit]).all(), (window, at, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_sizes_of_values(q1, dtype):
    # values that grow, fall and vanish along the context, logits up to some hundred, a row that one token rules
    rng = _rng(10)
    n = 700
    up = np.exp(rng.standard_normal((n, 1, 1))) * np.logspace(-8, 3, n)[:, None, None]
    for size in (up, up[::-1], np.full((n, 1, 1), 1e-7), np.where(np.arange(n) < 300, 0.0, 1.0)[:, None, None]):
        c = Cache(q1, [n], 2, 128, seed=12, v=[(rng.standard_normal((n, 2, 128)) * size)])
        check(q1, c, c.store(q1), [2], 4, dtype)
    c = Cache(q1, [n], 2, 128, seed=13, k=[20 * rng.standard_normal((n, 2, 128))])
    check(q1, c, c.store(q1), [2], 4, dtype, qsize=3.0)
    check(q1, c, c.store(q1), [2], 4, dtype, scale=-0.05)
    check(q1, c, c.store(q1), [2], 4, dtype, scale=0.0)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(q1):
    # the last pages of a cache of more than 2^32 bytes
    n_pages = (1 << 32) // (2 * 4 * 16 * 144) + 40
    c = Cache(q1, [130, 70], 2, 128, seed=14, n_pages=n_pages)
    cache = c.store(q1, noise=False)
    assert cache.numel() > 1 << 32
    check(q1, c, cache, [1, 2], 4)
    k, _ = q1.kv_load(cache, c.d_table(), c.d_lengths(), 70, dtype=torch.float32)
    assert np.array_equal(k[1].cpu().numpy(), c.kval[1])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 256])
def test_many_rows_that_see_nothing_and_small_hints(q1, D):
    # no tokens, fewer tokens than rows, missing pages (a whole tile's too), a short table; more row tiles than the hint foresees
    c = Cache(q1, [0, 30, 200, 320, 90], 1, D, page=32, seed=21)
    cache = c.store(q1)
    table = c.table.copy()
    table[2, [0, 2]] = [-1, c.n_pages]
    table[3, 0:4] = -1
    new = [40, 70, 130, 100, 5]
    check(q1, c, cache, new, 4, table=table, tiles=True)
    check(q1, c, cache, new, 4, table=np.ascontiguousarray(table[:, :3]), tiles=True)
    check(q1, c, cache, new, 4, "fp16", table=table, tiles=True, causal=False)
    check(q1, c, cache, new, 4, table=table, tiles=True, window=20)
    check(q1, c, cache, [0, 0, 200, 0, 90], 6, table=table, tiles=True, max_q=20)
    check(q1, c, cache, [0, 0, 200, 0, 90], 6, "fp16", tiles=True, max_q=13, max_len=1)
    assert q1.device_errors() == 0


@pytest.mark.gpu
def test_many_rows_beside_what_they_do_not_see(q1):
    # NaN everywhere but in the sequences; NaN in K and V of one token: only rows that see it become NaN
    c = Cache(q1, [300, 140], 1, 128, page=32, seed=22)
    nan = torch.full((1, 1, 128), float("nan"), device="cuda")
    for window, at, kv in ((0, 290, "v"), (0, 290, "k"), (50, 160, "v"), (50, 160, "k"), (50, 299, "v"), (0, 0, "v")):
        cache = torch.full((c.n_pages, 1, 2, 16 * (128 + 16)), 255, dtype=torch.uint8, device="cuda")
        rows = [torch.from_numpy(np.concatenate(x).astype(np.float32)).cuda() for x in (c.k, c.v)]
        cu = torch.tensor([0, 300, 440], dtype=torch.int32).cuda()
        q1.kv_store(cache, *rows, c.d_table(), c.d_lengths(), cu_seqlens=cu)
        one = [r[at:at + 1].clone() for r in rows]
        one[kv == "v"] = nan
        q1.kv_store(cache, *one, c.d_table(), torch.tensor([at + 1, 0], dtype=torch.int32).cuda(),
                    cu_seqlens=torch.tensor([0, 1, 1], dtype=torch.int32).cuda())
        q, qv = _rounded(_rng(9).standard_normal((280, 2, 128)), "bf16")
        o, lse = q1.kv_attention(q.cuda(), cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.tensor([0, 140, 280], dtype=torch.int32).cuda(),
                                 max_q=140, max_len=1 << 20, window=window, return_lse=True)
        for s in range(2):
            pos = np.arange(140) + c.lengths[s] - 140
            hit = (pos >= at) & ((pos < at + window) if window else True) if s == 0 else np.zeros(140, bool)
            want, _, size, _ = O.kv_attention(qv[140 * s:140 * s + 140], c.kval[s], c.vval[s], pos, 128 ** -0.5, True, window)
            got = o[140 * s:140 * s + 140].double().cpu().numpy()
            assert np.isnan(got[hit]).all()
            # check()'s bound with its logits' part below 2^-14
            assert (np.abs(got - want)[~hit] <= (2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size)[~hit]).all(), (window, at, kv, s)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_sizes_of_values_by_tiles(q1, dtype):
    rng = _rng(23)
    n = 500
    up = np.exp(rng.standard_normal((n, 1, 1))) * np.logspace(-8, 3, n)[:, None, None]
    for size in (up, up[::-1], np.full((n, 1, 1), 1e-3), np.where(np.arange(n) < 300, 0.0, 1.0)[:, None, None]):
        c = Cache(q1, [n], 1, 128, seed=24, v=[rng.standard_normal((n, 1, 128)) * size])
        check(q1, c, c.store(q1), [90], 2, dtype, tiles=True)
    c = Cache(q1, [n], 1, 128, seed=25, k=[20 * rng.standard_normal((n, 1, 128))])
    for kw in (dict(qsize=3.0), dict(scale=-0.05), dict(scale=0.0), dict(qsize=1e-4, scale=1e4), dict(qsize=1e4, scale=1e-6)):
        check(q1, c, c.store(q1), [90], 2, dtype, tiles=True, **kw)


@pytest.mark.gpu
def test_tiles_beyond_32_bits(q1):
    n_pages = (1 << 32) // (2 * 4 * 16 * 144) + 40
    c = Cache(q1, [200, 70], 2, 128, seed=26, n_pages=n_pages)
    check(q1, c, c.store(q1, noise=False), [200, 33], 2, tiles=True)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 256])
def test_stalled_expansion_times_out_and_recovers(q1, D):
    # no tile is expanded: the waits run out, the call returns, bit 3 reports it, and the next call is right
    c = Cache(q1, [300], 1, D, seed=27)
    cache = c.store(q1)
    assert q1.device_errors() == 0
    try:
        q1.set_wait_limit_ns(1_000_000)
        q1.set_stalled_producers(True)
        q1.kv_attention(torch.zeros(1, 300, 4, D, dtype=torch.bfloat16, device="cuda"), cache, c.d_table(), c.d_lengths(),
                        max_len=1 << 20)
        torch.cuda.synchronize()
        assert q1.device_errors() == 8
    finally:
        q1.set_stalled_producers(False)
        q1.set_wait_limit_ns(0)
    assert q1.device_errors() == 0
    check(q1, c, cache, [300], 4, tiles=True)
    assert q1.device_errors() == 0


@pytest.mark.gpu
def test_offsets_out_of_range_stay_inside(q1):
    # (results are undefined; nothing outside the arrays is touched, and the others are right)
    c = Cache(q1, [50, 60], 1, 64, seed=15)
    cache = c.store(q1)
    q = torch.randn(4, 2, 64, device="cuda")
    for cu in ([0, 9, 4], [-5, 2, 4], [3, 1, 1 << 30], [0, 0, 0], [4, 4, 4]):
        q1.kv_attention(q, cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(), max_q=2, max_len=60)
        q1.kv_load(cache, c.d_table(), c.d_lengths(), 4, cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
        q1.kv_attention(q.half().repeat(1, 64, 1), cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                        max_q=2, max_len=60)
    for lengths in ([-3, 60], [1 << 30, 60], [-(1 << 31), (1 << 31) - 1]):
        d = torch.tensor(lengths, dtype=torch.int32).cuda()
        q1.kv_attention(q, cache, c.d_table(), d, cu_seqlens=torch.tensor([0, 2, 4], dtype=torch.int32).cuda(), max_q=2, max_len=60)
    torch.cuda.synchronize()
    check(q1, c, cache, [2, 2], 2)


@pytest.mark.gpu
def test_step_by_step_in_a_graph(q1):
    # a captured decode step (store, then attend) replayed while lengths move on, on another stream: the rows of
    # one call over all tokens
    c = Cache(q1, [40, 21], 2, 128, page=16, seed=16)
    new = 12
    whole = c.store(q1)
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32).cuda()
    q = torch.randn(2, new, 6, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    want = q1.kv_attention(q.flatten(0, 1), whole, c.d_table(), c.d_lengths(), cu_seqlens=cu, max_q=new, max_len=48).view(2, new, 6, 128)
    # the same cache without its last tokens
    cache = whole.clone()
    lengths = c.d_lengths() - new
    fill = torch.full((2, new, 2, 128), float("nan"), device="cuda")
    q1.kv_store(cache, fill, fill, c.d_table(), c.d_lengths())
    k1, v1 = (torch.empty(2, 1, 2, 128, device="cuda") for _ in range(2))
    q_in, out = torch.empty(2, 1, 6, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 1, 6, 128, dtype=torch.bfloat16, device="cuda")
    table = c.d_table()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            lengths += 1
            q1.kv_store(cache, k1, v1, table, lengths)
            q1.kv_attention(q_in, cache, table, lengths, max_len=64, out=out)
        lengths.copy_(c.d_lengths() - new)
        for i in range(new):
            for b in range(2):
                at = c.lengths[b] - new + i
                k1[b, 0].copy_(torch.from_numpy(c.k[b][at].astype(np.float32)))
                v1[b, 0].copy_(torch.from_numpy(c.v[b][at].astype(np.float32)))
            q_in.copy_(q[:, i:i + 1])
            graph.replay()
            # two evaluations of the same sums in another order: their two roundings, and P's (two of 2^-11) with values
            # of at most 5
            assert (out[:, 0].float() - want[:, i].float()).abs().max() <= 2.0 ** -8 * want[:, i].float().abs().max() + 2 * 2.0 ** -11 * 5
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [1 << 20, 900])
def test_many_rows_in_a_graph_beside_rows_of_no_sequence(q1, max_len):
    # the tiles' form in parts (by the hint) and the few rows': what no sequence owns stays, a replay follows the lengths
    c = Cache(q1, [300, 900], 2, 128, seed=31)
    cache, table, lengths = c.store(q1), c.d_table(), c.d_lengths()
    cu = torch.tensor([5, 105, 170], dtype=torch.int32).cuda()
    q, qv = _rounded(_rng(32).standard_normal((200, 8, 128)), "bf16")
    q, out = q.cuda(), torch.full((200, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")

    def call():
        return q1.kv_attention(q, cache, table, lengths, cu_seqlens=cu, max_q=100, max_len=max_len, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now in ([300, 900], [150, 470], [40, 900]):
        lengths.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        got = out.double().cpu().numpy()
        assert (got[:5] == 7).all() and (got[170:] == 7).all()
        for b, (t0, t1) in enumerate(((5, 105), (105, 170))):
            n = now[b]
            want, _, size, _ = O.kv_attention(qv[t0:t1], c.kval[b][:n], c.vval[b][:n], np.arange(t1 - t0) + n - (t1 - t0), 128 ** -0.5)
            # check()'s bound with its logits' part below 2^-14 of what |bias|, at most 2 here, adds to the sizes
            assert (np.abs(got[t0:t1] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size + 2.0 ** -10).all(), (now, b)
    assert q1.device_errors() == 0


@pytest.mark.gpu
def test_calls_at_once(q1):
    # on two streams, each with its own workspace: the bits of one after the other
    c = Cache(q1, [2000], 2, 128, seed=33)
    cache, table, lengths = c.store(q1), c.d_table(), c.d_lengths()
    qs = [torch.randn(1, n, 8, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(n)).bfloat16() for n in (100, 1, 33, 100)]
    hints = (1 << 20, 2000, 1 << 20, 2000)
    want = [q1.kv_attention(q, cache, table, lengths, max_len=m) for q, m in zip(qs, hints)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(3):
        got = []
        for stream, q, m in zip(streams, qs, hints):
            with torch.cuda.stream(stream):
                got.append(q1.kv_attention(q, cache, table, lengths, max_len=m))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
def test_calls_that_share_a_workspace(q1):
    c = Cache(q1, [5000, 6000], 1, 128, seed=17)
    cache, ws = c.store(q1), torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    qs = [torch.randn(2, 1, 4, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).half() for i in range(4)]
    want = [q1.kv_attention(q, cache, c.d_table(), c.d_lengths(), max_len=6000) for q in qs]
    table, lengths = c.d_table(), c.d_lengths()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [q1.kv_attention(q, cache, table, lengths, max_len=6000, workspace=ws) for q in qs]
    for _ in range(2):
        ws.fill_(255)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- refusals (no GPU needed: validation comes before the library)
@pytest.fixture
def fake(monkeypatch):
    from bit_affine_quantized_g128_gb300 import q1 as mod

    def _forbidden(*a, **k):
        raise AssertionError("the library was reached with invalid arguments")
    monkeypatch.setattr(mod, "lib", _forbidden)
    monkeypatch.setattr(mod, "_lib", None)
    monkeypatch.setattr(mod, "load_library", _forbidden)
    monkeypatch.setattr(mod, "_is_cuda", lambda t: True)
    monkeypatch.setattr(mod, "_current_device", lambda: torch.device("cpu"))
    return mod


def _host(**kw):
    i32 = torch.int32
    a = dict(cache=torch.zeros(4, 2, 4, 2304, dtype=torch.uint8), block_table=torch.zeros(2, 3, dtype=i32),
             lengths=torch.zeros(2, dtype=i32), cu_seqlens=torch.zeros(3, dtype=i32), k=torch.zeros(6, 2, 128),
             v=torch.zeros(6, 2, 128), q=torch.zeros(6, 4, 128))
    return {**a, **kw}


COMMON = [
    (dict(cache=torch.zeros(4, 2, 4, 2304)), "uint8"),
    (dict(cache=torch.zeros(4, 2, 4, 2300, dtype=torch.uint8)), "kv_cache"),
    (dict(cache=torch.zeros(4, 2, 2304, dtype=torch.uint8)), "kv_cache"),
    (dict(cache=torch.zeros(4, 2, 8, 2304, dtype=torch.uint8)[:, :, ::2]), "contiguous"),
    (dict(cache=torch.zeros(4, 2, 3, 2304, dtype=torch.uint8)), "power of two"),
    (dict(cache=torch.zeros(4, 2, 0, 2304, dtype=torch.uint8)), "power of two"),
    (dict(block_table=torch.zeros(2, 3)), "block_table"),
    (dict(block_table=torch.zeros(6, dtype=torch.int32)), "block_table"),
    (dict(block_table=torch.zeros(0, 3, dtype=torch.int32)), "at least one"),
    (dict(lengths=torch.zeros(3, dtype=torch.int32)), "lengths"),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), "lengths"),
    (dict(lengths=None), "lengths"),
    (dict(cu_seqlens=torch.zeros(2, dtype=torch.int32)), "cu_seqlens"),
]


@pytest.mark.parametrize("change,match", COMMON + [
    (dict(k=torch.zeros(6, 2, 128, dtype=torch.float64), v=torch.zeros(6, 2, 128, dtype=torch.float64)), "bfloat16"),
    (dict(v=torch.zeros(6, 2, 128, dtype=torch.float16)), "agree"),
    (dict(v=torch.zeros(5, 2, 128)), "agree"),
    (dict(k=torch.zeros(6, 2, 64), v=torch.zeros(6, 2, 64)), "heads of 128"),
    (dict(k=torch.zeros(6, 3, 128), v=torch.zeros(6, 3, 128)), "2 heads"),
    (dict(cu_seqlens=None), "without cu_seqlens"),
    (dict(cu_seqlens=None, k=torch.zeros(3, 2, 2, 128), v=torch.zeros(3, 2, 2, 128)), "without cu_seqlens"),
])
def test_store_refuses(fake, change, match):
    a = _host(**change)
    with pytest.raises(ValueError, match=match):
        fake.kv_store(a["cache"], a["k"], a["v"], a["block_table"], a["lengths"], cu_seqlens=a["cu_seqlens"])


@pytest.mark.parametrize("change,match", COMMON + [(dict(rows=-1), "rows"), (dict(dtype=torch.int8), "bfloat16")])
def test_load_refuses(fake, change, match):
    a = _host(**{"rows": 6, "dtype": torch.float32, **change})
    with pytest.raises(ValueError, match=match):
        fake.kv_load(a["cache"], a["block_table"], a["lengths"], a["rows"], cu_seqlens=a["cu_seqlens"], dtype=a["dtype"])


@pytest.mark.parametrize("change,match", COMMON + [
    (dict(q=torch.zeros(6, 4, 128, dtype=torch.int32)), "bfloat16"),
    (dict(q=torch.zeros(6, 3, 128)), "multiple"),
    (dict(q=torch.zeros(6, 4, 64)), "heads of 128"),
    (dict(q=torch.zeros(6, 0, 128)), "multiple"),
    (dict(q=torch.zeros(2, 3, 4, 128)), "cu_seqlens"),
    (dict(cu_seqlens=None, q=torch.zeros(3, 2, 4, 128)), "without cu_seqlens"),
    (dict(window=-1), "window"), (dict(window=5, causal=False), "window"),
    (dict(out=torch.zeros(6, 4, 64)), "out"), (dict(out=torch.zeros(6, 4, 128).half()), "out"),
])
def test_attention_refuses(fake, change, match):
    a = _host(**change)
    kw = {n: a[n] for n in ("window", "causal", "out") if n in a}
    with pytest.raises(ValueError, match=match):
        fake.kv_attention(a["q"], a["cache"], a["block_table"], a["lengths"], cu_seqlens=a["cu_seqlens"], **kw)


def test_cache_sizes():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    assert mod.kv_cache(3, 2, 128, device="cpu").shape == (3, 2, 4, 2304)
    assert mod.kv_cache(0, 1, 64, page_size=16, device="cpu").shape == (0, 1, 1, 1152)
    assert mod.kv_cache(1, 1, 256, 32, 128, device="cpu").shape == (1, 1, 2, 4352)
    for bad in ((1, 1, 96), (1, 1, 64, 64, 128), (1, 1, 128, 64, 32), (1, 1, 128, 48), (1, 1, 128, 8), (1, 0, 128), (-1, 1, 128),
                (1, 1, 128, 64, 0)):
        with pytest.raises(ValueError):
            mod.kv_cache(*bad, device="cpu")


def test_refuses_host_tensors():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    a = _host()
    for call in (lambda: mod.kv_store(a["cache"], a["k"], a["v"], a["block_table"], a["lengths"], cu_seqlens=a["cu_seqlens"]),
                 lambda: mod.kv_load(a["cache"], a["block_table"], a["lengths"], 6, cu_seqlens=a["cu_seqlens"]),
                 lambda: mod.kv_attention(a["q"], a["cache"], a["block_table"], a["lengths"], cu_seqlens=a["cu_seqlens"])):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_workspace_size_by_sizes_alone():
    # no GPU and no pointers needed; 0 where the context is not split or the sizes are refused
    from bit_affine_quantized_g128_gb300 import q1 as mod
    size = mod.lib().q1_kv_attention_workspace_size
    sizes = dict(T=1, B=1, HK=2, D=128, group_size=64, page_size=64, n_pages=1000, table_width=900, table_stride=900)
    call = dict(HQ=8, dtype=0, causal=1, max_q=1, max_len=50000, scale=1.0)
    n = size(mod._CKvCache(**sizes), mod._CKvAttention(**call))
    assert n > 0 and n == size(mod._CKvCache(**sizes, data=4096, block_table=4096, lengths=4096),
                               mod._CKvAttention(**call, q=4096, o=4096, q_stride=1024, o_stride=1024))
    assert size(mod._CKvCache(**sizes), mod._CKvAttention(**{**call, "max_len": 100})) == 0
    for bad in (dict(D=96), dict(group_size=32), dict(page_size=48), dict(T=0), dict(B=0), dict(table_width=1 << 40)):
        assert size(mod._CKvCache(**{**sizes, **bad}), mod._CKvAttention(**call)) == 0
    for bad in (dict(HQ=3), dict(dtype=5), dict(window=3, causal=0)):
        assert size(mod._CKvCache(**sizes), mod._CKvAttention(**{**call, **bad})) == 0


@pytest.mark.gpu
def test_c_refusals(q1):
    p = torch.zeros(1 << 16, device="cuda").data_ptr()
    base = dict(data=p, block_table=p, lengths=p, cu_seqlens=None, n_pages=1, table_width=1, table_stride=1, T=2, B=2, HK=2, D=128,
                group_size=64, page_size=16)
    cases = [(dict(data=None), 1), (dict(block_table=None), 1), (dict(lengths=None), 1), (dict(D=96), 2), (dict(page_size=24), 2),
             (dict(page_size=8), 2), (dict(HK=0), 2), (dict(T=3), 2), (dict(B=0), 2), (dict(table_stride=0), 2), (dict(n_pages=-1), 2),
             (dict(table_width=1 << 40), 2), (dict(data=p + 8), 3), (dict(lengths=p + 2), 3), (dict(group_size=32), 5),
             (dict(D=64, group_size=128), 5)]

    def attend(c={}, **kw):  # noqa: B006
        a = dict(q=p, o=p, lse=None, q_stride=512, o_stride=512, max_q=1, max_len=10, HQ=4, dtype=0, causal=1, window=0, scale=1.0)
        a.update(kw)
        return q1.lib().q1_kv_attention(q1._CKvCache(**{**base, **c}), q1._CKvAttention(**a), None, 0, None)

    def store(c={}, k=p, ks=256, v=p, vs=256, dtype=0):  # noqa: B006
        return q1.lib().q1_kv_store(q1._CKvCache(**{**base, **c}), k, ks, v, vs, dtype, None)

    def load(c={}, k=p, ks=256, v=p, vs=256, dtype=0):  # noqa: B006
        return q1.lib().q1_kv_load(q1._CKvCache(**{**base, **c}), k, ks, v, vs, dtype, None)
    for c, status in cases:
        assert attend(c) == status and store(c) == status and load(c) == status, c
    for call in (store, load):
        for kw, status in ((dict(k=None), 1), (dict(v=None), 1), (dict(k=p + 4), 3), (dict(vs=260), 3), (dict(ks=128), 2), (dict(dtype=7), 4)):
            assert call(**kw) == status, kw
    for kw, status in ((dict(q=None), 1), (dict(o=None), 1), (dict(q=p + 8), 3), (dict(o_stride=516), 3), (dict(q_stride=256), 2),
                       (dict(HQ=3), 2), (dict(window=-1), 2), (dict(window=4, causal=0), 2), (dict(dtype=3), 4), (dict(lse=p + 2), 3)):
        assert attend(**kw) == status, kw
    assert attend(dict(T=2, B=2), max_len=100000) == 6      # the split context's workspace
    L = q1.lib()
    assert L.q1_kv_attention(None, None, None, 0, None) == 1 and L.q1_kv_store(None, p, 1, p, 1, 0, None) == 1
    assert L.q1_kv_attention(q1._CKvCache(**base), None, None, 0, None) == 1
