"""q1_kv_attention's form for many rows (tcgen05): cases that test_kv_cache.py does not bring there."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as O
from tests.test_kv_cache import DTYPES, Cache, _rng, _rounded, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q1():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    mod.load_library()
    return mod


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def parts_of(q1, c, T, HQ, dtype, max_q, max_len, window=0, causal=True):
    """The form that such a call takes: 0, or the tiles' with the context in so many parts."""
    B, width = c.table.shape
    cache = q1._CKvCache(T=T, B=B, HK=c.heads, D=c.D, group_size=c.gs, page_size=c.page, n_pages=c.n_pages, table_width=width, table_stride=width)
    return q1.lib().q1_kv_attention_parts(cache, q1._CKvAttention(HQ=HQ, dtype=list(DTYPES).index(dtype), max_q=max_q, max_len=max_len,
                                                                   causal=causal, window=window, scale=1.0))


def attend(q1, c, cache, q, new, few=False, whole=None, **kw):
    """o and lse (float64) of the rows q: by tiles (the context in one part or in several, as `whole` says, if given), or few."""
    kw = {"max_q": max(new), "max_len": 1 << 20, **kw}
    dtype = [n for n, t in DTYPES.items() if t == q.dtype][0]
    form = parts_of(q1, c, q.shape[0], q.shape[1], dtype, kw["max_q"], kw["max_len"], kw.get("window", 0), kw.get("causal", True))
    assert (form > 0) != few and whole in (None, form == 1)
    o, lse = q1.kv_attention(q.cuda(), cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.from_numpy(_starts(new)).cuda(),
                             return_lse=True, **kw)
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def bounds(c, b, qv, want, size, big, scale, dtype, least=2.0 ** -25):
    """Errors of o and lse of sequence b: those that test_kv_cache.check derives for tiles (least: half a step of V's smallest values)."""
    D, r, qv = c.D, qv.shape[1] // c.heads, qv.astype(np.float64)
    kb = np.abs(c.kq[b][2]).max(0).repeat(c.gs, -1).repeat(r, 0)
    logit = (D / 8 + 16) * 2.0 ** -24 * big + ((D / 8 + 16) * 2.0 ** -23 + 2.0 ** -22) * abs(scale) * (kb * np.abs(qv)).sum(-1)
    info = torch.finfo(DTYPES[dtype])
    floor = least + c.lengths[b] * 2.0 ** -32 * np.abs(c.vval[b]).max()
    return (info.eps / 2 * np.maximum(np.abs(want), info.tiny) + floor + 2.0 ** -10 * size + 2 * (2.0 ** -21 + logit)[..., None] * size,
            2.0 ** -21 + logit)


@pytest.mark.parametrize("D,HK,dtype,hint", [(64, 36, "bf16", 640), (64, 24, "fp16", 2000), (128, 24, "fp16", 640), (128, 16, "bf16", 2000),
                                             (256, 24, "bf16", 640), (256, 12, "fp16", 2000)])
def test_logits_that_jump_inside_a_tile(q1, D, HK, dtype, hint):
    # logits rise by 7 octaves at one column of every tile, 32, 64 or 96 of it: a piece of P that the softmax's reference does not
    # fit comes after pieces that are stored already (by their hints, the tiles' context is in one part, in two, in one, ..)
    n, new = 640, 300
    rng = _rng(D)
    tile = 128 if D == 64 else 64
    at = np.arange(n)
    for jump in range(32, tile, 32):
        level = at // tile + (at % tile >= jump)
        k = 0.02 * rng.standard_normal((n, HK, D)) + (7 * np.log(2) * D ** -0.5 * level)[:, None, None]
        c = Cache(q1, [n], HK, D, seed=D + jump, k=[k])
        q, qv = _rounded(1 + 0.02 * rng.standard_normal((new, 2 * HK, D)), dtype)
        o, lse = attend(q1, c, c.store(q1), q, [new], max_len=hint, whole=hint == n)
        some = [0, 1, 31, 32, 77, new - 1]
        want, want_lse, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], np.array(some) + n - new, D ** -0.5)
        err, lerr = bounds(c, 0, qv[some], want, size, big, D ** -0.5, dtype)
        assert (np.abs(o[some] - want) <= err).all() and (np.abs(lse[some] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse)).all(), jump
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,gs,dtype", [(64, 64, "bf16"), (128, 64, "bf16"), (128, 128, "fp16"), (256, 64, "fp16"), (256, 128, "bf16")])
def test_nan_in_one_group_of_v(q1, D, gs, dtype):
    # of a token in the middle, each group in turn (a CTA of a pair has half of the channels): the rows that see it have NaN in
    # that group's channels, the rows before it what they have without it
    n, HK, new, at = 500, 24, 300, 333
    c = Cache(q1, [n], HK, D, gs, seed=D + gs)
    cache = c.store(q1)
    q, qv = _rounded(_rng(D).standard_normal((new, 2 * HK, D)), dtype)
    pos = np.arange(new) + n - new
    some = [0, 100, int(np.argmax(pos == at)) - 1, int(np.argmax(pos == at)), 200, new - 1]
    want, _, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], pos[some], D ** -0.5)
    err, _ = bounds(c, 0, qv[some], want, size, big, D ** -0.5, dtype)
    hit = pos[some] >= at
    for g in range(D // gs):
        k, v = (torch.from_numpy(x[0][at:at + 1].astype(np.float32)).cuda() for x in (c.k, c.v))
        v[:, :, g * gs] = float("nan")
        one = cache.clone()
        q1.kv_store(one, k, v, c.d_table(), torch.tensor([at + 1], dtype=torch.int32).cuda(),
                    cu_seqlens=torch.tensor([0, 1], dtype=torch.int32).cuda())
        for hint in (n, 2000, 1 << 20):
            o, _ = attend(q1, c, one, q, [new], max_len=hint)
            assert np.isnan(o[pos >= at][:, :, g * gs:(g + 1) * gs]).all(), (g, hint)
            assert (np.abs(o[some] - want) <= err)[~hit].all() and not np.isnan(o[pos < at]).any(), (g, hint)
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,gs,dtype", [(64, 64, "fp16"), (128, 64, "fp16"), (128, 128, "bf16"), (256, 64, "bf16"), (256, 128, "fp16")])
def test_nan_in_v_keeps_to_its_group(q1, D, gs, dtype):
    # the other groups' channels, and lse, are what they are without it; by tiles in one part and in several, and by few rows
    n, HK, new, at = 500, 24, 300, 333
    c = Cache(q1, [n], HK, D, gs, seed=D + gs + 1)
    cache = c.store(q1)
    q, qv = _rounded(_rng(D).standard_normal((new, 2 * HK, D)), dtype)
    pos = np.arange(new) + n - new
    some = [0, 100, 200, new - 1]
    want, want_lse, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], pos[some], D ** -0.5)
    err, lerr = bounds(c, 0, qv[some], want, size, big, D ** -0.5, dtype)
    hit = pos[some] >= at
    for g in range(D // gs):
        k, v = (torch.from_numpy(x[0][at:at + 1].astype(np.float32)).cuda() for x in (c.k, c.v))
        v[:, :, g * gs + 5] = float("nan")
        one = cache.clone()
        q1.kv_store(one, k, v, c.d_table(), torch.tensor([at + 1], dtype=torch.int32).cuda(),
                    cu_seqlens=torch.tensor([0, 1], dtype=torch.int32).cuda())
        ch = np.zeros(D, bool)
        ch[g * gs:(g + 1) * gs] = True
        nan = hit[:, None, None] & ch
        for hint in (n, 2000, 1 << 20):
            o, lse = attend(q1, c, one, q, [new], max_len=hint)
            assert np.array_equal(np.isnan(o[some]), np.broadcast_to(nan, want.shape)), (g, hint)
            assert (np.abs(o[some] - want) <= err)[~np.broadcast_to(nan, want.shape)].all(), (g, hint)
            assert (np.abs(lse[some] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse)).all(), (g, hint)
        o, lse = attend(q1, c, one, q[-1:], [1], max_len=n, few=True)
        assert np.isnan(o[..., ch]).all() and (np.abs(o[0] - want[-1]) <= err[-1])[:, ~ch].all() and np.isfinite(lse).all()
    assert q1.device_errors() == 0


def scaled(c, cache, part, octaves):
    """The cache with all scales and biases of K (part 0) or V (part 1) times 2^octaves, and the oracle's values with them."""
    G = c.D // c.gs
    at = part * (2 * c.D + 16 * G) + 2 * c.D
    words = cache.view(torch.int32).clone()
    meta = words[..., at:at + 16 * G].contiguous().view(torch.bfloat16)
    words[..., at:at + 16 * G] = (meta.double() * 2.0 ** octaves).bfloat16().view(torch.int32)
    name, vals = (("kq", "kval"), ("vq", "vval"))[part]
    setattr(c, name, [(x, s * np.float32(2.0 ** octaves), b * np.float32(2.0 ** octaves)) for x, s, b in getattr(c, name)])
    setattr(c, vals, [x * np.float32(2.0 ** octaves) for x in getattr(c, vals)])
    return words.view(torch.uint8)


def small_bounds(c, b, qv, want, size, big, scale, dtype):
    """bounds() for sizes of any kind.  A power of two brings the largest scale or bias `top` of a head (of those that the rows of
    a tile see) to at least 2^-2 before scales, biases and values are rounded to fp16, whose steps end at 2^-24: half a step is
    2^-23 top.  A value of K or V has three such roundings, that of the scale up to 8 times: (8 + 1 + 1) 2^-23 < 2^-19 top."""
    r = qv.shape[1] // c.heads
    top = [np.maximum(np.abs(x[b][1]), np.abs(x[b][2])).max((0, 2)).repeat(r) for x in (c.kq, c.vq)]
    # (half a step among the sum's terms, not taken off a sum that holds 2^-25: in float64 that leaves nothing of terms below 2^-78)
    err, lerr = bounds(c, b, qv, want, size, big, scale, dtype, 2.0 ** -19 * top[1][:, None])
    more = abs(scale) * np.abs(qv.astype(np.float64)).sum(-1) * top[0] * 2.0 ** -19
    return err + 2 * more[..., None] * size, lerr + more


SIZES = [(0, -16), (0, -22), (0, -40), (0, -70), (-16, 0), (-20, 0), (-40, 0), (-18, -18), (12, 12), (40, 40)]    # octaves of K and V


@pytest.mark.parametrize("D,gs,HK,hint", [(64, 64, 36, 400), (64, 64, 24, 2000), (128, 64, 24, 400), (128, 128, 16, 2000), (256, 64, 24, 400),
                                          (256, 128, 12, 2000)])
def test_sizes_of_keys_and_values(q1, D, gs, HK, hint):
    # K and V of any size (of K with a softmax scale to match), by tiles in one part and in two: as right as those of size one
    n, new = 400, 300
    some = [0, 131, new - 1]
    for ke, ve in SIZES:
        c = Cache(q1, [n], HK, D, gs, seed=D + gs)
        cache = scaled(c, scaled(c, c.store(q1), 0, ke), 1, ve)
        dtype, scale = "bf16", D ** -0.5 * 2.0 ** -ke
        q, qv = _rounded(_rng(7).standard_normal((new, 2 * HK, D)), dtype)
        o, lse = attend(q1, c, cache, q, [new], max_len=hint, scale=scale, whole=hint == n)
        want, want_lse, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], np.array(some) + n - new, scale)
        err, lerr = small_bounds(c, 0, qv[some], want, size, big, scale, dtype)
        assert (np.abs(o[some] - want) <= err).all(), (ke, ve, float((np.abs(o[some] - want) / err).max()))
        assert (np.abs(lse[some] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse)).all(), (ke, ve)
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sizes_differ_between_heads_and_sequences(q1, D):
    # each head of each sequence with sizes of its own, a sequence of zeros, another of which rows see nothing; more row tiles than the
    # hint foresees; missing pages and a short table
    lengths, new, HK = [300, 260, 200, 20], [280, 90, 200, 60], 24
    rng = _rng(D + 1)
    ks, vs = (2.0 ** rng.integers(-24, 9, (4, 1, HK, 1)) for _ in range(2))
    for x in (ks, vs):
        x[2] = 0.0
    data = [[rng.standard_normal((n, HK, D)) * s[b] for b, n in enumerate(lengths)] for s in (ks, vs)]
    c = Cache(q1, lengths, HK, D, seed=5, k=data[0], v=data[1])
    c.table[1, 1] = -1
    cache = c.store(q1)
    # rows that bring each head's logits to some size: q against K's size
    q = rng.standard_normal((sum(new), HK, 2, D))
    cu = _starts(new)
    for b in range(4):
        q[cu[b]:cu[b + 1]] /= np.maximum(ks[b], 1e-9)[..., None] if b != 2 else 1.0
    q, qv = _rounded(q.reshape(sum(new), 2 * HK, D), "bf16")
    for kw in (dict(max_len=300), dict(max_len=2000), dict(max_len=2000, max_q=40)):
        o, lse = attend(q1, c, cache, q, new, **kw)
        for b, n in enumerate(new):
            some = np.array([0, n // 2, n - 1])
            rows, pos = cu[b] + some, some + lengths[b] - n
            there = np.array([0 <= c.table[b, p // c.page] < c.n_pages for p in range(lengths[b])])
            want, want_lse, size, big = O.kv_attention(qv[rows], c.kval[b], c.vval[b], pos, D ** -0.5, there=there)
            err, lerr = small_bounds(c, b, qv[rows], want, size, big, D ** -0.5, "bf16")
            assert (np.abs(o[rows] - want) <= err).all(), (kw, b, float((np.abs(o[rows] - want) / err).max()))
            empty = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(lse[rows]), empty)
            assert (np.abs(lse[rows][~empty] - want_lse[~empty]) <= (lerr + 2.0 ** -23 * np.abs(want_lse))[~empty]).all(), (kw, b)
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_sizes_beside_what_is_not_seen(q1, D):
    # small values in the window, the largest that are stored, infinities and NaN before it, behind the sequence and in the pages' rest
    n, HK, new, window = 700, 24, 300, 100
    rng = _rng(D + 2)
    first = n - new - window + 1                       # the first token that a row sees
    k, v = (rng.standard_normal((n, HK, D)) * 1e-6 for _ in range(2))
    for x, y in ((k, 3e4), (v, -3e4)):
        x[:first] = y * rng.random((first, HK, D))
    c = Cache(q1, [n], HK, D, page=32, seed=6, k=[k], v=[v])
    q, qv = _rounded(rng.standard_normal((new, 2 * HK, D)) * 1e6, "bf16")
    some = [0, 130, new - 1]
    pos = np.array(some) + n - new
    want, want_lse, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], pos, D ** -0.5, window=window)
    for x in ("kq", "vq"):                             # (the bounds go by what is seen)
        setattr(c, x, [tuple(a[first:] for a in getattr(c, x)[0])])
    c.vval = [c.vval[0][first:]]
    err, lerr = small_bounds(c, 0, qv[some], want, size, big, D ** -0.5, "bf16")
    cache = torch.full((c.n_pages, HK, 2, 16 * (D + 8 * (D // 64))), 255, dtype=torch.uint8, device="cuda")
    words = cache.view(torch.int32)
    words[::2] = 0x7F807F80                            # infinities in half of the pages, NaN in the others
    q1.kv_store(cache, torch.from_numpy(k.astype(np.float32)).cuda(), torch.from_numpy(v.astype(np.float32)).cuda(), c.d_table(), c.d_lengths(),
                cu_seqlens=torch.tensor([0, n], dtype=torch.int32).cuda())
    bad = cache.clone()
    nan = torch.full((new, HK, D), float("nan"), device="cuda")
    q1.kv_store(bad, nan, nan, c.d_table(), torch.tensor([first], dtype=torch.int32).cuda(), cu_seqlens=torch.tensor([0, new], dtype=torch.int32).cuda())
    for x in (cache, bad):
        o, lse = attend(q1, c, x, q, [new], max_len=n, window=window)
        assert (np.abs(o[some] - want) <= err).all(), float((np.abs(o[some] - want) / err).max())
        assert (np.abs(lse[some] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse)).all()
    assert q1.device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("octaves", [-16, -20, -27, -60, 9])
def test_sizes_of_keys_by_few_rows(q1, dtype, octaves):
    c = Cache(q1, [300, 41], 2, 128, seed=8)
    cache = scaled(c, c.store(q1), 0, octaves)

    class Stored:                                      # check() attends to the cache that it is given
        def __getattr__(self, name):
            return getattr(c, name)
    check(q1, Stored(), cache, [1, 2], 4, dtype, scale=128 ** -0.5 * 2.0 ** -octaves)


@pytest.mark.parametrize("T,new", [(40, [1, 0, 2, 1, 1]), (47, [20, 0, 13]), (200, [90, 33, 40]), (9, [0, 0]), (64, [0])])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_load_of_rows_of_no_sequence(q1, T, new, dtype):
    # before the first sequence and behind the last: zeros, by either form
    c = Cache(q1, [95] * len(new), 3, 64, seed=9)
    cache = c.store(q1)
    for first in {0, 3, T - sum(new)} if sum(new) else {0, 5, T}:
        cu = _starts(new) + first
        big = torch.full((1 << 22,), float("nan"), device="cuda")    # what the allocator hands out next
        del big
        for got, vals in zip(q1.kv_load(cache, c.d_table(), c.d_lengths(), T, cu_seqlens=torch.from_numpy(cu).cuda(), dtype=DTYPES[dtype]),
                             (c.kval, c.vval)):
            want = np.zeros((T, 3, 64), np.float32)
            for b, n in enumerate(new):
                want[cu[b]:cu[b + 1]] = vals[b][95 - n:]
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(DTYPES[dtype])), first


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_nan_of_vanishing_weight(q1, dtype):
    # a token whose weight is below fp32's least value is seen all the same: its NaN shows, in a block that the row sees all of
    # and in one that it sees in part, however the call's hints split the work
    n, D = 40, 128
    rng = _rng(10)
    for at in (5, 35):
        k, v = rng.standard_normal((n, 1, D)), rng.standard_normal((n, 1, D))
        k[:, 0, 0], k[at, 0, 0] = 10.0, -10.0
        v[at] = np.nan
        c = Cache(q1, [n], 1, D, seed=11, k=[k], v=[v])
        q = np.zeros((1, 2, D))
        q[..., 0] = 20.0
        for hint in (n, 1 << 20):
            o, lse = attend(q1, c, c.store(q1), _rounded(q, dtype)[0], [1], max_len=hint, scale=1.0, few=True)
            assert np.isnan(o).all() and np.isfinite(lse).all(), (at, hint)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [1e36, 1e-36])
def test_sizes_of_queries(q1, D, size):
    # rows as large and as small as bf16 and fp32 hold them, with a softmax scale to match, by both forms
    n, new, HK = 400, 300, 24
    c = Cache(q1, [n], HK, D, seed=D + 3)
    cache, scale = c.store(q1), D ** -0.5 / size
    some = [0, 131, new - 1]
    for dtype, first in (("bf16", 0), ("bf16", new - 2), ("fp32", new - 2)):
        q, qv = _rounded(_rng(12).standard_normal((new, 2 * HK, D)) * size, dtype)
        rows = [i for i in some if i >= first]
        o, lse = attend(q1, c, cache, q[first:], [new - first], max_len=n, scale=scale, few=first > 0)
        want, want_lse, wsize, big = O.kv_attention(qv[rows], c.kval[0], c.vval[0], np.array(rows) + n - new, scale)
        err, lerr = small_bounds(c, 0, qv[rows], want, wsize, big, scale, "bf16")
        rows = np.array(rows) - first
        assert (np.abs(o[rows] - want) <= err).all() and (np.abs(lse[rows] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse)).all(), dtype
    assert q1.device_errors() == 0


WINDOWS = [  # D, gs, HK, HQ / HK, page, dtype, window, whether the context is in one part
    (64, 64, 24, 2, 32, "fp16", 100, True), (64, 64, 12, 2, 64, "bf16", 1000, False), (64, 64, 24, 2, 16, "bf16", 1, True),
    (128, 64, 16, 2, 64, "bf16", 20, True), (128, 128, 8, 2, 16, "fp16", 600, False), (128, 64, 10, 3, 32, "bf16", 77, True),
    (256, 64, 12, 2, 32, "bf16", 100, True), (256, 128, 6, 2, 128, "fp16", 800, False), (256, 64, 8, 2, 64, "fp16", 1, True)]


@pytest.mark.parametrize("D,gs,HK,r,page,dtype,window,whole", WINDOWS)
def test_windows_by_tiles(q1, D, gs, HK, r, page, dtype, window, whole):
    lengths, new = [1200, 400, 33], [300, 40, 33]
    c = Cache(q1, lengths, HK, D, gs, page, seed=D + window)
    kw = dict(max_q=300, max_len=1200, window=window)
    parts = parts_of(q1, c, sum(new), HK * r, dtype, **kw)
    assert parts == 1 if whole else parts > 1
    check(q1, c, c.store(q1), new, HK * r, dtype, tiles=True, **kw)
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,gs,HK,r,page,dtype,window,whole", [w for w in WINDOWS if w[6] > 1])
def test_windows_by_tiles_beside_nan(q1, D, gs, HK, r, page, dtype, window, whole):
    # NaN in K or V of one token, behind the sequences and in pages of no sequence: rows whose window has left it, or not reached it
    n, new = 1200, 300
    at = n - new - window + 150                        # the first 150 rows see it, or as many as the window has
    c = Cache(q1, [n, 40], HK, D, gs, page, seed=D + window + 1)
    kept = torch.full((c.n_pages, HK, page // 16, 16 * (D + 8 * (D // gs))), 255, dtype=torch.uint8, device="cuda")
    rows = [torch.from_numpy(np.concatenate(x).astype(np.float32)).cuda() for x in (c.k, c.v)]
    q1.kv_store(kept, *rows, c.d_table(), c.d_lengths(), cu_seqlens=torch.tensor([0, n, n + 40], dtype=torch.int32).cuda())
    q, qv = _rounded(_rng(9).standard_normal((new, HK * r, D)), dtype)
    pos = np.arange(new) + n - new
    some = np.unique(np.clip([0, 149 - window, 150 - window, 149, 150, new - 1], 0, None))
    want, want_lse, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], pos[some], D ** -0.5, window=window)
    err, lerr = bounds(c, 0, qv[some], want, size, big, D ** -0.5, dtype)
    hit = (pos >= at) & (pos < at + window)
    for of_v in (False, True):
        one = [x[at:at + 1].clone() for x in rows]
        one[of_v][:] = float("nan")
        cache = kept.clone()
        q1.kv_store(cache, *one, c.d_table(), torch.tensor([at + 1, 0], dtype=torch.int32).cuda(),
                    cu_seqlens=torch.tensor([0, 1, 1], dtype=torch.int32).cuda())
        o, lse = attend(q1, c, cache, q, [new, 0], max_len=n, window=window, whole=whole)
        assert np.isnan(o[hit]).all() and not np.isnan(o[~hit]).any()
        assert (np.abs(o[some] - want) <= err)[~hit[some]].all()
        good = ~hit[some] | of_v
        assert (np.abs(lse[some] - want_lse) <= lerr + 2.0 ** -23 * np.abs(want_lse))[good].all() and (of_v or np.isnan(lse[hit]).all())
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,HK,whole", [(64, 36, True), (64, 16, False), (128, 24, True), (128, 12, False), (256, 24, True), (256, 8, False)])
def test_offsets_out_of_range_stay_inside_by_tiles(q1, D, HK, whole):
    # (results are undefined; nothing outside the arrays is touched, and the next call is right)
    n, T, hint = 400, 300, 400 if whole else 2000
    c = Cache(q1, [n, 90], HK, D, seed=15)
    cache, table = c.store(q1), c.d_table()
    q, qv = _rounded(_rng(16).standard_normal((T, 2 * HK, D)), "bf16")
    qd, out = q.cuda(), torch.zeros(T + 2, 2 * HK, D, dtype=torch.bfloat16, device="cuda")
    parts = parts_of(q1, c, T, 2 * HK, "bf16", T, hint)
    assert parts == 1 if whole else parts > 1
    out[0], out[-1] = 7.0, 7.0

    def call(cu, lengths):
        q1.kv_attention(qd, cache, table, torch.tensor(lengths, dtype=torch.int32).cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda(),
                        max_q=T, max_len=hint, out=out[1:-1])
    for cu in ([0, 900, 40], [-5, 200, 300], [300, 1, 1 << 30], [0, 0, 0], [300, 300, 300], [200, 100, 300], [1 << 30, -(1 << 31), 5]):
        call(cu, [n, 90])
    for lengths in ([-3, 90], [1 << 30, 90], [-(1 << 31), (1 << 31) - 1]):
        call([0, 290, 300], lengths)
    torch.cuda.synchronize()
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
    call([0, 290, 300], [n, 90])
    some = np.array([0, 130, 289])
    want, _, size, big = O.kv_attention(qv[some], c.kval[0], c.vval[0], some + n - 290, D ** -0.5)
    err, _ = bounds(c, 0, qv[some], want, size, big, D ** -0.5, "bf16")
    assert (np.abs(out[1:-1][some].double().cpu().numpy() - want) <= err).all()
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,HK,r,new,dtype,n", [(128, 19, 4, 512, "fp16", 200000), (128, 19, 4, 512, "fp16", 400000), (64, 38, 2, 500, "fp16", 150000), (256, 38, 2, 512, "bf16", 600000),
                                                (128, 1, 2, 1, "fp16", 1200000), (64, 200, 1, 1, "fp16", 700000)])
def test_long_sums_of_one_sign_in_16_bits(q1, D, HK, r, new, dtype, n):
    # contexts so long that what the tensor cores cut off their sums would show, with enough heads to fill the GPU without a split.
    # Relative to o of nearly equal weights: its rounding eps / 2, and in a part of 2^15 tokens with two products (fp16) or of 2^18 (bf16),
    # by few rows 2^15 per warp with two, 2^12 (2^14) additions that each cut at most 2^-23 of what has grown to half on average: 2^-12
    # (2^-10).  By tiles V's rounding, 2^-11: it does not average over the tokens, as nearly all of a channel's values have the same
    # code (the range of a group is -1 .. 1.05, its step 0.14), and so differ by the few values of their scale and bias in bf16.
    # P's roundings do, below 2^-14.
    g = torch.Generator(device="cuda").manual_seed(D)
    width = -(-n // 64)
    cache, table = q1.kv_cache(width, HK, D), torch.arange(width, dtype=torch.int32, device="cuda").view(1, -1)
    kept = torch.zeros(2, n, D, device="cuda")
    step = 1 << 14
    for t in range(0, n, step):
        m = min(step, n - t)
        k, v = 0.2 * torch.randn(1, m, HK, D, generator=g, device="cuda"), 1 + 0.05 * torch.rand(1, m, HK, D, generator=g, device="cuda")
        v[..., 5::64] = -1.0
        length = torch.tensor([t + m], dtype=torch.int32, device="cuda")
        q1.kv_store(cache, k, v, table, length)
        kept[:, t:t + m] = torch.stack([x[0, :, HK - 1] for x in q1.kv_load(cache, table, length, m, dtype=torch.float32)])
    q = torch.randn(1, new, HK * r, D, generator=g, device="cuda").to(DTYPES[dtype])
    o, lse = q1.kv_attention(q, cache, table, length, max_len=n, return_lse=True)
    k, v = kept.double()
    x = (k @ q[0, -1, -1].double()) * D ** -0.5
    want = torch.softmax(x, 0) @ v
    cut = 2.0 ** -12 if dtype == "fp16" else 2.0 ** -10
    of_v = 2.0 ** -11 if new > 1 else 0.0
    assert ((o[0, -1, -1].double() - want).abs() <= (torch.finfo(DTYPES[dtype]).eps / 2 + of_v + cut + 2.0 ** -14) * want.abs()).all()
    assert abs(float(lse[0, -1, -1]) - float(torch.logsumexp(x, 0))) <= 2.0 ** -18
    assert q1.device_errors() == 0


@pytest.mark.parametrize("D,HK,hint", [(64, 36, 600), (64, 24, 2000), (128, 24, 600), (128, 16, 2000), (256, 24, 600), (256, 12, 2000)])
def test_values_enter_fp16_rows_exactly(q1, D, HK, hint):
    # equal weights, which are powers of two, over values of two sizes per channel: what o is off beyond its own rounding (2^-11) is
    # what the values were, and sums of 600 tokens in two products, below 2^-16 of what they add up in size
    n, new = 600, 300
    base = _rng(D).standard_normal((1, HK, D))
    c = Cache(q1, [n], HK, D, seed=D, k=[_rng(D + 1).standard_normal((n, HK, D))], v=[base * np.where(np.arange(n) % 2, 1.37, 1.0)[:, None, None]])
    o, lse = attend(q1, c, c.store(q1), torch.zeros(new, 2 * HK, D, dtype=torch.float16), [new], max_len=hint, causal=False, whole=hint == n)
    v = c.vval[0].astype(np.float64)
    want = v.mean(0).repeat(2, 0)
    size = (np.abs(v - np.repeat(c.vq[0][2], 64, -1)) + np.abs(np.repeat(c.vq[0][2], 64, -1))).mean(0).repeat(2, 0)
    assert (np.abs(o - want) <= 2.0 ** -11 * np.maximum(np.abs(want), 2.0 ** -14) + 2.0 ** -16 * size).all()
    assert (np.abs(lse - np.log(n)) <= 2.0 ** -20).all()
