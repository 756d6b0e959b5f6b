"""q1_kv_attention's form for many rows (tcgen05): cases that test_kv_cache.py does not bring there."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as O
from tests.test_kv_cache import DTYPES, Cache, _rng, _rounded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q1():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    mod.load_library()
    return mod


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int32)


def attend(q1, c, cache, q, new, **kw):
    """o and lse (float64) of the rows q, the tiles' form by the hint max_len (a long context has few rows take it, in parts)."""
    kw = {"max_q": max(new), "max_len": 1 << 20, **kw}
    o, lse = q1.kv_attention(q.cuda(), cache, c.d_table(), c.d_lengths(), cu_seqlens=torch.from_numpy(_starts(new)).cuda(),
                             return_lse=True, **kw)
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def bounds(c, b, qv, want, size, big, scale, dtype):
    """Errors of o and lse of sequence b: those that test_kv_cache.check derives for tiles."""
    D, r = c.D, qv.shape[1] // c.heads
    kb = np.abs(c.kq[b][2]).max(0).repeat(c.gs, -1).repeat(r, 0)
    logit = (D / 8 + 16) * 2.0 ** -24 * big + ((D / 8 + 16) * 2.0 ** -23 + 2.0 ** -22) * abs(scale) * (kb * np.abs(qv)).sum(-1)
    info = torch.finfo(DTYPES[dtype])
    floor = 2.0 ** -25 + c.lengths[b] * 2.0 ** -32 * np.abs(c.vval[b]).max()
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
        o, lse = attend(q1, c, c.store(q1), q, [new], max_len=hint)
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
        o, lse = attend(q1, c, one, q[-1:], [1], max_len=n)
        assert np.isnan(o[..., ch]).all() and (np.abs(o[0] - want[-1]) <= err[-1])[:, ~ch].all() and np.isfinite(lse).all()
    assert q1.device_errors() == 0


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
            o, lse = attend(q1, c, c.store(q1), _rounded(q, dtype)[0], [1], max_len=hint, scale=1.0)
            assert np.isnan(o).all() and np.isfinite(lse).all(), (at, hint)
