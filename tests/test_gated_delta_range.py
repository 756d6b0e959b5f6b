"""q1.gated_delta where values of very different size meet in one chunk.

Bounds, per element of o and per column of the state, are relative to the sizes at
the token itself (oracle.serving_oracle.delta_sizes: the largest norm that the column
had, decayed by the gates since), so that a large value does not widen the
bounds of what comes after it has faded:
  * 2^-17 of scale |q_t| size_t, and of the size after the last token.  Every fp32
    operand of the chunked form is a pair of fp16 values, 2^-22 of its own value, and
    a token's result goes through at most eight of them (A, its inverse, T, P', the
    state, R, the scaled U, the gates: 2^-19 if all pull the same way); a quarter
    is left for the sums over up to 64 earlier tokens.  Token by token in fp32 it
    is 2^-24 a few times per token: the same bound covers both forms and all types.
  * 2^-36 of the largest size in the sequence: fp16 values end at 2^-24, 2^-39 of
    the largest value of a row that is scaled to [2^14, 2^15); eight times that
    for a sum over 64 of them.
  * half a unit in the last place of o (finfo.eps / 2), and fp16's smallest step.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as O

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def q1():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    mod.load_library()
    return mod


def _np(x):
    return x.double().numpy()


def _inputs(L, dtype, seed, HK=2, HV=4, DK=128, DV=128):
    """One sequence of ordinary values: keys and values of size 1, slow decays."""
    g = torch.Generator().manual_seed(seed)
    a = dict(q=torch.randn(L, HK, DK, generator=g), k=torch.randn(L, HK, DK, generator=g),
             v=torch.randn(L, HV, DV, generator=g), g=-0.02 * torch.rand(L, HV, generator=g),
             beta=torch.sigmoid(torch.randn(L, HV, generator=g)), state=0.3 * torch.randn(1, HV, DK, DV, generator=g))
    return a, DT[dtype]


def _run(q1, a, dt, l2norm=True, scale=None, arith=2.0 ** -17, least=2.0 ** -36):
    q, k, v = (a[n].to(dt) for n in "qkv")
    L, _, DK = q.shape
    scale = DK ** -0.5 if scale is None else scale
    args = [_np(x) for x in (q, k, v, a["g"], a["beta"], a["state"])]
    want_o, want_s, _ = O.gated_delta(*args, [0, L], scale, l2norm)
    sizes, last = O.delta_sizes(*args[1:], [0, L], l2norm)
    sd = a["state"].cuda()
    o = q1.gated_delta(q.cuda(), k.cuda(), v.cuda(), a["g"].cuda(), a["beta"].cuda(), sd, max_len=L, scale=scale,
                       qk_l2norm=l2norm, cu_seqlens=torch.tensor([0, L], dtype=torch.int32).cuda())
    o, s = _np(o.cpu()), _np(sd.cpu())
    assert q1.device_errors() == 0
    assert np.isfinite(o).all() and np.isfinite(s).all()
    floor = least * np.maximum(sizes.max(0), np.linalg.norm(args[5][0], axis=1))
    e = np.linalg.norm(s[0] - want_s[0], axis=1) / (arith * last[0] + floor + 1e-37)
    assert (e <= 1).all(), f"state off by {e.max():.3g} bounds"
    qn = np.ones(q.shape[:2]) if l2norm else np.linalg.norm(args[0], axis=-1)
    qn = np.repeat(qn, v.shape[1] // q.shape[1], 1)[:, :, None]
    inner = abs(scale) * qn * (arith * sizes + floor)
    half = torch.finfo(dt).eps / 2
    e = np.abs(o - want_o) / (half * (np.abs(want_o) + inner) + inner + (6e-8 if dt == torch.float16 else 1e-37))
    assert (e <= 1).all(), f"o off by {e.max():.3g} bounds at token {int(e.max((1, 2)).argmax())}"


both = pytest.mark.parametrize("dtype", ["bf16", "fp16"])
lengths = pytest.mark.parametrize("L", [20, 64, 130])   # token by token, one chunk, three


@pytest.mark.gpu
@both
@lengths
@pytest.mark.parametrize("factor", [10.0, 100.0, 1000.0, 1e4])
@pytest.mark.parametrize("HK,HV,DK,DV", [(2, 4, 128, 128), (1, 3, 64, 64)])
def test_one_large_value_that_fades(q1, HK, HV, DK, DV, factor, L, dtype):
    for at in (3, 13):
        a, dt = _inputs(L, dtype, 5, HK, HV, DK, DV)
        a["g"] -= 0.3
        a["v"][at] *= factor
        _run(q1, a, dt)


@pytest.mark.gpu
@both
@lengths
def test_one_large_value_late(q1, L, dtype):
    # what lies before it in its chunk does not see it
    a, dt = _inputs(L, dtype, 6)
    a["v"][L - 3] *= 1e4
    _run(q1, a, dt)


@pytest.mark.gpu
@both
@lengths
@pytest.mark.parametrize("before,after", [(1.0, 1.0), (1000.0, 1.0), (1000.0, 0.0)])
def test_a_strong_decay_inside(q1, before, after, L, dtype):
    # what was written before is left at 2^-14 of its size; without new values, all of it
    for at in (9, L // 2, L // 2 + 3):
        a, dt = _inputs(L, dtype, 7)
        a["g"][at] = -10.0
        a["v"][:at] *= before
        a["state"] *= before
        a["v"][at:] *= after
        _run(q1, a, dt)


@pytest.mark.gpu
@both
@lengths
@pytest.mark.parametrize("HK,HV,DK,DV", [(2, 4, 128, 128), (2, 2, 64, 128), (1, 3, 128, 64)])
def test_a_large_entry_overwritten(q1, HK, HV, DK, DV, L, dtype):
    # a state of 1000 under a key, a token that writes an ordinary value under it, and
    # queries for it: the parts of o from the state and from the chunk nearly cancel
    a, dt = _inputs(L, dtype, 8, HK, HV, DK, DV)
    key = a["k"][4]
    a["q"][4:] = key
    unit = (key.to(dt).float() / key.to(dt).float().norm(dim=-1, keepdim=True)).repeat_interleave(HV // HK, 0)
    a["state"][0] += 1000.0 * unit[:, :, None] * torch.sign(a["v"][0])[:, None, :]
    a["beta"][4] = 1.0
    _run(q1, a, dt)
    # the same, written inside the chunk
    a, dt = _inputs(L, dtype, 9, HK, HV, DK, DV)
    a["k"][11] = a["k"][4]
    a["q"][11:] = a["k"][4]
    a["v"][4] *= 1000.0
    a["beta"][4] = a["beta"][11] = 1.0
    _run(q1, a, dt)


@pytest.mark.gpu
@both
@lengths
def test_a_large_entry_that_is_not_asked_for(q1, L, dtype):
    a, dt = _inputs(L, dtype, 10)
    a["state"][0, :, 5] *= 3000.0
    a["k"][:, :, 5] = 0.0
    a["q"][:, :, 5] = 0.0
    _run(q1, a, dt)


@pytest.mark.gpu
@both
@lengths
@pytest.mark.parametrize("small", [1e-4, 1e-6])
def test_small_beta_behind_large_ones(q1, small, L, dtype):
    for at in (2, 6):
        a, dt = _inputs(L, dtype, 11)
        a["beta"][at:] = small * (0.5 + 0.5 * a["beta"][at:])
        a["g"][at] = -14.0
        a["state"] *= 0.0
        _run(q1, a, dt)


@pytest.mark.gpu
@both
@pytest.mark.parametrize("L", [18, 64, 100])
@pytest.mark.parametrize("bk2", [2.05, 3.0])
def test_keys_that_overshoot(q1, bk2, L, dtype):
    # beta |k|^2 above 2: every token's correction grows what it corrects.  The sums
    # over earlier tokens no longer shrink: 2^-15.
    a, dt = _inputs(L, dtype, 12)
    a["k"] *= bk2 ** 0.5 / a["k"].norm(dim=-1, keepdim=True)
    a["beta"][:] = 1.0
    _run(q1, a, dt, l2norm=False, scale=0.1, arith=2.0 ** -15)


@pytest.mark.gpu
@both
@pytest.mark.parametrize("L", [18, 64, 100])
def test_one_key_that_overshoots(q1, L, dtype):
    # beta |k|^2 = r + 1 = 2.2 with one key throughout: what lies under it changes its sign
    # and grows by r = 1.2 with every token, and so does every error.  Each of L tokens
    # then adds 2^-19 of the terms that it sums, and of a series of alternating signs and
    # ratio r the terms are (r + 1) / (r - 1) = 11 times their sum.  (The recurrence in fp32,
    # 2^-24 per step, is 1e-4 off after 64 tokens.)
    a, dt = _inputs(L, dtype, 12)
    a["k"][:] = a["k"][:1]
    a["k"] *= 2.2 ** 0.5 / a["k"].norm(dim=-1, keepdim=True)
    a["beta"][:] = 1.0
    # fp16 outputs end at 65504
    _run(q1, a, dt, l2norm=False, scale=0.1 if dt == torch.bfloat16 else 1e-4, arith=11 * L * 2.0 ** -19)


@pytest.mark.gpu
@both
@pytest.mark.parametrize("L", [64, 130])
@pytest.mark.parametrize("total,steps", [(-5.0, 64), (-30.0, 64), (-30.0, 1), (-45.0, 3)])
def test_a_state_that_only_decays(q1, total, steps, L, dtype):
    # nothing is written: the state is e^G of what it was, however small, and o reads it.
    # Chunk by chunk a factor of 2^-22 and a product's rounding, and an operand's 2^-22;
    # nothing is summed that has not decayed as far.
    a, dt = _inputs(L, dtype, 14)
    a["beta"][:] = 0.0
    a["g"][:] = 0.0
    a["g"][5:5 + steps] = total / steps * (0.75 + 0.5 * torch.rand(steps, 4, generator=torch.Generator().manual_seed(15)))[:L - 5]
    _run(q1, a, dt, arith=2.0 ** -20, least=0.0)


@pytest.mark.gpu
@both
@lengths
def test_gates_that_grow(q1, L, dtype):
    # positive log decays, e^6 over a chunk
    a, dt = _inputs(L, dtype, 13)
    a["g"] = a["g"].abs() + 0.08
    _run(q1, a, dt, arith=2.0 ** -15)
