"""q1.gated_delta against the token-by-token float64 oracle.

Bounds, per element of o: half a unit in the last place of the output type
(finfo.eps / 2 relative), plus the arithmetic's own error.  That is fp32
(2^-24 per operation) wherever a state or a correction is formed; the operands
of the chunked form's matrix products are fp16 pairs (22 bits), except that the
weights of a chunk's own tokens in o are a single fp16 (2^-11 relative).  What
an error in them is relative to is the size of the terms, at most
scale |q| max_t |S_t[:, c]| times a small constant for the chunk's partial sums:
4 is allowed.  The state: 2^-20 per chunk of products, and 2^-24 a few times per
token, relative to the largest norm that the head's state had.
"""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as O

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _inputs(lengths, HK, HV, DK, DV, dtype, seed, pool=None, strided=True, keys="random", decay="mixed"):
    g = torch.Generator().manual_seed(seed)
    T = sum(lengths)
    row = torch.randn(T, 2 * HK * DK + HV * DV, generator=g)
    if keys == "same":       # every key of a head alike: the worst conditioned chunk
        row[:, HK * DK:2 * HK * DK] = row[:1, HK * DK:2 * HK * DK]
    if keys == "tiny":
        row *= 1e-4
    if keys == "large":
        row *= 300.0
    row = row.to(DT[dtype])
    if not strided:
        q, k, v = (x.contiguous() for x in row.split([HK * DK, HK * DK, HV * DV], 1))
    else:
        q, k, v = row.split([HK * DK, HK * DK, HV * DV], 1)
    q, k, v = q.unflatten(1, (HK, DK)), k.unflatten(1, (HK, DK)), v.unflatten(1, (HV, DV))
    step = torch.exp(torch.rand(T, HV, generator=g) * 6.0 - 7.0)
    gate = {"mixed": -(1 + 8 * torch.rand(HV, generator=g)) * step, "none": torch.zeros(T, HV),
            "strong": -40.0 * torch.rand(T, HV, generator=g),
            "reset": torch.where(torch.rand(T, HV, generator=g) < 0.1, -float("inf"), -step)}[decay]
    beta = torch.sigmoid(torch.randn(T, HV, generator=g))
    state = 0.3 * torch.randn(pool or len(lengths), HV, DK, DV, generator=g)
    starts = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return q, k, v, gate, beta, state, starts


def _np(x):
    return x.double().numpy()


def _check(o, state, want_o, want_state, colmax, q, dtype, starts, scale, l2norm, slots, fresh=None):
    assert torch.isfinite(o.float()).all() and torch.isfinite(state).all()
    qn = np.ones(q.shape[:2]) if l2norm else np.linalg.norm(_np(q), axis=-1)
    qn = np.repeat(qn, want_o.shape[1] // q.shape[1], 1)
    eps = torch.finfo(DT[dtype]).eps / 2
    arith = 2.0 ** -19 if dtype == "fp32" else 2.0 ** -11
    for b in range(len(starts) - 1):
        s = slice(starts[b], starts[b + 1])
        L = starts[b + 1] - starts[b]
        size = abs(scale) * qn[s][:, :, None] * colmax[b][None]
        bound = eps * np.abs(want_o[s]) + 4 * arith * size + (6e-8 if dtype == "fp16" else 1e-37)
        err = np.abs(_np(o.cpu())[s] - want_o[s])
        assert (err <= bound).all(), f"sequence {b} (L = {L}): o off by {(err / bound).max():.2f} bounds"
        if slots[b] is None:
            continue
        fro = np.linalg.norm(colmax[b], axis=-1)
        e = np.linalg.norm((_np(state.cpu())[slots[b]] - want_state[slots[b]]).reshape(len(fro), -1), axis=-1)
        assert (e <= 2.0 ** -20 * (4 + L / 16) * fro + 1e-37).all(), \
            f"sequence {b} (L = {L}): state off by {(e / fro).max():.2e}"


def _run(q1, lengths, HK, HV, DK, DV, dtype, seed, l2norm=True, scale=None, slots=None, fresh=None, pool=None, **kw):
    q, k, v, g, beta, state, starts = _inputs(lengths, HK, HV, DK, DV, dtype, seed, pool, **kw)
    scale = DK ** -0.5 if scale is None else scale
    want_o, want_s, colmax = O.gated_delta(_np(q), _np(k), _np(v), _np(g), _np(beta), _np(state), starts, scale, l2norm,
                                           slots, fresh)
    d = "cuda"
    row = torch.cat([x.flatten(1) for x in (q, k, v)], 1).to(d)   # columns of one row, as a projection gives
    n = [q.shape[1] * DK, k.shape[1] * DK, v.shape[1] * DV]
    qd, kd, vd = (x.unflatten(1, (-1, D)) for x, D in zip(row.split(n, 1), (DK, DK, DV)))
    if not kw.get("strided", True):
        qd, kd, vd = qd.contiguous(), kd.contiguous(), vd.contiguous()
    sd = state.to(d)
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=d)  # noqa: E731
    o = q1.gated_delta(qd, kd, vd, g.to(d), beta.to(d), sd, cu_seqlens=i32(starts.tolist()), max_len=max(lengths + [1]),
                       slots=i32(slots), fresh=i32(fresh), scale=scale, qk_l2norm=l2norm)
    entries = list(range(len(lengths))) if slots is None else [s if 0 <= s < state.shape[0] else None for s in slots]
    _check(o, sd, want_o, want_s, colmax, q, dtype, starts, scale, l2norm, entries)
    untouched = [i for i in range(state.shape[0]) if i not in entries]
    assert torch.equal(sd.cpu()[untouched], state[untouched])
    return o, sd


@pytest.fixture(scope="module")
def q1():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    mod.load_library()
    return mod


SHAPES = [(2, 4, 128, 128), (3, 3, 64, 64), (1, 3, 128, 64), (2, 2, 64, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("HK,HV,DK,DV", SHAPES)
@pytest.mark.parametrize("lengths", [[1], [1, 1, 1], [2, 5, 0, 1], [8, 7], [17, 33]], ids=str)
def test_short_sequences(q1, lengths, HK, HV, DK, DV, dtype):
    _run(q1, lengths, HK, HV, DK, DV, dtype, seed=11 + len(lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("HK,HV,DK,DV", SHAPES)
@pytest.mark.parametrize("lengths", [[64], [63, 65], [128, 1, 0, 191], [257], [3, 200, 64]], ids=str)
def test_long_sequences(q1, lengths, HK, HV, DK, DV, dtype):
    _run(q1, lengths, HK, HV, DK, DV, dtype, seed=23 + len(lengths))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("HK,HV,DK,DV", [(4, 8, 128, 128), (8, 16, 128, 128), (8, 16, 64, 128), (16, 16, 128, 64)])
def test_many_heads(q1, HK, HV, DK, DV, dtype):
    # more heads than SMs hold at once, and between half as many and that
    _run(q1, [70, 1, 130, 64, 0, 200, 33, 65, 128, 90], HK, HV, DK, DV, dtype, seed=61, slots=[9, 3, 4, 0, 1, 2, 8, -1, 6, 7],
         fresh=[0, 0, 1, 0, 0, 1, 0, 0, 0, 0], pool=10)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("decay", ["none", "strong", "reset"])
@pytest.mark.parametrize("lengths", [[5], [150, 70]], ids=str)
def test_decays(q1, lengths, decay, dtype):
    _run(q1, lengths, 2, 4, 128, 128, dtype, seed=5, decay=decay)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,keys", [("bf16", "same"), ("fp16", "same"), ("bf16", "tiny"), ("bf16", "large"),
                                        ("fp16", "large")])
@pytest.mark.parametrize("lengths", [[6], [130]], ids=str)
def test_keys(q1, lengths, dtype, keys):
    _run(q1, lengths, 2, 4, 128, 128, dtype, seed=7, keys=keys)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[3, 1, 4], [100, 65, 90]], ids=str)
def test_without_norm_and_with_a_scale(q1, lengths):
    # keys of length about 1, as a caller that normalises itself passes them
    q, k, v, g, beta, state, starts = _inputs(lengths, 2, 4, 128, 128, "bf16", 3)
    k = (k.float() / k.float().norm(dim=-1, keepdim=True)).bfloat16()
    want_o, want_s, colmax = O.gated_delta(_np(q), _np(k), _np(v), _np(g), _np(beta), _np(state), starts, 0.25, False)
    sd = state.cuda()
    o = q1.gated_delta(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), sd,
                       cu_seqlens=torch.from_numpy(starts).cuda(), max_len=max(lengths), scale=0.25)
    _check(o, sd, want_o, want_s, colmax, q, "bf16", starts, 0.25, False, [0, 1, 2])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("decay", ["none", "mixed"])
def test_keys_that_nearly_stop_contracting(q1, dtype, decay):
    # beta |k|^2 up to 1.9: a token's own correction overshoots, the state keeps its size
    q, k, v, g, beta, state, starts = _inputs([200, 50], 2, 4, 128, 128, dtype, 57, decay=decay)
    k = (k.float() / k.float().norm(dim=-1, keepdim=True) * 1.37).to(DT[dtype])
    want_o, want_s, colmax = O.gated_delta(_np(q), _np(k), _np(v), _np(g), _np(beta), _np(state), starts, 0.1, False)
    sd = state.cuda()
    o = q1.gated_delta(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), sd, cu_seqlens=torch.from_numpy(starts).cuda(),
                       max_len=200, scale=0.1)
    _check(o, sd, want_o, want_s, colmax, q, dtype, starts, 0.1, False, [0, 1])


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[1, 1, 1, 1], [70, 1, 130, 5]], ids=str)
def test_slots_fresh_and_missing_entries(q1, lengths):
    _run(q1, lengths, 2, 4, 128, 128, "bf16", seed=9, slots=[5, -1, 2, 0], fresh=[0, 0, 1, 0], pool=7)
    _run(q1, lengths, 2, 4, 128, 128, "bf16", seed=9, slots=[5, 7, 2, 0], fresh=[1, 1, 1, 1], pool=7)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 3, 96])
def test_equal_lengths_without_offsets(q1, L):
    q, k, v, g, beta, state, starts = _inputs([L] * 3, 2, 4, 128, 128, "bf16", 31)
    b4 = lambda x: x.unflatten(0, (3, L)).cuda()  # noqa: E731
    sd, se = state.cuda(), state.cuda()
    o = q1.gated_delta(b4(q), b4(k), b4(v), b4(g), b4(beta), sd, qk_l2norm=True)
    e = q1.gated_delta(q.cuda(), k.cuda(), v.cuda(), g.cuda(), beta.cuda(), se, max_len=L,
                       cu_seqlens=torch.from_numpy(starts).cuda(), qk_l2norm=True)
    assert o.shape == (3, L, 4, 128)
    assert torch.equal(o.flatten(0, 1), e) and torch.equal(sd, se)


@pytest.mark.gpu
@pytest.mark.parametrize("lengths", [[9, 4], [140, 77]], ids=str)
def test_in_pieces_equals_whole(q1, lengths):
    # the state carries a sequence over a cut
    q, k, v, g, beta, state, starts = _inputs(lengths, 2, 4, 128, 128, "bf16", 41)
    cut = [n // 2 for n in lengths]
    ids = [torch.cat([torch.arange(starts[b], starts[b] + cut[b]) for b in range(2)]),
           torch.cat([torch.arange(starts[b] + cut[b], starts[b + 1]) for b in range(2)])]
    want_o, want_s, colmax = O.gated_delta(_np(q), _np(k), _np(v), _np(g), _np(beta), _np(state), starts, 128 ** -0.5, True)
    sd = state.cuda()
    o = torch.empty(v.shape, dtype=v.dtype)
    for part, ns in zip(ids, (cut, [n - c for n, c in zip(lengths, cut)])):
        cu = torch.tensor([0, ns[0], ns[0] + ns[1]], dtype=torch.int32, device="cuda")
        o[part] = q1.gated_delta(q[part].cuda(), k[part].cuda(), v[part].cuda(), g[part].cuda(), beta[part].cuda(), sd,
                                 cu_seqlens=cu, max_len=max(ns), qk_l2norm=True).cpu()
    _check(o, sd, want_o, want_s, colmax, q, "bf16", starts, 128 ** -0.5, True, [0, 1])


@pytest.mark.gpu
def test_neighbours_do_not_leak(q1):
    # a sequence full of infinities and NaN next to a clean one changes nothing in it
    lengths = [70, 90, 3]
    q, k, v, g, beta, state, starts = _inputs(lengths, 2, 4, 128, 128, "bf16", 43)
    args = [x.cuda() for x in (q.contiguous(), k.contiguous(), v.contiguous(), g, beta)]
    cu = torch.from_numpy(starts).cuda()
    s0 = state.cuda()
    o0 = q1.gated_delta(*args, s0, cu_seqlens=cu, max_len=90, qk_l2norm=True)
    for x, bad in zip(args, (float("inf"), float("nan"), float("inf"), float("nan"), float("nan"))):
        x[starts[1]:starts[2]] = bad
    s1 = state.cuda()
    o1 = q1.gated_delta(*args, s1, cu_seqlens=cu, max_len=90, qk_l2norm=True)
    for b in (0, 2):
        assert torch.equal(o0[starts[b]:starts[b + 1]], o1[starts[b]:starts[b + 1]])
        assert torch.equal(s0[b], s1[b])


@pytest.mark.gpu
def test_offsets_out_of_range_stay_inside(q1):
    # results are undefined; the call returns, and nothing outside the arrays is touched
    q, k, v, g, beta, state, starts = _inputs([80, 50], 2, 4, 128, 128, "bf16", 47)
    args = [x.cuda() for x in (q, k, v, g, beta)]
    for bad in ([0, 500, 130], [-5, 80, 130], [90, 20, 1 << 30], [130, 0, 130]):
        for ml in (1, 130):
            q1.gated_delta(*args, state.cuda(), cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), max_len=ml)
    torch.cuda.synchronize()
    assert q1.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("L", [1, 100])
def test_other_stream_and_graph(q1, L):
    q, k, v, g, beta, state, starts = _inputs([L, L], 2, 4, 128, 128, "bf16", 51)
    args = [x.cuda() for x in (q.contiguous(), k.contiguous(), v.contiguous(), g, beta)]
    cu = torch.from_numpy(starts).cuda()
    s0 = state.cuda()
    o0 = q1.gated_delta(*args, s0, cu_seqlens=cu, max_len=L, qk_l2norm=True)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        s1 = state.cuda()
        o1 = q1.gated_delta(*args, s1, cu_seqlens=cu, max_len=L, qk_l2norm=True)
    st.synchronize()
    assert torch.equal(o0, o1) and torch.equal(s0, s1)
    s2, graph = state.cuda(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2 = q1.gated_delta(*args, s2, cu_seqlens=cu, max_len=L, qk_l2norm=True)
    s2.copy_(state.cuda())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o0, o2) and torch.equal(s0, s2)


@pytest.mark.gpu
def test_stalled_copies_time_out_and_recover(q1):
    # nothing is copied for the chunked form: its waits run out, the call returns,
    # bit 2 reports it, the states keep their values, and the next call is right
    q, k, v, g, beta, state, starts = _inputs([100, 70], 2, 4, 128, 128, "bf16", 53)
    args = [x.cuda() for x in (q, k, v, g, beta)]
    cu = torch.from_numpy(starts).cuda()
    want = state.cuda()
    o = q1.gated_delta(*args, want, cu_seqlens=cu, max_len=100, qk_l2norm=True)
    assert q1.device_errors() == 0
    sd = state.cuda()
    try:
        q1.set_wait_limit_ns(1_000_000)
        q1.set_stalled_producers(True)
        q1.gated_delta(*args, sd, cu_seqlens=cu, max_len=100, qk_l2norm=True)
        torch.cuda.synchronize()
        assert q1.device_errors() == 4
        assert torch.equal(sd.cpu(), state)
    finally:
        q1.set_stalled_producers(False)
        q1.set_wait_limit_ns(0)
    assert q1.device_errors() == 0
    again = q1.gated_delta(*args, sd, cu_seqlens=cu, max_len=100, qk_l2norm=True)
    assert torch.equal(o, again) and torch.equal(sd, want)
    assert q1.device_errors() == 0


def _long(lengths, HK, HV, DK, DV, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(lengths)
    q, k = (torch.randn(T, HK, DK, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    v = torch.randn(T, HV, DV, generator=g).to(DT[dtype]).cuda()
    gate, beta = -0.2 * torch.rand(T, HV, generator=g).cuda(), torch.rand(T, HV, generator=g).cuda()
    state = 0.3 * torch.randn(len(lengths) + 1, HV, DK, DV, generator=g).cuda()
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32, device="cuda")
    return (q, k, v, gate, beta), state, cu


# few heads and many chunks: done in two, three or four slabs, whose chunk
# kernels run beside the chain; a hint of 64 tokens gives one slab
@pytest.mark.gpu
@pytest.mark.parametrize("lengths,HK,HV,DK,DV,dtype", [
    ([2113], 16, 32, 128, 128, "bf16"), ([2113], 32, 32, 64, 64, "fp16"), ([5300], 8, 32, 128, 128, "fp16"),
    ([13000], 8, 32, 128, 64, "bf16"), ([40, 8200, 0, 1500], 3, 9, 128, 128, "bf16"), ([17000], 2, 38, 64, 128, "bf16"),
    ([3000, 64, 3000], 4, 24, 128, 64, "fp16")], ids=str)
def test_slabs_equal_one_walk(q1, lengths, HK, HV, DK, DV, dtype):
    args, state, cu = _long(lengths, HK, HV, DK, DV, dtype, seed=71)
    B = len(lengths)
    slots = torch.tensor([B, -1, 0, 1][:B], dtype=torch.int32, device="cuda")  # the second has none
    for fresh in (None, torch.tensor([1, 1, 0, 0][:B], dtype=torch.int32, device="cuda")):
        kw = dict(cu_seqlens=cu, slots=slots, fresh=fresh, qk_l2norm=True)
        s0, s1, s2 = state.clone(), state.clone(), state.clone()
        o0 = q1.gated_delta(*args, s0, max_len=64, **kw)
        o1 = q1.gated_delta(*args, s1, max_len=max(lengths), **kw)
        o2 = q1.gated_delta(*args, s2, **kw)
        assert torch.isfinite(o0.float()).all()
        assert torch.equal(o0, o1) and torch.equal(s0, s1)
        assert torch.equal(o0, o2) and torch.equal(s0, s2)
    assert q1.device_errors() == 0


@pytest.mark.gpu
def test_slabs_against_the_oracle(q1):
    _run(q1, [2100], 2, 38, 64, 64, "bf16", seed=73)


@pytest.mark.gpu
def test_slabs_one_call_after_another(q1):
    # calls that share one workspace, without a wait between them, and in a graph
    args, state, cu = _long([4500], 16, 32, 128, 128, "bf16", seed=79)
    other, _, _ = _long([4500], 16, 32, 128, 128, "bf16", seed=83)
    want, ws = state.clone(), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    outs = [q1.gated_delta(*x, want, cu_seqlens=cu, max_len=64, qk_l2norm=True) for x in (args, other, args, other)]
    got = state.clone()
    again = [q1.gated_delta(*x, got, cu_seqlens=cu, max_len=4500, qk_l2norm=True, workspace=ws)
             for x in (args, other, args, other)]
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(outs, again))
    graph, got = torch.cuda.CUDAGraph(), state.clone()
    with torch.cuda.graph(graph):
        again = [q1.gated_delta(*x, got, cu_seqlens=cu, max_len=4500, qk_l2norm=True, workspace=ws)
                 for x in (args, other, args, other)]
    for _ in range(2):
        got.copy_(state)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(outs, again))


@pytest.mark.gpu
def test_stalled_copies_in_slabs_keep_the_states(q1):
    args, state, cu = _long([5300], 8, 32, 128, 128, "bf16", seed=89)
    want, sd = state.clone(), state.clone()
    o = q1.gated_delta(*args, want, cu_seqlens=cu, max_len=5300, qk_l2norm=True)
    assert q1.device_errors() == 0
    try:
        q1.set_wait_limit_ns(1_000_000)
        q1.set_stalled_producers(True)
        q1.gated_delta(*args, sd, cu_seqlens=cu, max_len=5300, qk_l2norm=True)
        torch.cuda.synchronize()
        assert q1.device_errors() == 4
        assert torch.equal(sd, state)
    finally:
        q1.set_stalled_producers(False)
        q1.set_wait_limit_ns(0)
    again = q1.gated_delta(*args, sd, cu_seqlens=cu, max_len=5300, qk_l2norm=True)
    assert torch.equal(o, again) and torch.equal(sd, want)
    assert q1.device_errors() == 0


# ---- refusals (no GPU needed: validation comes before the library)
@pytest.fixture
def fake(monkeypatch):
    from bit_affine_quantized_g128_gb300 import q1 as mod

    def _forbidden(*a, **k):
        raise AssertionError("the library was reached with invalid arguments")
    monkeypatch.setattr(mod, "lib", _forbidden)
    monkeypatch.setattr(mod, "load_library", _forbidden)
    monkeypatch.setattr(mod, "_is_cuda", lambda t: True)
    monkeypatch.setattr(mod, "_current_device", lambda: torch.device("cpu"))
    return mod


def _host(T=6, HK=2, HV=4, DK=64, DV=64, dtype=torch.bfloat16, B=2):
    return dict(q=torch.zeros(T, HK, DK, dtype=dtype), k=torch.zeros(T, HK, DK, dtype=dtype),
                v=torch.zeros(T, HV, DV, dtype=dtype), g=torch.zeros(T, HV), beta=torch.zeros(T, HV),
                state=torch.zeros(B, HV, DK, DV), cu_seqlens=torch.tensor([0, 3, 6], dtype=torch.int32))


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros(6, 2, 64, dtype=torch.float64)), "bfloat16"),
    (dict(k=torch.zeros(6, 2, 64)), "one dtype"),
    (dict(g=torch.zeros(6, 4, dtype=torch.bfloat16)), "float32"),
    (dict(beta=torch.zeros(6, 3)), "agree"),
    (dict(v=torch.zeros(5, 4, 64, dtype=torch.bfloat16)), "agree"),
    (dict(v=torch.zeros(6, 3, 64, dtype=torch.bfloat16), g=torch.zeros(6, 3), beta=torch.zeros(6, 3)), "multiple of HK"),
    (dict(v=torch.zeros(6, 4, 96, dtype=torch.bfloat16)), "64 or 128"),
    (dict(state=torch.zeros(2, 4, 64, 64, dtype=torch.bfloat16)), "state"),
    (dict(state=torch.zeros(2, 4, 64, 128)[..., ::2]), "contiguous"),
    (dict(state=torch.zeros(1, 4, 64, 64)), "entries"),
    (dict(cu_seqlens=torch.tensor([0, 6])), "cu_seqlens"),
    (dict(cu_seqlens=torch.tensor([0], dtype=torch.int32)), "at least one"),
    (dict(cu_seqlens=None), "without cu_seqlens"),
    (dict(slots=torch.zeros(3, dtype=torch.int32)), "slots"),
    (dict(fresh=torch.zeros(2)), "fresh"),
    (dict(out=torch.zeros(6, 4, 64)), "out"),
])
def test_refuses(fake, change, match):
    with pytest.raises(ValueError, match=match):
        fake.gated_delta(**{**_host(), **change})


def test_refuses_host_tensors():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    with pytest.raises(ValueError, match="CUDA"):
        mod.gated_delta(**_host())


def test_workspace_size_before_the_tensors_exist():
    # by sizes alone (no GPU needed): with and without pointers the same
    from bit_affine_quantized_g128_gb300 import q1 as mod
    size = mod.lib().q1_gated_delta_workspace_size
    sizes = dict(T=300, B=2, HK=2, HV=4, DK=64, DV=64, max_len=200, dtype=0)
    full = dict(q=4096, k=4096, v=4096, o=4096, g=4096, beta=4096, state=4096, cu_seqlens=4096, n_slots=2, q_stride=128,
                k_stride=128, v_stride=256, o_stride=256, g_stride=4, beta_stride=4)
    n = size(mod._CDelta(**sizes, **full))
    assert n > 0 and size(mod._CDelta(**sizes)) == n
    assert size(mod._CDelta(**{**sizes, "T": 301})) > 0        # two unequal sequences: the offsets come later
    for none in (dict(max_len=1), dict(dtype=2), dict(T=0), dict(DK=96), dict(HV=3), dict(B=0)):
        assert size(mod._CDelta(**{**sizes, **none})) == 0


@pytest.mark.parametrize("B,DK,DV,last", [(1, 128, 128, 36), (1, 64, 64, 36), (8, 128, 128, 20), (8, 64, 128, 24),
                                          (8, 128, 64, 32), (8, 64, 64, 40)])
def test_longest_sequences_that_go_token_by_token(B, DK, DV, last):
    # those need no workspace: by the number of heads and, once they fill the GPU, their size
    from bit_affine_quantized_g128_gb300 import q1 as mod
    size = lambda L: mod.lib().q1_gated_delta_workspace_size(  # noqa: E731
        mod._CDelta(T=B * L, B=B, HK=16, HV=48, DK=DK, DV=DV, max_len=L, dtype=0))
    assert size(last) == 0 and size(last + 1) > 0


@pytest.mark.gpu
def test_c_refusals(q1):
    z = torch.zeros(1 << 16, device="cuda")
    p = z.data_ptr()

    def call(**kw):
        a = dict(q=p, k=p, v=p, o=p, g=p, beta=p, state=p, cu_seqlens=None, slots=None, fresh=None, q_stride=128,
                 k_stride=128, v_stride=256, o_stride=256, g_stride=4, beta_stride=4, T=2, B=2, n_slots=2, max_len=1,
                 HK=2, HV=4, DK=64, DV=64, dtype=0, qk_l2norm=1, scale=1.0)
        a.update(kw)
        return q1.lib().q1_gated_delta(q1._CDelta(**a), None, 0, None)
    for kw, status in [(dict(q=None), 1), (dict(state=None), 1), (dict(DK=96), 2), (dict(HV=3), 2), (dict(HK=0), 2),
                       (dict(T=3), 2), (dict(B=0), 2), (dict(n_slots=1), 2), (dict(v_stride=128), 2),
                       (dict(q=p + 2), 3), (dict(k_stride=132), 3), (dict(state=p + 8), 3), (dict(dtype=3), 4)]:
        assert call(**kw) == status, kw
    assert q1.lib().q1_gated_delta(None, None, 0, None) == 1
    # the chunked form without its workspace, or with too small a one
    assert call(T=200, max_len=100) == 6
