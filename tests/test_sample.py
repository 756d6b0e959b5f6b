"""q1.sample against a float64 oracle, row by row: tokens equal, probabilities
to fp32 rounding (2^-24) plus the weights' 2^-33.

The inputs are seeded; a draw within 1e-9 (relative) of a border between two
tokens would be a coin toss between the two implementations, so the oracle's
inputs avoid none on purpose but none is that close.
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


def _compare(q1, logits, u, **settings):
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in settings.items()}
    token, prob = q1.sample(logits if logits.is_cuda else logits.cuda(), u.cuda(), **dev)
    token, prob = token.cpu().numpy(), prob.cpu().double().numpy()
    x = logits.float().cpu().numpy()
    for b in range(x.shape[0]):
        # the settings as the call takes them: fp32
        s = {k: float(v[b] if isinstance(v, torch.Tensor) else np.float32(v)) for k, v in settings.items()}
        if "top_k" in s:
            s["top_k"] = int(s["top_k"])
        t, p = O.sample_row(x[b], float(u[b]), **s)
        assert token[b] == t, f"row {b} {s}: token {token[b]}, oracle {t}"
        assert abs(prob[b] - p) <= 2.0 ** -23 * p, f"row {b}: prob {prob[b]}, oracle {p}"


def _logits(B, V, dtype, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    x = std * torch.randn(B, V, generator=g)
    x[torch.arange(B), torch.randint(0, V, (B,), generator=g)] += 6.0
    return x.to(DT[dtype]), torch.rand(B, generator=g), g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4099, 32003, 152064])
def test_temperature_only(q1, V, dtype):
    x, u, _ = _logits(6, V, dtype, 100 + V)
    _compare(q1, x, u)
    _compare(q1, x, u, temperature=0.7)
    _compare(q1, x, u, temperature=torch.tensor([0.2, 0.5, 1.0, 1.5, 5.0, 100.0]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("V", [5, 1003, 32003])
@pytest.mark.parametrize("std", [0.3, 3.0])
def test_truncations(q1, V, dtype, std):
    x, u, g = _logits(9, V, dtype, 7 * V, std)
    k = torch.tensor([1, 2, 3, 17, 50, 400, V, 0, V + 5], dtype=torch.int32)
    p = torch.tensor([0.1, 0.5, 0.9, 0.95, 0.99, 0.999, 1.0, 1e-6, 0.0])
    m = torch.tensor([0.5, 0.1, 0.05, 0.01, 1e-3, 1e-6, 0.0, 1.0, 3.0])
    t = 0.5 + torch.rand(9, generator=g)
    _compare(q1, x, u, top_k=k)
    _compare(q1, x, u, top_p=p)
    _compare(q1, x, u, min_p=m)
    _compare(q1, x, u, temperature=t, top_k=k, top_p=p.flip(0), min_p=m)
    _compare(q1, x, u, temperature=t, top_k=k.flip(0), top_p=p, min_p=m.flip(0))
    _compare(q1, x, u, top_k=20, top_p=0.9, min_p=0.02, temperature=0.8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [32003, 262144])
def test_wide_nuclei(q1, V, dtype):
    # top-p that ends among tokens of tiny weight, flat rows, and large top-k before it
    x, u, _ = _logits(6, V, dtype, V + 1)
    p = torch.tensor([0.99, 0.9999, 0.99999, 0.999999, 1 - 2.0 ** -24, 0.5])
    _compare(q1, x, u, top_p=p)
    _compare(q1, x, u, top_p=p.flip(0), temperature=50.0)
    _compare(q1, x, u, top_p=p, temperature=0.05)
    _compare(q1, x, u, top_k=torch.tensor([1500, 3000, 9000, 20000, 31000, 32002], dtype=torch.int32), top_p=p.flip(0), temperature=3.0)
    _compare(q1, x, u, top_k=torch.tensor([1025, 2048, 5000, 10000, 20000, 32000], dtype=torch.int32), min_p=1e-4)


@pytest.mark.gpu
def test_ties_go_to_the_lowest_index(q1):
    V = 20000   # more equal logits in one place than the sorted list holds
    x = torch.zeros(8, V)
    x[1, ::2] = 1.0
    x[2, 100:16100] = 3.0
    x[3, 5000:] = -0.0
    x[4, ::3] = 2.0
    x[5, -1] = 4.0
    u = torch.tensor([0.0, 0.25, 0.5, 0.999, 0.3, 0.9, 0.75, 0.125])
    k = torch.tensor([5000, 9000, 15000, 3, 6000, 4000, 19999, 1], dtype=torch.int32)
    _compare(q1, x, u, top_k=k)
    _compare(q1, x, u, top_p=torch.tensor([0.5, 0.25, 0.5, 0.75, 0.3, 0.9, 0.5, 0.125]))
    _compare(q1, x, u, top_k=k, top_p=0.5)
    _compare(q1, x.bfloat16(), u, top_k=k, top_p=0.25, min_p=0.5)
    _compare(q1, x, u, temperature=0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1030, 2100, 20000])
def test_nuclei_of_equal_logits_many_times(q1, V):
    # top-p that ends among more equal logits than the sorted list holds: every CTA of
    # a row forms the same sums before they go on to bisect for the end.  Short slices
    # leave the least time between the two; enough rows run to fill the GPU.
    for B in (1, 64, 400):
        x = torch.zeros(B, V)
        x[:, 0] = (torch.arange(B) % 3).float()          # rows differ
        u = (0.137 + 0.7548776662 * torch.arange(B)) % 1.0
        p = 0.2 + 0.6 * ((torch.arange(B) * 0.6180339887) % 1.0)
        # one weight of exp(l_0) at index 0, then V - 1 ones: the kept ones are 0 .. n - 1
        # (all rows' sums are far from a border between two tokens: checked here)
        w0 = torch.exp(x[:, 0].double())
        total = w0 + (V - 1)
        over = p.float().double() * total - w0           # ones needed beyond index 0
        assert ((over - over.round()).abs() > 2e-6).all()
        kept = w0 + torch.ceil(over).clamp(min=0)
        at = u.float().double() * kept - w0
        assert ((at - at.round()).abs() > 2e-6).all()
        want = torch.where(at < 0, 0.0, torch.floor(at) + 1).int()
        xd, ud, pd = x.cuda(), u.cuda(), p.cuda()
        for _ in range(20):
            token, _ = q1.sample(xd, ud, top_p=pd)
            assert torch.equal(token.cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masked_rows(q1, dtype):
    V, inf = 3000, float("inf")
    x, u, _ = _logits(9, V, dtype, 3)
    x[0, :] = -inf                          # nothing left
    x[1, :] = float("nan")
    x[2, 1:] = -inf                         # one token
    x[3, ::2] = -inf
    x[4, 1::2] = float("nan")
    x[5, 7] = inf                           # infinities share the weight
    x[5, 2900] = inf
    x[6, :2000] = torch.finfo(DT[dtype]).min
    x[7, :] = torch.finfo(DT[dtype]).min    # a mask by the type's lowest value over the whole row
    x[8, :] = torch.finfo(DT[dtype]).min
    x[8, 55] = torch.finfo(DT[dtype]).max
    for kw in (dict(), dict(top_k=5), dict(top_p=0.9), dict(min_p=0.1), dict(temperature=0.0),
               dict(temperature=0.5, top_k=40, top_p=0.8, min_p=0.05)):
        _compare(q1, x, u, **kw)


@pytest.mark.gpu
def test_temperatures_and_numbers_at_the_ends(q1):
    x, u, _ = _logits(8, 5000, "fp32", 77)
    t = torch.tensor([1e-45, 1e-20, 1e-3, 0.0, -1.0, 1e6, 1e30, float("inf")])
    _compare(q1, x, u, temperature=t)
    ends = torch.tensor([0.0, 1e-30, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1e-10, 2.0 ** -40])
    _compare(q1, x, ends)
    _compare(q1, x, ends, top_k=3)
    token, _ = q1.sample(x.cuda(), torch.tensor([1.0, 2.0, float("inf"), -1.0, float("nan"), 0.0, 0.0, 0.0]).cuda())
    last = [int(torch.nonzero(torch.exp(x[b].double() - x[b].max()) > 0)[-1]) for b in range(3)]
    assert token.cpu().tolist()[:3] == last
    assert token.cpu().tolist()[3:] == [0] * 5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 3, 5])
def test_strides_and_alignment(q1, dtype, offset):
    big, u, _ = _logits(5, 3011, dtype, 13)
    view = big.cuda()[:, offset:offset + 3001 - 2 * offset]
    _compare(q1, view, u, top_k=30, top_p=0.9)
    _compare(q1, big.cuda().t().contiguous().t(), u, top_p=0.9)   # column order: copied by the binding


@pytest.mark.gpu
def test_batches(q1):
    for B in (0, 1, 2, 37, 300):
        x, u, _ = _logits(B, 2000, "bf16", B) if B else (torch.zeros(0, 2000, dtype=torch.bfloat16), torch.zeros(0), None)
        _compare(q1, x, u, top_k=50, top_p=0.9, temperature=0.9)


@pytest.mark.gpu
def test_frequencies(q1):
    # many uniform numbers over one row: each token's share is its probability
    V, n = 50, 4000
    x = torch.linspace(-2, 2, V)
    u = (torch.arange(n) + 0.5) / n
    token, prob = q1.sample(x[None].expand(n, V).contiguous().cuda(), u.cuda())
    share = torch.bincount(token.cpu().long(), minlength=V) / n
    p = torch.softmax(x.double(), 0)
    assert (share - p).abs().max() <= 1.0 / n
    assert (prob.cpu().double() - p[token.cpu().long()]).abs().max() <= 2.0 ** -22


@pytest.mark.gpu
def test_graph_replay(q1):
    x, u, _ = _logits(4, 9000, "bf16", 21)
    xd, ud = x.cuda(), u.cuda()
    want = q1.sample(xd, ud, top_p=0.9)[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, _ = q1.sample(xd, ud, top_p=0.9)
    graph.replay()
    assert torch.equal(token, want)
    ud.copy_(torch.rand(4))
    graph.replay()
    assert torch.equal(token, q1.sample(xd, ud, top_p=0.9)[0])


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


@pytest.mark.parametrize("logits,u,kw,match", [
    (torch.zeros(3), torch.zeros(3), {}, "2-D"),
    (torch.zeros(3, 4, dtype=torch.float64), torch.zeros(3), {}, "bfloat16"),
    (torch.zeros(3, 0), torch.zeros(3), {}, "V"),
    (torch.zeros(1, (1 << 18) + 1, dtype=torch.bfloat16), torch.zeros(1), {}, "V"),
    (torch.zeros(3, 4), torch.zeros(2), {}, "u must"),
    (torch.zeros(3, 4), torch.zeros(3, dtype=torch.float64), {}, "u must"),
    (torch.zeros(3, 4), None, {}, "u must"),
    (torch.zeros(3, 4), torch.zeros(3), dict(top_k=torch.zeros(3)), "top_k"),
    (torch.zeros(3, 4), torch.zeros(3), dict(top_p=torch.zeros(2)), "top_p"),
    (torch.zeros(3, 4), torch.zeros(3), dict(temperature=torch.zeros(3, dtype=torch.float16)), "temperature"),
])
def test_refuses(fake, logits, u, kw, match):
    with pytest.raises(ValueError, match=match):
        fake.sample(logits, u, **kw)


def test_refuses_host_tensors():
    from bit_affine_quantized_g128_gb300 import q1 as mod
    with pytest.raises(ValueError, match="CUDA"):
        mod.sample(torch.zeros(2, 4), torch.zeros(2))


@pytest.mark.gpu
def test_c_refusals(q1):
    z = torch.zeros(64, device="cuda")
    p = z.data_ptr()

    def call(**kw):
        a = dict(logits=p, u=p, token=p, B=1, V=8, row_stride=8, dtype=2, temperature_value=1.0, top_p_value=1.0)
        a.update(kw)
        return q1.lib().q1_sample(q1._CSample(**a), None)
    for kw, status in [(dict(logits=None), 1), (dict(u=None), 1), (dict(token=None), 1), (dict(V=0), 2),
                       (dict(V=(1 << 18) + 1, row_stride=1 << 19), 2), (dict(B=-1), 2), (dict(B=2, row_stride=7), 2),
                       (dict(logits=p + 1), 3), (dict(dtype=5), 4)]:
        assert call(**kw) == status, kw
