"""examples/hybrid_decoder.py with attention layers: Q1 products, gated delta rule, 4-bit cache, attention
and sampler as one decoder, each attention call and each token against the oracle."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from bit_affine_quantized_g128_gb300 import synth
from oracle import serving_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decoder.py")
    spec = importlib.util.spec_from_file_location("hybrid_decoder_attention", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_calls_are_the_oracles(example, monkeypatch):
    q1 = example.q1
    calls, draws = [], []

    def store(cache, k, v, table, lengths, **kw):
        calls.append([k.clone(), v.clone(), kw["cu_seqlens"].tolist(), lengths.tolist()])
        return real_store(cache, k, v, table, lengths, **kw)

    def attention(q, *args, **kw):
        o = real_attention(q, *args, **kw)
        calls[-1] += [q.clone(), o.clone()]
        return o

    def sample(logits, u, **kw):
        token, extra = real_sample(logits, u, **kw)
        draws.append((logits.clone(), u.clone(), token.clone()))
        return token, extra

    real_store, real_attention, real_sample = q1.kv_store, q1.kv_attention, q1.sample
    monkeypatch.setattr(q1, "kv_store", store)
    monkeypatch.setattr(q1, "kv_attention", attention)
    monkeypatch.setattr(q1, "sample", sample)
    prompts = [synth.token_ids(n, 4096, seed=n).tolist() for n in (5, 170, 33)]
    model = example.HybridDecoder(slots=3, seed=3, attend=2, max_tokens=200)
    g = torch.Generator(device="cuda").manual_seed(7)
    tokens = model.generate(prompts, 5, g, temperature=0.5, top_k=30, top_p=0.75)
    assert tokens.shape == (5, 3) and len(calls) == 6 and len(draws) == 5
    seen = [[np.zeros((0, 2, 128)), np.zeros((0, 2, 128))] for _ in prompts]
    for k, v, cu, lengths, q, o in calls:
        k, v, q, o = (x.double().cpu().numpy() for x in (k, v, q, o))
        for b in range(3):
            rows = slice(cu[b], cu[b + 1])
            seen[b] = [np.concatenate([x, y[rows]]) for x, y in zip(seen[b], (k, v))]
            n = cu[b + 1] - cu[b]
            assert lengths[b] == len(seen[b][0])
            kq, vq = (O.kv_quantise(x, 64) for x in seen[b])
            want, _, size, big = O.kv_attention(q[rows], O.kv_values(*kq), O.kv_values(*vq), np.arange(n) + lengths[b] - n, 128 ** -0.5)
            bias = np.abs(vq[2]).max(0).repeat(64, -1).repeat(2, 0)
            # bf16's half step, 2^-8; weights and values as fp16, 2^-11 each; the logits' fp32 sums,
            # their code and bias parts apart
            kb = np.abs(kq[2]).max(0).repeat(64, -1).repeat(2, 0)
            logit = 32 * 2.0 ** -24 * big + (32 * 2.0 ** -23 + 2.0 ** -22) * 128 ** -0.5 * (kb * np.abs(q[rows])).sum(-1)
            bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * (size + bias) + 2 * (2.0 ** -21 + logit)[..., None] * (size + bias) + 2.0 ** -24
            assert (np.abs(o[rows] - want) <= bound).all(), b
    for logits, u, token in draws:
        for b in range(3):
            assert int(token[b]) == O.sample_row(logits[b].float().cpu().numpy(), float(u[b]), 0.5, 30, 0.75)[0]
    assert q1.device_errors() == 0


def test_room_and_slots(example):
    model = example.HybridDecoder(slots=2, seed=4, attend=1, max_tokens=70)
    with pytest.raises(ValueError, match="room for 70"):
        model.generate([[1] * 60], 11)
    # a slot used again starts afresh
    g = torch.Generator(device="cuda")
    first = model.generate([[5, 6, 7], list(range(60))], 6, g.manual_seed(3), temperature=0.7)
    again = model.generate([[5, 6, 7], list(range(60))], 6, g.manual_seed(3), temperature=0.7)
    assert torch.equal(first, again) and model.lengths.tolist() == [9, 66]


def test_command(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["hybrid_decoder.py", "--tokens", "4", "--batch", "2", "--attend", "2"])
    example.main()
    assert "tokens/s" in capsys.readouterr().out
