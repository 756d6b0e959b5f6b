"""examples/hybrid_decoder.py: embedding, Q1 products, gated delta rule, tied head
and sampler as one decoder."""
import importlib.util
import os

import pytest
import torch

from bit_affine_quantized_g128_gb300 import synth
from oracle import serving_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_decoder.py")
    spec = importlib.util.spec_from_file_location("hybrid_decoder", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_decoding_follows_the_prefill(example):
    # tokens generated one by one, then the whole text in one prefill: the hidden
    # states of the last token agree, and so do the recurrent states
    prompts = [synth.token_ids(n, 4096, seed=n).tolist() for n in (5, 70, 33)]
    model = example.HybridDecoder(slots=3, seed=3)
    g = torch.Generator(device="cuda").manual_seed(7)
    tokens = model.generate(prompts, 6, g, temperature=0.9, top_k=40, top_p=0.95)
    assert tokens.shape == (6, 3) and int(tokens.min()) >= 0 and int(tokens.max()) < 4096
    states = [s.clone() for s in model.states]
    whole = [p + tokens[:, b].tolist() for b, p in enumerate(prompts)]
    lengths = [len(w) for w in whole]
    cu = torch.tensor([0, lengths[0], lengths[0] + lengths[1], sum(lengths)], dtype=torch.int32, device="cuda")
    ids = torch.tensor(sum(whole, []), dtype=torch.int32, device="cuda")
    h = model.forward(ids, cu, max(lengths), torch.arange(3, dtype=torch.int32, device="cuda"),
                      torch.ones(3, dtype=torch.int32, device="cuda"))
    assert torch.isfinite(h.float()).all()
    # bf16 activations in between, rounded in different places by the two paths
    # (narrow and prefill products, token by token and chunked): 2^-8 a rounding,
    # some forty of them in a row on the way through two layers, adding like noise
    for a, b in zip(states, model.states):
        assert (a - b).norm() <= 40 ** 0.5 * 2.0 ** -8 * b.norm()


def test_sampled_tokens_are_the_oracles(example):
    model = example.HybridDecoder(slots=4, seed=5)
    h = example.rms_norm(torch.randn(4, 512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))).bfloat16()
    logits = model.logits(h)
    u = torch.tensor([0.1, 0.4, 0.7, 0.95])
    token, _ = example.q1.sample(logits, u.cuda(), temperature=0.5, top_k=30, top_p=0.75)
    for b in range(4):
        want, _ = O.sample_row(logits[b].float().cpu().numpy(), float(u[b]), 0.5, 30, 0.75)
        assert int(token[b]) == want


def test_command(example, capsys, monkeypatch):
    monkeypatch.setattr("sys.argv", ["hybrid_decoder.py", "--tokens", "4", "--batch", "2"])
    example.main()
    assert "tokens/s" in capsys.readouterr().out
