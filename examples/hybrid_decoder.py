"""A small decoder whose linears are Q1 and whose token mixer is the gated delta rule.

    python examples/hybrid_decoder.py [--tokens 32] [--batch 4]

Random weights (there is no checkpoint here): it shows how the calls go together,
from packed weights to sampled tokens.  Per layer: RMS norm, one Q1 projection to
q, k, v and the two gates, the gated delta rule on its recurrent states, a Q1
projection back; RMS norm and the Q1 feed-forward block.  The head is tied to the
Q1 embedding, and each row's token is drawn with its own settings.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_affine_quantized_g128_gb300 import q1, synth  # noqa: E402


def rms_norm(x, eps=1e-6):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)).to(x.dtype)


class HybridDecoder:
    """n_layers of (gated delta rule, feed-forward), hidden size D, HK key and HV value heads of `dim`."""

    def __init__(self, n_layers=2, D=512, HK=2, HV=4, dim=128, F=1024, vocab=4096, slots=8, seed=0, device="cuda"):
        self.D, self.HK, self.HV, self.dim, self.device = D, HK, HV, dim, device

        def weight(N, K, i):
            return q1.Q1Weight.from_host(synth.q1_tensor(N, K, seed=seed + 97 * i, affine=False), device)

        self.embedding = weight(vocab, D, 1)
        self.n_qkv = 2 * HK * dim + HV * dim
        self.n_in = -(-(self.n_qkv + 2 * HV) // 128) * 128   # q, k, v, then the gates' inputs; rows of 16 bytes
        self.layers = []
        for i in range(n_layers):
            w = [weight(self.n_in, D, 10 * i + 2), weight(D, HV * dim, 10 * i + 3), weight(F, D, 10 * i + 4),
                 weight(F, D, 10 * i + 5), weight(D, F, 10 * i + 6)]
            a = torch.linspace(1.0, 8.0, HV, device=device)      # decay rates
            self.layers.append((w, a))
        # one recurrent state per layer and slot
        self.states = [torch.zeros(slots, HV, dim, dim, device=device) for _ in range(n_layers)]

    def forward(self, ids, cu_seqlens, max_len, slots, fresh):
        """Hidden states [T, D] of the packed tokens `ids`; the sequences' states move on."""
        x, _ = q1.embed_gather(self.embedding, ids)
        x = rms_norm(x)
        HK, HV, d = self.HK, self.HV, self.dim
        for ((w_in, w_out, gate, up, down), a), state in zip(self.layers, self.states):
            row = q1.qmm(w_in, rms_norm(x))
            q, k, v = row[:, :self.n_qkv].split([HK * d, HK * d, HV * d], 1)
            gates = row[:, self.n_qkv:self.n_qkv + 2 * HV].float()
            decay = -a * torch.nn.functional.softplus(gates[:, :HV] - 4.0)
            beta = torch.sigmoid(gates[:, HV:])
            o = q1.gated_delta(q.unflatten(1, (HK, d)), k.unflatten(1, (HK, d)), v.unflatten(1, (HV, d)), decay, beta, state,
                               cu_seqlens=cu_seqlens, max_len=max_len, slots=slots, fresh=fresh, qk_l2norm=True)
            x = x + q1.qmm(w_out, rms_norm(o.flatten(1)))
            h = rms_norm(x)
            if h.shape[0] <= 8:
                x = x + q1.ffn_fused(gate, up, down, h)
            else:
                x = x + q1.qmm(down, torch.nn.functional.silu(q1.qmm(gate, h)) * q1.qmm(up, h))
        return rms_norm(x)

    def logits(self, h):
        return q1.qmm(self.embedding, h)

    def generate(self, prompts, n_tokens, generator=None, **settings):
        """n_tokens tokens after each of `prompts` (lists of ids): int32 [n_tokens, B] on the device."""
        B = len(prompts)
        lengths = [len(p) for p in prompts]
        ids = torch.tensor(sum(prompts, []), dtype=torch.int32, device=self.device)
        cu = torch.tensor([sum(lengths[:i]) for i in range(B + 1)], dtype=torch.int32, device=self.device)
        slots = torch.arange(B, dtype=torch.int32, device=self.device)
        fresh = torch.ones(B, dtype=torch.int32, device=self.device)
        h = self.forward(ids, cu, max(lengths), slots, fresh)
        last = h[(cu[1:] - 1).long()].contiguous()
        one = torch.arange(B + 1, dtype=torch.int32, device=self.device)
        out = []
        for _ in range(n_tokens):
            u = torch.rand(B, device=self.device, generator=generator)
            token, _ = q1.sample(self.logits(last), u, **settings)
            out.append(token)
            last = self.forward(token, one, 1, slots, None)
        return torch.stack(out)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=32)
    p.add_argument("--batch", type=int, default=4)
    args = p.parse_args()
    model = HybridDecoder(slots=args.batch)
    prompts = [synth.token_ids(40 + 90 * b, 4096, seed=b).tolist() for b in range(args.batch)]
    g = torch.Generator(device="cuda").manual_seed(1)
    model.generate(prompts, 2, g)
    torch.cuda.synchronize()
    t = time.perf_counter()
    tokens = model.generate(prompts, args.tokens, g, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02)
    torch.cuda.synchronize()
    print(tokens.t().cpu().tolist())
    print(f"{args.batch * args.tokens / (time.perf_counter() - t):.0f} tokens/s")


if __name__ == "__main__":
    main()
