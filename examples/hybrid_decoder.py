"""A small decoder whose linears are Q1 and whose token mixer is the gated delta rule,
in some layers, if asked for, softmax attention over a 4-bit cache.

    python examples/hybrid_decoder.py [--tokens 32] [--batch 4] [--attend 2]

Random weights (there is no checkpoint here): it shows how the calls go together,
from packed weights to sampled tokens.  Per layer: RMS norm, one Q1 projection to
q, k, v and the two gates, the gated delta rule on its recurrent states, a Q1
projection back; RMS norm and the Q1 feed-forward block.  An attention layer stores its
new keys and values and attends to all that its sequence has in the cache, without a
code of the positions (the recurrent layers know the order).  The head is tied to the
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
    """n_layers of (gated delta rule, feed-forward), hidden size D, HK key and HV value heads of `dim`.  Every `attend`-th layer
    (0: none) is attention, HV query heads over HK of keys and values, with room for max_tokens per slot."""

    def __init__(self, n_layers=2, D=512, HK=2, HV=4, dim=128, F=1024, vocab=4096, slots=8, seed=0, device="cuda", attend=0,
                 max_tokens=1024):
        self.D, self.HK, self.HV, self.dim, self.device = D, HK, HV, dim, device

        def weight(N, K, i):
            return q1.Q1Weight.from_host(synth.q1_tensor(N, K, seed=seed + 97 * i, affine=False), device)

        self.embedding = weight(vocab, D, 1)
        self.n_qkv = 2 * HK * dim + HV * dim
        self.n_in = -(-(self.n_qkv + 2 * HV) // 128) * 128   # q, k, v, then the gates' inputs; rows of 16 bytes
        self.layers = []
        for i in range(n_layers):
            mixes = attend == 0 or (i + 1) % attend != 0    # (else it attends: q, k, v)
            w = [weight(self.n_in if mixes else (HV + 2 * HK) * dim, D, 10 * i + 2), weight(D, HV * dim, 10 * i + 3), weight(F, D, 10 * i + 4),
                 weight(F, D, 10 * i + 5), weight(D, F, 10 * i + 6)]
            a = torch.linspace(1.0, 8.0, HV, device=device)      # decay rates
            self.layers.append((w, a if mixes else None))
        # per layer one recurrent state per slot, or the pages of all slots
        page = 64
        width = -(-max_tokens // page)
        self.max_tokens = max_tokens
        self.states = [torch.zeros(slots, HV, dim, dim, device=device) if a is not None
                       else q1.kv_cache(slots * width, HK, dim, page, device=device) for _, a in self.layers]
        self.pages = torch.arange(slots * width, dtype=torch.int32, device=device).view(slots, width)
        self.lengths = torch.zeros(slots, dtype=torch.int32, device=device)

    def forward(self, ids, cu_seqlens, max_len, slots, fresh):
        """Hidden states [T, D] of the packed tokens `ids`; the sequences' states move on."""
        x, _ = q1.embed_gather(self.embedding, ids)
        x = rms_norm(x)
        HK, HV, d = self.HK, self.HV, self.dim
        if any(a is None for _, a in self.layers):
            slot = slots.long()
            before = self.lengths[slot] if fresh is None else self.lengths[slot] * (fresh == 0)
            lengths = before + cu_seqlens.diff()
            self.lengths[slot] = lengths
            pages = self.pages[slot]
        for ((w_in, w_out, gate, up, down), a), state in zip(self.layers, self.states):
            row = q1.qmm(w_in, rms_norm(x))
            if a is None:
                q, k, v = row.split([HV * d, HK * d, HK * d], 1)
                q1.kv_store(state, k.unflatten(1, (HK, d)), v.unflatten(1, (HK, d)), pages, lengths, cu_seqlens=cu_seqlens)
                o = q1.kv_attention(q.unflatten(1, (HV, d)), state, pages, lengths, cu_seqlens=cu_seqlens, max_q=max_len)
            else:
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
        if any(a is None for _, a in self.layers) and max(lengths) + n_tokens > self.max_tokens:
            raise ValueError(f"the cache has room for {self.max_tokens} tokens per sequence")
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
    p.add_argument("--attend", type=int, default=0, help="every so many-th layer attends over a 4-bit cache")
    args = p.parse_args()
    model = HybridDecoder(slots=args.batch, attend=args.attend)
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
