"""The hints of q1_kv_attention: any value picks a plan that can be launched."""
import pytest

from bit_affine_quantized_g128_gb300 import q1 as mod


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("B,D", [(1, 128), (7, 64), (300, 256)])
def test_any_max_len_has_a_plan(dtype, B, D):
    # (no GPU needed) from 2^31 on the plan is that of the longest sequence that there can be
    size = mod.lib().q1_kv_attention_workspace_size
    c = mod._CKvCache(T=B, B=B, HK=2, D=D, group_size=64, page_size=64, n_pages=1000, table_width=900, table_stride=900)

    def plan(max_len):
        return size(c, mod._CKvAttention(HQ=8, dtype=dtype, causal=1, max_q=1, scale=1.0, max_len=max_len))
    want = plan((1 << 31) - 1)
    assert want < 1 << 30
    for max_len in (1 << 31, 152 << 32, 304 << 32, 0x98000000000, 0x130000000000, 1 << 62, (1 << 63) - 1):
        assert plan(max_len) == want, hex(max_len)


def test_cases_for_tiles_go_by_tiles():
    # (no GPU needed) the lists of test_kv_cache.py that are meant for the form for many rows: all without a window in parts, or in one
    # part; with a window those of WHOLE
    from tests.test_kv_cache import DTYPES, MANY, WHOLE
    for cases, whole in ((MANY, False), (WHOLE, True)):
        for D, gs, HK, r, page, dtype, lengths, new, window in cases:
            c = mod._CKvCache(T=sum(new), B=len(new), HK=HK, D=D, group_size=gs, page_size=page, n_pages=99, table_width=99, table_stride=99)
            a = mod._CKvAttention(HQ=HK * r, dtype=list(DTYPES).index(dtype), causal=1, max_q=max(new), window=window, scale=1.0,
                                  max_len=max(lengths) if whole else 1 << 20)
            parts = mod.lib().q1_kv_attention_parts(c, a)
            assert parts == 1 if whole else window > 0 or parts > 1, (D, HK, r, new)
    a = mod._CKvAttention(HQ=3, dtype=0, causal=1, max_q=1, max_len=1, scale=1.0)
    assert mod.lib().q1_kv_attention_parts(c, a) == -1 and mod.lib().q1_kv_attention_parts(None, a) == -1


@pytest.mark.gpu
def test_many_sequences_without_max_q():
    # 60000 sequences of a row each, their longest unknown: as with the hint, and not refused
    import torch
    B, HK, r, D = 60000, 1, 16, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    cache, table = mod.kv_cache(B, HK, D, page_size=16), torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    lengths = torch.randint(1, 17, (B,), generator=g, device="cuda", dtype=torch.int32)
    kv = torch.randn(2, B, 16, HK, D, generator=g, device="cuda").bfloat16()
    mod.kv_store(cache, kv[0], kv[1], table, torch.full_like(lengths, 16))
    q = torch.randn(B, HK * r, D, generator=g, device="cuda").bfloat16()
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    want = mod.kv_attention(q, cache, table, lengths, cu_seqlens=cu, max_q=1, max_len=16)
    assert torch.equal(mod.kv_attention(q, cache, table, lengths, cu_seqlens=cu, max_len=16), want)


@pytest.mark.gpu
@pytest.mark.parametrize("r,dtype", [(16, "float32"), (64, "float16")])
def test_a_prompt_among_many_tokens(r, dtype):
    # few rows, and tiles (fp16): more row tiles of one sequence than the grid has for each, with the hint and without; rows behind
    # the last sequence
    import numpy as np
    import torch

    from oracle import serving_oracle as O
    B, n, D = 3000, 4001, 64
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.ones(B, dtype=torch.int32, device="cuda")
    rows[1234] = n
    cu = torch.cat([rows[:1] * 0, rows.cumsum(0).int()])
    T = int(cu[-1])
    width = -(-n // 64)
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    table[:, 0] = torch.arange(B)
    table[1234, 1:] = B + torch.arange(width - 1)
    cache = mod.kv_cache(B + width - 1, 1, D)
    kv = torch.randn(2, T, 1, D, generator=g, device="cuda")
    mod.kv_store(cache, kv[0], kv[1], table, rows, cu_seqlens=cu)
    q = torch.randn(T + 5, r, D, generator=g, device="cuda").to(getattr(torch, dtype))
    out = [torch.full_like(q, 7.0) for _ in range(3)]
    for o, max_q in zip(out, (n, None, 1)):
        mod.kv_attention(q, cache, table, rows, cu_seqlens=cu, max_q=max_q, max_len=n, out=o)
    assert torch.equal(out[0], out[1]) and all(bool((o[T:] == 7).all()) for o in out)
    k, v = (x[1234:1234 + n].double().cpu().numpy() for x in mod.kv_load(cache, table, rows, T, cu_seqlens=cu, dtype=torch.float32))
    some = np.array([0, 5, 1000, n - 1])
    want, _, size, _ = O.kv_attention(q[1234 + some].double().cpu().numpy(), k, v, some, D ** -0.5)
    # fp16 outputs and, by tiles, weights and values: three roundings; logits below 2^-14
    bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -10 * size + 2.0 ** -13 * size
    for o in out:
        assert (np.abs(o[1234 + some].double().cpu().numpy() - want) <= bound).all()
    assert mod.device_errors() == 0


def test_out_must_not_overlap_q(monkeypatch):
    # (no GPU needed) a row is read by several CTAs; columns beside q's are none of it
    import torch
    reached = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: reached.append(name) or 0
    monkeypatch.setattr(mod, "_lib", Library())
    monkeypatch.setattr(mod, "_is_cuda", lambda t: True)
    monkeypatch.setattr(mod, "_current_device", lambda: torch.device("cpu"))
    monkeypatch.setattr(mod, "_raw_stream", lambda i: 0)
    cache, table = torch.zeros(4, 2, 4, 2304, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32)
    lengths, cu = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    n = 4 * 128
    flat = torch.zeros(64 * n, dtype=torch.bfloat16)

    def call(T, stride, at, out):
        q = flat[at * n:].as_strided((T, 4, 128), (stride * n, 128, 1))
        mod.kv_attention(q, cache, table, lengths, cu_seqlens=cu, out=flat[out * n:(out + T) * n].view(T, 4, 128))
    for T, stride, at, out in ((6, 1, 8, 2), (6, 1, 8, 14), (1, 1, 8, 7), (1, 1, 8, 9), (3, 8, 8, 9), (3, 8, 8, 13), (3, 8, 8, 5), (3, 8, 8, 25)):
        call(T, stride, at, out)
    assert len(reached) == 8
    for T, stride, at, out in ((6, 1, 8, 8), (6, 1, 8, 3), (6, 1, 8, 13), (1, 1, 8, 8), (3, 8, 8, 14), (3, 8, 8, 6), (3, 8, 8, 24), (3, 2, 8, 9)):
        with pytest.raises(ValueError, match="overlap"):
            call(T, stride, at, out)
    assert len(reached) == 8
