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
