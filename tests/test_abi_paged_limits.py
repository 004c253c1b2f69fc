"""Sizes of the paged calls beyond their kernels' 32-bit arithmetic are refused before anything is enqueued."""
import pytest

from test_abi_paged import APPEND, DECODE, PREFILL, cache, call, layer, m, ref  # noqa: F401


@pytest.mark.parametrize("n_q,n_kv", [(65536, 4096), (131070, 65535), (1048560, 65535)])
def test_q_heads(m, n_q, n_kv):
    lay = layer(m, n_q_heads=n_q, n_kv_heads=n_kv, head_dim=64, rope_dims=64)
    c = cache(m, n_kv=n_kv, D=64, page=16)
    assert call(m.lib.kvq_paged_append, APPEND, ref(lay), ref(c)) == 2 and "65535" in m.kvq_last_error()
    assert call(m.lib.attn_paged_decode, DECODE, ref(lay), ref(c)) == 2
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(lay), ref(c)) == 2
    assert m.attn_paged_decode_workspace_bytes(lay, c, 4, 100) == 0
    assert m.attn_paged_prefill_workspace_bytes(lay, c, 4, 9, 9, 100) == 0
