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


@pytest.mark.parametrize("n_kv,window,max_pos,n", [(65535, 0, (1 << 24) - 1, 1), (16384, 0, (1 << 24) - 1, 4),
                                                   (65535, 1 << 23, (1 << 24) - 1, 1), (4096, 0, (1 << 24) - 1, 1 << 23)])
def test_places_of_keys(m, n_kv, window, max_pos, n):
    """A unit's (kv head, key tile) places in 32 bits, all of a call's in 64 with the CTAs."""
    lay = layer(m, n_q_heads=n_kv, n_kv_heads=n_kv, head_dim=64, rope_dims=64, window=window)
    c = cache(m, n_kv=n_kv, D=64, page=16)
    kw = dict(n_seqs=n, max_pages=1 << 20, max_pos=max_pos)
    assert call(m.lib.attn_paged_decode, DECODE, ref(lay), ref(c), **kw) == 2 and "too many" in m.kvq_last_error()
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(lay), ref(c), n_rows=n, **kw) == 2
    assert m.attn_paged_decode_workspace_bytes(lay, c, n, max_pos) == 0
    assert m.attn_paged_prefill_workspace_bytes(lay, c, n, n, 9, max_pos) == 0


def test_largest_calls_have_workspaces(m):
    """What one GPU's memory can hold the rows of is far below the limits."""
    lay, c = layer(m, n_q_heads=128, n_kv_heads=8, head_dim=128, rope_dims=128, window=0), cache(m, n_kv=8, D=128)
    assert m.attn_paged_decode_workspace_bytes(lay, c, 1 << 20, (1 << 24) - 1) > 0
    assert m.attn_paged_prefill_workspace_bytes(lay, c, 1 << 10, 1 << 20, 1 << 20, (1 << 24) - 1) > 0
