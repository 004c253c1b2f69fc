"""The size of attn_train_backward's workspace against the limit that
include/kvq.h states, to the longest passes the call takes (host only)."""
import pytest

MIB = 1 << 20


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def limit(n_q, n_kv, D, window, n_blocks, n_rows, max_rows):
    """A row sees the prefix (max_rows at most) and its own block up to itself,
    or its window."""
    keys = min(n_rows, max_rows * (2 if n_blocks > 1 else 1))
    keys = min(keys, window) if window else keys
    tiles = max(1 << 30, 2048 * keys) if keys > 500_000 else 1 << 30
    return (tiles + max(256 * MIB, 8 * n_rows * n_kv * D) + 4 * n_rows * n_q + 104 * n_rows + 8 * n_blocks +
            4 * MIB)


@pytest.mark.parametrize("n_q,n_kv,D", [(16, 1, 512), (8, 2, 256), (8, 8, 64), (1, 1, 128), (64, 4, 64)])
@pytest.mark.parametrize("window", [0, 1, 512, 100_000])
def test_workspace_stays_within_its_limit(m, n_q, n_kv, D, window):
    lay = m.layer(n_q, n_kv, D, window, 0, 1e4)
    f = m.attn_train_backward_workspace_bytes
    sized = 0
    for n_rows in (1, 77, 2048, 5800, 60_001, 524_288, 700_001, 1_000_000, 2_000_000, 4_000_000, (1 << 24) - 1):
        for n_blocks in (1, 2, 9, 1000, 65535):
            for max_rows in {n_rows, (n_rows + 1) // 2, (n_rows + n_blocks - 1) // n_blocks}:
                b = f(lay, n_blocks, n_rows, max_rows)
                assert b <= limit(n_q, n_kv, D, window, n_blocks, n_rows, max_rows), (n_rows, n_blocks, max_rows)
                sized += b > 0
    assert sized >= 50                                  # (the rest are refused: too many tiles)


def test_workspace_of_long_passes(m):
    """Two million rows without a window (the limit was once stated as 1 GB and
    the sums): the tiles alone take 3.8 GiB; with a window they stay at 1 GiB."""
    n = 2_000_000
    rest = 8 * n * 512 + n * (4 * 16 + 104) + 4 * MIB
    f = m.attn_train_backward_workspace_bytes
    b = f(m.layer(16, 1, 512, 0, 0, 1e4), 1, n, n)
    assert 3.8 * (1 << 30) <= b - 8 * n * 512 and b <= 2048 * n + rest
    assert f(m.layer(16, 1, 512, 1024, 0, 1e4), 1, n, n) <= (1 << 30) + rest


@pytest.mark.parametrize("ratio", [3, 12, 17, 32, 64, 128])
def test_ratios_a_layer_or_a_tile_does_not_take(m, ratio):
    """q heads per kv head: 1, 2, 4, 8 or 16."""
    import ctypes
    lay = m.layer(ratio, 1, 256, 0, 0, 1e4)
    p = 1 << 20                                                       # a fake address: never dereferenced
    read = (1, p, 4, 4, p, p, p, p, 1, p, p, p, p, p, 0, 0, p, 1 << 40, None)
    assert m.lib.attn_train_backward(ctypes.byref(lay), *read) == 2
    assert m.attn_train_backward_workspace_bytes(lay, 1, 4, 4) == 0
    if ratio > 16:
        prep = (1, p, 4) + (p,) * 5 + (None,) * 5 + (0,) + (None,) * 3 + (p, 1 << 40, None)
        assert m.lib.kvq_train_prep_backward(ctypes.byref(lay), *prep) == 2
        assert m.kvq_train_prep_backward_workspace_bytes(lay, 4) == 0
