"""Workspaces of the paged reads: a call that asks for less fits the workspace of one that asks for more, and what
pieces of the keys take is bounded by the GPU, not by the call."""
import numpy as np
import pytest

from test_abi_paged import cache, layer, m  # noqa: F401

# n_q, n_kv, D, window
SHAPES = [(8, 2, 256, 0), (8, 2, 256, 512), (32, 8, 128, 0), (4, 4, 64, 0), (16, 1, 512, 0), (6, 2, 128, 100),
          (14, 2, 512, 0)]


def need(m, shape, n_seqs, n_rows, most, max_pos):
    n_q, n_kv, D, W = shape
    return m.attn_paged_prefill_workspace_bytes(layer(m, n_q_heads=n_q, n_kv_heads=n_kv, head_dim=D, window=W,
                                                      rope_dims=D),
                                                cache(m, n_kv=n_kv, D=D), n_seqs, n_rows, most, max_pos)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_smaller_call_fits(m, shape):
    """Each of the four sizes falls alone, then all of them together."""
    g = np.random.default_rng(shape[2])
    for _ in range(300):
        n_rows = int(2 ** g.uniform(0, 16))
        n_seqs = int(min(2 ** g.uniform(0, 10), 4 * n_rows))
        most, max_pos = int(g.integers(1, n_rows + 1)), int(2 ** g.uniform(0, 23))
        whole = need(m, shape, n_seqs, n_rows, most, max_pos)
        assert whole > 0
        fewer = [int(g.integers(1, x + 1)) for x in (n_seqs, n_rows, most, max_pos)]
        for at in range(4):
            one = [n_seqs, n_rows, most, max_pos]
            one[at] = fewer[at]
            assert need(m, shape, *one) <= whole, (one, (n_seqs, n_rows, most, max_pos))
        assert need(m, shape, *fewer) <= whole


def test_the_rest_of_a_chunked_prompt_fits(m):
    """Chunks of 500 rows and what is left, one workspace."""
    whole = need(m, SHAPES[0], 1, 500, 500, 16383)
    assert all(need(m, SHAPES[0], 1, rows, rows, 16383) <= whole for rows in range(1, 501))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("n_seqs,n_rows", [(1, 64), (16, 64), (16, 256), (64, 64), (256, 300), (1000, 8000)])
def test_pieces_are_bounded(m, shape, n_seqs, n_rows):
    """Rows' own data (q as f16, a place per group of rows, at most two groups a row and sequence) and at most 64 MB
    of pieces: 2 of 16 rows a CTA of the row kernel, 256 KB a pair of CTAs of the prompt kernel."""
    n_q, n_kv, D, W = shape
    rows = n_rows * n_q * D * 2 + 16 * (n_rows + n_seqs)
    assert need(m, shape, n_seqs, n_rows, -(-n_rows // n_seqs), 100000) <= rows + (64 << 20)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_smaller_decode_fits(m, shape):
    n_q, n_kv, D, W = shape
    lay, c = layer(m, n_q_heads=n_q, n_kv_heads=n_kv, head_dim=D, window=W, rope_dims=D), cache(m, n_kv=n_kv, D=D)
    sizes = [(n, p) for n in (1, 2, 3, 7, 16, 64, 300, 5000) for p in (0, 1, 63, 64, 500, 511, 512, 4095, 100000)]
    got = {x: m.attn_paged_decode_workspace_bytes(lay, c, *x) for x in sizes}
    assert all(got[a] <= got[b] for a in sizes for b in sizes if a[0] <= b[0] and a[1] <= b[1])


@pytest.mark.parametrize("shape", SHAPES)
def test_rows_of_a_sequence_without_a_bound(m, shape):
    """max_rows_per_seq may be far above the rows of the call."""
    want = need(m, shape, 3, 500, 500, 9000)
    for most in (1 << 20, 1 << 28, 1 << 29, 1 << 30, (1 << 31) - 1):
        assert need(m, shape, 3, 500, most, 9000) == want
