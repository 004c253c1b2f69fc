"""attn_train_backward on passes that are long beside their window, and on
windows whose reach ends at a block's, a tile's or the prefix's edge."""
import numpy as np
import pytest

import workloads as W
from test_gpu_train_backward import ReadCase, offsets, spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


@pytest.mark.parametrize("window", [1, 2, 57, 58, 63, 64, 72, 73, 74, 127, 128, 129, 200, 201, 256, 257])
@pytest.mark.parametrize("D,n_q,n_kv", [(64, 16, 1), (128, 2, 1)])
def test_windows_that_end_at_edges(m, window, D, n_q, n_kv):
    """Prefix tiles whose last key is or is not seen by a branch's first row
    (the prefix's second tile holds 72 keys: windows 72 to 74, and its first
    from 73 on), branches of one and two tiles, an empty one, one of one row."""
    c = ReadCase(m, spec(n_q, n_kv, D, window), [200, 130, 0, 1, 257])
    c.run()
    c.verify(norm=False)


def read_time(m, n_q, n_kv, D, window, blocks):
    """Least of five event times (ms) of one call."""
    T = sum(blocks)
    gen = torch.Generator(device="cuda").manual_seed(41)

    def rows(heads, scale):
        return torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=gen)

    q, out, do = rows(n_q, 0.2), rows(n_q, 0.5), rows(n_q, 0.01)
    k, v = rows(n_kv, 0.2), rows(n_kv, 1.0)
    lse = torch.full((T, n_q), 8.0, device="cuda")        # (any finite statistics will do)
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    lay, offs = m.layer(n_q, n_kv, D, window, 0, 1e4), offsets(blocks)
    ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), T, max(blocks))
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    times = []
    for _ in range(6):
        start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        start.record()
        m.attn_train_backward(lay, len(blocks), offs, T, max(blocks), q, k, v, out, 0, lse, do, dq, dk, dv, 0, 0, ws,
                              ws_bytes)
        stop.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(stop))
    assert int(ws[:4].cpu().numpy().view(np.uint32)[0]) == 0
    return min(times[1:])


@pytest.mark.parametrize("n_q,n_kv,D,window,blocks", [
    (16, 1, 64, 16, [16384]),
    (8, 2, 256, 512, [32768]),
])
def test_windowed_time_grows_with_the_rows(m, n_q, n_kv, D, window, blocks):
    """A window leaves each row the same work however long the pass is: sixteen
    times the rows take sixteen times the time, not more than 1.5 times that
    (they took 3.6 and 1.9 times that when every key tile's list was looked for
    among all the rows after it)."""
    short = read_time(m, n_q, n_kv, D, window, blocks)
    long = read_time(m, n_q, n_kv, D, window, [16 * b for b in blocks])
    assert long <= 1.5 * 16 * short, (short, long, long / (16 * short))
