"""attn_train_backward on passes that are long beside their window, on
windows whose reach ends at a block's, a tile's or the prefix's edge, and on
passes whose P and dS tiles take more than one chunk of the workspace."""
import numpy as np
import pytest

import oracle as O
from test_gpu_train_backward import ReadCase, dense_gradient, offsets, spec

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


@pytest.mark.parametrize("n_q,n_kv,D,window,blocks,tiles,f32_sums", [
    (16, 1, 512, 0, [3000, 1500, 1, 2100], 18000, True),         # two output halves, operands not kept in shared memory
    (16, 1, 512, 0, [6600], 18000, False),
    (16, 16, 128, 0, [6000], 18000, True),
    (16, 2, 128, 2500, [2000, 3000, 40, 2900], 17000, False),
])
def test_several_chunks_at_128_and_512(m, n_q, n_kv, D, window, blocks, tiles, f32_sums):
    """More tiles than a chunk's 16384 (counted here by the mask: `tiles` at
    least): sums over chunks, added to what was there; against the definition
    in 64 bits (2-norms: P or dS and the output rounded to bf16, 5e-3)."""
    gen = torch.Generator(device="cuda").manual_seed(51)
    T = sum(blocks)
    off = np.concatenate([[0], np.cumsum(blocks)])
    see = torch.from_numpy(O.train_mask(off, window)).cuda()
    per, count = 128 * n_kv // n_q, 0                    # rows of a tile; tiles do not span blocks
    for b0, b1 in zip(off[:-1], off[1:]):
        for r in range(b0, b1, per):
            row = see[r:min(r + per, b1)].any(0)
            for keys in ([row[:off[1]]] if b0 == 0 else [row[:off[1]], row[b0:b1]]):
                count += int(torch.nn.functional.pad(keys, (0, -len(keys) % 128)).view(-1, 128).any(1).sum())
    assert count * n_kv > tiles

    def rows(heads, scale):
        return (torch.randn(T, heads, D, generator=gen, device="cuda") * scale).bfloat16()

    q, k, v, do = rows(n_q, 0.15), rows(n_kv, 1.0), rows(n_kv, 1.0), rows(n_q, 0.01)
    dq, dk, dv, out, lse = dense_gradient(*(x.double() for x in (q, k, v, do)), see)
    lay = m.layer(n_q, n_kv, D, window, 0, 1e4)
    ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), T, max(blocks))
    assert ws_bytes > (1 << 30)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    kind = torch.float32 if f32_sums else torch.bfloat16
    start = torch.randn(2, T, n_kv, D, generator=gen, device="cuda").to(kind)
    got = [torch.empty_like(q), start[0].clone(), start[1].clone()]
    m.attn_train_backward(lay, len(blocks), offsets(blocks), T, max(blocks), q, k, v, out.float(), 1, lse.float(), do,
                          *got, f32_sums, f32_sums, ws, ws_bytes)
    torch.cuda.synchronize()
    assert int(ws[:4].cpu().numpy().view(np.uint32)[0]) == 0
    for name, x, w, s in zip(("dq", "dk", "dv"), got, (dq, dk, dv), (None, start[0], start[1])):
        added = f32_sums and s is not None
        x = x.double() - (s.double() if added else 0.0)
        # (the fp32 addition to `start`, of size 1, rounds by 2^-24 of it)
        room = 5e-3 * w.norm() + (2.0 ** -24 * s.double().norm() if added else 0.0)
        assert (x - w).norm() <= room, (name, float((x - w).norm() / w.norm()))
