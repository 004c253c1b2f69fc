"""Calls of the paged cache that a program may make and a single read does not show: batches padded behind their last
sequence, more groups than a block plans by itself, many short sequences beside long ones, outputs on element
boundaries, steps issued one behind the other without a synchronization, and prompt rows in captured graphs."""
import numpy as np
import pytest

import oracle as O
from paged_ref import F32
from test_gpu_paged import GUARD, Read, append_rows, ask, bf16, check, dev, filled, lay, m, offsets, spec  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("last", ["reads", "idle", "past the table"])
@pytest.mark.parametrize("rows", [3, 90])
def test_rows_behind_the_last_sequence(m, rows, last):
    """n_rows above row_offsets[n_seqs]: those rows' outputs stay as they were, whatever the last sequence is."""
    layer = spec(8, 2, 128)
    gpu, tables, g = filled(m, layer, 32, "i8", [70, 300], 5)
    start = [50, {"reads": 300 - rows, "idle": -1, "past the table": 32 * tables.shape[1] - 1}[last]]
    off, behind = offsets([2, rows]), 11
    end = int(off[-1])
    q, w = ask(g, layer, end + behind, 3.0)
    r = Read(m, layer, gpu, tables, start, [2, rows], q, w, True, off, max_pos=32 * tables.shape[1] - 1)
    got = r.run()
    assert (got[end:] == 77).all() and not r.prepped()[end:].any()
    check(layer, gpu, tables, q, w, got, [(0, 0, 50), (1, 0, 51)], True, r.prepped())
    if last == "reads":
        check(layer, gpu, tables, q, w, got, [(2, 1, 300 - rows), (end - 1, 1, 299)], True, r.prepped())
    elif last == "idle":
        assert not got[2:end].any()
    else:
        assert np.isnan(got[3:end]).all()
    # the write and the read-back
    k, v, wk = bf16(g, (end + behind, 2, 128)), bf16(g, (end + behind, 2, 128)), bf16(g, 128, 1.0, 0.1)
    before = {c: gpu.codes[c].clone() for c in "kv"}
    idle = dev(np.int32([-1, -1]))
    pre = torch.full((2, end + behind, 2, 128), 77, dtype=torch.int16, device="cuda")
    args = (dev(tables), tables.shape[1], 2, dev(off))
    m.kvq_paged_append(lay(m, layer), gpu.cache, *args, idle, end + behind, dev(k), dev(v), dev(wk), pre)
    out = [torch.full((end + behind, 2, 128), 77, dtype=torch.int16, device="cuda") for _ in range(2)]
    m.kvq_paged_gather(gpu.cache, *args, dev(np.int32([50, 0])), end + behind, out[0], out[1])
    torch.cuda.synchronize()
    assert bool((pre == 77).all()) and all(torch.equal(before[c], gpu.codes[c]) for c in "kv")
    for c, o in zip("kv", out):
        assert bool((o[end:] == 77).all())
        want = np.stack([gpu.p.values(c, tables[1], h, np.arange(rows)) for h in range(2)], 1)
        assert np.array_equal(O.bf16_to_f64(o[2:end].cpu().numpy().view(np.uint16)),
                              O.rn_bf16(want.astype(F32).astype(np.float64)))


def test_more_groups_than_a_block_plans(m):
    """1100 sequences: decode and windows of two rows."""
    layer = spec(4, 2, 64)
    g0 = np.random.default_rng(2)
    lens = [int(x) for x in g0.integers(2, 40, 1100)]
    lens[3], lens[700], lens[1099] = 700, 300, 65
    gpu, tables, g = filled(m, layer, 16, "i8", lens, 9)
    pos = [n - 1 for n in lens]
    pos[10] = -1
    q, w = ask(g, layer, 1100, 3.0)
    r = Read(m, layer, gpu, tables, pos, [1] * 1100, q, w)
    got = r.run()
    assert r.status() == 0 and not got[10].any()
    some = [0, 3, 9, 11, 511, 699, 700, 701, 1022, 1023, 1024, 1025, 1098, 1099]
    check(layer, gpu, tables, q, w, got, [(s, s, pos[s]) for s in some], True)
    q, w = ask(g, layer, 2200, 3.0)
    start = [n - 2 for n in lens]
    r = Read(m, layer, gpu, tables, start, [2] * 1100, q, w, True, offsets([2] * 1100))
    got = r.run()
    assert r.status() == 0
    check(layer, gpu, tables, q, w, got, [(2 * s + t, s, start[s] + t) for s in some for t in (0, 1)], True)


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 2, 1), (128, 8, 2), (256, 4, 1), (512, 4, 1)])
def test_short_sequences_beside_long_ones(m, D, n_q, n_kv):
    """Shares of the keys that hold many units, and that begin and end anywhere in them."""
    layer = spec(n_q, n_kv, D)
    lens = [1 + i % 7 for i in range(150)]
    lens[20], lens[21], lens[149] = 3000, 130, 900
    gpu, tables, g = filled(m, layer, 64, "i8", lens, D + 1)
    pos = [n - 1 for n in lens]
    q, w = ask(g, layer, 150, 3.0)
    r = Read(m, layer, gpu, tables, pos, [1] * 150, q, w)
    got = r.run()
    assert r.status() == 0
    check(layer, gpu, tables, q, w, got, [(s, s, p) for s, p in enumerate(pos)], True)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("D,rows", [(128, 5), (128, 150), (256, 150)])
def test_outputs_on_element_boundaries(m, D, rows, f32):
    layer = spec(8, 2, D)
    gpu, tables, g = filled(m, layer, 32, "e4m3", [400], D)
    q, w = ask(g, layer, rows, 3.0)
    for offs in (offsets([rows]), None):
        n = rows if offs is not None else 1
        r = Read(m, layer, gpu, tables, [400 - n], [n], q[:n], w, f32, offs)
        r.run()
        want, qp = r.full.clone(), r.qp.clone()
        r.full, r.qp = (torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")[1:] for t in (r.full, r.qp))
        r.full.fill_(77)
        r.call()                                          # (the call takes the tensors that the object holds)
        torch.cuda.synchronize()
        assert torch.equal(r.full, want) and torch.equal(r.qp, qp)


@pytest.mark.parametrize("D", [64, 128, 512])
def test_steps_behind_one_another(m, D):
    """Append and read of 40 steps, their positions moved on by the stream, with and without a wait after each call."""
    layer = spec(4, 1, D)
    lens, steps = [100, 1, 900], 40
    outs = []
    for wait in (True, False):
        gpu, tables, g = filled(m, layer, 16, "i8", lens, 4, spare=9, max_pages=60)
        free = [p for p in range(gpu.p.n_pages) if p not in set(tables[tables >= 0])]
        assert len(free) >= 9
        for s, n in enumerate(lens):                      # room for the steps
            for i in range(-(-n // 16), -(-(n + steps) // 16)):
                tables[s, i] = free.pop()
        raw = [bf16(g, (3 * steps, 1, D)) for _ in "kv"]
        k, v = (dev(x) for x in raw)
        q, w = ask(g, layer, 3, 3.0)
        off, wk = dev(offsets([1, 1, 1])), dev(bf16(g, D, 1.0, 0.1))
        r = Read(m, layer, gpu, tables, lens, [1, 1, 1], q, w, max_pos=959)
        got = []
        for i in range(steps):
            m.kvq_paged_append(lay(m, layer), gpu.cache, r.keep[0], tables.shape[1], 3, off, r.keep[1], 3,
                               k[3 * i:3 * i + 3], v[3 * i:3 * i + 3], wk, None)
            if wait:
                torch.cuda.synchronize()
            r.call()
            if wait:
                torch.cuda.synchronize()
            got.append(r.full[:-GUARD].clone())
            r.keep[1].add_(1)
        torch.cuda.synchronize()
        outs.append(torch.stack(got))
    assert bool(outs[0].isfinite().all()) and torch.equal(outs[0], outs[1])


def test_prompt_rows_in_a_graph(m):
    """Two reads of prompt rows on two streams of one capture, each with its workspace, replayed with other rows."""
    layer = spec(8, 2, 128)
    gpu, tables, g = filled(m, layer, 32, "e4m3", [300, 260], 3)
    off = offsets([200, 60])
    q, w = ask(g, layer, 260, 3.0)
    a, b = (Read(m, layer, gpu, tables, [100, 200], [200, 60], q, w, True, off) for _ in range(2))
    a.run()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        a.call()
        with torch.cuda.stream(side):
            b.call()
        torch.cuda.current_stream().wait_stream(side)
    new = [ask(g, layer, 260, 3.0)[0] for _ in range(2)]
    starts = [[37, -1], [0, 200]]
    for r, x, s in zip((a, b), new, starts):
        r.keep[2].copy_(dev(x))
        r.keep[1].copy_(dev(np.int32(s)))
        r.full.fill_(77)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for r, x, s in zip((a, b), new, starts):
        got = r.full[:-GUARD].cpu().numpy().astype(np.float64).reshape(r.shape)
        check(layer, gpu, tables, x, w, got, [(t, 0, s[0] + t) for t in (0, 64, 199)], True)
        if s[1] < 0:
            assert not got[200:].any()
        else:
            check(layer, gpu, tables, x, w, got, [(200, 1, 200), (259, 1, 259)], True)
