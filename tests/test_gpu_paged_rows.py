"""The paged reads row by row: table entries that name no page whatever number they hold, value scales of 0 beside
small ones, rows that are NaN only where they themselves see a position without a page, and chunks cut along their keys."""
import numpy as np
import pytest

from paged_ref import F32
from test_gpu_paged import GUARD, Gpu, Read, ask, bf16, check, dev, filled, lay, m, offsets, spec  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-2, -1, -2 ** 31, 2 ** 31 - 1, "n_pages"])
@pytest.mark.parametrize("rows", [1, 3, 100])
@pytest.mark.parametrize("D,kind", [(64, "e4m3"), (128, "i8"), (256, "e4m3"), (512, "i8")])
def test_no_number_outside_the_pool_is_a_page(m, D, kind, rows, entry):
    layer = spec(4, 1, D)
    gpu, tables, g = filled(m, layer, 16, kind, [300, 300], D)
    q, w = ask(g, layer, 2 * rows, 3.0)
    start = [300 - rows] * 2
    off = offsets([rows] * 2) if rows > 1 else None
    good = Read(m, layer, gpu, tables, start, [rows] * 2, q, w, True, off)
    want = good.run()
    assert good.status() == 0
    bad = tables.copy()
    bad[0, 5] = gpu.p.n_pages if entry == "n_pages" else entry
    r = Read(m, layer, gpu, bad, start, [rows] * 2, q, w, True, off)
    got = r.run()
    assert r.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert np.isnan(got[:rows]).all() and np.array_equal(got[rows:], want[rows:])


@pytest.mark.parametrize("sharp", [2.0, 6.0])
@pytest.mark.parametrize("rows", [1, 4, 150])
@pytest.mark.parametrize("D,kind", [(64, "i8"), (128, "e4m3"), (256, "i8"), (512, "e4m3")])
def test_zero_scales_beside_the_smallest(m, D, kind, rows, sharp):
    """Value scales 0, 2^-40 and 2^-33: a page of zeros takes its weight and leaves the others' values their bits."""
    layer = spec(16, 4, D, rope_dims=0)
    gpu, tables, g = filled(m, layer, 16, kind, [300], 78)
    for i, page in enumerate(tables[0]):
        gpu.p.scales["v"][page] = [0.0, 2.0 ** -40, 2.0 ** -33][i % 3]
    gpu = Gpu(m, gpu.p)                                        # (the codes of the zero pages stay: their rows read as zeros)
    q, w = ask(g, layer, rows, sharp)
    r = Read(m, layer, gpu, tables, [300 - rows], [rows], q, w, True, offsets([rows]) if rows > 1 else None)
    got = r.run()
    assert r.status() == 0
    check(layer, gpu, tables, q, w, got, [(t, 0, 300 - rows + t) for t in range(0, rows, 7)], True)


@pytest.mark.parametrize("rows", [1, 60])
@pytest.mark.parametrize("D,kind", [(64, "i8"), (128, "e4m3"), (256, "i8"), (512, "e4m3")])
def test_scales_of_zero_read_as_zeros(m, D, kind, rows):
    """Whatever the codes: keys of scale 0 score 0, values of scale 0 add nothing, and with nothing else the output is 0."""
    layer = spec(4, 1, D, rope_dims=0)
    gpu, tables, g = filled(m, layer, 16, kind, [200, 90], 79)
    gpu.p.scales["k"][tables[0][::2]] = 0.0
    gpu.p.scales["v"][tables[0][1::3]] = 0.0
    gpu.p.scales["v"][tables[1][:6]] = 0.0
    gpu = Gpu(m, gpu.p)
    q, w = ask(g, layer, 2 * rows, 2.0)
    r = Read(m, layer, gpu, tables, [200 - rows, 90 - rows], [rows] * 2, q, w, True,
             offsets([rows] * 2) if rows > 1 else None)
    got = r.run()
    assert r.status() == 0 and not got[rows:].any()
    check(layer, gpu, tables, q, w, got, [(t, 0, 200 - rows + t) for t in range(0, rows, 7)], True)


# n_q, n_kv, D, window, first position, rows, places of the table that name no page (of 16 positions), codes
MISSING = [(8, 2, 128, 0, 200, 40, [14], "i8"), (8, 2, 128, 20, 200, 40, [12], "e4m3"), (8, 2, 128, 8, 200, 64, [12, 15], "i8"),
           (4, 1, 64, 0, 0, 300, [9, 11], "e4m3"), (4, 4, 64, 33, 100, 200, [6, 13], "i8"),
           (8, 2, 256, 0, 100, 120, [12], "i8"), (8, 2, 256, 50, 90, 150, [5, 13], "e4m3"),
           (16, 1, 512, 0, 60, 70, [7], "i8"), (16, 1, 512, 30, 60, 70, [4], "e4m3"),
           (8, 2, 128, 0, 5000, 100, [316], "i8"), (8, 2, 256, 0, 4990, 100, [317], "e4m3"), (4, 4, 128, 0, 0, 400, [20], "i8"),
           # windows of few rows, and ratios that take 16 rows at a time
           (8, 2, 128, 0, 220, 6, [14], "i8"), (4, 1, 64, 9, 230, 8, [13], "e4m3"), (8, 2, 256, 10, 230, 8, [13], "i8"),
           (16, 1, 512, 0, 223, 2, [14], "i8"), (6, 2, 128, 0, 200, 40, [14], "e4m3"), (6, 2, 256, 20, 200, 40, [12], "i8"),
           (8, 2, 128, 0, 4990, 8, [312], "e4m3")]


@pytest.mark.parametrize("n_q,n_kv,D,window,start,rows,places,kind", MISSING)
def test_only_rows_that_see_a_missing_page(m, n_q, n_kv, D, window, start, rows, places, kind):
    """A chunk or window with pages missing among its keys: the rows before them (or, under a window, past them) are as
    with all pages, bit for bit."""
    layer = spec(n_q, n_kv, D, window)
    gpu, tables, g = filled(m, layer, 16, kind, [start + rows], D + rows, fill=0x7F)
    p, spare = gpu.p, min(set(range(gpu.p.n_pages)) - set(tables[0]))
    for x in (p.codes["k"], p.codes["v"], p.scales["k"], p.scales["v"]):
        x[[0, spare]] = x[[spare, 0]]                          # (page 0 holds bytes that read as NaN)
    tables[tables == 0] = spare
    gpu = Gpu(m, p)
    q, w = ask(g, layer, rows, 3.0)
    off = offsets([rows])
    want = Read(m, layer, gpu, tables, [start], [rows], q, w, True, off).run()
    bad = tables.copy()
    bad[0, places] = [-1, gpu.p.n_pages][:len(places)]
    r = Read(m, layer, gpu, bad, [start], [rows], q, w, True, off)
    got = r.run()
    pos = start + np.arange(rows)
    first = np.maximum(0, pos - window + 1) if window else np.zeros_like(pos)
    sees = np.zeros(rows, bool)
    for i in places:
        sees |= (first <= 16 * i + 15) & (pos >= 16 * i)
    assert sees.any() and not sees.all() and r.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert np.isnan(got[sees]).all()
    assert np.array_equal(got[~sees], want[~sees])
    check(layer, gpu, tables, q, w, got, [(int(t), 0, int(pos[t])) for t in np.flatnonzero(~sees)[::9]], True)


@pytest.mark.parametrize("n_q,n_kv,D,kind,copies", [(8, 2, 256, "i8", 1), (8, 2, 256, "e4m3", 5), (16, 1, 512, "i8", 2),
                                                    (16, 4, 128, "e4m3", 2), (4, 1, 64, "i8", 9)])
def test_short_chunks_cut_along_their_keys(m, n_q, n_kv, D, kind, copies):
    """Chunks of few rows behind keys from one tile to dozens: pieces whose places lie one behind the other, more than
    there are places for (5 and 9 copies) or fewer."""
    layer = spec(n_q, n_kv, D)
    lens = [40, 2600, 90, 1500, 130, 700, 300, 200] * copies
    rows = [10, 33, 9, 12, 11, 10, 17, 10] * copies
    gpu, tables, g = filled(m, layer, 64, kind, lens, D + copies)
    start, off = [n - r for n, r in zip(lens, rows)], offsets(rows)
    q, w = ask(g, layer, int(off[-1]), 3.0)
    r = Read(m, layer, gpu, tables, start, rows, q, w, True, off)
    got = r.run()
    assert r.status() == 0 and np.array_equal(got, r.run())
    at = [(int(off[s]) + t, s, start[s] + t) for s in range(len(lens)) for t in (0, rows[s] - 1)]
    check(layer, gpu, tables, q, w, got, at if copies < 3 else at[::3], True)


def test_one_workspace_for_a_chunked_prompt(m):
    """Chunks of 500 rows and the rest, all in the workspace of the first."""
    layer = spec(8, 2, 256)
    total, most = 1064, 500
    gpu, tables, g = filled(m, layer, 64, "i8", [total], 6)
    q, w = ask(g, layer, total, 3.0)
    L, dq, dw, t = lay(m, layer), dev(q), dev(w), dev(tables)
    need = m.attn_paged_prefill_workspace_bytes(L, gpu.cache, 1, most, most, total - 1)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    out = torch.empty((total, 8, 256), dtype=torch.float32, device="cuda")
    for at in range(0, total, most):
        n = min(most, total - at)
        m.attn_paged_prefill(L, gpu.cache, t, tables.shape[1], 1, dev(offsets([n])), dev(np.int32([at])), n, n,
                             total - 1, dq[at:at + n], dw, out[at:at + n], True, None, ws, need)
        torch.cuda.synchronize()
        assert int(ws[:4].cpu().numpy().view(np.uint32)[0]) == 0
    check(layer, gpu, tables, q, w, out.cpu().numpy().astype(np.float64),
          [(p, 0, p) for p in (0, 1, 499, 500, 777, 999, 1000, 1063)], True)
