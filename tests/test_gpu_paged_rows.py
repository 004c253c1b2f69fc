"""The paged reads row by row: table entries that name no page whatever number they hold, value scales of 0 beside
small ones, and rows that are NaN only where they themselves see a position without a page."""
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
