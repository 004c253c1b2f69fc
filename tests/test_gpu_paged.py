"""The paged 8-bit cache on the GPU: appended codes and scales bit for bit,
attention over pages within the bounds its roundings leave, against a numpy
cache in 64 bits; idle sequences, windows, tables that name no page, slots that
hold bytes no read may use, other streams and captured graphs."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from paged_ref import F32, Pages, attend, bound, prep

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 256


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def spec(n_q, n_kv, D, window=0, rope_dims=None, theta=1e4, k_eq_v=False):
    return W.LayerSpec(n_q, n_kv, D, window, D if rope_dims is None else rope_dims, theta, k_eq_v)


def lay(m, s):
    return m.layer(s.n_q_heads, s.n_kv_heads, s.head_dim, s.window, s.rope_dims, s.rope_theta, s.rms_eps, s.k_eq_v)


def bf16(g, shape, loc=0.0, scale=1.0):
    return W.bf16_bits_from_f32((loc + scale * g.standard_normal(shape)).astype(F32))


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a.copy()).cuda()


class Gpu:
    """A numpy cache's pages on the GPU."""

    def __init__(self, m, pages):
        self.p = pages
        self.codes = {c: dev(pages.codes[c]) for c in "kv"}
        self.scales = {c: dev(pages.scales[c]) for c in "kv"}
        self.cache = m.paged_cache(self.codes["k"], self.codes["v"], self.scales["k"], self.scales["v"], pages.n_pages,
                                   pages.P, pages.n_kv, pages.D, m.KVQ_CODE_E4M3 if pages.kind == "e4m3" else
                                   m.KVQ_CODE_I8)

    def same(self):
        for c in "kv":
            assert np.array_equal(self.scales[c].cpu().numpy(), self.p.scales[c], equal_nan=True), c
            got = self.codes[c].cpu().numpy()
            assert np.array_equal(got, self.p.codes[c]), (c, np.argwhere(got != self.p.codes[c])[:4])


def tables_for(lens, P, n_pages, seed, max_pages=None):
    """Scattered pages for sequences of these lengths."""
    order = list(np.random.default_rng(seed).permutation(n_pages))
    need = [-(-n // P) for n in lens]
    t = np.full((len(lens), max_pages or max(1, max(need))), -1, np.int32)
    for s, n in enumerate(need):
        for i in range(n):
            t[s, i] = order.pop()
    return t


def offsets(rows):
    return np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)


def append_rows(m, layer, gpu, tables, start, rows, g, scale=1.0, prepped=True, only=None):
    """Appends rows on the GPU and in numpy; returns nothing, the caller compares."""
    n, n_kv, D = int(sum(rows)), layer.n_kv_heads, layer.head_dim
    k = bf16(g, (n, n_kv, D))
    v = None if layer.k_eq_v else bf16(g, (n, n_kv, D))
    w = bf16(g, D, 1.0, 0.1 * scale)
    off = offsets(rows)
    dk, dv = dev(k), dev(v) if v is not None else None
    out = torch.full((2 * n * n_kv * D + GUARD,), 77, dtype=torch.int16, device="cuda") if prepped else None
    m.kvq_paged_append(lay(m, layer), gpu.cache, dev(tables), tables.shape[1], len(rows), dev(off),
                       dev(np.int32(start)), n, dk, dv, dev(w), out)
    torch.cuda.synchronize()
    for s, r in enumerate(rows):
        if r and start[s] >= 0 and (only is None or s in only):
            pos = np.arange(start[s], start[s] + r)
            kh = prep(k[off[s]:off[s + 1]], w, pos, layer)
            vh = prep((k if v is None else v)[off[s]:off[s + 1]], None, pos, layer)
            gpu.p.append(tables[s], start[s], kh, vh)
            if prepped:
                got = out[:-GUARD].view(2, n, n_kv, D)[:, off[s]:off[s + 1]].cpu().numpy().view(np.uint16)
                assert np.array_equal(got[0], O.f64_to_bf16(kh)) and np.array_equal(got[1], O.f64_to_bf16(vh))
    if prepped:
        assert bool((out[-GUARD:] == 77).all())


# D, n_kv, rope dims, K = V, page tokens, codes
SHAPES = [(64, 2, 64, False, 16, "i8"), (64, 5, 24, False, 128, "e4m3"), (128, 8, 128, False, 32, "e4m3"),
          (128, 1, 0, True, 64, "i8"), (256, 2, 256, False, 64, "i8"), (256, 3, 64, True, 16, "e4m3"),
          (512, 1, 128, True, 64, "i8"), (512, 2, 512, False, 128, "e4m3"), (64, 17, 64, False, 32, "i8")]


@pytest.mark.parametrize("D,n_kv,rope,kv,P,kind", SHAPES)
def test_append_bit_for_bit(m, D, n_kv, rope, kv, P, kind):
    """Chunks of prompts and single rows, into begun and new pages, so that scales grow and old rows move."""
    g = np.random.default_rng(D + n_kv)
    layer = spec(n_kv, n_kv, D, rope_dims=rope, k_eq_v=kv)
    n_pages = 40
    gpu = Gpu(m, Pages(n_pages, n_kv, P, D, kind, seed=3))
    end = [3 * P, P + 1, 1, 2 * P + 5]
    tables = tables_for(end, P, n_pages, 4, max_pages=5)
    lens = [0, 0, 0, 0]
    for rows in ([P + 3, 1, 0, 5], [1, 1, 1, 1], [1, P - 1, 0, P], [P + 1, 0, 0, 0], [1, 0, 0, P - 1]):
        append_rows(m, layer, gpu, tables, lens, rows, g)
        lens = [a + b for a, b in zip(lens, rows)]
        gpu.same()


def test_append_of_one_row_a_page_at_a_time(m):
    """Each new row larger than the last: the scale grows every time."""
    layer = spec(1, 1, 64)
    for kind in ("i8", "e4m3"):
        gpu = Gpu(m, Pages(4, 1, 16, 64, kind, seed=9))
        tables = np.int32([[2, 0]])
        for p in range(18):
            x = np.zeros((1, 1, 64))
            x[0, 0, :2 + 60 * (p % 2)] = 1.0                    # peaked rows have larger entries once normed
            k = W.bf16_bits_from_f32((x * (p + 1)).astype(F32))
            w = W.bf16_bits_from_f32(np.full(64, 0.5 + 0.25 * p, F32))
            m.kvq_paged_append(lay(m, layer), gpu.cache, dev(tables), 2, 1, dev(offsets([1])), dev(np.int32([p])), 1,
                               dev(k), dev(k), dev(w))
            gpu.p.append(tables[0], p, prep(k, w, [p], layer), prep(k, None, [p], layer))
        torch.cuda.synchronize()
        gpu.same()


def test_append_zero_and_tiny_rows(m):
    """A page of zeros has scale 0; rows below the smallest scale read as zeros, and later rows find both."""
    layer = spec(1, 1, 64, rope_dims=0)
    gpu = Gpu(m, Pages(4, 1, 16, 64, "i8", seed=2))
    tables = np.int32([[1], [3]])
    for step, rows in enumerate((np.zeros((2, 64)), np.full((2, 64), 2.0 ** -60), np.ones((2, 64)))):
        k = W.bf16_bits_from_f32(rows[:, None].astype(F32))
        w = W.bf16_bits_from_f32(np.ones(64, F32))
        m.kvq_paged_append(lay(m, layer), gpu.cache, dev(tables), 1, 2, dev(offsets([1, 1])), dev(np.int32([step] * 2)),
                           2, dev(k), dev(k), dev(w))
        for s in range(2):
            gpu.p.append(tables[s], step, prep(k[s:s + 1], w, [step], layer), prep(k[s:s + 1], None, [step], layer))
    torch.cuda.synchronize()
    gpu.same()


def test_append_passes_over_what_has_no_page(m):
    """Idle sequences, rows past the table and pages it does not name: nothing is written for them."""
    g = np.random.default_rng(5)
    layer = spec(2, 2, 64)
    gpu = Gpu(m, Pages(8, 2, 16, 64, "i8", seed=6))
    tables = np.int32([[0, 1], [2, 3], [-1, 4], [8, 5], [6, 7]])
    rows, start = [3, 4, 10, 5, 5], [0, -1, 14, 2, 30]
    k, v, w = bf16(g, (27, 2, 64)), bf16(g, (27, 2, 64)), bf16(g, 64, 1.0, 0.1)
    m.kvq_paged_append(lay(m, layer), gpu.cache, dev(tables), 2, 5, dev(offsets(rows)), dev(np.int32(start)), 27,
                       dev(k), dev(v), dev(w))
    torch.cuda.synchronize()
    off = offsets(rows)

    def put(s, first, last):                                   # positions first .. last - 1 of sequence s
        i = off[s] + first - start[s]
        at = slice(i, i + last - first)
        pos = np.arange(first, last)
        gpu.p.append(tables[s], first, prep(k[at], w, pos, layer), prep(v[at], None, pos, layer))

    put(0, 0, 3)
    put(2, 16, 24)                                             # its first page is none
    put(4, 30, 32)                                             # the rest is past the table
    gpu.same()


def test_gather_reads_back(m):
    g = np.random.default_rng(11)
    for D, n_kv, rope, kv, P, kind in SHAPES[1:6]:
        layer = spec(n_kv, n_kv, D, rope_dims=rope, k_eq_v=kv)
        gpu = Gpu(m, Pages(30, n_kv, P, D, kind, seed=3))
        lens = [P + 7, 2 * P, 1]
        tables = tables_for(lens, P, 30, 1, max_pages=3)
        append_rows(m, layer, gpu, tables, [0, 0, 0], lens, g, prepped=False)
        start, rows = [3, P - 2, -1], [P + 4, 3, 2]
        n, off = sum(rows), offsets(rows)
        out = [torch.full((n * n_kv * D + GUARD,), 77, dtype=torch.int16, device="cuda") for _ in range(2)]
        m.kvq_paged_gather(gpu.cache, dev(tables), 3, 3, dev(off), dev(np.int32(start)), n, out[0], out[1])
        torch.cuda.synchronize()
        for c, o in zip("kv", out):
            got = O.bf16_to_f64(o[:-GUARD].view(n, n_kv, D).cpu().numpy().view(np.uint16))
            assert bool((o[-GUARD:] == 77).all())
            for s in range(2):
                pos = np.arange(start[s], start[s] + rows[s])
                want = np.stack([gpu.p.values(c, tables[s], h, pos) for h in range(n_kv)], 1)
                want = O.rn_bf16(want.astype(F32).astype(np.float64))
                assert np.array_equal(got[off[s]:off[s + 1]], want)
            assert np.isnan(got[off[2]:]).all()


# ---- attention ----

def filled(m, layer, P, kind, lens, seed, spare=3, fill=None, max_pages=None):
    """Pages holding `lens` tokens a sequence, appended on the GPU; everything else keeps its bytes (and NaN scales)."""
    g = np.random.default_rng(seed)
    n_pages = sum(-(-n // P) for n in lens) + spare
    gpu = Gpu(m, Pages(n_pages, layer.n_kv_heads, P, layer.head_dim, kind, seed=seed, fill=fill))
    tables = tables_for(lens, P, n_pages, seed, max_pages)
    append_rows(m, layer, gpu, tables, [0] * len(lens), lens, g, prepped=False)
    gpu.same()
    return gpu, tables, g


def ask(g, layer, rows, sharp):
    q = bf16(g, (rows, layer.n_q_heads, layer.head_dim))
    w = bf16(g, layer.head_dim, sharp / np.sqrt(layer.head_dim), 0.1 * sharp / np.sqrt(layer.head_dim))
    return q, w


class Read:
    """A read of rows on the GPU: outputs in fp32 or bf16 with guards, workspace and q_prepped."""

    def __init__(self, m, layer, gpu, tables, pos, rows, q, w, f32=True, offs=None, max_pos=None, stream=None):
        self.n = n = q.shape[0]
        top = max(0, max(p + max(1, r) - 1 for p, r in zip(pos, rows)))
        self.max_pos = top if max_pos is None else max_pos
        size = n * layer.n_q_heads * layer.head_dim
        self.full = torch.full((size + GUARD,), 77, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        self.qp = torch.zeros(size + GUARD, dtype=torch.int16, device="cuda")
        L = lay(m, layer)
        self.keep = [dev(tables), dev(np.int32(pos)), dev(q), dev(w)]
        t, p, dq, dw = self.keep
        if offs is None:
            need = m.attn_paged_decode_workspace_bytes(L, gpu.cache, n, self.max_pos)
            self.ws = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
            self.call = lambda: m.attn_paged_decode(L, gpu.cache, t, tables.shape[1], n, p, self.max_pos, dq, dw,
                                                    self.full, f32, self.qp, self.ws, need, stream)
        else:
            self.keep.append(dev(offs))
            most = max(1, max(rows))
            need = m.attn_paged_prefill_workspace_bytes(L, gpu.cache, len(rows), n, most, self.max_pos)
            self.ws = torch.full((need + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
            self.call = lambda: m.attn_paged_prefill(L, gpu.cache, t, tables.shape[1], len(rows), self.keep[-1], p, n,
                                                     most, self.max_pos, dq, dw, self.full, f32, self.qp, self.ws,
                                                     need, stream)
        self.shape, self.need = (n, layer.n_q_heads, layer.head_dim), need

    def run(self):
        self.call()
        torch.cuda.synchronize()
        assert bool((self.full[-GUARD:] == 77).all()) and bool((self.ws[self.need:] == 0xA5).all())
        assert bool((self.qp[-GUARD:] == 0).all())
        return self.full[:-GUARD].float().cpu().numpy().astype(np.float64).reshape(self.shape)

    def status(self):
        return int(self.ws[:4].cpu().numpy().view(np.uint32)[0])

    def prepped(self):
        return self.qp[:-GUARD].cpu().numpy().view(np.uint16).reshape(self.shape)


def check(layer, gpu, tables, q, w, got, at, f32, prepped=None):
    """at: (row, sequence, position) to compare."""
    for row, s, p in at:
        q_hat = prep(q[row:row + 1], w, [p], layer)[0]
        if prepped is not None:
            assert np.array_equal(prepped[row], O.f64_to_bf16(q_hat))
        out, mag, big = attend(gpu.p, tables[s], q_hat, p, layer.window)
        n = min(p + 1, layer.window) if layer.window else p + 1
        lim = bound(out, mag, big, n, layer.head_dim, not f32)
        off = np.abs(got[row] - out)
        assert (off <= lim).all(), (row, s, p, float((off / lim).max()), np.argwhere(off > lim)[:3])


# n_q, n_kv, D, window, rope dims, K = V, page, codes
HEADS = [(4, 2, 64, 0, 64, False, 16, "i8"), (16, 1, 64, 0, 32, False, 32, "e4m3"), (5, 1, 64, 100, 64, False, 64, "i8"),
         (8, 8, 128, 0, 128, False, 32, "e4m3"), (32, 8, 128, 37, 128, False, 16, "i8"),
         (6, 2, 128, 0, 64, True, 128, "e4m3"), (8, 2, 256, 64, 256, False, 64, "i8"),
         (16, 1, 256, 0, 64, False, 16, "e4m3"), (16, 1, 512, 0, 128, True, 64, "i8"),
         (3, 3, 512, 130, 512, False, 128, "e4m3"), (14, 2, 512, 0, 0, False, 32, "i8")]


@pytest.mark.parametrize("n_q,n_kv,D,window,rope,kv,P,kind", HEADS)
def test_decode(m, n_q, n_kv, D, window, rope, kv, P, kind):
    """One to several hundred keys, tile and page borders, an idle slot, and bytes that read as NaN where no row is."""
    layer = spec(n_q, n_kv, D, window, rope, k_eq_v=kv)
    lens = [1, 2, 16, 63, 64, 65, 128, 200, 517]
    gpu, tables, g = filled(m, layer, P, kind, lens, D + n_q, fill=0x7F)
    pos = [n - 1 for n in lens]
    pos[2] = -1
    q, w = ask(g, layer, len(lens), 4.0)
    at = [(s, s, p) for s, p in enumerate(pos) if p >= 0]
    for f32 in (True, False):
        r = Read(m, layer, gpu, tables, pos, [1] * len(lens), q, w, f32)
        got = r.run()
        assert r.status() == 0 and not got[2].any()
        check(layer, gpu, tables, q, w, got, at, f32, r.prepped())
        assert np.array_equal(got, r.run())


@pytest.mark.parametrize("sharp", [0.0, 0.3, 30.0])
@pytest.mark.parametrize("D,kind", [(128, "i8"), (256, "e4m3"), (512, "i8")])
def test_decode_long_and_sharp(m, sharp, D, kind):
    """Thousands of keys cut over many CTAs, from equal weights to one key that takes all."""
    layer = spec(8 if D < 512 else 16, 1, D)
    lens = [5000, 1300]
    gpu, tables, g = filled(m, layer, 32, kind, lens, D)
    q, w = ask(g, layer, 2, sharp)
    r = Read(m, layer, gpu, tables, [4999, 1299], [1, 1], q, w)
    got = r.run()
    assert r.status() == 0
    check(layer, gpu, tables, q, w, got, [(0, 0, 4999), (1, 1, 1299)], True)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_scales_far_apart(m, D):
    """Pages whose scales differ by 2^40: the largest weights may sit on the smallest values."""
    layer = spec(4, 1, D, rope_dims=0)
    lens = [300]
    gpu, tables, g = filled(m, layer, 16, "i8", lens, 77)
    for i, page in enumerate(tables[0]):
        gpu.p.scales["v"][page] = [2.0 ** -40, 2.0 ** 3, 0.0, 2.0 ** -20][i % 4]
        if i % 4 == 2:
            gpu.p.codes["v"][page] = 0
    gpu = Gpu(m, gpu.p)
    q, w = ask(g, layer, 1, 2.0)
    r = Read(m, layer, gpu, tables, [299], [1], q, w)
    got = r.run()
    check(layer, gpu, tables, q, w, got, [(0, 0, 299)], True)


def test_decode_tables_that_name_no_page(m):
    """Such rows are NaN and flagged; the others are as without them."""
    layer = spec(8, 2, 128)
    lens = [100, 100, 100, 40, 70]
    gpu, tables, g = filled(m, layer, 16, "i8", lens, 31, max_pages=7)
    q, w = ask(g, layer, 5, 3.0)
    pos = [99, 99, 99, 39, 69]
    good = Read(m, layer, gpu, tables, pos, [1] * 5, q, w).run()
    bad = tables.copy()
    bad[1, 3] = -1
    bad[2, 0] = gpu.p.n_pages
    r = Read(m, layer, gpu, bad, [99, 99, 99, 39, 112], [1] * 5, q, w)     # 112 is past seven pages
    got = r.run()
    assert r.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert np.isnan(got[[1, 2, 4]]).all() and np.array_equal(got[[0, 3]], good[[0, 3]])
    r = Read(m, layer, gpu, tables, pos, [1] * 5, q, w, max_pos=69)        # positions above the bound
    got = r.run()
    assert r.status() == m.KVQ_STATUS_SEQ_SKIPPED and np.isnan(got[:3]).all()
    check(layer, gpu, tables, q, w, got, [(3, 3, 39), (4, 4, 69)], True)


def test_pages_behind_a_window_may_be_gone(m):
    layer = spec(8, 2, 64, window=50)
    gpu, tables, g = filled(m, layer, 16, "e4m3", [200], 8)
    q, w = ask(g, layer, 1, 3.0)
    tables[0, :9] = -1                                         # positions below 144; 150 is the oldest seen
    r = Read(m, layer, gpu, tables, [199], [1], q, w)
    got = r.run()
    assert r.status() == 0
    check(layer, gpu, tables, q, w, got, [(0, 0, 199)], True)


PREFILL = HEADS + [(128, 8, 64, 0, 64, False, 32, "e4m3"), (2, 2, 128, 16, 128, False, 32, "i8")]


@pytest.mark.parametrize("n_q,n_kv,D,window,rope,kv,P,kind", PREFILL)
def test_prefill(m, n_q, n_kv, D, window, rope, kv, P, kind):
    """Whole prompts, later chunks that start inside pages, verify windows, single rows, none, idle sequences."""
    layer = spec(n_q, n_kv, D, window, rope, k_eq_v=kv)
    lens, rows = [150, 300, 64, 1, 33, 40, 20], [150, 37, 4, 1, 0, 17, 5]
    gpu, tables, g = filled(m, layer, P, kind, lens, D + n_q + 1, fill=0x7F)
    start = [n - r for n, r in zip(lens, rows)]
    start[5] = -1
    off = offsets(rows)
    q, w = ask(g, layer, int(off[-1]), 4.0)
    at = [(off[s] + t, s, start[s] + t) for s in range(7) for t in range(rows[s]) if start[s] >= 0]
    for f32 in (True, False):
        r = Read(m, layer, gpu, tables, start, rows, q, w, f32, off)
        got = r.run()
        assert r.status() == 0 and not got[off[5]:off[6]].any()
        check(layer, gpu, tables, q, w, got, at[::3] if f32 else at[::17], f32, r.prepped())
        assert np.array_equal(got, r.run())


@pytest.mark.parametrize("D,n_q,n_kv,window,kind", [(64, 4, 4, 0, "i8"), (128, 8, 2, 0, "e4m3"), (256, 8, 2, 0, "i8"),
                                                    (128, 16, 1, 300, "i8"), (512, 16, 1, 0, "e4m3")])
def test_prefill_long(m, D, n_q, n_kv, window, kind):
    """Chunks over thousands of keys, a whole long prompt beside them."""
    layer = spec(n_q, n_kv, D, window)
    lens, rows = [2500, 1100], [260, 1100]
    gpu, tables, g = filled(m, layer, 64, kind, lens, D)
    start, off = [2240, 0], offsets(rows)
    q, w = ask(g, layer, 1360, 3.0)
    r = Read(m, layer, gpu, tables, start, rows, q, w, True, off)
    got = r.run()
    assert r.status() == 0
    at = [(t, 0, 2240 + t) for t in (0, 1, 63, 127, 128, 200, 259)]
    at += [(260 + t, 1, t) for t in (0, 1, 31, 127, 128, 500, 767, 1099)]
    check(layer, gpu, tables, q, w, got, at, True)


@pytest.mark.parametrize("rows", [6, 200])
def test_prefill_tables_that_name_no_page(m, rows):
    layer = spec(8, 2, 128)
    gpu, tables, g = filled(m, layer, 16, "i8", [250, 250], 31, max_pages=16)
    start, off = [250 - rows] * 2, offsets([rows] * 2)
    q, w = ask(g, layer, 2 * rows, 3.0)
    good = Read(m, layer, gpu, tables, start, [rows] * 2, q, w, True, off).run()
    bad = tables.copy()
    bad[0, 2] = -7
    r = Read(m, layer, gpu, bad, start, [rows] * 2, q, w, True, off)
    got = r.run()
    assert r.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert np.isnan(got[rows - 1]).all() and np.array_equal(got[rows:], good[rows:])
    # rows past the table, in a chunk whose first rows are in it
    r = Read(m, layer, gpu, tables, [250 - rows, 256 - rows + 3], [rows] * 2, q, w, True, off)
    got = r.run()
    assert r.status() == m.KVQ_STATUS_SEQ_SKIPPED and np.isnan(got[2 * rows - 3:]).all()
    assert np.array_equal(got[:rows], good[:rows])


@pytest.mark.parametrize("n_q", [4, 8])
def test_decode_is_the_last_row_of_a_prompt(m, n_q):
    """The two reads of one row agree within both bounds, whatever path each takes."""
    layer = spec(n_q, 2, 128)
    gpu, tables, g = filled(m, layer, 32, "e4m3", [400], 3)
    q, w = ask(g, layer, 400, 3.0)
    whole = Read(m, layer, gpu, tables, [0], [400], q, w, True, offsets([400])).run()
    one = Read(m, layer, gpu, tables, [399], [1], q[-1:], w).run()
    q_hat = prep(q[-1:], w, [399], layer)[0]
    out, mag, big = attend(gpu.p, tables[0], q_hat, 399, 0)
    assert (np.abs(whole[-1] - one[0]) <= 2 * bound(out, mag, big, 400, 128, False)).all()


def test_elements_past_32_bits(m):
    """Pages more than 2^32 bytes into the codes."""
    layer = spec(8, 4, 256)
    n_pages, P = 40000, 128                                    # 5.2 GB of codes each
    small = Pages(3, 4, P, 256, "i8", seed=1)
    codes = {c: torch.zeros((n_pages, 4, P, 256), dtype=torch.uint8, device="cuda") for c in "kv"}
    scales = {c: torch.zeros((n_pages, 4), dtype=torch.float32, device="cuda") for c in "kv"}
    cache = m.paged_cache(codes["k"], codes["v"], scales["k"], scales["v"], n_pages, P, 4, 256, m.KVQ_CODE_I8)
    g = np.random.default_rng(1)
    far, near = np.int32([[39999, 33000]]), np.int32([[0, 2]])
    k, v, w = bf16(g, (150, 4, 256)), bf16(g, (150, 4, 256)), bf16(g, 256, 1.0, 0.1)
    m.kvq_paged_append(lay(m, layer), cache, dev(far), 2, 1, dev(offsets([150])), dev(np.int32([0])), 150, dev(k),
                       dev(v), dev(w))
    pos = np.arange(150)
    small.append(near[0], 0, prep(k, w, pos, layer), prep(v, None, pos, layer))
    for a, b in zip(far[0], near[0]):
        assert np.array_equal(scales["k"][int(a)].cpu().numpy(), small.scales["k"][b])
    assert np.array_equal(codes["v"][33000, :, :22].cpu().numpy(), small.codes["v"][2, :, :22])

    class Far:
        pass

    gpu = Far()
    gpu.cache, gpu.p = cache, small
    q, w = ask(g, layer, 150, 3.0)
    got = Read(m, layer, gpu, far, [149], [1], q[-1:], w).run()
    check(layer, gpu, near, q[-1:], w, got, [(0, 0, 149)], True)
    got = Read(m, layer, gpu, far, [0], [150], q, w, True, offsets([150])).run()
    check(layer, gpu, near, q, w, got, [(0, 0, 0), (130, 0, 130), (149, 0, 149)], True)
    del codes, cache, gpu
    torch.cuda.empty_cache()


def test_streams_and_graphs(m):
    """A decode step on another stream, two steps at once on two streams, and captured and replayed with new data."""
    layer = spec(8, 2, 128)
    gpu, tables, g = filled(m, layer, 32, "i8", [300, 77], 3)
    q, w = ask(g, layer, 2, 3.0)
    want = Read(m, layer, gpu, tables, [299, 76], [1, 1], q, w).run()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ra = Read(m, layer, gpu, tables, [299, 76], [1, 1], q, w, stream=a)
    rb = Read(m, layer, gpu, tables, [299, 76], [1, 1], q, w, stream=b)
    torch.cuda.synchronize()
    for _ in range(10):
        ra.call()
        rb.call()
    torch.cuda.synchronize()
    shape = ra.shape
    for r in (ra, rb):
        assert np.array_equal(r.full[:-GUARD].cpu().numpy().reshape(shape), want.astype(F32))
    r = Read(m, layer, gpu, tables, [299, 76], [1, 1], q, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.call()
    other = dev(ask(g, layer, 2, 3.0)[0])
    r.keep[2].copy_(other)
    r.keep[1].copy_(dev(np.int32([150, -1])))
    r.full.fill_(77)
    graph.replay()
    torch.cuda.synchronize()
    got = r.full[:-GUARD].cpu().numpy().astype(np.float64).reshape(shape)
    check(layer, gpu, tables, other.cpu().numpy().view(np.uint16), w, got, [(0, 0, 150)], True)
    assert not got[1].any()
