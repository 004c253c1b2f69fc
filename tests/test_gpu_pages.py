"""The pool of pages on the GPU against its bookkeeping one sequence after
another: random programs of reserving, forking, freeing and compacting, pools
that run out, contents that move with their pages, and a serving run (prompt,
decode, fork, decode, free, compact) whose reads stay what they were."""
import numpy as np
import pytest

from paged_ref import Pages, Pool
from test_gpu_paged import Gpu, Read, append_rows, ask, check, dev, spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


class GpuPool:
    def __init__(self, m, n_seqs, max_pages, n_pages, P, caches):
        """caches: (n_kv, head_dim) of each."""
        self.m, self.ref = m, Pool(n_seqs, max_pages, n_pages, P)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables = torch.full((n_seqs, max_pages), -1, **i32)
        self.lens, self.refs = torch.zeros(n_seqs, **i32), torch.zeros(n_pages, **i32)
        self.pool = m.page_pool(self.tables, self.lens, self.refs, n_seqs, max_pages, n_pages, P)
        self.start, self.granted = torch.zeros(n_seqs, **i32), torch.zeros(n_seqs, **i32)
        self.map, self.live = torch.zeros(n_pages, **i32), torch.zeros(1, **i32)
        g = torch.Generator(device="cuda").manual_seed(n_pages)
        self.data, list_ = [], []
        for n_kv, D in caches:
            c = [torch.randint(0, 256, (n_pages, n_kv, P, D), generator=g, dtype=torch.uint8, device="cuda")
                 for _ in range(2)]
            s = [torch.rand((n_pages, n_kv), generator=g, device="cuda") for _ in range(2)]
            self.data += c + s
            list_.append(m.paged_cache(c[0], c[1], s[0], s[1], n_pages, P, n_kv, D, m.KVQ_CODE_I8))
        self.caches = m.paged_caches(list_)
        self.need = m.kvq_pages_workspace_bytes(self.pool)
        self.ws = torch.full((self.need + 256,), 0xA5, dtype=torch.uint8, device="cuda")

    def same(self):
        torch.cuda.synchronize()
        assert self.tables.cpu().tolist() == self.ref.tables
        assert self.lens.cpu().tolist() == self.ref.lens and self.refs.cpu().tolist() == self.ref.refs
        assert bool((self.ws[self.need:] == 0xA5).all())

    def copied(self, before, pairs):
        for a, b in zip(before, self.data):
            for src, dst in pairs:
                a[dst] = a[src].clone()
            assert torch.equal(a, b)

    def reserve(self, n_new):
        before = [t.clone() for t in self.data]
        self.m.kvq_pages_reserve(self.pool, self.caches, dev(np.int32(n_new)), self.start, self.granted, self.ws,
                                 self.need)
        granted, start, copies = self.ref.reserve(n_new)
        self.same()
        assert self.granted.cpu().tolist() == granted and self.start.cpu().tolist() == start
        self.copied(before, copies)
        return granted

    def fork(self, parents, children):
        got = torch.full((len(parents),), 9, dtype=torch.int32, device="cuda")
        self.m.kvq_pages_fork(self.pool, dev(np.int32(parents)), dev(np.int32(children)), len(parents), got)
        granted = self.ref.fork(parents, children)
        self.same()
        assert got.cpu().tolist() == granted
        return granted

    def free(self, seqs, keep=None):
        self.m.kvq_pages_free(self.pool, dev(np.int32(seqs)), None if keep is None else dev(np.int32(keep)), len(seqs))
        self.ref.free(seqs, keep)
        self.same()

    def compact(self, with_map=True):
        before = [t.clone() for t in self.data]
        self.m.kvq_pages_compact(self.pool, self.caches, self.map if with_map else None, self.live, self.ws, self.need)
        live, to, moves = self.ref.compact()
        self.same()
        assert int(self.live) == live
        if with_map:
            assert self.map.cpu().tolist() == to
        self.copied(before, moves)


@pytest.mark.parametrize("n_seqs,max_pages,n_pages,P,caches,seed", [
    (12, 9, 60, 16, [(1, 64)], 0), (40, 30, 700, 32, [(3, 128), (2, 64)], 1), (7, 5, 33, 128, [(17, 64), (1, 512)], 2),
    (300, 4, 900, 64, [(1, 64)], 3)])
def test_random_programs(m, n_seqs, max_pages, n_pages, P, caches, seed):
    g = np.random.default_rng(seed)
    p = GpuPool(m, n_seqs, max_pages, n_pages, P, caches)
    for step in range(25):
        what = g.integers(0, 5)
        if what <= 1:
            top = int(g.choice([2, P, 2 * P]))
            p.reserve((g.integers(-1, top, n_seqs) * (g.random(n_seqs) < 0.7)).tolist())
        elif what == 2:
            k = int(g.integers(1, n_seqs + 1))
            p.fork(g.integers(-1, n_seqs + 1, k).tolist(), g.integers(-1, n_seqs + 1, k).tolist())
        elif what == 3:
            k = int(g.integers(1, n_seqs))
            seqs = g.integers(-1, n_seqs + 1, k).tolist()
            p.free(seqs, None if g.random() < 0.5 else g.integers(-2, 3 * P, k).tolist())
        else:
            p.compact(bool(step % 2))


def test_a_pool_that_runs_out(m):
    p = GpuPool(m, 6, 4, 7, 16, [(2, 64)])
    assert p.reserve([16, 40, 64, 1, 0, 65]) == [1, 1, 0, 0, 1, 0]        # 1, 3, 4 of the 3 left; past four pages
    assert p.fork([1, 1], [2, 3]) == [1, 1]
    assert p.reserve([0, 1, 1, 1, 0, 1]) == [1, 1, 1, 1, 1, 0]            # three copies take what is left
    # sequence 0's page, the shared page that all three left, and the copy of sequence 1 are free: 1, 1, 1, none
    p.free([0, 1])
    assert p.reserve([16, 0, 9, 9, 0, 16]) == [1, 1, 1, 1, 1, 0]
    p.compact()
    p.free(list(range(6)))
    p.compact()
    assert p.ref.refs == [0] * 7


def test_references_of_the_program_itself(m):
    """A page that no sequence holds but the program counted is not taken, and moves."""
    p = GpuPool(m, 3, 4, 12, 16, [(1, 64)])
    for page in (0, 9):
        p.refs[page] = p.ref.refs[page] = 1
    p.reserve([20, 16, 50])
    assert 0 not in p.ref.tables[0]
    p.free([0, 1])
    p.compact()
    assert p.ref.refs.count(1) == 6 and p.ref.refs[6:] == [0] * 6


def test_forks_of_an_empty_and_of_a_full_page(m):
    p = GpuPool(m, 5, 3, 9, 16, [(2, 64)])
    p.reserve([32, 0, 0, 0, 0])
    assert p.fork([0, 4, 0], [1, 2, 0]) == [0, 1, 0]       # 0 is a child of the call: nothing may be forked from it
    assert p.fork([0, 4], [1, 2]) == [1, 1]
    p.reserve([1, 1, 1, 0, 0])                             # full pages stay shared
    assert p.ref.tables[0][:2] == p.ref.tables[1][:2] and p.ref.tables[0][2] != p.ref.tables[1][2]
    p.free([1], [20])                                      # back into a shared page
    p.reserve([0, 3, 0, 0, 0])                             # which is copied before it is written
    assert p.ref.tables[0][1] != p.ref.tables[1][1]


def test_a_large_pool(m):
    g = np.random.default_rng(4)
    p = GpuPool(m, 600, 200, 100000, 16, [(1, 64)])
    p.reserve(g.integers(0, 200 * 16, 600).tolist())
    p.free(g.permutation(600)[:250].tolist())
    p.compact()
    p.reserve(g.integers(0, 400, 600).tolist())
    p.fork(list(range(0, 100)), list(range(500, 600)))


@pytest.mark.parametrize("kind,P", [("i8", 16), ("e4m3", 32)])
def test_a_serving_run(m, kind, P):
    """Two layers over one pool: prompts, decode steps, a fork whose branches diverge, a rollback, compaction."""
    g = np.random.default_rng(1)
    layers = [spec(8, 2, 64, window=40), spec(4, 1, 128, rope_dims=64, k_eq_v=True)]
    n_seqs, max_pages, n_pages = 4, 8, 30
    p = GpuPool(m, n_seqs, max_pages, n_pages, P, [])
    gpus = [Gpu(m, Pages(n_pages, s.n_kv_heads, P, s.head_dim, kind, seed=i)) for i, s in enumerate(layers)]
    p.caches = m.paged_caches([x.cache for x in gpus])

    def copy_ref(pairs):
        for x in gpus:
            for a, b in pairs:
                for c in "kv":
                    x.p.codes[c][b], x.p.scales[c][b] = x.p.codes[c][a], x.p.scales[c][a]

    def grow(n_new):
        m.kvq_pages_reserve(p.pool, p.caches, dev(np.int32(n_new)), p.start, p.granted, p.ws, p.need)
        granted, start, copies = p.ref.reserve(n_new)
        assert granted == [1] * n_seqs
        copy_ref(copies)
        p.same()
        for layer, x in zip(layers, gpus):
            append_rows(m, layer, x, np.int32(p.ref.tables), start, n_new, g, prepped=False)
            x.same()
        return start

    def look(start, rows, prompt):
        tables, off = np.int32(p.ref.tables), np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        for layer, x in zip(layers, gpus):
            q, w = ask(g, layer, int(off[-1]) if prompt else n_seqs, 3.0)
            if prompt:
                r = Read(m, layer, x, tables, start, rows, q, w, True, off)
                at = [(off[s] + t, s, start[s] + t) for s in range(n_seqs) for t in range(rows[s])]
            else:
                pos = [a if n else -1 for a, n in zip(start, rows)]
                r = Read(m, layer, x, tables, pos, [1] * n_seqs, q, w)
                at = [(s, s, a) for s, a in enumerate(pos) if a >= 0]
            got = r.run()
            assert r.status() == 0
            check(layer, x, tables, q, w, got, at[::5] if prompt else at, True)

    look(grow([45, 1, 20, 0]), [45, 1, 20, 0], True)
    look(grow([1, 1, 1, 0]), [1, 1, 1, 0], False)
    p.fork([0], [3])
    look(grow([1, 1, 0, 1]), [1, 1, 0, 1], False)          # both copies of the shared page go their own way
    look(grow([3, 4, 0, 2]), [3, 4, 0, 2], True)
    p.free([0, 2], [47, 0])                                # a rollback of two drafted rows, and a sequence done
    live, _, moves = p.ref.compact()
    m.kvq_pages_compact(p.pool, p.caches, None, p.live, p.ws, p.need)
    copy_ref(moves)
    p.same()
    assert int(p.live) == live
    look(grow([1, 1, 30, 1]), [1, 1, 0, 1], False)


def test_captured_with_the_reads(m):
    """A decode step of the pool, the append and the read as one graph, replayed."""
    layer, P, g = spec(8, 2, 64), 16, np.random.default_rng(2)
    p = GpuPool(m, 2, 6, 20, P, [])
    x = Gpu(m, Pages(20, 2, P, 64, "i8", seed=1))
    p.caches = m.paged_caches([x.cache])
    L = m.layer(8, 2, 64, 0, 64, 1e4)
    k, v = (torch.from_numpy(g.standard_normal((2, 2, 64)).astype(np.float32)).cuda().bfloat16() for _ in range(2))
    q = torch.from_numpy(g.standard_normal((2, 8, 64)).astype(np.float32)).cuda().bfloat16()
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    one, off = dev(np.int32([1, 1])), dev(np.int32([0, 1, 2]))
    need = m.attn_paged_decode_workspace_bytes(L, x.cache, 2, 6 * P - 1)
    ws, out = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(2, 8, 64, device="cuda")

    def step():
        m.kvq_pages_reserve(p.pool, p.caches, one, p.start, p.granted, p.ws, p.need)
        m.kvq_paged_append(L, x.cache, p.tables, 6, 2, off, p.start, 2, k, v, w)
        m.attn_paged_decode(L, x.cache, p.tables, 6, 2, p.start, 6 * P - 1, q, w, out, 1, None, ws, need)

    step()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(40):
        graph.replay()
    torch.cuda.synchronize()
    assert p.lens.cpu().tolist() == [41, 41] and p.refs.cpu().tolist() == [1] * 6 + [0] * 14
    # the same value in every row: its quantized form is the answer at every length, up to the weights' rounding to f16
    assert torch.allclose(out, first, rtol=2.0 ** -10, atol=1e-5)
