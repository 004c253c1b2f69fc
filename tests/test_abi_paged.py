"""Host-side argument checks of the paged cache's calls (nothing is enqueued),
and the numpy reference of the GPU tests against hand-worked values."""
import ctypes

import numpy as np
import pytest

from paged_ref import E4M3, Pages, Pool, code_values, encode

P = 1 << 20          # a fake, aligned "device address": never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__.build()
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def layer(m, **kw):
    d = dict(n_q_heads=8, n_kv_heads=2, head_dim=256, window=512, rope_dims=256, rope_theta=1e4)
    d.update(kw)
    return m.layer(**d)


def cache(m, **kw):
    d = dict(k=P, v=P, ks=P, vs=P, n_pages=10, page=64, n_kv=2, D=256, kind=0)
    d.update(kw)
    return m.paged_cache(*d.values())


def pool(m, **kw):
    d = dict(tables=P, lens=P, refs=P, n_seqs=4, max_pages=3, n_pages=10, page=64)
    d.update(kw)
    return m.page_pool(*d.values())


def ref(x):
    return ctypes.byref(x) if x is not None else None


CACHES = [(dict(k=None), 1), (dict(k=P + 8), 1), (dict(v=P + 4), 1), (dict(ks=None), 1), (dict(vs=P + 2), 1),
          (dict(n_pages=0), 1), (dict(page=8), 2), (dict(page=48), 2), (dict(page=256), 2), (dict(D=96), 2),
          (dict(kind=2), 1), (dict(kind=-1), 1), (dict(n_kv=0), 1)]
LAYERS = [(dict(head_dim=128), 1), (dict(n_kv_heads=4), 1), (dict(rot_signs=P), 2), (dict(n_q_heads=34), 2),
          (dict(head_dim=96), 2)]

APPEND = dict(tables=P, max_pages=3, n_seqs=4, offs=P, start=P, n_rows=9, k=P, v=P, w=P, prepped=None)
DECODE = dict(tables=P, max_pages=3, n_seqs=4, pos=P, max_pos=100, q=P, w=P, out=P, f32=0, prepped=None, ws=P,
              ws_bytes=BIG)
PREFILL = dict(tables=P, max_pages=3, n_seqs=4, offs=P, start=P, n_rows=9, max_rows=9, max_pos=100, q=P, w=P, out=P,
               f32=0, prepped=None, ws=P, ws_bytes=BIG)
GATHER = dict(tables=P, max_pages=3, n_seqs=4, offs=P, start=P, n_rows=9, k=P, v=P)


def call(fn, defaults, *first, **kw):
    d = dict(defaults)
    d.update(kw)
    return fn(*first, *d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), 1), (dict(tables=P + 2), 1), (dict(max_pages=0), 1), (dict(n_seqs=-1), 1), (dict(n_seqs=0), 1),
    (dict(n_rows=-1), 1), (dict(n_rows=1 << 24), 1), (dict(offs=None), 1), (dict(offs=P + 1), 1), (dict(start=None), 1),
    (dict(k=None), 1), (dict(k=P + 8), 1), (dict(v=None), 1), (dict(v=P + 2), 1), (dict(w=None), 1), (dict(w=P + 1), 1),
    (dict(prepped=P + 1), 1)])
def test_append_refusals(m, kw, status):
    assert call(m.lib.kvq_paged_append, APPEND, ref(layer(m)), ref(cache(m)), **kw) == status
    assert m.kvq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), 1), (dict(max_pages=-1), 1), (dict(n_seqs=-1), 1), (dict(pos=None), 1), (dict(pos=P + 2), 1),
    (dict(max_pos=-1), 1), (dict(max_pos=1 << 24), 1), (dict(q=None), 1), (dict(q=P + 8), 1), (dict(w=None), 1),
    (dict(out=None), 1), (dict(out=P + 2, f32=1), 1), (dict(out=P + 1), 1), (dict(f32=2), 1), (dict(prepped=P + 1), 1),
    (dict(ws=None), 1), (dict(ws=P + 16), 1), (dict(ws_bytes=0), 4)])
def test_decode_refusals(m, kw, status):
    assert call(m.lib.attn_paged_decode, DECODE, ref(layer(m)), ref(cache(m)), **kw) == status
    assert m.kvq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(tables=P + 1), 1), (dict(offs=None), 1), (dict(offs=P + 2), 1), (dict(start=None), 1), (dict(n_rows=-3), 1),
    (dict(max_rows=0), 1), (dict(max_pos=1 << 24), 1), (dict(q=P + 4), 1), (dict(w=P + 1), 1), (dict(out=None), 1),
    (dict(ws=P + 128), 1), (dict(ws_bytes=1000), 4), (dict(n_seqs=0), 1)])
def test_prefill_refusals(m, kw, status):
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(layer(m)), ref(cache(m)), **kw) == status
    assert m.kvq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), 1), (dict(max_pages=0), 1), (dict(offs=P + 2), 1), (dict(start=None), 1), (dict(n_rows=-1), 1),
    (dict(k=None), 1), (dict(k=P + 8), 1), (dict(v=P + 2), 1), (dict(n_seqs=0), 1)])
def test_gather_refusals(m, kw, status):
    assert call(m.lib.kvq_paged_gather, GATHER, ref(cache(m)), **kw) == status
    assert m.kvq_last_error()


@pytest.mark.parametrize("kw,status", CACHES)
def test_cache_refusals(m, kw, status):
    c = cache(m, **kw)
    assert call(m.lib.kvq_paged_append, APPEND, ref(layer(m)), ref(c)) == status
    assert call(m.lib.attn_paged_decode, DECODE, ref(layer(m)), ref(c)) == status
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(layer(m)), ref(c)) == status
    assert call(m.lib.kvq_paged_gather, GATHER, ref(c)) == status
    caches = m.paged_caches([cache(m), c])
    assert m.lib.kvq_pages_compact(ref(pool(m)), caches, 2, None, P, P, BIG, None) == status
    assert m.lib.attn_paged_decode_workspace_bytes(ref(layer(m)), ref(c), 4, 100) == 0
    assert m.lib.attn_paged_prefill_workspace_bytes(ref(layer(m)), ref(c), 4, 9, 9, 100) == 0


@pytest.mark.parametrize("kw,status", LAYERS)
def test_layer_refusals(m, kw, status):
    lay = layer(m, **kw)
    assert call(m.lib.kvq_paged_append, APPEND, ref(lay), ref(cache(m))) == status
    assert call(m.lib.attn_paged_decode, DECODE, ref(lay), ref(cache(m))) == status
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(lay), ref(cache(m))) == status
    assert m.lib.attn_paged_decode_workspace_bytes(ref(lay), ref(cache(m)), 4, 100) == 0


def test_keys_equal_values_layers_take_no_values(m):
    lay = layer(m, k_eq_v=True)
    assert call(m.lib.kvq_paged_append, APPEND, ref(lay), ref(cache(m))) == 1
    assert call(m.lib.kvq_paged_append, APPEND, ref(lay), ref(cache(m)), v=None, n_rows=0) == 0


def test_nothing_to_do(m):
    lay, c = layer(m), cache(m)
    assert call(m.lib.kvq_paged_append, APPEND, ref(lay), ref(c), n_rows=0) == 0
    assert call(m.lib.kvq_paged_gather, GATHER, ref(c), n_rows=0) == 0
    assert call(m.lib.attn_paged_decode, DECODE, ref(lay), ref(c), n_seqs=0) == 0
    assert call(m.lib.attn_paged_prefill, PREFILL, ref(lay), ref(c), n_rows=0) == 0
    assert m.lib.kvq_pages_free(ref(pool(m)), None, None, 0, None) == 0
    assert m.lib.kvq_pages_fork(ref(pool(m)), None, None, 0, None, None) == 0
    for first in ((None, ref(c)), (ref(lay), None)):
        assert call(m.lib.kvq_paged_append, APPEND, *first) == 1
        assert call(m.lib.attn_paged_decode, DECODE, *first) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(tables=None), 1), (dict(lens=P + 2), 1), (dict(refs=None), 1), (dict(n_seqs=0), 1), (dict(max_pages=0), 1),
    (dict(n_pages=0), 1), (dict(page=24), 2), (dict(n_seqs=1 << 20, max_pages=1 << 20), 2)])
def test_pool_refusals(m, kw, status):
    p, caches = pool(m, **kw), m.paged_caches([cache(m)])
    assert m.lib.kvq_pages_free(ref(p), P, None, 1, None) == status
    assert m.lib.kvq_pages_fork(ref(p), P, P, 1, None, None) == status
    assert m.lib.kvq_pages_reserve(ref(p), caches, 1, P, P, P, P, BIG, None) == status
    assert m.lib.kvq_pages_compact(ref(p), caches, 1, None, P, P, BIG, None) == status
    assert m.lib.kvq_pages_workspace_bytes(ref(p)) == 0


def test_pool_call_refusals(m):
    p, one = ref(pool(m)), m.paged_caches([cache(m)])
    free, fork, reserve, compact = (m.lib.kvq_pages_free, m.lib.kvq_pages_fork, m.lib.kvq_pages_reserve,
                                    m.lib.kvq_pages_compact)
    assert free(None, P, None, 1, None) == 1 and free(p, None, None, 1, None) == 1
    assert free(p, P, P + 2, 1, None) == 1 and free(p, P, None, -1, None) == 1
    assert fork(p, None, P, 1, None, None) == 1 and fork(p, P, P + 1, 1, None, None) == 1
    assert fork(p, P, P, 1, P + 2, None) == 1 and fork(p, P, P, -1, None, None) == 1
    assert reserve(p, None, 1, P, P, P, P, BIG, None) == 1 and reserve(p, one, 0, P, P, P, P, BIG, None) == 1
    assert reserve(p, one, 129, P, P, P, P, BIG, None) == 1
    for at in range(3):
        args = [P, P, P]
        args[at] = None
        assert reserve(p, one, 1, *args, P, BIG, None) == 1
    assert reserve(p, one, 1, P, P, P, P + 16, BIG, None) == 1 and reserve(p, one, 1, P, P, P, P, 100, None) == 4
    assert compact(p, one, 1, P + 1, P, P, BIG, None) == 1 and compact(p, one, 1, None, None, P, BIG, None) == 1
    assert compact(p, one, 1, None, P, None, BIG, None) == 1 and compact(p, one, 1, None, P, P, 0, None) == 4
    for kw in (dict(n_pages=11), dict(page=32)):
        other = m.paged_caches([cache(m), cache(m, **kw)])
        assert compact(p, other, 2, None, P, P, BIG, None) == 1
        assert reserve(p, other, 2, P, P, P, P, BIG, None) == 1


def test_workspaces_grow_with_the_call(m):
    lay, c = layer(m), cache(m)
    d = [m.attn_paged_decode_workspace_bytes(lay, c, n, pos) for n, pos in ((1, 0), (1, 1000), (4, 1000), (64, 5000))]
    assert 0 < d[0] <= d[1] <= d[2] <= d[3]
    f = [m.attn_paged_prefill_workspace_bytes(lay, c, n, r, r, 5000) for n, r in ((1, 1), (1, 100), (4, 400), (4, 4000))]
    assert 0 < f[0] <= f[1] <= f[2] <= f[3]
    assert m.attn_paged_decode_workspace_bytes(lay, c, -1, 0) == 0 == m.attn_paged_decode_workspace_bytes(lay, c, 1, -1)
    assert m.attn_paged_prefill_workspace_bytes(lay, c, 1, 1, 1, 1 << 24) == 0
    assert m.kvq_pages_workspace_bytes(pool(m)) >= 3 * 4 * 10


def test_struct_layouts(m):
    assert ctypes.sizeof(m.KvqPagedCache) == 56 and m.KvqPagedCache.code_type.offset == 48
    assert ctypes.sizeof(m.KvqPagePool) == 40 and m.KvqPagePool.page_tokens.offset == 36


# ---- the reference itself ----

def test_reference_codes():
    assert E4M3[0x7E] == 448 and E4M3[0x01] == 2.0 ** -9 and E4M3[0x38] == 1 and E4M3[0xB8] == -1
    every = np.arange(256, dtype=np.uint8)
    finite = every[(every & 127) != 127]
    assert np.array_equal(encode(code_values(finite, "e4m3").astype(np.float32), "e4m3"), finite)
    # halfway values go to the even code, beyond the top they stop there
    assert np.array_equal(encode(np.float32([17, 19, 2.0 ** -10, 3 * 2.0 ** -10, 500, -460]), "e4m3"),
                          np.uint8([0x58, 0x5A, 0x00, 0x02, 0x7E, 0xFE]))
    assert np.array_equal(encode(np.float32([0.5, 1.5, -2.5, 200, -127.6]), "i8").view(np.int8), [0, 2, -2, 127, -127])


def test_reference_scale_growth():
    pg = Pages(2, 1, 16, 64, "i8", seed=1)
    one, two = np.zeros((1, 1, 64)), np.zeros((1, 1, 64))
    one[0, 0, :3] = [127.0, -64.0, 1.0]
    two[0, 0, 0] = 254.0
    pg.append([1], 0, one, one)
    assert pg.scales["k"][1, 0] == 1 and list(pg.codes["k"][1, 0, 0, :3].view(np.int8)) == [127, -64, 1]
    pg.append([1], 1, two, one)
    assert pg.scales["k"][1, 0] == 2 and pg.scales["v"][1, 0] == 1
    assert list(pg.codes["k"][1, 0, 0, :3].view(np.int8)) == [64, -32, 0]          # 63.5 and 0.5 go to the even code
    assert np.array_equal(pg.values("v", [1], 0, [0, 1])[:, :3], [[127, -64, 1]] * 2)
    pg.append([0], 0, np.full((1, 1, 64), 2.0 ** -41), two)                          # below the smallest scale
    assert pg.scales["k"][0, 0] == 0 and not pg.codes["k"][0, 0, 0].any()


def test_reference_pool():
    p = Pool(4, 4, 6, 16)
    assert p.reserve([20, 0, 0, 0]) == ([1, 1, 1, 1], [0, 0, 0, 0], [])
    assert p.tables[0] == [0, 1, -1, -1] and p.refs == [1, 1, 0, 0, 0, 0]
    assert p.fork([0, 0, 2, 1], [1, 1, 2, 3]) == [1, 0, 0, 0]        # listed twice; itself; from a child of the call
    assert p.refs == [2, 2, 0, 0, 0, 0] and p.lens == [20, 20, 0, 0]
    granted, start, copies = p.reserve([1, 13, 17, 16])              # 1, 1 + 1, 2 of 4 free pages; the last is refused
    assert granted == [1, 1, 0, 0] and start == [20, 20, 0, 0] and copies == [(1, 2), (1, 3)]
    assert p.tables[1] == [0, 3, 4, -1] and p.refs == [2, 0, 1, 1, 1, 0]
    assert p.compact() == (4, [0, -1, 2, 3, 1, -1], [(4, 1)]) and p.tables[1] == [0, 3, 1, -1]
    p.free([1, 1, 9], [18, 0, 0])
    assert p.lens == [21, 18, 0, 0] and p.tables[1] == [0, 3, -1, -1] and p.refs == [2, 0, 1, 1, 0, 0]
