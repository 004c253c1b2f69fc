"""Host-side argument checks of the training read's gradient calls (nothing is
enqueued)."""
import ctypes

import pytest

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


READ = dict(n_blocks=1, offs=P, n_rows=4, max_rows=4, q=P, k=P, v=P, out=P, out_f32=1, lse=P, do=P, dq=P, dk=P, dv=P,
            dkv_f32=0, acc=0, ws=P, ws_bytes=BIG)


def read(m, lay, **kw):
    d = dict(READ)
    d.update(kw)
    return m.lib.attn_train_backward(ctypes.byref(lay) if lay else None, *d.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n_blocks=0), 1), (dict(n_blocks=65536), 1), (dict(offs=None), 1), (dict(offs=P + 2), 1),
    (dict(n_rows=-1), 1), (dict(n_rows=1 << 24), 1), (dict(max_rows=0), 1), (dict(max_rows=5), 1),
    (dict(q=None), 1), (dict(q=P + 8), 1), (dict(k=None), 1), (dict(k=P + 2), 1), (dict(v=P + 4), 1),
    (dict(out=None), 1), (dict(out=P + 2), 1), (dict(out=P + 1, out_f32=0), 1), (dict(out_f32=2), 1),
    (dict(lse=None), 1), (dict(lse=P + 2), 1), (dict(do=P + 8), 1), (dict(dq=None), 1), (dict(dq=P + 1), 1),
    (dict(dk=None), 1), (dict(dk=P + 1), 1), (dict(dv=P + 2, dkv_f32=1), 1), (dict(dkv_f32=3), 1),
    (dict(acc=1), 1),                                    # bf16 gradients are not added to
    (dict(acc=2, dkv_f32=1), 1), (dict(ws=None), 1), (dict(ws=P + 16), 1), (dict(ws_bytes=0), 4),
])
def test_read_backward_refusals(m, kw, status):
    assert read(m, layer(m), **kw) == status
    assert m.kvq_last_error()


def test_read_backward_layers(m):
    assert read(m, None) == 1
    assert read(m, layer(m, n_q_heads=6, n_kv_heads=2)) == 2           # ratio 3 does not divide 128
    assert read(m, layer(m, head_dim=96)) == 2
    rotated = layer(m, rot_signs=P)
    assert read(m, rotated) == 2
    assert read(m, layer(m), n_rows=0, max_rows=0) == 0                # nothing to do
    f = m.attn_train_backward_workspace_bytes
    assert f(layer(m, head_dim=96), 1, 4, 4) == 0 and f(layer(m), 0, 4, 4) == 0 and f(layer(m), 1, -1, 1) == 0
    assert f(layer(m), 1, 4, 5) == 0 and f(layer(m), 1, 4, 0) == 0
    need = f(layer(m), 1, 4, 4)
    assert need > 0 and read(m, layer(m), ws_bytes=need - 1) == 4


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 2, 2), (128, 16, 2), (256, 8, 2), (512, 16, 1)])
def test_read_backward_workspace_grows(m, D, n_q, n_kv):
    lay = layer(m, head_dim=D, n_q_heads=n_q, n_kv_heads=n_kv, window=0, rope_dims=0)
    f = m.attn_train_backward_workspace_bytes
    last = 0
    for n in list(range(1, 400)) + [1000, 4097, 20000, 100001, 500001]:
        b = f(lay, 1, n, n)
        assert b >= last
        last = b


def test_read_backward_too_many_tiles(m):
    """Tiles are counted in 32 bits: a pass that may have more is refused, one
    of as many rows in short blocks is not."""
    lay = layer(m, head_dim=512, n_q_heads=16, n_kv_heads=1, window=0, rope_dims=0)
    f = m.attn_train_backward_workspace_bytes
    rows = (1 << 24) - 1
    assert f(lay, 1, rows, rows) == 0
    assert read(m, lay, n_rows=rows, max_rows=rows) == 2 and b"tiles" in m.lib.kvq_last_error()
    assert f(lay, 65535, rows, 300) > 0
    windowed = layer(m, head_dim=512, n_q_heads=16, n_kv_heads=1, window=1024, rope_dims=0)
    assert f(windowed, 1, rows, rows) > 0


def test_lse_refusals(m):
    lay = layer(m)
    L = ctypes.byref(lay)
    f = m.lib.attn_train_forward_lse
    assert f(L, 1, P, 4, 4, P, P, P, P, P, 1, None, None, P, BIG, None) == 1       # lse NULL
    assert f(L, 1, P, 4, 4, P, P, P, P, P, 1, None, P + 2, P, BIG, None) == 1
    assert f(L, 1, P, 4, 4, P, P, P, P, None, 1, None, P, P, BIG, None) == 1       # out NULL
    assert f(L, 1, P, 4, 4, P, P, P, P, P, 1, None, P, P, 0, None) == 4
    assert f(L, 1, P, 0, 0, P, P, P, P, P, 1, None, None, P, BIG, None) == 0
    g = m.lib.attn_train_donor_forward_lse
    assert g(L, 1, P, 4, 4, P, P, P, P, P, P, P, P, 1, None, None, P, BIG, None) == 1
    assert g(L, 1, P, 4, 4, P, P, None, P, P, P, P, P, 1, None, P, P, BIG, None) == 1   # v_raw missing


PREP = dict(n_blocks=1, offs=P, n_rows=4, q=P, q_w=P, dqh=P, dq=P, dqw=P, k=P, v=P, k_w=P, dkh=P, dvh=P, f32=0, dk=P,
            dv=P, dkw=P, ws=P, ws_bytes=BIG)
NO_Q = dict(q=None, q_w=None, dqh=None, dq=None, dqw=None)
NO_KV = dict(k=None, v=None, k_w=None, dkh=None, dvh=None, dk=None, dv=None, dkw=None)


def prep(m, lay, **kw):
    d = dict(PREP)
    d.update(kw)
    return m.lib.kvq_train_prep_backward(ctypes.byref(lay) if lay else None, *d.values(), None)


@pytest.mark.parametrize("kw", [
    dict(n_blocks=0), dict(offs=None), dict(n_rows=-1), dict(f32=2), {**NO_Q, **NO_KV}, {**NO_Q, "dq": P},
    {**NO_KV, "dkw": P}, dict(q=P + 8), dict(q_w=None), dict(q_w=P + 1), dict(dqh=P + 8), dict(dq=P + 2),
    dict(dqw=P + 2), dict(dqw=None), dict(k=P + 8), dict(v=None), dict(v=P + 8), dict(k_w=None), dict(dkh=P + 8),
    dict(dvh=None), dict(dk=P + 8), dict(dv=None), dict(dv=P + 8), dict(dkw=None), dict(ws=None), dict(ws=P + 128),
])
def test_prep_backward_refusals(m, kw):
    assert prep(m, layer(m), **kw) == 1
    assert m.kvq_last_error()


def test_prep_backward_layers(m):
    assert prep(m, None) == 1
    keqv = layer(m, k_eq_v=True)
    assert prep(m, keqv) == 1                                          # v_raw given with K = V
    assert prep(m, keqv, v=None) == 1                                  # dv_raw given
    assert prep(m, layer(m, rot_signs=P)) == 2
    need = m.kvq_train_prep_backward_workspace_bytes(layer(m), 4)
    assert need > 0 and prep(m, layer(m), ws_bytes=need - 1) == 4
    assert prep(m, layer(m), n_rows=0) == 0
    assert prep(m, layer(m), n_rows=0, **NO_KV) == 0
    assert m.kvq_train_prep_backward_workspace_bytes(layer(m, head_dim=96), 4) == 0
    assert m.kvq_train_prep_backward_workspace_bytes(layer(m), -1) == 0
