"""Calls of the training read's gradients that their documentation allows and
ordinary passes do not make: buffers of more than 2^32 elements, 65535 blocks,
operands aligned to their elements alone, in-place gradients at every head
shape, a bf16 out with the log-sum-exp, captured graphs, event pairs."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from test_gpu_train_backward import PREP_CASES, PrepCase, bits, dense_gradient, f32, offsets, spec

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def status(ws):
    return int(ws[:4].cpu().numpy().view(np.uint32)[0])


def test_offsets_past_32_bits(m):
    """The rows of the last branches lie past 2^32 elements (8 GB) of q, out,
    d_out and their gradients.  There is no prefix, so a branch's gradients are
    those of a pass of its own, but for fp32 sums cut otherwise: one bf16 step,
    2^-7 of a value at most, and where a sum of some 3000 terms cancels 3000 * 2^-24
    of its terms' sizes, which 1e-3 of the largest value holds (a row taken from
    or put to a wrong place is off by values of their own size)."""
    n_q, n_kv, D, window, branch = 64, 4, 512, 64, 2048
    blocks = [0] + [branch] * 67
    T = sum(blocks)
    assert (T - 2 * branch) * n_q * D > 1 << 32
    lay = m.layer(n_q, n_kv, D, window, D, 1e4)
    gen = torch.Generator(device="cuda").manual_seed(71)

    def rows(heads, scale):
        return torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda").normal_(0, scale, generator=gen)

    q, out, do, k, v = rows(n_q, 0.15), rows(n_q, 0.3), rows(n_q, 0.01), rows(n_kv, 1.0), rows(n_kv, 1.0)
    q_w, k_w = (torch.ones(D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = torch.full((T, n_q), 5.0, device="cuda")       # (any finite statistics will do)

    def read(blocks, at):
        n = sum(blocks)
        x = [t[at:at + n] for t in (q, k, v, out, lse, do)]
        got = [torch.zeros_like(t) for t in x[:3]]
        ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), n, branch)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
        m.attn_train_backward(lay, len(blocks), offsets(blocks), n, branch, x[0], x[1], x[2], x[3], 0, x[4], x[5],
                              *got, 0, 0, ws, ws_bytes)
        torch.cuda.synchronize()
        assert status(ws) == 0
        return got

    def prep(blocks, at, dq_hat, dk_hat, dv_hat):
        n = sum(blocks)
        x = [t[at:at + n] for t in (q, k, v)]
        got = [torch.zeros_like(t) for t in x]
        dw = [torch.zeros(D, device="cuda") for _ in range(2)]
        ws_bytes = m.kvq_train_prep_backward_workspace_bytes(lay, n)
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
        m.kvq_train_prep_backward(lay, len(blocks), offsets(blocks), n, x[0], q_w, dq_hat, got[0], dw[0], x[1], x[2],
                                  k_w, dk_hat, dv_hat, False, got[1], got[2], dw[1], ws, ws_bytes)
        torch.cuda.synchronize()
        assert status(ws) == 0
        return got

    whole = read(blocks, 0)
    raw = prep(blocks, 0, *whole)
    for b in (0, 31, 33, 65, 66):                        # the first, either side of 2^31 elements, the last two
        at = b * branch
        own = read([0, branch], at)
        for x, y in zip(whole, own):
            x, y = x[at:at + branch].float(), y.float()
            assert y.abs().max() > 0
            assert bool(((x - y).abs() <= 2.0 ** -7 * y.abs() + 1e-3 * y.abs().max()).all())
        # the preps' rows do not share sums: the same bits from the same gradients
        again = prep([0, branch], at, *(x[at:at + branch].contiguous() for x in whole))
        assert all(torch.equal(x[at:at + branch], y) for x, y in zip(raw, again))


def test_65535_blocks(m):
    """A prefix of 300 rows and the most branches a layout may have, of no or one
    row each but the last (200 rows)."""
    n_branches = 65534
    blocks = np.zeros(n_branches + 1, dtype=np.int64)
    blocks[0], blocks[2::8], blocks[-1] = 300, 1, 200
    blocks = blocks.tolist()
    T, D = sum(blocks), 64
    assert T > 8000
    gen = torch.Generator(device="cuda").manual_seed(72)
    q, k, v, do = ((torch.randn(T, 1, D, generator=gen, device="cuda") * x).bfloat16() for x in (0.4, 1.0, 1.0, 0.01))
    off = np.concatenate([[0], np.cumsum(blocks)])
    see = torch.from_numpy(O.train_mask(off, 0)).cuda()
    want = dense_gradient(*(x.double() for x in (q, k, v, do)), see)
    lay = m.layer(1, 1, D, 0, D, 1e4)
    ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), T, 300)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    got = [torch.empty_like(x) for x in (q, k, v)]
    m.attn_train_backward(lay, len(blocks), offsets(blocks), T, 300, q, k, v, want[3].float(), 1, want[4].float(), do,
                          *got, 0, 0, ws, ws_bytes)
    torch.cuda.synchronize()
    assert status(ws) == 0
    for name, x, w in zip(("dq", "dk", "dv"), got, want):   # (P or dS and the output rounded to bf16)
        assert (x.double() - w).norm() <= 5e-3 * w.norm(), name
    # and the preps, whose rows' positions come from the layout
    c = PrepCase(m, spec(2, 1, D, 0, D), blocks)
    c.run()
    c.verify()


@pytest.mark.parametrize("name", ["d512-keqv-partial", "d256-full-rope", "d64-rope-2", "one-row"])
def test_prep_weights_aligned_to_their_elements(m, name):
    """Norm weights one bf16, their gradients one float past a 16-byte boundary:
    the same bits."""
    sp, blocks, kw = PREP_CASES[name]
    c = PrepCase(m, sp, blocks, **kw)
    c.run()
    want = [t.t.clone() for t in (c.dq, c.dq_w, c.dk, c.dk_w)]
    D = sp.head_dim
    q_w, k_w = (torch.zeros(D + 1, dtype=torch.int16, device="cuda") for _ in range(2))
    q_w[1:], k_w[1:] = bits(c.q_w), bits(c.k_w)
    dw = torch.full((2, D + 4), 77.0, device="cuda")
    kind = f32 if c.kv_f32 else bits
    for t in (c.dq, c.dk):
        t.t.fill_(5)
    m.kvq_train_prep_backward(c.lay, c.n_blocks, c.offs, c.T, bits(c.q), q_w[1:], bits(c.dq_hat), c.dq.t, dw[0, 1:],
                              bits(c.k), None if c.v is None else bits(c.v), k_w[1:], kind(c.dk_hat), kind(c.dv_hat),
                              c.kv_f32, c.dk.t, None if c.dv is None else c.dv.t, dw[1, 1:], c.ws, c.ws_bytes)
    torch.cuda.synchronize()
    assert c.status() == 0
    for x, y in zip((c.dq.t, dw[0, 1:D + 1], c.dk.t, dw[1, 1:D + 1]), want):
        assert torch.equal(x, y)
    assert bool((dw[:, 0] == 77).all()) and bool((dw[:, D + 1:] == 77).all())


@pytest.mark.parametrize("sp,blocks", [(spec(16, 1, 512, 0, 128, 1e6, True), [65, 40]), (spec(4, 2, 512, 0, 512), [50]),
                                       (spec(6, 2, 128, 0, 6), [0, 33, 20]), (spec(2, 2, 64, 0, 0), [40])])
def test_prep_in_place_at_every_head_dim(m, sp, blocks):
    """Gradients of raw rows written over those of the prepped rows (bf16); on a
    K = V layer over the keys'."""
    c = PrepCase(m, sp, blocks)
    c.run()
    dq, dk, dv = bits(c.dq_hat), bits(c.dk_hat), bits(c.dv_hat)
    dq_w, dk_w = torch.empty_like(c.dq_w.t), torch.empty_like(c.dk_w.t)
    m.kvq_train_prep_backward(c.lay, c.n_blocks, c.offs, c.T, bits(c.q), bits(c.q_w), dq, dq, dq_w, bits(c.k),
                              None if c.v is None else bits(c.v), bits(c.k_w), dk, dv, False, dk,
                              None if c.v is None else dv, dk_w, c.ws, c.ws_bytes)
    torch.cuda.synchronize()
    pairs = [(dq, c.dq), (dk, c.dk), (dq_w, c.dq_w), (dk_w, c.dk_w)] + ([] if c.v is None else [(dv, c.dv)])
    assert all(torch.equal(x, y.t) for x, y in pairs)


@pytest.mark.parametrize("sp,blocks", [(spec(8, 2, 256, 64, 256), [130, 60, 77]),
                                       (spec(16, 1, 512, 0, 128, 1e6, True), [90, 30]),
                                       (spec(4, 4, 128, 0, 64), [1])])
def test_whole_step_captured_in_one_graph(m, sp, blocks):
    """Donor forward with the log-sum-exp, read backward and prep backward in one
    graph, replayed on other inputs and twice: the bits of plain calls."""
    from quantized_kv_attention_quant_gb300 import harness
    gen = torch.Generator(device="cuda").manual_seed(73)
    T = int(sum(blocks))

    def case(seed):
        d = (torch.randn(T, sp.n_q_heads, sp.head_dim, generator=gen, device="cuda") * 0.01).bfloat16()
        return harness.TrainGradCase(W.TrainWorkload("graph", seed, sp, blocks), d.view(torch.int16))

    def results(c):
        return [t for t in (c.out, c.lse, c.dq, c.dq_w, c.dk, c.dv, c.dk_w) if t is not None]

    a, b = case(83), case(84)
    b.forward(), b.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in results(b)]
    a.forward(), a.backward()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        a.forward(), a.backward()
    for x, y in ((a.q, b.q), (a.q_w, b.q_w), (a.k, b.k), (a.v, b.v), (a.k_w, b.k_w), (a.d_out, b.d_out)):
        if x is not None:
            x.copy_(y)
    for _ in range(2):
        for t in results(a):
            t.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert a.status_word() == a.grad_status() == 0
        assert all(torch.equal(x, y) for x, y in zip(results(a), want))


@pytest.mark.parametrize("sp,blocks", [(spec(8, 2, 256, 64), [200, 70, 1, 0, 150]), (spec(16, 1, 512), [100, 40])])
def test_lse_with_a_bf16_out(m, sp, blocks):
    """out as bf16: the same bits as without the log-sum-exp, which is the one
    that a call with an fp32 out leaves."""
    from quantized_kv_attention_quant_gb300 import harness
    wl = W.TrainWorkload("lse-bf16", 85, sp, blocks)
    a = harness.TrainCase(wl, out_f32=False, keep_prepped=True)
    a.step()
    b = harness.TrainGradCase(wl, torch.zeros_like(a.q))
    b.forward()
    lse, out = torch.empty_like(b.lse), torch.empty_like(a.out)
    m.attn_train_forward_lse(b.lay, b.n_blocks, b.offs, b.n_rows, b.max_rows, b.q, b.q_w, b.k_hat, b.v_hat, out,
                             False, None, lse, b.ws, b.ws_bytes)
    torch.cuda.synchronize()
    assert torch.equal(out, a.out) and torch.equal(lse, b.lse)
    assert torch.equal(out, b.out.bfloat16().view(torch.int16))


def test_event_pairs_of_the_lse_forwards(m):
    """kvq_profile_next_read: the forwards that keep the log-sum-exp record the
    pair around their attention kernel as the plain ones do."""
    from quantized_kv_attention_quant_gb300 import harness
    sp, blocks = spec(8, 2, 256, 0), [700, 300]
    c = harness.TrainGradCase(W.TrainWorkload("events", 86, sp, blocks), torch.zeros(1000, 8, 256, dtype=torch.int16, device="cuda"))
    c.forward()

    def alone():
        m.attn_train_forward_lse(c.lay, c.n_blocks, c.offs, c.n_rows, c.max_rows, c.q, c.q_w, c.k_hat, c.v_hat, c.out,
                                 True, c.q_prepped, c.lse, c.ws, c.ws_bytes)

    for call in (c.forward, alone):
        k0, k1, c0, c1 = (torch.cuda.Event(enable_timing=True) for _ in range(4))
        k0.record(), k1.record()
        torch.cuda.synchronize()
        c0.record()
        m.kvq_profile_next_read(k0, k1)
        call()
        c1.record()
        torch.cuda.synchronize()
        assert 0 < k0.elapsed_time(k1) <= c0.elapsed_time(c1)
