"""attn_train_backward, the forward's log-sum-exp and kvq_train_prep_backward
on the GPU against the float64 oracle, within the bounds their roundings
leave: head shapes and layouts from one row to several tiles, windows that
cut into the prefix, rows that see one key, sharp and flat softmaxes, fp32
sums that several layers add to, layouts that break the rules, other streams,
a captured graph, and a donor with its sharer as a training step."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from train_backward_ref import (F32, bf16_normal, close, prep_bounds, prep_gradient, read_bounds, read_gradient,
                                within)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 512             # elements after every output that must stay as they are


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import quantized_kv_attention_quant_gb300 as pkg
    return pkg


def spec(n_q, n_kv, D, window=0, rope_dims=0, theta=1e4, k_eq_v=False):
    return W.LayerSpec(n_q, n_kv, D, window, rope_dims, theta, k_eq_v)


def bits(x):
    return torch.from_numpy(O.f64_to_bf16(x).view(np.int16)).cuda()


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda()


def offsets(blocks):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(blocks)]).astype(np.int32)).cuda()


def values(t):
    if t.dtype == torch.int16:
        return O.bf16_to_f64(t.cpu().numpy().view(np.uint16))
    return t.cpu().numpy().astype(np.float64)


class Out:
    """An output tensor with guard elements behind it."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        self.all = torch.full((n + GUARD,), 77, dtype=dtype, device="cuda")
        self.t = self.all[:n].view(*shape)
        if fill is not None:
            self.t.copy_(fill)

    def untouched(self):
        return bool((self.all == 77).all())

    def check(self):
        assert bool((self.all[self.t.numel():] == 77).all()), "written past its end"
        return values(self.t)


class ReadCase:
    """Random prepped rows; out and lse as fp32 from the oracle."""

    def __init__(self, m, sp, blocks, seed=5, q_scale=None, out_f32=True, dkv_f32=False):
        rng = np.random.default_rng(seed)
        T = int(sum(blocks))
        self.m, self.sp, self.blocks, self.T = m, sp, list(blocks), T
        self.lay = m.layer(sp.n_q_heads, sp.n_kv_heads, sp.head_dim, sp.window, sp.rope_dims, sp.rope_theta,
                           sp.rms_eps, sp.k_eq_v)
        scale = np.linspace(0.1, 1.0, sp.n_q_heads)[None, :, None] if q_scale is None else q_scale
        qs, ks = (T, sp.n_q_heads, sp.head_dim), (T, sp.n_kv_heads, sp.head_dim)
        self.q, self.k, self.v = bf16_normal(rng, qs, scale), bf16_normal(rng, ks), bf16_normal(rng, ks)
        self.do = bf16_normal(rng, qs, 0.01)
        self.want = read_gradient(sp, blocks, self.q, self.k, self.v, self.do)
        self.out_f32, self.dkv_f32 = out_f32, dkv_f32
        self.dev = dict(q=bits(self.q), k=bits(self.k), v=bits(self.v), do=bits(self.do), offs=offsets(blocks),
                        out=f32(self.want["out"]) if out_f32 else bits(O.rn_bf16(self.want["out"])),
                        lse=f32(self.want["lse"]))
        self.max_rows = max(1, max(blocks))
        kind = torch.float32 if dkv_f32 else torch.int16
        self.dq, self.dk, self.dv = Out(qs, torch.int16), Out(ks, kind), Out(ks, kind)
        self.workspace()

    def workspace(self):
        self.ws_bytes = self.m.attn_train_backward_workspace_bytes(self.lay, len(self.blocks), self.T, self.max_rows)
        assert self.ws_bytes > 0
        self.ws = torch.full((self.ws_bytes + GUARD,), 77, dtype=torch.uint8, device="cuda")

    def run(self, accumulate=False, stream=None, dq=None, dk=None, dv=None):
        d = self.dev
        self.m.attn_train_backward(self.lay, len(self.blocks), d["offs"], self.T, self.max_rows, d["q"], d["k"],
                                   d["v"], d["out"], self.out_f32, d["lse"], d["do"],
                                   self.dq.t if dq is None else dq, self.dk.t if dk is None else dk,
                                   self.dv.t if dv is None else dv, self.dkv_f32, accumulate, self.ws,
                                   self.ws_bytes, stream)

    def status(self):
        assert bool((self.ws[self.ws_bytes:] == 77).all()), "the workspace was written past its end"
        return int(self.ws[:4].cpu().numpy().view(np.uint32)[0])

    def verify(self, out_err=0.0, norm=True):
        torch.cuda.synchronize()
        assert self.status() == 0
        bounds = read_bounds(self.q, self.k, self.v, self.do, self.want, out_err=out_err)
        for name, o, b in zip(("dq", "dk", "dv"), (self.dq, self.dk, self.dv), bounds):
            got = o.check()
            within(got, self.want[name], b, not self.dkv_f32 or name == "dq", name)
            if norm and np.linalg.norm(self.want[name]) > 0:
                close(got, self.want[name], name)


READ_CASES = {
    # a prefix shared by ragged branches (an empty one, a one-row one), a window that cuts into the prefix
    "d256-sliding-prefix": (spec(8, 2, 256, 64), [200, 70, 1, 0, 150]),
    # 16 q heads per kv head: 8 rows per 128-row tile
    "d512-g16": (spec(16, 1, 512), [100, 40, 70]),
    "d512-sliding": (spec(16, 1, 512, 96), [150, 130]),
    "d512-mha-two-kv": (spec(4, 4, 512), [130, 3]),
    # one causal block over several key tiles
    "d128-causal": (spec(4, 2, 128), [333]),
    "d128-g8-window-past-the-end": (spec(16, 2, 128, 1000), [64, 64, 63]),
    "d128-window-one-tile": (spec(4, 4, 128, 128), [257, 129]),
    # no prefix: every branch alone
    "d64-g16-no-prefix": (spec(32, 2, 64), [0, 90, 45]),
    "d64-window2": (spec(2, 2, 64, 2), [20, 5]),
    "d256-g1-tile-edges": (spec(2, 2, 256), [128, 129, 127]),
    "d256-g2": (spec(8, 4, 256, 300), [256, 1, 1, 1, 255]),
    "d64-long": (spec(2, 1, 64), [700, 300]),
}


@pytest.mark.parametrize("name", sorted(READ_CASES))
def test_read_backward(m, name):
    sp, blocks = READ_CASES[name]
    c = ReadCase(m, sp, blocks)
    c.run()
    c.verify()


@pytest.mark.parametrize("blocks", [[1], [0, 1], [2], [3, 0, 0], [5, 1, 1, 1], [0, 0, 7]])
@pytest.mark.parametrize("D,n_q,n_kv", [(64, 2, 1), (128, 4, 4), (256, 8, 2), (512, 16, 1)])
def test_read_backward_tiny(m, blocks, D, n_q, n_kv):
    c = ReadCase(m, spec(n_q, n_kv, D), blocks)
    c.run()
    c.verify(norm=False)


@pytest.mark.parametrize("D", [64, 256, 512])
def test_rows_that_see_one_key_have_no_score_gradient(m, D):
    """Window 1: P = 1 and dS = 0 exactly, so dq and dk are 0 and dv is the
    sum of the group's d_out."""
    c = ReadCase(m, spec(4, 2, D, 1), [40, 9])
    c.run()
    c.verify(norm=False)
    assert not c.dq.check().any() and not c.dk.check().any()


@pytest.mark.parametrize("q_scale", [0.0, 0.02, 1.0, 4.0])
def test_read_backward_flat_and_sharp(m, q_scale):
    """From equal scores to rows that see one key almost alone."""
    c = ReadCase(m, spec(4, 2, 256, 0), [150, 60], q_scale=q_scale)
    c.run()
    c.verify(norm=q_scale <= 1.0)


def test_bf16_out(m):
    """out rounded to bf16: delta is off by its rounding."""
    c = ReadCase(m, spec(8, 2, 128), [140, 33], out_f32=False)
    c.run()
    c.verify(out_err=2.0 ** -8, norm=False)


@pytest.mark.parametrize("D,G", [(256, 4), (512, 16), (64, 1)])
def test_fp32_sums_and_accumulate(m, D, G):
    c = ReadCase(m, spec(2 * G, 2, D, 70), [120, 50], dkv_f32=True)
    c.run()
    c.verify()
    first = c.dk.t.clone(), c.dv.t.clone()
    c.run(accumulate=True)
    torch.cuda.synchronize()
    assert c.status() == 0
    # x + x is exact
    assert torch.equal(c.dk.t, 2 * first[0]) and torch.equal(c.dv.t, 2 * first[1])
    c.dk.check(), c.dv.check()


def test_bf16_gradients_are_the_rounded_sums(m):
    a = ReadCase(m, spec(8, 2, 256, 100), [160, 90], dkv_f32=True)
    b = ReadCase(m, spec(8, 2, 256, 100), [160, 90])
    a.run(), b.run()
    torch.cuda.synchronize()
    for x, y in ((a.dk, b.dk), (a.dv, b.dv)):
        assert torch.equal(x.t.bfloat16().view(torch.int16), y.t)
    assert torch.equal(a.dq.t, b.dq.t)


@pytest.mark.parametrize("D,window", [(64, 0), (256, 40)])
def test_hundreds_of_branches(m, D, window):
    """More blocks, tiles and pairs of tiles than the plan keeps on chip; a few
    blocks are empty."""
    c = ReadCase(m, spec(1, 1, D, window), [130] + [1] * 300 + [0] * 7 + [2] * 220 + [257])
    c.run()
    c.verify()


@pytest.mark.parametrize("D,n_q,n_kv,f32_sums", [(64, 4, 2, False), (128, 2, 2, True), (512, 16, 1, True), (256, 8, 2, False)])
def test_outputs_and_out_aligned_to_their_elements(m, D, n_q, n_kv, f32_sums):
    """dq, dk, dv and out one element past a 16-byte boundary: the same bits,
    with and without pieces to join (a sum of one piece, several)."""
    for blocks in ([70, 30], [1100, 300] if D <= 128 else [300, 60]):
        c = ReadCase(m, spec(n_q, n_kv, D, 0), blocks, dkv_f32=f32_sums)
        c.run()
        want = [o.t.clone() for o in (c.dq, c.dk, c.dv)]
        off = []
        for o in (c.dq, c.dk, c.dv):
            n = o.t.numel()
            whole = torch.full((n + 9,), 77, dtype=o.t.dtype, device="cuda")
            off.append((whole, whole[1:1 + n].view(o.t.shape)))
        flat = torch.empty(c.dev["out"].numel() + 1, dtype=c.dev["out"].dtype, device="cuda")
        flat[1:].copy_(c.dev["out"].reshape(-1))
        c.dev["out"] = flat[1:].view(c.dev["out"].shape)
        c.run(dq=off[0][1], dk=off[1][1], dv=off[2][1])
        torch.cuda.synchronize()
        assert c.status() == 0
        for (whole, t), w in zip(off, want):
            assert torch.equal(t, w)
            assert int(whole[0]) == 77 and bool((whole[1 + t.numel():] == 77).all())
        if f32_sums:                                     # x + x is exact
            c.run(accumulate=True, dq=off[0][1], dk=off[1][1], dv=off[2][1])
            torch.cuda.synchronize()
            assert torch.equal(off[1][1], 2 * want[1]) and torch.equal(off[2][1], 2 * want[2])


def test_scores_of_millions_stay_finite(m):
    """Norm weights of 256 allow scores of 10^7, which fp32 holds to steps of 1:
    P = exp(S - lse) is then off by a factor, the gradients stay finite."""
    c = ReadCase(m, spec(4, 2, 512, 0), [90, 40], q_scale=256.0)
    c.dev["k"] = bits(c.k * 256.0)
    s = np.einsum("ihd,jhd->hij", c.q, np.repeat(c.k, 2, axis=1) * 256.0)
    see = O.train_mask(np.array([0, 90, 130]), 0)
    top = np.where(see[None], s, -np.inf).max(2).T       # the log-sum-exp of scores this far apart
    c.dev["lse"] = f32(top)
    c.run()
    torch.cuda.synchronize()
    assert c.status() == 0
    for o in (c.dq, c.dk, c.dv):
        assert np.isfinite(o.check()).all()


def test_same_call_same_bits_and_max_block_rows(m):
    """Twice the same bits, on another stream, and with a looser bound of the
    block rows (another workspace and grid)."""
    c = ReadCase(m, spec(16, 2, 128, 0), [300, 70, 31])
    c.run()
    torch.cuda.synchronize()
    first = [o.t.clone() for o in (c.dq, c.dk, c.dv)]
    side = torch.cuda.Stream()
    for loose in (False, True):
        if loose:
            c.max_rows = c.T
            c.workspace()
        for o in (c.dq, c.dk, c.dv):
            o.t.fill_(5)
        side.wait_stream(torch.cuda.current_stream())
        c.run(stream=side)
        side.synchronize()
        if not loose:
            assert all(torch.equal(x, o.t) for x, o in zip(first, (c.dq, c.dk, c.dv)))
    c.verify()


def test_captured_graph_replays_on_new_inputs(m):
    a = ReadCase(m, spec(8, 2, 256, 100), [160, 90], seed=6)
    b = ReadCase(m, spec(8, 2, 256, 100), [160, 90], seed=7)
    a.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(stream=torch.cuda.current_stream())
    for name in ("q", "k", "v", "do", "out", "lse"):
        a.dev[name].copy_(b.dev[name])
    g.replay()
    b.run()
    torch.cuda.synchronize()
    for x, y in ((a.dq, b.dq), (a.dk, b.dk), (a.dv, b.dv)):
        assert torch.equal(x.t, y.t)


@pytest.mark.parametrize("offs,n_rows,max_rows", [
    ([0, 50, 40], 100, 100),         # block 1 runs backwards
    ([0, 50, 90], 100, 100),         # rows left over
    ([1, 50, 100], 100, 100),        # the prefix does not start at 0
    ([0, 50, 101], 100, 100),        # past the rows
    ([0, -5, 100], 100, 100),
    ([0, 50, 100], 100, 49),         # a block longer than max_block_rows
    ([0, 60, 40, 100], 100, 100),    # a branch that starts inside the prefix
])
def test_bad_layouts_write_nothing(m, offs, n_rows, max_rows):
    sp = spec(4, 2, 128)
    c = ReadCase(m, sp, [n_rows])
    c.blocks = offs[1:]
    c.dev["offs"] = torch.tensor(offs, dtype=torch.int32, device="cuda")
    c.max_rows = max_rows
    c.workspace()
    c.run()
    torch.cuda.synchronize()
    assert c.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert c.dq.untouched() and c.dk.untouched() and c.dv.untouched()
    # the same workspace then serves a valid call
    c.dev["offs"] = torch.tensor([0] + [n_rows] * (len(offs) - 1), dtype=torch.int32, device="cuda")
    c.max_rows = n_rows
    c.workspace()
    c.run()
    c.verify()


def test_two_streams_with_their_own_workspaces(m):
    cases = [ReadCase(m, spec(8, 2, 256, 0), [300, 100], seed=s) for s in (8, 9)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c in cases:
        c.verify()


@pytest.mark.parametrize("D,n_q,n_kv,window,blocks", [(512, 16, 1, 0, [512, 300, 301]), (128, 8, 8, 0, [1501])])
def test_same_bits_beside_another_stream(m, D, n_q, n_kv, window, blocks):
    """CTAs draw their sums' pieces from a counter: with calls on two streams at
    once they draw them in another order each time, and the bits stay."""
    gen = torch.Generator(device="cuda").manual_seed(31)
    T = sum(blocks)
    lay, offs = m.layer(n_q, n_kv, D, window, 0, 1e4), offsets(blocks)
    ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), T, max(blocks))

    def case():
        q, do, out = (torch.randn(T, n_q, D, generator=gen, device="cuda") * x for x in (0.2, 0.01, 0.5))
        k, v = (torch.randn(T, n_kv, D, generator=gen, device="cuda") * x for x in (0.2, 1.0))
        lse = torch.full((T, n_q), 8.0, device="cuda")    # (any finite statistics will do)
        got = [torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (n_q, n_kv, n_kv)]
        return [x.bfloat16() for x in (q, k, v)], out, lse, do.bfloat16(), got, torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")

    def run(c, stream):
        (q, k, v), out, lse, do, got, ws = c
        m.attn_train_backward(lay, len(blocks), offs, T, max(blocks), q, k, v, out, 1, lse, do, *got, 0, 0, ws, ws_bytes,
                              stream)

    cases, streams = [case(), case()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    first = []
    for c in cases:
        run(c, streams[0])
        torch.cuda.synchronize()
        first.append([t.clone() for t in c[4]])
    for _ in range(10):
        for c in cases:
            for t in c[4]:
                t.zero_()
        torch.cuda.synchronize()
        for c, st in zip(cases, streams):
            run(c, st)
        torch.cuda.synchronize()
        for c, f in zip(cases, first):
            assert all(torch.equal(x, y) for x, y in zip(c[4], f))
            assert int(c[5][:4].view(torch.int32)[0]) == 0


@pytest.mark.parametrize("kind", ["sliding", "full"])
def test_read_backward_of_the_stack(m, kind):
    """The 42-layer stack's layer shapes over its training pass (prefix 1024,
    four branches of 256)."""
    sliding, full = W.workload_train_prefix_shared()
    wl = sliding if kind == "sliding" else full
    c = ReadCase(m, wl.layer, wl.blocks)
    c.run()
    c.verify()


# ---------------------------------------------------------------------------
# the forward's log-sum-exp
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["d256-sliding-prefix", "d512-g16", "d128-causal", "d64-g16-no-prefix"])
@pytest.mark.parametrize("donor", [False, True])
def test_forward_lse(m, name, donor):
    from quantized_kv_attention_quant_gb300 import harness
    sp, blocks = READ_CASES[name]
    wl = W.TrainWorkload("lse-" + name, 81, sp, blocks)
    a = harness.TrainCase(wl, keep_prepped=True)
    a.step(fused=donor)
    d_out = torch.zeros_like(a.q)
    b = harness.TrainGradCase(wl, d_out)
    if donor:
        b.forward()
    else:
        b.prep_kv()
        m.attn_train_forward_lse(b.lay, b.n_blocks, b.offs, b.n_rows, b.max_rows, b.q, b.q_w, b.k_hat, b.v_hat,
                                 b.out, True, b.q_prepped, b.lse, b.ws, b.ws_bytes)
    torch.cuda.synchronize()
    assert a.status_word() == b.status_word() == 0
    for x, y in ((a.out, b.out), (a.q_prepped, b.q_prepped), (a.k_hat, b.k_hat), (a.v_hat, b.v_hat)):
        assert torch.equal(x, y)
    q, k = values(b.q_prepped), values(b.k_hat)
    want = read_gradient(sp, blocks, q, k, values(b.v_hat), np.zeros_like(q))["lse"]
    # S within D F32 |q||k|, each exponential within 8 F32 and their sum of T terms within T F32 of itself
    G, D = sp.n_q_heads // sp.n_kv_heads, sp.head_dim
    size = np.stack([(np.abs(q[:, h]) @ np.abs(k[:, h // G]).T).max(1) for h in range(sp.n_q_heads)], 1)
    room = D * F32 * size + (8 + wl.n_rows) * F32 + 4 * F32 * np.abs(want)
    assert (np.abs(b.lse.cpu().numpy() - want) <= room).all()


# ---------------------------------------------------------------------------
# the preps' gradient
# ---------------------------------------------------------------------------

class PrepCase:
    def __init__(self, m, sp, blocks, q_side=True, kv_side=True, kv_f32=False, seed=15, x_scale=1.0):
        rng = np.random.default_rng(seed)
        T, D = int(sum(blocks)), sp.head_dim
        self.m, self.sp, self.T = m, sp, T
        self.off = np.concatenate([[0], np.cumsum(blocks)])
        self.lay = m.layer(sp.n_q_heads, sp.n_kv_heads, D, sp.window, sp.rope_dims, sp.rope_theta, sp.rms_eps,
                           sp.k_eq_v)
        self.offs, self.n_blocks = offsets(blocks), len(blocks)
        self.kv_f32 = kv_f32
        qs, ks = (T, sp.n_q_heads, D), (T, sp.n_kv_heads, D)
        self.q_side, self.kv_side = q_side, kv_side
        if q_side:
            self.q, self.dq_hat = bf16_normal(rng, qs, x_scale), bf16_normal(rng, qs, 0.01)
            self.q_w = bf16_normal(rng, (D,), 0.1) + 1.0
            self.q_w = O.rn_bf16(self.q_w)
            self.dq, self.dq_w = Out(qs, torch.int16), Out((D,), torch.float32)
        if kv_side:
            self.k, self.k_w = bf16_normal(rng, ks, x_scale), O.rn_bf16(1.0 + 0.1 * rng.normal(size=D))
            self.v = None if sp.k_eq_v else bf16_normal(rng, ks, x_scale)
            self.dk_hat, self.dv_hat = bf16_normal(rng, ks, 0.01), bf16_normal(rng, ks, 0.01)
            if kv_f32:
                self.dk_hat = self.dk_hat * np.float32(1.0 / 3.0)
                self.dk_hat = self.dk_hat.astype(np.float32).astype(np.float64)
            self.dk, self.dk_w = Out(ks, torch.int16), Out((D,), torch.float32)
            self.dv = None if sp.k_eq_v else Out(ks, torch.int16)
        self.ws_bytes = m.kvq_train_prep_backward_workspace_bytes(self.lay, T)
        self.ws = torch.full((self.ws_bytes + GUARD,), 77, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        kind = f32 if self.kv_f32 else bits
        q = (bits(self.q), bits(self.q_w), bits(self.dq_hat), self.dq.t, self.dq_w.t) if self.q_side else (None,) * 5
        kv = (None, None, None, None, None, False, None, None, None)
        if self.kv_side:
            kv = (bits(self.k), None if self.v is None else bits(self.v), bits(self.k_w), kind(self.dk_hat),
                  kind(self.dv_hat), self.kv_f32, self.dk.t, None if self.dv is None else self.dv.t, self.dk_w.t)
        self.m.kvq_train_prep_backward(self.lay, self.n_blocks, self.offs, self.T, *q, *kv, self.ws, self.ws_bytes,
                                       stream)
        torch.cuda.synchronize()

    def status(self):
        assert bool((self.ws[self.ws_bytes:] == 77).all())
        return int(self.ws[:4].cpu().numpy().view(np.uint32)[0])

    def verify(self):
        assert self.status() == 0
        sp = self.sp
        if self.q_side:
            dx, dw = prep_gradient(sp, self.off, self.q, self.q_w, self.dq_hat, True)
            bx, bw = prep_bounds(sp, self.q, self.q_w, self.dq_hat, dx)
            within(self.dq.check(), dx, bx, True, "dq")
            within(self.dq_w.check(), dw, bw, False, "dq_w")
        if self.kv_side:
            dk, dkw = prep_gradient(sp, self.off, self.k, self.k_w, self.dk_hat, True)
            bk, bw = prep_bounds(sp, self.k, self.k_w, self.dk_hat, dk)
            x = self.k if sp.k_eq_v else self.v
            dv, _ = prep_gradient(sp, self.off, x, None, self.dv_hat, False)
            bv, _ = prep_bounds(W.LayerSpec(1, 1, sp.head_dim, 0, 0, 1e4, False), x, None, self.dv_hat, dv)
            within(self.dk_w.check(), dkw, bw, False, "dk_w")
            if sp.k_eq_v:
                within(self.dk.check(), dk + dv, bk + bv, True, "dk")
            else:
                within(self.dk.check(), dk, bk, True, "dk")
                within(self.dv.check(), dv, bv, True, "dv")


PREP_CASES = {
    "d256-full-rope": (spec(8, 2, 256, 0, 256), [90, 31, 1, 0, 8], {}),
    "d512-keqv-partial": (spec(16, 1, 512, 0, 128, 1e6, True), [65, 40], dict(kv_f32=True)),
    "d512-full-rope": (spec(4, 2, 512, 0, 512), [50], {}),
    "d512-rope-320": (spec(4, 2, 512, 0, 320), [50], {}),
    "d128-ratio3-odd-pairs": (spec(6, 2, 128, 0, 6), [0, 33, 20], dict(kv_f32=True)),
    "d128-rope-64": (spec(12, 4, 128, 0, 64), [77], {}),
    "d64-no-rope": (spec(2, 2, 64, 0, 0), [40], {}),
    "d64-rope-2": (spec(1, 1, 64, 0, 2), [700, 300], {}),
    "d64-rope-62": (spec(1, 1, 64, 0, 62), [33], dict(kv_f32=True)),
    "d256-sharer": (spec(8, 2, 256, 0, 256), [300, 45], dict(kv_side=False)),
    "d256-keys-alone": (spec(8, 2, 256, 0, 64), [64, 45], dict(q_side=False)),
    "one-row": (spec(8, 2, 256, 0, 256), [1], {}),
    "small-raw-rows": (spec(4, 2, 128, 0, 128), [25], dict(x_scale=2.0 ** -12)),
    "large-raw-rows": (spec(4, 2, 128, 0, 128), [25], dict(x_scale=2.0 ** 20)),
    "many-rows": (spec(2, 1, 64, 0, 64), [11000, 1234], {}),
}


@pytest.mark.parametrize("name", sorted(PREP_CASES))
def test_prep_backward(m, name):
    sp, blocks, kw = PREP_CASES[name]
    c = PrepCase(m, sp, blocks, **kw)
    c.run()
    c.verify()


def test_prep_backward_in_place(m):
    """Gradients written over those they come from."""
    sp, blocks, _ = PREP_CASES["d256-full-rope"]
    c = PrepCase(m, sp, blocks)
    c.run()
    dq, dk, dv = bits(c.dq_hat), bits(c.dk_hat), bits(c.dv_hat)
    dq_w, dk_w = torch.empty_like(c.dq_w.t), torch.empty_like(c.dk_w.t)
    m.kvq_train_prep_backward(c.lay, c.n_blocks, c.offs, c.T, bits(c.q), bits(c.q_w), dq, dq, dq_w, bits(c.k),
                              bits(c.v), bits(c.k_w), dk, dv, False, dk, dv, dk_w, c.ws, c.ws_bytes)
    torch.cuda.synchronize()
    for x, y in ((dq, c.dq), (dk, c.dk), (dv, c.dv), (dq_w, c.dq_w), (dk_w, c.dk_w)):
        assert torch.equal(x, y.t)


def test_prep_backward_bad_layout_writes_nothing(m):
    sp, blocks, _ = PREP_CASES["d256-full-rope"]
    c = PrepCase(m, sp, blocks)
    c.offs = torch.tensor([0, 90, 80, 122, 122, 130], dtype=torch.int32, device="cuda")
    c.run()
    assert c.status() == m.KVQ_STATUS_SEQ_SKIPPED
    assert all(o.untouched() for o in (c.dq, c.dk, c.dv, c.dq_w, c.dk_w))


# ---------------------------------------------------------------------------
# a training step: a donor and the layer that reads its keys and values
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("sp,blocks", [(spec(8, 2, 256, 64, 256), [130, 60, 77]),
                                       (spec(16, 1, 512, 0, 128, 1e6, True), [90, 30])])
def test_training_step_of_donor_and_sharer(m, sp, blocks):
    """The sharer's key and value gradients are added to the donor's, which
    carries the sums through its preps.  The chain's oracle takes the prepped
    rows the GPU wrote (bit-exact by the forward's own tests); the fp32 out
    comes from P rounded to f16, so out is off by 2 * 2^-11 of sum P |v|."""
    from quantized_kv_attention_quant_gb300 import harness
    rng = np.random.default_rng(16)
    T = int(sum(blocks))
    shape = (T, sp.n_q_heads, sp.head_dim)
    do = [bf16_normal(rng, shape, 0.01) for _ in range(2)]
    wl = W.TrainWorkload("grad-step", 82, sp, blocks)
    donor = harness.TrainGradCase(wl, bits(do[0]), layer_id=3, adds=True)
    sharer = harness.TrainGradCase(wl, bits(do[1]), donor_case=donor, layer_id=9)
    for c in (donor, sharer):
        c.forward()
    for c in (sharer, donor):
        c.backward()
    torch.cuda.synchronize()
    assert donor.status_word() == sharer.status_word() == donor.grad_status() == sharer.grad_status() == 0
    k, v = values(donor.k_hat), values(donor.v_hat)
    off = np.concatenate([[0], np.cumsum(blocks)])
    dk, dv = 0.0, 0.0
    for c, d in zip((donor, sharer), do):
        g = read_gradient(sp, blocks, values(c.q_prepped), k, v, d)
        close(values(c.dq_hat), g["dq"], "dq_hat", 8e-3)
        dq, dq_w = prep_gradient(sp, off, values(c.q), values(c.q_w), g["dq"], True)
        close(values(c.dq), dq, "dq", 1e-2)
        close(values(c.dq_w), dq_w, "dq_w", 1e-2)
        dk, dv = dk + g["dk"], dv + g["dv"]
    close(values(donor.dk_hat), dk, "dk_hat", 8e-3)
    close(values(donor.dv_hat), dv, "dv_hat", 8e-3)
    gk, gk_w = prep_gradient(sp, off, values(donor.k), values(donor.k_w), dk, True)
    gv, _ = prep_gradient(sp, off, values(donor.k if sp.k_eq_v else donor.v), None, dv, False)
    close(values(donor.dk_w), gk_w, "dk_w", 1e-2)
    if sp.k_eq_v:
        close(values(donor.dk), gk + gv, "dk", 1e-2)
    else:
        close(values(donor.dk), gk, "dk", 1e-2)
        close(values(donor.dv), gv, "dv", 1e-2)


def test_training_step_of_the_stack_runs(m):
    """Forward and backward pass of all 42 layers: every status word clean,
    every gradient finite, the donors' sums those of their sharers in order."""
    from quantized_kv_attention_quant_gb300 import harness
    gen = torch.Generator(device="cuda").manual_seed(3)

    def d_outs(i, sp, rows):
        t = torch.randn(rows, sp.n_q_heads, sp.head_dim, generator=gen, device="cuda") * 0.01
        return t.bfloat16().view(torch.int16)

    stack = harness.TrainGradStackCase([64, 20, 12], d_outs)
    stack.step()
    torch.cuda.synchronize()
    for c in stack.layers:
        assert c.status_word() == 0 and c.grad_status() == 0
        for t in (c.dq, c.dq_w) + ((c.dk, c.dk_w) if c.donor else ()):
            assert np.isfinite(values(t)).all() and values(t).any()


# ---------------------------------------------------------------------------
# passes whose P and dS tiles do not fit one chunk of the workspace
# ---------------------------------------------------------------------------

def dense_gradient(q, k, v, do, see):
    """The definition in 64 bits on the GPU, head by head: dq, dk, dv, out, lse."""
    G = q.shape[1] // k.shape[1]
    dq, dk, dv, out = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    for h in range(q.shape[1]):
        s = (q[:, h] @ k[:, h // G].T).masked_fill_(~see, -float("inf"))
        lse[:, h] = torch.logsumexp(s, 1)
        p = (s - lse[:, h, None]).exp_()
        dp = do[:, h] @ v[:, h // G].T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        dq[:, h], out[:, h] = ds @ k[:, h // G], p @ v[:, h // G]
        dk[:, h // G] += ds.T @ q[:, h]
        dv[:, h // G] += p.T @ do[:, h]
    return dq, dk, dv, out, lse


@pytest.mark.parametrize("D,n_q,n_kv,window,blocks,f32_sums", [
    (64, 128, 8, 0, [2100], True),                       # one causal block
    (64, 128, 8, 700, [900, 700, 600, 500], False),      # branches, a window into the prefix
    (256, 64, 4, 0, [1500, 40, 1500], True),
])
def test_read_backward_in_several_chunks(m, D, n_q, n_kv, window, blocks, f32_sums):
    """More than 16384 tiles: dk and dv are summed over chunks, accumulated to
    what was there; against the definition in 64 bits (2-norms)."""
    gen = torch.Generator(device="cuda").manual_seed(21)
    T = sum(blocks)

    def rows(heads, scale):
        x = torch.randn(T, heads, D, generator=gen, device="cuda") * scale
        return x.bfloat16()

    q, k, v, do = rows(n_q, 0.4), rows(n_kv, 1.0), rows(n_kv, 1.0), rows(n_q, 0.01)
    see = torch.from_numpy(O.train_mask(np.concatenate([[0], np.cumsum(blocks)]), window)).cuda()
    want = dense_gradient(*(x.double() for x in (q, k, v, do)), see)
    out, lse = want[3].float(), want[4].float()
    lay = m.layer(n_q, n_kv, D, window, 0, 1e4)
    ws_bytes = m.attn_train_backward_workspace_bytes(lay, len(blocks), T, max(blocks))
    assert ws_bytes > (1 << 30)                          # a full chunk: 16384 tiles of 64 KB
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    kind = torch.float32 if f32_sums else torch.bfloat16
    dq = torch.empty_like(q)
    start = torch.randn(2, T, n_kv, D, generator=gen, device="cuda").to(kind) if f32_sums else None
    dk, dv = (start[0].clone(), start[1].clone()) if f32_sums else (torch.empty_like(k), torch.empty_like(v))
    m.attn_train_backward(lay, len(blocks), offsets(blocks), T, max(blocks), q, k, v, out, 1, lse, do, dq, dk, dv,
                          f32_sums, f32_sums, ws, ws_bytes)
    torch.cuda.synchronize()
    assert int(ws[:4].cpu().numpy().view(np.uint32)[0]) == 0
    for name, got, w, s in (("dq", dq, want[0], None), ("dk", dk, want[1], 0), ("dv", dv, want[2], 1)):
        got = got.double() - (start[s].double() if f32_sums and s is not None else 0.0)
        # (the fp32 addition to `start`, of size 1, rounds by 2^-24 of it)
        room = 5e-3 * w.norm() + (2.0 ** -24 * start[s].double().norm() if f32_sums and s is not None else 0.0)
        assert (got - w).norm() <= room, (name, float((got - w).norm() / w.norm()))
