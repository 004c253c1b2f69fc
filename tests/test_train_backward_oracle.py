"""The oracle's gradients of the training read and of the preps against
central differences of the forward definitions (without their roundings)."""
import numpy as np
import pytest

import oracle as O
import workloads as W

STEP = 1e-5


def spec(n_q, n_kv, D, window):
    return W.LayerSpec(n_q, n_kv, D, window, 0, 1e4, False)


def numeric(f, x):
    """Central differences of the scalar f by every element of x: off from the
    gradient by the third derivative times STEP^2 and by rounding over STEP
    (values of order 1..100: 1e-10 and 1e-9), well inside the 1e-6 asked."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        old = x[i]
        x[i] = old + STEP
        up = f()
        x[i] = old - STEP
        g[i] = (up - f()) / (2 * STEP)
        x[i] = old
    return g


def naive_read(sp, q, k, v, off):
    """The read row by row from the oracle's own visibility rule."""
    out = np.zeros_like(q)
    G = sp.n_q_heads // sp.n_kv_heads
    for r in range(q.shape[0]):
        vis = O.train_visible(off, r, sp.window)
        for h in range(q.shape[1]):
            s = k[vis, h // G] @ q[r, h]
            e = np.exp(s - s.max())
            out[r, h] = (e / e.sum()) @ v[vis, h // G]
    return out


@pytest.mark.parametrize("blocks,window,n_q,n_kv", [([5], 0, 2, 1), ([3, 2, 0, 2], 0, 2, 2), ([4, 3, 1], 3, 4, 2),
                                                    ([0, 3, 2], 2, 1, 1), ([2, 2], 1, 2, 1)])
def test_read_gradient_against_differences(blocks, window, n_q, n_kv):
    rng = np.random.default_rng(11)
    sp, D = spec(n_q, n_kv, 4, window), 4
    off = np.concatenate([[0], np.cumsum(blocks)])
    T = int(off[-1])
    q, k, v = rng.normal(size=(T, n_q, D)), rng.normal(size=(T, n_kv, D)), rng.normal(size=(T, n_kv, D))
    do = rng.normal(size=(T, n_q, D))
    got = O.train_attend_backward(sp, q, k, v, do, off)
    assert np.allclose(got["out"], naive_read(sp, q, k, v, off), atol=1e-12)

    def f():
        return float((naive_read(sp, q, k, v, off) * do).sum())

    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        assert np.abs(got[name] - numeric(f, x)).max() < 1e-6, name
    # a row that sees one key: its dS is 0
    one = [r for r in range(T) if len(O.train_visible(off, r, window)) == 1]
    assert one and np.abs(got["dq"][one]).max() < 1e-14


def test_lse_is_the_log_of_the_summed_exponentials():
    rng = np.random.default_rng(12)
    sp, off = spec(2, 1, 8, 0), [0, 3, 5]
    q, k, v = rng.normal(size=(5, 2, 8)), rng.normal(size=(5, 1, 8)), rng.normal(size=(5, 1, 8))
    got = O.train_attend_backward(sp, q, k, v, q, off)
    for r in range(5):
        vis = O.train_visible(off, r, 0)
        assert np.allclose(got["lse"][r], np.log(np.exp(q[r] @ k[vis, 0].T).sum(axis=1)), atol=1e-12)


@pytest.mark.parametrize("rope_dims", [0, 4, 8])
@pytest.mark.parametrize("weighted", [True, False])
def test_prep_gradient_against_differences(rope_dims, weighted):
    rng = np.random.default_rng(13)
    T, H, D, eps, theta = 3, 2, 8, 1e-3, 1e4
    pos = np.array([0, 7, 100003])
    x, dz = rng.normal(size=(T, H, D)), rng.normal(size=(T, H, D))
    w = 1 + 0.1 * rng.normal(size=D) if weighted else None
    half = rope_dims // 2
    ang = pos[:, None] * O.rope_inv_freq(theta, D, rope_dims)[None, :]

    def f():
        y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
        y = y * w if weighted else y
        z = y.copy()
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        z[..., :half] = y[..., :half] * c - y[..., half:rope_dims] * s
        z[..., half:rope_dims] = y[..., half:rope_dims] * c + y[..., :half] * s
        return float((z * dz).sum())

    dx, dw = O.rms_norm_backward(x, w, O.unrope(dz, pos, theta, rope_dims), eps)
    assert np.abs(dx - numeric(f, x)).max() < 1e-6
    if weighted:
        assert np.abs(dw - numeric(f, w)).max() < 1e-6
    # along x itself only eps counts: x . dx = r (g . x) (1 - r^2 mean(x^2)) = r^3 eps (g . x), g = w dy
    r = 1.0 / np.sqrt((x * x).mean(axis=-1) + eps)
    gx = (O.unrope(dz, pos, theta, rope_dims) * (w if weighted else 1.0) * x).sum(axis=-1)
    assert np.abs((dx * x).sum(axis=-1) - r ** 3 * eps * gx).max() < 1e-12
