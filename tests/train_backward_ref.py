"""Expected gradients of the training read and of its preps (float64 oracle),
with the bounds the kernels' roundings leave."""
from __future__ import annotations

import numpy as np

import oracle as O

F16 = 2.0 ** -11        # of an f16 rounding
BF16 = 2.0 ** -8        # half a step of a bf16 rounding, relative to the value
F32 = 2.0 ** -24
TINY = 2.0 ** -126      # the smallest normal float: a smaller P may be taken as 0


def bf16_normal(rng, shape, scale=1.0):
    """bf16 values (as float64) of normal draws."""
    return O.rn_bf16(rng.normal(size=shape) * scale)


def read_bounds(q, k, v, do, g, out_err=0.0, lse_err=0.0):
    """Element-wise bounds of |dq|, |dk|, |dv| errors before the output's own
    rounding, for the gradient `g` of train_attend_backward.

    Per score: the fp32 products of a row sum D terms, each partial sum within
    F32 of its size, so S is off by at most D F32 |q||k| (likewise dP, and
    delta with out off by out_err); lse by F32 |lse| + lse_err; the exponential
    by 4 F32 of itself.  P and dS each enter a product rounded to bf16; a sum
    of n products in fp32 adds n F32 of the sum of their sizes.  P below the
    smallest normal float, TINY, may be flushed to 0 by the exponential: P is
    off by TINY at most beside the relative errors, dS by TINY (|dP| + |delta|).
    For dS, P is rounded to f16 times 2^15 first: off by F16 of itself, or by
    half the smallest f16 step, 2^-25, over 2^15 where it is subnormal there
    (2^-40, which holds TINY too)."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    aq, ak, av, ado, aout = (np.abs(x) for x in (q, k, v, do, g["out"]))
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for kvh in range(Hkv):
        for i in range(G):
            h = kvh * G + i
            p, ds = g["p"][kvh][:, i], np.abs(g["ds"][kvh][:, i])
            e_p = D * F32 * (aq[:, h] @ ak[:, kvh].T) + (F32 * np.abs(g["lse"][:, h]) + lse_err)[:, None] + 4 * F32
            e_dp = D * F32 * (ado[:, h] @ av[:, kvh].T)
            e_delta = D * F32 * (ado[:, h] * aout[:, h]).sum(1) + (ado[:, h] * out_err * aout[:, h]).sum(1)
            size = ado[:, h] @ av[:, kvh].T + (ado[:, h] * aout[:, h]).sum(1)[:, None]     # >= |dP| + |delta|
            e_ds = ds * (BF16 + F16 + e_p) + 2.0 ** -40 * (p > 0) * size + p * (1 + BF16 + F16 + e_p) * (e_dp + e_delta[:, None])
            one = (p > 0).sum(1) == 1                       # one visible key: dS is 0
            e_ds[one] = 0.0
            n = T * G * F32
            bq[:, h] = (e_ds + n * ds) @ ak[:, kvh]
            bk[:, kvh] += (e_ds + n * ds).T @ aq[:, h]
            bv[:, kvh] += (p * (BF16 + e_p + n) + TINY * (p > 0)).T @ ado[:, h]
    return bq, bk, bv


def within(got, want, bound, bf16_out=True, what=""):
    """|got - want| <= bound, plus the output's own rounding."""
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == want.shape, what
    assert np.isfinite(got).all(), (what, "not finite")
    room = bound + (BF16 if bf16_out else F32) * (np.abs(want) + bound) + 1e-38
    off = np.abs(got - want) - room
    assert (off <= 0).all(), (what, float(np.max(np.abs(got - want))), float(np.max(np.abs(got - want) / room)),
                              np.unravel_index(int(np.argmax(off)), off.shape))


def close(got, want, what="", most=5e-3):
    """2-norm of the error against the result's.  P (or dS) and the output are
    each rounded to bf16, errors uniform within half a step and unrelated to
    the values: each is BF16 / sqrt(3) = 2.3e-3 of a value at most in the root
    mean square, the two together 3.2e-3; 5e-3 leaves room for few samples."""
    got = np.asarray(got, dtype=np.float64)
    size = np.linalg.norm(want)
    off = np.linalg.norm(got - want)
    assert off <= most * size, (what, float(off / max(size, 1e-300)))


def read_gradient(spec, blocks, q, k, v, do):
    off = np.concatenate([[0], np.cumsum(blocks)])
    return O.train_attend_backward(spec, q, k, v, do, off)


def prep_gradient(spec, off, x, w, dz, rotated):
    """(dx, dw) of a prepped row's raw values; F32-accurate kernels."""
    _, pos = O.layout_positions(off)
    dy = O.unrope(dz, pos, spec.rope_theta, spec.rope_dims) if rotated else np.asarray(dz, dtype=np.float64)
    return O.rms_norm_backward(x, w, dy, float(np.float32(spec.rms_eps)))


def prep_bounds(spec, x, w, dz, dx):
    """Bounds of dx and dw before the output's rounding: fp32 arithmetic with
    sums of D terms; the rotation's cosine and sine within 4 F32 of 1, so a
    rotated dim within 8 F32 of its pair's size; the norm's r within D F32."""
    D = x.shape[-1]
    R = spec.rope_dims
    az = np.abs(dz)
    pair = az.copy()
    if R:
        both = az[..., :R // 2] + az[..., R // 2:R]
        pair[..., :R // 2], pair[..., R // 2:R] = both, both
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(spec.rms_eps)))
    aw = np.ones(D) if w is None else np.abs(w)
    g = aw * pair
    e = (D + 16) * F32
    bx = e * (r * g + np.abs(x) * r ** 3 * (g * np.abs(x)).mean(-1, keepdims=True)) * 2
    n = x.shape[0] * x.shape[1] * F32
    bw = ((2 * e + n) * pair * np.abs(x) * r).sum((0, 1))
    return bx, bw
