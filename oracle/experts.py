"""CPU oracle of the expert operators (numpy, float64) -- TEST INFRASTRUCTURE ONLY.

Only the tests and ``__graft_entry__.smoke()`` may import this module; the CUDA library never uses
it and it uses nothing from the library.

MXFP4 follows the OCP Microscaling Formats specification, version 1.0: blocks of 32 elements, a
shared scale 2^X with X = floor(log2 max|x|) - 2 held to -127..127, elements rounded to the nearest
of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the code with an even last bit, larger magnitudes to 6).
"""
from __future__ import annotations

import numpy as np

from . import gating

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])


def mx_quantize(x: np.ndarray):
    """(codes [R, K/2] uint8, scales [R, ceil(K/64), 2] uint8) of x [R, K]; codes of a block with a
    NaN or an infinity are 0."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    v = np.zeros((R, 64 * ((K + 63) // 64)))
    v[:, :K] = x
    v = v.reshape(R, -1, 32)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    m = np.abs(v).max(axis=2)
    X = np.where(m == 0, -127, np.maximum(-127, np.frexp(m)[1] - 1 - 2))
    a = np.ldexp(np.abs(v), -X[..., None])
    best, code = np.full(a.shape, np.inf), np.zeros(a.shape, np.uint8)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):                                # even codes first: they keep the ties
        d = np.abs(a - MAGNITUDES[c])
        code, best = np.where(d < best, c, code).astype(np.uint8), np.minimum(d, best)
    code = (code + 8 * (np.signbit(v) & ~bad[..., None])).astype(np.uint8).reshape(R, v.shape[1] * 32)[:, :K]
    scales = np.where(bad, 255, X + 127)
    scales[:, (K + 31) // 32:] = 127
    return code[:, 0::2] | (code[:, 1::2] << 4), scales.astype(np.uint8).reshape(R, v.shape[1] // 2, 2)


def mx_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values [..., K] of codes [..., K/2] with scales [..., ceil(K/64), 2]."""
    codes, s = np.asarray(codes), np.asarray(scales).astype(np.int64)
    K = 2 * codes.shape[-1]
    v = np.empty(codes.shape[:-1] + (K,))
    v[..., 0::2] = VALUES[codes & 15]
    v[..., 1::2] = VALUES[codes >> 4]
    m = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127)).reshape(s.shape[:-2] + (2 * s.shape[-2],))
    return v * np.repeat(m, 32, axis=-1)[..., :K]


def silu(x):
    return x / (1.0 + np.exp(-x))


def sum_error(n: int, squares: np.ndarray) -> np.ndarray:
    """A bound on the error of a sum of n products held in float32, added 16 at a time with each
    addition cut (not rounded) to 24 bits: n / 16 + 32 cuts of at most 2^-23 of a partial sum, which
    stays under 4 times the root of the sum of the squared products (``squares``)."""
    return (n / 16 + 32) * 2.0 ** -23 * 4 * np.sqrt(squares)


def gated(x, w13, I):
    """(h, bound on its float32 sums' effect) of x [R, K] and w13 [2 I, K] in float64."""
    K = x.shape[1]
    y, e = x @ w13.T, sum_error(K, (x * x) @ (w13 * w13).T)
    g, u = y[:, :I], y[:, I:]
    h = silu(g) * u
    # |silu'| <= 1.1; exp and the division cost a few units in the last place of float32
    return h, 1.1 * e[:, :I] * np.abs(u) + np.abs(silu(g)) * e[:, I:] + 2.0 ** -20 * np.abs(h)


def grouped(x, counts, w, *, gate=False, row_weight=None):
    """(y, bound) of expert-major rows x [A, K] (float64 values) and w [E, N or 2 N, K]; the bound
    leaves out the result's own rounding."""
    N = w.shape[1] // (2 if gate else 1)
    y, e, at = np.zeros((x.shape[0], N)), np.zeros((x.shape[0], N)), 0
    for j, c in enumerate(counts):
        rows = slice(at, at + int(c))
        at += int(c)
        if gate:
            y[rows], e[rows] = gated(x[rows], w[j], N)
        else:
            y[rows] = x[rows] @ w[j].T
            e[rows] = sum_error(x.shape[1], (x[rows] ** 2) @ (w[j] ** 2).T)
    if row_weight is not None:
        y, e = y * row_weight[:, None], e * np.abs(row_weight[:, None])
    return y, e + 2.0 ** -22 * np.abs(y)


def routing(x, wr, k, **kw):
    """Oracle gating on float64 logits, and for each token whether its experts stay the same when
    the logits move by as much as float32 sums may move them."""
    logits = x @ wr.T
    e = sum_error(x.shape[1], (x * x) @ (wr * wr).T) + 2.0 ** -21 * np.abs(logits)
    ref = gating.gating_topk(logits, k, **kw)
    sure = np.ones(len(x), bool)
    rng = np.random.default_rng(0)
    for _ in range(6):
        z = logits + 2 * e * rng.choice([-1.0, 1.0], size=e.shape)
        sure &= (gating.gating_topk(z, k, **kw)["expert_idx"] == ref["expert_idx"]).all(axis=1)
    return ref["y_out"], ref["expert_idx"], sure, e.max(axis=1)


def layer(x, weights, experts, weight_error, w13, w2, h_unit):
    """(y [T, H], bound) for the given routing: float64 values throughout, ``h_unit`` the largest
    relative error of rounding h between the products, ``weight_error`` [T] that of the weights.
    The result's own rounding is left out of the bound."""
    T, H = x.shape
    I = w2.shape[2]
    y, var, worst = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    squares = np.zeros((T, H))
    for t in range(T):
        for w, e in zip(weights[t], experts[t]):
            h, eh = gated(x[t:t + 1], w13[e], I)
            y[t] += w * (w2[e] @ h[0])
            # errors of different i are independent: they add up as the root of their squares
            var[t] += w * w * ((w2[e] ** 2) @ (eh[0] + h_unit * np.abs(h[0])) ** 2)
            squares[t] += w * w * ((w2[e] ** 2) @ h[0] ** 2)
            worst[t] += weight_error[t] * abs(w) * np.abs(w2[e] @ h[0])
    return y, 5 * np.sqrt(var) + worst + sum_error(I * len(experts[0]), squares) + 2.0 ** -20 * np.abs(y)
