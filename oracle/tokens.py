"""CPU oracle of the operators around the experts (numpy, float64) -- TEST INFRASTRUCTURE ONLY.

Only the tests and ``__graft_entry__.smoke()`` may import this module; the CUDA library never uses
it and it uses nothing from the library.

Beside a result most functions give its size: the same formula with every term's magnitude and every
difference made a sum.  Errors of float32 arithmetic are small multiples of 2^-24 of it, however much cancels.
"""
from __future__ import annotations

import numpy as np

from . import experts, gating


def sort_tokens(expert_idx, E, first=0):
    """(row_idx [T, k], token_idx [T k], counts [E]) by walking the experts and, for each, all slots."""
    flat = np.asarray(expert_idx).astype(object).reshape(-1)      # Python integers: no wrap-around
    row_idx, token_idx, counts, at = np.full(flat.size, -1), np.full(flat.size, -1), np.zeros(E, np.int64), 0
    for e in range(E):
        for i, v in enumerate(flat):
            if v - first == e:
                row_idx[i], token_idx[at] = at, i
                counts[e] += 1
                at += 1
    return row_idx.reshape(np.shape(expert_idx)), token_idx, counts


def sort_tokens_at_once(expert_idx, E, first=0):
    """The same for many slots, by a stable sort (the tests hold the two together)."""
    idx = np.asarray(expert_idx)
    key = np.where((idx >= first) & (idx < first + E), idx.astype(np.int64) - first, E).reshape(-1)
    order = np.argsort(key, kind="stable")
    token_idx = np.where(key[order] < E, order, -1)
    row_idx = np.full(key.size, -1)
    row_idx[token_idx[token_idx >= 0]] = np.nonzero(token_idx >= 0)[0]
    return row_idx.reshape(idx.shape), token_idx, np.bincount(key, minlength=E + 1)[:E]


def move(values, token_idx, per=1):
    """The rows of values (one for each slot, or each `per` slots) in the order of token_idx; zeros for -1."""
    values = np.asarray(values)
    out = np.zeros((len(token_idx), *values.shape[1:]), values.dtype)
    for r, i in enumerate(token_idx):
        if i >= 0:
            out[r] = values[i // per]
    return out


def combine(rows, row_idx, weight=None):
    """(y [T, H], size)."""
    T, k = row_idx.shape
    y, size = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= row_idx[t, j] < len(rows):
                term = rows[row_idx[t, j]] * (1.0 if weight is None else weight[t, j])
                y[t] += term
                size[t] += np.abs(term)
    return y, size


def combine_grad(grad_y, rows, row_idx, weight=None):
    """(grad_rows [R, H], grad_weight [T, k], its size)."""
    T, k = row_idx.shape
    grad_rows, grad_weight, size = np.zeros(rows.shape), np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            r = row_idx[t, j]
            if 0 <= r < len(rows):
                grad_rows[r] = grad_y[t] * (1.0 if weight is None else weight[t, j])
                grad_weight[t, j] = grad_y[t] @ rows[r]
                size[t, j] = np.abs(grad_y[t]) @ np.abs(rows[r])
    return grad_rows, grad_weight, size


def add_rms_norm(x, weight, residual=None, eps=1e-6):
    """(y, h)."""
    h = x if residual is None else x + residual
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight, h


def add_rms_norm_grad(grad_y, h, weight, grad_h=None, eps=1e-6):
    """(grad_x, its size, grad_weight, its size)."""
    H = h.shape[1]
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    g = grad_y * weight
    gx = r * g - h * r ** 3 * (g * h).sum(1, keepdims=True) / H
    size = np.abs(r * g) + np.abs(h) * r ** 3 * np.abs(g * h).sum(1, keepdims=True) / H
    if grad_h is not None:
        gx, size = gx + grad_h, size + np.abs(grad_h)
    terms = grad_y * h * r
    return gx, size, terms.sum(0), np.abs(terms).sum(0)


E4M3 = np.array([i * 2.0 ** -9 for i in range(8)]
                + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:119])      # 0 .. 448
BLOCK = {"int8": 0, "e4m3": 0, "e4m3_128": 128, "mxfp8": 32, "mxfp4": 32}     # 0: the whole row
VALUES = {"int8": np.arange(128.0), "e4m3": E4M3, "e4m3_128": E4M3, "mxfp8": E4M3, "mxfp4": experts.MAGNITUDES}


def nearest(v, values):
    """v rounded to +-values (ascending), ties to the even index, larger magnitudes to the largest."""
    a = np.abs(v)
    i = np.clip(np.searchsorted(values, a), 1, len(values) - 1)
    lo, hi = values[i - 1], values[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return np.copysign(np.where(up, hi, lo), v)


def block_scales(y, quant):
    """[T, blocks] scales, NaN where a block holds a NaN or an infinity."""
    T, H = y.shape
    block = BLOCK[quant] or H
    v = np.zeros((T, -(-H // block) * block))
    v[:, :H] = np.abs(y)
    v = v.reshape(T, -1, block)
    bad = ~np.isfinite(v).all(2)
    m = np.where(bad, 0.0, v.max(2, where=np.isfinite(v), initial=0.0))
    if quant.startswith("mx"):
        X = np.where(m == 0, -127, np.maximum(-127, np.frexp(m)[1] - 1 - (8 if quant == "mxfp8" else 2)))
        s = np.ldexp(1.0, X)
    else:
        s = np.maximum(m / VALUES[quant][-1], 2.0 ** -126)
    return np.where(bad, np.nan, s)


def spread(s, quant, H):
    """Block scales [T, blocks] as one for each element [T, H]."""
    return np.repeat(s, BLOCK[quant] or H, axis=1)[:, :H]


def gating_grad(grad_y, x, expert_idx, *, bias=None, additional_bias=None, mask=None, grad_out=None, scale=1.0, eps=1e-20,
                norm_type=0):
    """(grad_x, its size, grad_bias, its size, grad_additional_bias, its size); entries of expert_idx outside
    0 .. e - 1 count as none."""
    T, e = x.shape
    n = gating.normalize(x, norm_type)
    gx, size = np.zeros((T, e)), np.zeros((T, e))
    sums = np.zeros((2, 2, e))
    for t in range(T):
        extra = additional_bias is not None and mask is not None and bool(mask[t])
        b = additional_bias if extra else bias
        s = n[t] + (0.0 if b is None else b)
        js = [j for j in range(expert_idx.shape[1]) if 0 <= expert_idx[t, j] < e]
        P = sum(s[expert_idx[t, j]] for j in js) + eps
        inner = sum(grad_y[t, j] * s[expert_idx[t, j]] for j in js) / P
        inner_size = sum(abs(grad_y[t, j] * s[expert_idx[t, j]]) for j in js) / abs(P)
        ds = np.zeros(e) if grad_out is None else grad_out[t].astype(np.float64).copy()
        ds_size = np.abs(ds)
        for j in js:
            ds[expert_idx[t, j]] += scale / P * (grad_y[t, j] - inner)
            ds_size[expert_idx[t, j]] += abs(scale / P) * (abs(grad_y[t, j]) + inner_size)
        if norm_type == 0:
            gx[t] = n[t] * (ds - ds @ n[t])
            size[t] = n[t] * (ds_size + ds_size @ n[t])
        else:
            slope = 1 / (1 + np.exp(-x[t]))
            if norm_type == 1:
                slope = slope / (1 + np.exp(x[t]))
            gx[t], size[t] = ds * slope, ds_size * slope
        sums[int(extra), 0] += ds
        sums[int(extra), 1] += ds_size
    return gx, size, sums[0, 0], sums[0, 1], sums[1, 0], sums[1, 1]
