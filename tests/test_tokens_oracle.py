"""Pins of the oracle of the operators around the experts (oracle/tokens.py), on the CPU: hand-worked cases,
brute force, and gradients against differences."""
import numpy as np
import pytest

from oracle import gating
from oracle import tokens as ox


def test_sort_by_hand():
    """Three tokens with two experts each, experts 1..3 held: expert 1 has slots 1 and 4, expert 2 none, expert 3 slots
    0 and 5; slots 2 (expert 0) and 3 (-1) have no row."""
    row, token, counts = ox.sort_tokens(np.array([[3, 1], [0, -1], [1, 3]]), 3, 1)
    assert row.tolist() == [[2, 0], [-1, -1], [1, 3]]
    assert token.tolist() == [1, 4, 0, 5, -1, -1]
    assert counts.tolist() == [2, 0, 2]
    x = np.array([10, 20, 30])
    assert ox.move(x, token, 2).tolist() == [10, 30, 10, 30, 0, 0]


@pytest.mark.parametrize("T,k,E,first", [(1, 1, 1, 0), (17, 3, 5, 0), (9, 4, 3, 2), (30, 2, 40, -7)])
def test_sort_is_a_stable_sort(T, k, E, first):
    rng = np.random.default_rng(T)
    idx = rng.integers(first - 2, first + E + 2, (T, k))
    row, token, counts = ox.sort_tokens(idx, E, first)
    key = np.where((idx >= first) & (idx < first + E), idx - first, E).reshape(-1)
    order = np.argsort(key, kind="stable")
    n = int((key < E).sum())
    assert np.array_equal(token[:n], order[:n]) and (token[n:] == -1).all()
    assert np.array_equal(counts, np.bincount(key, minlength=E + 1)[:E])
    for a, b in zip((row, token, counts), ox.sort_tokens_at_once(idx, E, first)):
        assert np.array_equal(a, b)
    for i, r in enumerate(row.reshape(-1)):
        assert (r == -1) == (key[i] == E) and (r == -1 or token[r] == i)


def test_sort_does_not_wrap():
    big = np.iinfo(np.int64)
    row, _, counts = ox.sort_tokens(np.array([[big.min, big.max, 5]]), 4, 2)
    assert row.tolist() == [[-1, -1, 0]] and counts.tolist() == [0, 0, 0, 1]


def difference(f, at, step):
    """Central differences of the scalar f at every element of `at`."""
    g = np.zeros(at.shape)
    for i in np.ndindex(at.shape):
        hi, lo = at.copy(), at.copy()
        hi[i] += step
        lo[i] -= step
        g[i] = (f(hi) - f(lo)) / (2 * step)
    return g


@pytest.mark.parametrize("weighted", [False, True])
def test_combine_grad_is_the_difference(weighted):
    rng = np.random.default_rng(2)
    row, token, _ = ox.sort_tokens(np.array([[0, 2], [1, 5], [2, 2]]), 3)
    rows, gy = rng.standard_normal((6, 4)), rng.standard_normal((3, 4))
    w = rng.standard_normal((3, 2)) if weighted else None
    grad_rows, grad_weight, _ = ox.combine_grad(gy, rows, row, w)
    assert np.allclose(difference(lambda v: (ox.combine(v, row, w)[0] * gy).sum(), rows, 1e-3), grad_rows, atol=1e-9)
    if weighted:
        assert np.allclose(difference(lambda v: (ox.combine(rows, row, v)[0] * gy).sum(), w, 1e-3), grad_weight, atol=1e-9)
    # the gradient of the move to expert order is the unweighted way back
    x = rng.standard_normal((3, 4))
    assert np.allclose(difference(lambda v: (ox.move(v, token, 2) * rows).sum(), x, 1e-3), ox.combine(rows, row)[0], atol=1e-9)


@pytest.mark.parametrize("residual", [False, True])
def test_norm_grad_is_the_difference(residual):
    rng = np.random.default_rng(3)
    x, w, gy = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7))
    res, gh = (rng.standard_normal((3, 7)), rng.standard_normal((3, 7))) if residual else (None, None)

    def loss(x, w):
        y, h = ox.add_rms_norm(x, w, res, 0.1)
        return (y * gy).sum() + (0.0 if gh is None else (h * gh).sum())

    h = ox.add_rms_norm(x, w, res, 0.1)[1]
    gx, _, gw, _ = ox.add_rms_norm_grad(gy, h, w, gh, 0.1)
    assert np.allclose(difference(lambda v: loss(v, w), x, 1e-5), gx, atol=1e-8)
    assert np.allclose(difference(lambda v: loss(x, v), w, 1e-5), gw, atol=1e-8)


def test_norm_by_hand():
    y, h = ox.add_rms_norm(np.array([[1.0, 3.0]]), np.array([1.0, 2.0]), np.array([[2.0, 1.0]]), 0.0)
    assert np.allclose(h, [[3, 4]]) and np.allclose(y, np.array([[3, 8]]) / np.sqrt(12.5))


@pytest.mark.parametrize("norm_type", [0, 1, 2])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("out", [False, True])
def test_gating_grad_is_the_difference(norm_type, masked, out):
    rng = np.random.default_rng(4 + norm_type)
    T, e, k = 4, 6, 3
    x, gy = rng.standard_normal((T, e)), rng.standard_normal((T, k))
    go = rng.standard_normal((T, e)) if out else None
    idx = np.array([rng.permutation(e)[:k] for _ in range(T)])
    idx[0, 1] = idx[0, 0]                                  # one expert twice in a row
    bias, extra = rng.random(e), rng.random(e)
    mask = np.array([False, True, False, True]) if masked else None

    def loss(x, bias, extra):
        total = 0.0
        for t in range(T):
            s = gating.normalize(x[t], norm_type) + (extra if masked and mask[t] else bias)
            p = s[idx[t]]
            total += (p / (p.sum() + 0.01) * 2.5 * gy[t]).sum() + (0.0 if go is None else (s * go[t]).sum())
        return total

    gx, _, gb, _, ge, _ = ox.gating_grad(gy, x, idx, bias=bias, additional_bias=extra, mask=mask, grad_out=go, scale=2.5,
                                         eps=0.01, norm_type=norm_type)
    assert np.allclose(difference(lambda v: loss(v, bias, extra), x, 1e-5), gx, atol=1e-7)
    assert np.allclose(difference(lambda v: loss(x, v, extra), bias, 1e-5), gb, atol=1e-7)
    assert np.allclose(difference(lambda v: loss(x, bias, v), extra, 1e-5), ge, atol=1e-7)


def test_e4m3_values_and_ties():
    assert len(ox.E4M3) == 127 and ox.E4M3[-1] == 448 and ox.E4M3[1] == 2.0 ** -9 and ox.E4M3[8] == 2.0 ** -6
    assert ox.nearest(np.array([17.0, 19.0, -17.0, 500.0, 2.0 ** -10, 3 * 2.0 ** -10]), ox.E4M3).tolist() == [
        16, 20, -16, 448, 0, 2 * 2.0 ** -9]
    assert ox.nearest(np.array([0.5, 1.5, 2.5, -2.5, 130.0]), ox.VALUES["int8"]).tolist() == [0, 2, 2, -2, 127]


def test_block_scales():
    y = np.zeros((2, 40))
    y[0, 0], y[0, 35], y[1, 3] = 254.0, -7.0, np.nan
    assert ox.block_scales(y, "int8").tolist()[0] == [2.0] and np.isnan(ox.block_scales(y, "int8")[1]).all()
    assert ox.block_scales(y, "mxfp8")[0].tolist() == [2.0 ** -1, 2.0 ** -6]
    assert np.array_equal(np.isnan(ox.block_scales(y, "mxfp8")), [[False, False], [True, False]])
    assert ox.block_scales(y, "mxfp4")[0].tolist() == [2.0 ** 5, 1.0] and ox.block_scales(y, "mxfp8")[1, 1] == 2.0 ** -127
    assert ox.spread(ox.block_scales(y, "mxfp8"), "mxfp8", 40)[0, 31:33].tolist() == [0.5, 2.0 ** -6]
