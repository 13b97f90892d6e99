"""The operators around the experts on the GPU against the float64 oracle (oracle/tokens.py).

What is moved must be equal.  What is computed is held to a bound on float32 arithmetic, n * 2^-24 of the
oracle's size of the result (the same formula on magnitudes, so whatever cancels), plus the result's own rounding: at most
half a step, 2^-8 for bfloat16, 2^-11 for float16, 2^-24 for float32, and half of the least subnormal.  n is
the length of the longest chain of additions plus a few products and functions of at most 2 units each: a sum over a
row of H elements is cut among 64 partial sums or more, one over T rows among 64 or more where T is above 64.
"""
import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from moe_expert_token_gb300 import tokens as tk
from oracle import experts as oe
from oracle import tokens as ox
from test_experts_gpu import LEAST, UNIT, down, up

pytestmark = pytest.mark.gpu

FLOATS = ["float16", "bfloat16", "float32"]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


def row_ops(n):
    """The n of the module's bound for a sum over a row of n elements."""
    return n / 64 + 40


def close(got, ref, size, ops, dt):
    """got (a tensor of dtype name dt) within ops * 2^-24 * size and its own rounding of ref, where ref is finite."""
    g = down(got)
    assert g.shape == ref.shape
    fine = np.isfinite(ref)
    assert np.array_equal(np.isfinite(g), fine) and np.array_equal(np.isnan(g), np.isnan(ref))
    err = ops * 2.0 ** -24 * size
    room = (err * (1 + UNIT[dt]) + UNIT[dt] * np.abs(ref) + LEAST[dt])[fine]
    off = np.abs(g - ref)[fine]
    assert np.all(off <= room), f"{np.max(off / room)} times the bound"


def offset(t, n):
    """A copy of the tensor that starts n elements into an allocation."""
    import torch

    flat = torch.zeros(t.numel() + n, dtype=t.dtype, device="cuda")
    flat[n:] = t.reshape(-1)
    return flat[n:].view(t.shape)


def ints(a, dtype):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).to(getattr(torch, dtype)).cuda()


# ----------------------------------------------------------------------------- sort

def check_sort(x, idx, E, first=0, scales=None, weight=None, kind="int32", cumsum=False, **kw):
    """moe_sort_tokens against the oracle, bit for bit; x, scales, weight: device tensors, idx: numpy [T, k]."""
    import torch

    T, k = idx.shape
    row, token, counts = ox.sort_tokens_at_once(idx, E, first)
    got = moe.moe_sort_tokens(x, ints(idx, kind), E, first_expert=first, per_token_scales=scales, expert_topk_weight=weight,
                              expert_token_num_type=0 if cumsum else 1, **kw)
    sx, ss, gt, gr, num, sw = got
    assert num.dtype == getattr(torch, kind) and gt.dtype == gr.dtype == torch.int32
    assert np.array_equal(num.cpu().numpy(), np.cumsum(counts) if cumsum else counts)
    assert np.array_equal(gr.cpu().numpy(), row)
    assert np.array_equal(gt.cpu().numpy(), token)
    at = torch.from_numpy(token).cuda()
    used, at = at >= 0, at.clamp(min=0)

    def moved(src, to):
        bits = lambda t: t.contiguous().view(torch.uint8).reshape(t.shape[0], -1)  # noqa: E731
        want = bits(src)[to] * used[:, None].to(torch.uint8)
        return torch.equal(bits(got_rows), want)

    got_rows = sx
    assert sx.dtype == x.dtype and moved(x, torch.div(at, k, rounding_mode="floor"))
    if scales is None:
        assert ss is None
    else:
        got_rows = ss
        assert ss.shape == (T * k, *scales.shape[1:]) and moved(scales, torch.div(at, k, rounding_mode="floor"))
    if weight is None:
        assert sw is None
    else:
        assert sw.shape == (T * k, 1)
        got_rows = sw
        assert moved(weight.float().reshape(-1, 1), at)
    return got


def experts(rng, T, k, E, wrong=0.0):
    idx = rng.integers(0, E, (T, k))
    if wrong:
        idx = np.where(rng.random((T, k)) < wrong, rng.choice([-1, -2 ** 31, E, 2 ** 31 - 1], (T, k)), idx)
    return idx


# few and many slots (4096 is the most that one launch takes), experts from 1 to 4096, k to 64
SORTS = [(1, 1, 1, 8), (1, 8, 256, 7168), (3, 2, 4, 33), (5, 64, 70, 16), (64, 64, 4096, 20), (512, 8, 256, 40), (4096, 1, 3, 12),
         (4097, 1, 5, 18), (513, 8, 256, 100), (65, 64, 4096, 6), (2000, 6, 60, 130), (30000, 4, 17, 8)]


@pytest.mark.parametrize("T,k,E,H", SORTS)
@pytest.mark.parametrize("dt,kind", [("bfloat16", "int32"), ("int8", "int64")])
def test_sort(T, k, E, H, dt, kind):
    import torch

    rng = np.random.default_rng(T + E)
    x = torch.from_numpy(rng.integers(-128, 128, (T, H))).to(getattr(torch, dt)).cuda()
    scales = up(rng.random(T), "float32") if dt == "int8" else None
    check_sort(x, experts(rng, T, k, E), E, scales=scales, weight=up(rng.random((T, k)), "float32"), kind=kind)


@pytest.mark.parametrize("T,k,E,H", [(1, 4, 3, 64), (40, 3, 9, 50), (3000, 3, 9, 50), (1500, 8, 300, 96)])
@pytest.mark.parametrize("kind", ["int32", "int64"])
@pytest.mark.parametrize("cumsum", [False, True])
def test_sort_slots_without_rows(T, k, E, H, kind, cumsum):
    """Padded tokens, experts held elsewhere, the integer types' extremes: rows of zeros behind the others."""
    rng = np.random.default_rng(T)
    idx = experts(rng, T, k, E, wrong=0.4)
    idx[T // 2:T // 2 + 3] = -1
    for first, held in ((0, E), (E // 3, max(1, E // 3)), (E, 5)):
        check_sort(up(rng.standard_normal((T, H)), "float16"), idx, held, first,
                   scales=up(rng.integers(0, 255, (T, (H + 63) // 64, 2)).astype(np.uint8)),
                   weight=up(rng.random((T, k)), "bfloat16"), kind=kind, cumsum=cumsum)


def test_sort_wide_integers():
    """int64 experts whose low half alone would be held, and a first expert near the type's end."""
    idx = np.array([[1 << 32, 2, -(1 << 63)], [(1 << 63) - 1, (1 << 32) + 2, 1]])
    x = up(np.arange(8.0).reshape(2, 4), "float32")
    check_sort(x, idx, 4, kind="int64")
    first = (1 << 63) - 4097
    check_sort(x, np.array([[first, first + 4], [first - 1, -(1 << 63)]]), 5, first, kind="int64")
    with pytest.raises(ValueError):
        moe.moe_sort_tokens(x, ints(idx, "int64"), 4, first_expert=1 << 63)


@pytest.mark.parametrize("T", [300, 9000])
def test_sort_one_expert_and_none(T):
    rng = np.random.default_rng(T)
    x = up(rng.standard_normal((T, 24)), "bfloat16")
    check_sort(x, np.full((T, 2), 6), 8)
    check_sort(x, np.full((T, 2), -1), 8)
    check_sort(x, np.repeat(np.arange(T)[::-1, None] % 8, 2, axis=1), 8, cumsum=True)


@pytest.mark.parametrize("T", [5, 2500])
@pytest.mark.parametrize("off", [0, 1, 2, 4, 8])
def test_sort_strides_and_alignment(T, off):
    """Rows that begin at any byte, with gaps between them, and scales beside every alignment."""
    import torch

    rng = np.random.default_rng(off)
    idx = experts(rng, T, 3, 7, wrong=0.1)
    for H in (48, 37):
        x = offset(torch.from_numpy(rng.integers(0, 256, (T, 64)).astype(np.uint8)).cuda(), off)[:, 5:5 + H]
        for cols in (3, 4, 224):
            scales = offset(torch.from_numpy(rng.integers(0, 256, (T, cols)).astype(np.uint8)).cuda(), off)
            check_sort(x, idx, 7, scales=scales)
    check_sort(offset(up(rng.standard_normal((T, 96)), "bfloat16"), off), idx, 7, weight=offset(up(rng.random((T, 3)), "float16"), off))


def test_sort_empty():
    import torch

    x = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    for cumsum in (0, 1):
        got = moe.moe_sort_tokens(x, torch.empty((0, 2), dtype=torch.int64, device="cuda"), 3, expert_token_num_type=cumsum)
        assert got[0].shape == (0, 16) and got[4].tolist() == [0, 0, 0]


def test_sort_indices_only():
    """The C entry without rows."""
    import torch

    rng = np.random.default_rng(0)
    for T in (7, 5000):
        idx = experts(rng, T, 2, 5)
        e, token, row = ints(idx, "int32"), torch.empty(2 * T, dtype=torch.int32, device="cuda"), torch.empty(2 * T, dtype=torch.int32, device="cuda")
        num = torch.empty(5, dtype=torch.int32, device="cuda")
        n = moe.moe_sort_workspace(T, 2, 5)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        st = moe.moe_sort_run(e.data_ptr(), 0, T, 2, 0, 5, None, 0, 0, None, 0, None, 0, None, None, None, token.data_ptr(),
                              row.data_ptr(), num.data_ptr(), 1, ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
        assert st == m.MRR_OK
        want = ox.sort_tokens_at_once(idx, 5)
        assert np.array_equal(row.cpu().numpy().reshape(T, 2), want[0]) and np.array_equal(token.cpu().numpy(), want[1])
        assert np.array_equal(num.cpu().numpy(), want[2])


def test_sort_past_32_bits():
    """More than 2^32 bytes of rows."""
    import torch

    T, k, H = 70000, 8, 8192
    x = torch.zeros((T, H), dtype=torch.uint8, device="cuda")
    mark = torch.arange(T, device="cuda")
    x[:, 0], x[:, 1], x[:, H - 1] = mark % 251, mark // 251 % 251, mark % 13
    idx = np.random.default_rng(1).integers(0, 40, (T, k))
    rows, _, token, row, _, _ = moe.moe_sort_tokens(x, ints(idx, "int32"), 40)
    assert np.array_equal(row.cpu().numpy(), ox.sort_tokens_at_once(idx, 40)[0])
    t = torch.div(token.long(), k, rounding_mode="floor")
    for c in (0, 1, H - 1):
        assert torch.equal(rows[:, c], x[t, c])


# ----------------------------------------------------------------------------- combine

def combine_case(rng, T, k, R, H, dt, weight_dt, wrong=0.2):
    row = rng.permutation(max(R, T * k))[:T * k].reshape(T, k)       # no row twice
    row = np.where(rng.random((T, k)) < wrong, -1, row)
    rows = up(rng.standard_normal((R, H)), dt)
    w = None if weight_dt is None else up(rng.standard_normal((T, k)), weight_dt)
    return rows, row, w


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 7168), (3, 2, 33), (7, 9, 130), (2, 64, 24), (40, 33, 10), (130, 4, 264), (600, 6, 2050)])
@pytest.mark.parametrize("dt", FLOATS)
@pytest.mark.parametrize("weight_dt", [None, *FLOATS])
def test_combine(T, k, H, dt, weight_dt):
    rng = np.random.default_rng(T * H + k)
    R = T * k - (T * k) // 3
    rows, row, w = combine_case(rng, T, k, R, H, dt, weight_dt)      # some rows are past R
    row[T // 2] = -1
    y = moe.moe_combine_tokens(rows, ints(row, "int32"), w)
    ref, size = ox.combine(down(rows), row, None if w is None else down(w))
    close(y, ref, size, k + 2, dt)
    assert not np.any(down(y)[T // 2])
    if w is None:
        import torch

        assert torch.equal(moe.moe_sort_tokens_grad(rows, ints(row, "int32")), y)


def test_combine_leaves_out_what_has_no_row():
    """Weights of slots without a row, and rows that no slot names, hold NaN: neither shows."""
    import torch

    rows = torch.full((9, 40), float("nan"), dtype=torch.bfloat16, device="cuda")
    rows[2], rows[5] = 1.0, 2.0
    row = np.array([[2, -1, 5], [-1, -5, 9], [100, 5, -2 ** 31]])
    w = torch.tensor([[0.5, float("nan"), 2.0], [float("nan")] * 3, [float("inf"), 1.0, float("nan")]], device="cuda")
    y = moe.moe_combine_tokens(rows, ints(row, "int32"), w)
    assert torch.equal(y[:, 0].float().cpu(), torch.tensor([4.5, 0.0, 2.0])) and bool((y == y[:, :1]).all())
    row = np.array([[2, -1, 5], [-1, -5, 9], [100, -1, -2 ** 31]])
    grad, gw = moe.moe_combine_tokens_grad(torch.ones(3, 40, dtype=torch.bfloat16, device="cuda"), rows, ints(row, "int32"),
                                           ints(np.array([-1, -1, 0, -1, -1, 2, -1, -1, -1]), "int32"), w)
    assert gw[0].tolist() == [40.0, 0.0, 80.0] and not gw[1:].any()
    assert grad[2, 0] == 0.5 and grad[5, 0] == 2.0 and not grad[[0, 1, 3, 4, 6, 7, 8]].any()


def test_combine_infinities_follow_the_formula():
    import torch

    rows = up(np.array([[1.0, np.inf], [2.0, -np.inf], [np.nan, 3.0]]), "float32")
    y = moe.moe_combine_tokens(rows, ints(np.array([[0, 1], [2, -1], [0, 0]]), "int32"))
    want = torch.tensor([[3.0, float("nan")], [float("nan"), 3.0], [2.0, float("inf")]])
    assert torch.equal(torch.nan_to_num(y.cpu(), 7.0), torch.nan_to_num(want, 7.0))


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_combine_alignment(off, dt):
    import torch

    rng = np.random.default_rng(off)
    rows, row, w = combine_case(rng, 9, 4, 36, 264, dt, "float32")
    idx = ints(row, "int32")
    token = ints(ox_token(row, 36), "int32")
    gy = up(rng.standard_normal((9, 264)), dt)
    want, (grows, gw) = moe.moe_combine_tokens(rows, idx, w), moe.moe_combine_tokens_grad(gy, rows, idx, token, w)
    assert torch.equal(moe.moe_combine_tokens(offset(rows, off), offset(idx, 1), offset(w, 1)), want)
    a, b = moe.moe_combine_tokens_grad(offset(gy, off), offset(rows, off), offset(idx, 1), offset(token, 3), offset(w, 1))
    assert torch.equal(a, grows)
    ref, size = ox.combine_grad(down(gy), down(rows), row, down(w))[1:]
    close(b, ref, size, row_ops(264), "float32")


def ox_token(row, R):
    """token_idx [R] of row_idx [T, k]."""
    token = np.full(R, -1)
    for i, r in enumerate(row.reshape(-1)):
        if 0 <= r < R:
            token[r] = i
    return token


@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 7168), (3, 2, 33), (7, 9, 130), (2, 64, 24), (40, 33, 10), (130, 4, 264), (300, 6, 2050)])
@pytest.mark.parametrize("dt", FLOATS)
@pytest.mark.parametrize("weight_dt", [None, *FLOATS])
def test_combine_grad(T, k, H, dt, weight_dt):
    rng = np.random.default_rng(T * H + k)
    R = T * k + 5
    rows, row, w = combine_case(rng, T, k, R, H, dt, weight_dt)
    gy = up(rng.standard_normal((T, H)), dt)
    grows, gw = moe.moe_combine_tokens_grad(gy, rows, ints(row, "int32"), ints(ox_token(row, R), "int32"), w)
    ref_rows, ref_w, size = ox.combine_grad(down(gy), down(rows), row, None if w is None else down(w))
    close(grows, ref_rows, np.abs(ref_rows), 2, dt)
    if w is None:
        assert gw is None
    else:
        close(gw, ref_w, size, row_ops(H), weight_dt)


def test_combine_empty():
    import torch

    rows = torch.ones((4, 24), device="cuda")
    y = moe.moe_combine_tokens(rows, torch.empty((0, 3), dtype=torch.int32, device="cuda"))
    assert y.shape == (0, 24)
    none = torch.empty((0, 24), device="cuda")
    y = moe.moe_combine_tokens(none, ints(np.zeros((2, 3)), "int32"), torch.ones((2, 3), device="cuda"))
    assert y.shape == (2, 24) and not y.any()
    grows, gw = moe.moe_combine_tokens_grad(none, rows, torch.empty((0, 3), dtype=torch.int32, device="cuda"),
                                            ints(np.full(4, -1), "int32"), torch.empty((0, 3), device="cuda"))
    assert not grows.any() and gw.shape == (0, 3)


def test_combine_past_32_bits():
    import torch

    R, H, k = 270000, 8192, 8                                       # 2^31 elements and more
    rows = torch.zeros((R, H), dtype=torch.bfloat16, device="cuda")
    row = np.stack([R - 1 - np.arange(k * 3).reshape(3, k), np.arange(k * 3).reshape(3, k)]).reshape(6, k)
    v = up(np.random.default_rng(0).standard_normal((6, k, H)), "bfloat16")
    rows[torch.from_numpy(row).cuda()] = v
    y = moe.moe_combine_tokens(rows, ints(row, "int32"))
    close(y, down(v).sum(1), np.abs(down(v)).sum(1), k + 2, "bfloat16")
    token = torch.full((R,), -1, dtype=torch.int32, device="cuda")
    token[torch.from_numpy(row).cuda().reshape(-1)] = torch.arange(6 * k, dtype=torch.int32, device="cuda")
    w = torch.full((6, k), 2.0, device="cuda")
    grows, gw = moe.moe_combine_tokens_grad(v[:, 0].contiguous(), rows, ints(row, "int32"), token, w)
    assert torch.equal(grows[row[0, 3]], 2 * v[0, 0]) and torch.equal(grows[row[5, 0]], 2 * v[5, 0])
    assert int((grows != 0).any(1).sum()) == 6 * k
    terms = down(v) * down(v[:, :1])
    close(gw, terms.sum(2), np.abs(terms).sum(2), row_ops(H), "float32")


# ----------------------------------------------------------------------------- norm

NORMS = [(1, 1), (1, 2), (3, 8), (2, 31), (5, 250), (4, 256), (9, 264), (3, 1000), (3, 1026), (1, 7168), (2, 2050), (310, 2048),
         (305, 1998), (1, 8200), (2, 20000), (307, 4104), (2, 65536), (1, 40001)]


def norm_inputs(T, H, dt, weight_dt, residual, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H)) * np.exp2(rng.integers(-3, 4, (T, 1)))
    res = up(rng.standard_normal((T, H)), dt) if residual else None
    return rng, up(x, dt), up(1 + 0.2 * rng.standard_normal(H), weight_dt or dt), res


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dt,weight_dt", [("float16", None), ("bfloat16", None), ("float32", None), ("bfloat16", "float32"),
                                          ("float16", "float32")])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(T, H, dt, weight_dt, residual):
    rng, x, w, res = norm_inputs(T, H, dt, weight_dt, residual, H)
    y, h, q, s = moe.moe_add_rms_norm(x, w, res, eps=1e-5)
    assert q is None and s is None
    ry, rh = ox.add_rms_norm(down(x), down(w), None if res is None else down(res), 1e-5)
    # relative to |x| + |residual| in h, as the sum may cancel; y's elements are multiples of it
    size = np.abs(down(x)) + (0 if res is None else np.abs(down(res)))
    scale = np.abs(ry) / np.where(rh == 0, 1, np.abs(rh))
    close(y, ry, np.abs(ry) * row_ops(H) + size * scale, 1, dt)
    if residual:
        close(h, rh, size, 1, dt)
    else:
        assert h is x


@pytest.mark.parametrize("T,H", NORMS)
@pytest.mark.parametrize("dt,weight_dt", [("float16", None), ("bfloat16", "float32"), ("float32", None)])
@pytest.mark.parametrize("through", [False, True])
def test_norm_grad(T, H, dt, weight_dt, through):
    rng, h, w, gh = norm_inputs(T, H, dt, weight_dt, through, H + 1)
    gy = up(rng.standard_normal((T, H)), dt)
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=gh, eps=1e-5)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w), None if gh is None else down(gh), 1e-5)
    close(gx, rx, sx, row_ops(H), dt)
    close(gw, rw, sw, row_ops(H) + T / 64 + 60, weight_dt or dt)


@pytest.mark.parametrize("H", [64, 4096])
def test_norm_grad_of_many_rows(H):
    T = 3001
    rng, h, w, gh = norm_inputs(T, H, "bfloat16", "float32", True, H)
    gy = up(rng.standard_normal((T, H)), "bfloat16")
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=gh)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w), down(gh))
    close(gx, rx, sx, row_ops(H), "bfloat16")
    close(gw, rw, sw, row_ops(H) + T / 64 + 60, "float32")


def test_norm_grad_is_the_difference():
    """Along a random direction, against the forward pass itself in float32."""
    import torch

    rng, x, w, res = norm_inputs(40, 600, "float32", None, True, 5)
    gy, gh, d = (up(rng.standard_normal((40, 600)), "float32") for _ in range(3))
    dw = up(rng.standard_normal(600), "float32")

    def loss(step):
        y, h, _, _ = moe.moe_add_rms_norm(x + step * d, w + step * dw, res)
        return float((y.double() * gy.double()).sum() + (h.double() * gh.double()).sum())

    h = moe.moe_add_rms_norm(x, w, res)[1]
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=gh)
    slope = float((gx.double() * d.double()).sum() + (gw.double() * dw.double()).sum())
    # step 2^-6: the second difference is step^2 / 6 of third derivatives of the size of the terms, float32 noise 2^-24 / step
    size = float((gx.abs().double() * d.abs().double()).sum() + (gw.abs().double() * dw.abs().double()).sum())
    assert abs((loss(2.0 ** -6) - loss(-(2.0 ** -6))) / 2.0 ** -5 - slope) <= 2.0 ** -11 * size


def check_quant(q, s, y, quant, ops):
    """Scales and codes of y (float64, exact up to ops * 2^-24): each is what some y within that bound gives."""
    import torch

    tol, H = (ops + 4) * 2.0 ** -24, y.shape[1]
    ref, got = ox.block_scales(y, quant), s.cpu().numpy()
    if quant.startswith("mx"):
        raw = got.reshape(len(got), -1)
        blocks = ref.shape[1]
        assert (raw[:, blocks:] == 127).all()
        got = np.where(raw == 255, np.nan, np.ldexp(1.0, raw.astype(np.int64) - 127))[:, :blocks]
        ok = (got == ox.block_scales(y * (1 + tol), quant)) | (got == ox.block_scales(y * (1 - tol), quant))
    else:
        got = got.astype(np.float64).reshape(ref.shape)
        ok = np.abs(got - ref) <= (tol + 2.0 ** -22) * ref
    bad = np.isnan(ref)
    assert np.array_equal(np.isnan(got), bad) and ok[~bad].all()
    each = ox.spread(got, quant, H)
    if quant == "mxfp4":
        c = q.cpu().numpy()
        codes = np.empty(y.shape)
        codes[:, 0::2], codes[:, 1::2] = oe.VALUES[c & 15], oe.VALUES[c >> 4]
    else:
        codes = q.to(torch.float32).cpu().numpy().astype(np.float64)
    fine = ~np.isnan(each)
    with np.errstate(invalid="ignore"):
        v = np.where(fine, y / each, 0.0)
    lo, hi = ox.nearest(np.abs(v) * (1 - tol), ox.VALUES[quant]), ox.nearest(np.abs(v) * (1 + tol), ox.VALUES[quant])
    a = np.abs(codes)
    assert ((a >= lo) & (a <= hi))[fine].all()
    assert (np.sign(codes) == np.sign(v))[fine & (lo > 0)].all()
    return codes, each


QUANTS = ["int8", "e4m3", "e4m3_128", "mxfp8", "mxfp4"]


@pytest.mark.parametrize("T,H", [(1, 2), (3, 30), (2, 32), (5, 96), (7, 130), (4, 256), (9, 1000), (3, 1026), (1, 7168), (2, 2050), (310, 2048),
                                 (306, 1998), (2, 20000), (2, 65536)])
@pytest.mark.parametrize("quant", QUANTS)
@pytest.mark.parametrize("dt", FLOATS)
def test_norm_quantised(T, H, quant, dt):
    import torch

    rng, x, w, res = norm_inputs(T, H, dt, None, H % 4 == 0, H)
    w[H // 3] = 40.0                                                # one loud channel
    y, h, q, s = moe.moe_add_rms_norm(x, w, res, eps=1e-5, quant=quant)
    # of the float32 sum, whose own error is relative to x and residual and not to what they cancel to
    h32 = down(x.float() if res is None else x.float() + res.float())
    codes, each = check_quant(q, s, ox.add_rms_norm(h32, down(w), None, 1e-5)[0], quant, row_ops(H) + 64)
    for out in FLOATS:
        if quant == "mxfp4":
            back = moe.moe_mx_dequantize(q, s, getattr(torch, out))
        else:
            back = moe.moe_dequantize_rows(q, s, getattr(torch, out))
        exact = torch.from_numpy(codes * each)                      # a float32 product, rounded to float32 first
        assert torch.equal(back.cpu(), exact.float().to(getattr(torch, out)))
    only = moe.moe_add_rms_norm(x, w, res, eps=1e-5, quant=quant, return_y=False)
    assert only[0] is None and torch.equal(only[2].view(torch.uint8), q.view(torch.uint8)) and torch.equal(only[3], s)


@pytest.mark.parametrize("quant", QUANTS)
def test_norm_mx_rows_are_the_quantiser_s(quant):
    """MXFP4 rows of float32 y are those of moe_mx_quantize; the others keep y to half a step."""
    import torch

    _, x, w, _ = norm_inputs(50, 640, "float32", None, False, 1)
    y, _, q, s = moe.moe_add_rms_norm(x, w, quant=quant)
    if quant == "mxfp4":
        qq, ss = moe.moe_mx_quantize(y)
        assert torch.equal(q, qq) and torch.equal(s, ss)
    else:
        back = moe.moe_dequantize_rows(q, s, torch.float32)
        step = 2.0 ** -4 * y.abs() + y.abs().amax(1, keepdim=True) * (1 / 254 if quant == "int8" else 2.0 ** -17)
        if quant == "mxfp8":                                        # what is above 448 of 512 of the scale's range is cut to it
            step = torch.maximum(step, y.abs() / 8)
        assert bool(((back - y).abs() <= step * (1 + 1e-5)).all())


@pytest.mark.parametrize("quant", [None, *QUANTS])
@pytest.mark.parametrize("H", [160, 4096])
def test_norm_of_zeros_nan_and_infinity(quant, H):
    """A row with a NaN is lost whole; one with an infinity holds NaN there and zeros beside; zeros stay zeros."""
    import torch

    rng, x, w, _ = norm_inputs(5, H, "bfloat16", None, False, 2)
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, H - 2] = float("inf")
    y, _, q, s = moe.moe_add_rms_norm(x, w, quant=quant)
    assert not y[1].any() and bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3, H - 2])) and not y[3, :H - 2].any()
    clean = moe.moe_add_rms_norm(x[[0, 4]].contiguous(), w, quant=quant)
    assert torch.equal(y[[0, 4]], clean[0])
    if quant:
        assert torch.equal(q.view(torch.uint8)[[0, 4]], clean[2].view(torch.uint8)) and torch.equal(s[[0, 4]], clean[3])
        back = (moe.moe_mx_dequantize if quant == "mxfp4" else moe.moe_dequantize_rows)(q, s, torch.float32)
        assert not back[1].any() and bool(torch.isnan(back[2]).all())
        block = ox.BLOCK[quant] or H
        lost = torch.zeros(H, dtype=torch.bool)
        lost[(H - 2) // block * block:] = True
        assert torch.equal(torch.isnan(back[3]).cpu(), lost) and not back[3][~lost.cuda()].any()


def test_norm_zero_rows_without_eps():
    """0 / 0: NaN, as the formula says."""
    import torch

    y = moe.moe_add_rms_norm(torch.zeros((2, 48), device="cuda"), torch.ones(48, device="cuda"), eps=0.0)[0]
    assert bool(torch.isnan(y).all())


@pytest.mark.parametrize("quant", ["int8", "e4m3", "e4m3_128"])
def test_norm_smallest_scales(quant):
    """Weights so small that a scale would leave float32's normal range: it stops at 2^-126, and codes go to zero."""
    import torch

    x = up(np.random.default_rng(0).standard_normal((3, 256)), "float32")
    for e in (-120, -130, -149):
        w = torch.full((256,), 2.0 ** e, device="cuda")
        y, _, q, s = moe.moe_add_rms_norm(x, w, quant=quant)
        assert bool((s >= 2.0 ** -126).all())
        back = moe.moe_dequantize_rows(q, s, torch.float32)
        assert bool(((back - y).abs() <= 2.0 ** -126 + y.abs().amax() / 16).all())


@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("T", [3, 400])
def test_norm_strides_and_alignment(off, dt, T):
    import torch

    rng, big, w, res = norm_inputs(T, 1500, dt, None, True, off)
    x, r = offset(big, off)[:, 3:1203], offset(res, off)[:, :1200]
    w = offset(w[:1200].contiguous(), off)
    want = moe.moe_add_rms_norm(x.contiguous(), w.clone(), r.contiguous(), quant="e4m3")
    got = moe.moe_add_rms_norm(x, w, r, quant="e4m3")
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    gy = up(rng.standard_normal((T, 1200)), dt)
    want = moe.moe_add_rms_norm_grad(gy, want[1], w.clone(), grad_h=gy)
    got = moe.moe_add_rms_norm_grad(offset(gy, off), offset(got[1], off), w, grad_h=offset(gy, off))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_norm_empty():
    import torch

    x, w = torch.empty((0, 96), device="cuda"), torch.ones(96, device="cuda")
    for quant in (None, *QUANTS):
        y, h, q, s = moe.moe_add_rms_norm(x, w, x, quant=quant)
        assert y.shape == h.shape == (0, 96)
        if quant and quant != "mxfp4":
            assert moe.moe_dequantize_rows(q, s).shape == (0, 96)
    gx, gw = moe.moe_add_rms_norm_grad(x, x, w)
    assert gx.shape == (0, 96) and not gw.any()


def test_dequantize_every_code():
    """All 256 codes under many scales, NaN ones among them."""
    import torch

    q = torch.arange(256, dtype=torch.uint8, device="cuda").repeat(3, 1)
    f8 = q.view(torch.float8_e4m3fn).float().double().cpu().numpy()
    i8 = q.view(torch.int8).double().cpu().numpy()
    s = torch.tensor([0.37, 2.0 ** -126, float("nan")], device="cuda")
    for codes, ref in ((q.view(torch.int8), i8), (q.view(torch.float8_e4m3fn), f8)):
        for sc in (s, s[:, None]) if codes.dtype == torch.int8 else (s,):
            got = moe.moe_dequantize_rows(codes, sc, torch.float32)
            assert np.array_equal(down(got), (ref * down(s)[:, None]).astype(np.float32).astype(np.float64), equal_nan=True)
    s = torch.tensor([[0.5, 3.0], [1.0, float("nan")], [7.0, 0.1]], device="cuda")
    got = moe.moe_dequantize_rows(q.view(torch.float8_e4m3fn), s, torch.float32)
    assert np.array_equal(down(got), (f8 * np.repeat(down(s), 128, axis=1)).astype(np.float32).astype(np.float64), equal_nan=True)
    b = torch.randint(0, 256, (3, 4, 2), dtype=torch.uint8, device="cuda")
    b[0, 0, 0], b[1, 0, 0] = 255, 0
    got = moe.moe_dequantize_rows(q.view(torch.float8_e4m3fn), b, torch.float32)
    e = b.cpu().numpy().reshape(3, 8).astype(np.int64)
    scale = np.repeat(np.where(e == 255, np.nan, np.ldexp(1.0, e - 127)), 32, axis=1)
    with np.errstate(over="ignore"):
        assert np.array_equal(down(got), (f8 * scale).astype(np.float32).astype(np.float64), equal_nan=True)


# ----------------------------------------------------------------------------- the routing's gradient

@pytest.mark.parametrize("T,e,k", [(1, 1, 1), (3, 4, 4), (9, 60, 6), (5, 64, 64), (40, 128, 8), (700, 256, 8), (6, 513, 33), (7, 1024, 2),
                                   (5000, 20, 3)])
@pytest.mark.parametrize("dt", FLOATS)
@pytest.mark.parametrize("norm_type", [0, 1, 2])
def test_gating_grad(T, e, k, dt, norm_type):
    rng = np.random.default_rng(T + e + norm_type)
    x, gy = up(2 * rng.standard_normal((T, e)), dt), up(rng.standard_normal((T, k)), dt)
    bias, extra = up(0.1 * rng.random(e), dt), up(0.3 * rng.random(e), dt)
    idx = np.stack([rng.permutation(e)[:k] for _ in range(T)])
    for case in range(3):
        kw, ref_kw = {}, {}
        if case:
            kw, ref_kw = {"bias": bias}, {"bias": down(bias)}
        if case == 2:
            mask = rng.random(T) < 0.5
            out = up(rng.standard_normal((T, e)), "float32")
            kw |= {"additional_bias": extra, "additional_token_mask": up(mask), "grad_out": out}
            ref_kw |= {"additional_bias": down(extra), "mask": mask, "grad_out": down(out)}
        gx, gb, ge = moe.moe_gating_top_k_grad(gy, x, ints(idx, "int32"), routed_scaling_factor=2.5, norm_type=norm_type, **kw)
        rx, sx, rb, sb, re, se = ox.gating_grad(down(gy), down(x), idx, scale=2.5, norm_type=norm_type, **ref_kw)
        ops = 3 * (e / 32 + k / 32) + 120
        close(gx, rx, sx, ops, dt)
        assert (gb is None) == (case == 0) and (ge is None) == (case < 2)
        if case:
            close(gb, rb, sb, ops + T / 64 + 60, dt)
        if case == 2:
            close(ge, re, se, ops + T / 64 + 60, dt)


def test_gating_grad_follows_the_forward_pass():
    """moe_gating_top_k's own choice, its weights along a direction, and a 3-D batch."""
    import torch

    rng = np.random.default_rng(0)
    x, d, gy = up(rng.standard_normal((2, 30, 64)), "float32"), up(rng.standard_normal((2, 30, 64)), "float32"), up(rng.standard_normal((2, 30, 6)), "float32")
    bias = up(0.1 * rng.random(64), "float32")
    kw = dict(bias=bias, norm_type=1, routed_scaling_factor=2.5)
    _, idx, _ = moe.moe_gating_top_k(x, 6, k_group=4, group_count=8, **kw)
    gx, gb, _ = moe.moe_gating_top_k_grad(gy, x, idx, **kw)
    assert gx.shape == x.shape and gb.shape == (64,)
    step = 2.0 ** -12

    def weights(v):                                                 # the same experts, by the forward formula
        s = torch.sigmoid(v.double()) + bias.double()
        p = s.gather(2, idx.long())
        return p / p.sum(2, keepdim=True) * 2.5

    y = moe.moe_gating_top_k(x, 6, k_group=4, group_count=8, **kw)[0]
    assert torch.allclose(y.double(), weights(x), rtol=1e-5)
    slope = ((weights(x.double() + step * d.double()) - weights(x.double() - step * d.double())) / (2 * step) * gy.double()).sum()
    size = float((gx.abs() * d.abs()).double().sum())
    assert abs(float((gx.double() * d.double()).sum()) - float(slope)) <= 2.0 ** -14 * size


def test_gating_grad_repeated_and_missing_experts():
    """One expert several times in a row (hash routing), entries out of range, k of more than one warp."""
    rng = np.random.default_rng(3)
    T, e, k = 50, 70, 40
    idx = rng.integers(0, 5, (T, k))
    idx[3] = -1
    idx[4, ::2] = e
    idx[5, 7] = -2 ** 31
    x, gy = up(rng.standard_normal((T, e)), "float32"), up(rng.standard_normal((T, k)), "float32")
    for norm_type in (0, 1, 2):
        gx, _, _ = moe.moe_gating_top_k_grad(gy, x, ints(idx, "int32"), norm_type=norm_type)
        rx, sx, *_ = ox.gating_grad(down(gy), down(x), idx, norm_type=norm_type)
        close(gx, rx, sx, 3 * e / 32 + 160 + k, "float32")


def test_gating_grad_of_saturated_scores():
    """Logits at which a sigmoid is 1 in float32: its slope is still right."""
    x = up(np.array([[20.0, -20.0, 60.0, -60.0, 0.0, 12.0]]), "float32")
    gy = up(np.array([[1.0, -1.0]]), "float32")
    idx = np.array([[0, 4]])
    for norm_type in (0, 1, 2):
        gx, _, _ = moe.moe_gating_top_k_grad(gy, x, ints(idx, "int32"), norm_type=norm_type)
        rx, sx, *_ = ox.gating_grad(down(gy), down(x), idx, norm_type=norm_type)
        close(gx, rx, sx, 130 + 61 * 4, "float32")                  # expf's argument carries 61 units in the worst of them


def test_gating_grad_empty():
    import torch

    x = torch.empty((0, 8), device="cuda")
    gx, gb, ge = moe.moe_gating_top_k_grad(torch.empty((0, 2), device="cuda"), x, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                                           bias=torch.ones(8, device="cuda"))
    assert gx.shape == (0, 8) and not gb.any() and ge is None


# ----------------------------------------------------------------------------- streams, graphs, the same bits

def whole_pass(x, res, w, logits, wsort=None, wgrad=None, stream=None):
    import torch

    kw = {"stream": stream}
    y, h, q, s = moe.moe_add_rms_norm(x, w, res, quant="mxfp8", **kw)
    with torch.cuda.stream(stream):                                 # moe_gating_top_k allocates on the current stream
        weight, idx, _ = moe.moe_gating_top_k(logits, 4, norm_type=1)
    rows, scales, token, row, num, sw = moe.moe_sort_tokens(y, idx, logits.shape[1], per_token_scales=s, expert_topk_weight=weight,
                                                            workspace=wsort, **kw)
    z = moe.moe_combine_tokens(rows, row, weight, **kw)
    grows, gweight = moe.moe_combine_tokens_grad(z, rows, row, token, weight, **kw)
    gy = moe.moe_sort_tokens_grad(grows, row, **kw)
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=z, workspace=wgrad, **kw)
    glogits, _, _ = moe.moe_gating_top_k_grad(gweight, logits, idx, norm_type=1, **kw)
    back = moe.moe_dequantize_rows(q, s, x.dtype, **kw)
    return [y, h, back, rows, scales, token, row, num, sw, z, grows, gweight, gy, gx, gw, glogits]


def pass_inputs(T, H, E, seed):
    rng = np.random.default_rng(seed)
    return (up(rng.standard_normal((T, H)), "bfloat16"), up(rng.standard_normal((T, H)), "bfloat16"), up(rng.random(H) + 0.5, "bfloat16"),
            up(rng.standard_normal((T, E)), "bfloat16"))


def same(a, b):
    import torch

    return all(torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8)) for p, q in zip(a, b))


@pytest.mark.parametrize("T", [5, 1300])
def test_a_graph_replays_with_new_inputs(T):
    import torch

    first, second = pass_inputs(T, 520, 32, 0), pass_inputs(T, 520, 32, 1)
    want = [whole_pass(*first), whole_pass(*second)]
    held = [t.clone() for t in first]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        whole_pass(*held)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = whole_pass(*held)
    for inputs, ref in ((second, want[1]), (first, want[0]), (second, want[1])):
        for t, v in zip(held, inputs):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, ref)


@pytest.mark.parametrize("T", [5, 1300])
def test_streams_at_once(T):
    """Calls on several streams at the same time, named or current, give the bits of calls alone."""
    import torch

    inputs = [pass_inputs(T, 520, 32, i) for i in range(3)]
    want = [whole_pass(*i) for i in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for i, s in zip(inputs, streams):
            got.append(whole_pass(*i, stream=s))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(streams[0]):
        again = whole_pass(*inputs[1])
    torch.cuda.synchronize()
    assert same(again, want[1])


def test_workspaces():
    import torch

    T, H, E = 1300, 520, 32
    inputs = pass_inputs(T, H, E, 0)
    want = whole_pass(*inputs)
    n, g = moe.moe_sort_workspace(T, 4, E), moe.moe_add_rms_norm_grad_workspace(T, H)
    assert n > 0 and moe.moe_sort_workspace(5, 4, E) == 0
    ws = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((g // 4,), float("nan"), device="cuda")]
    for _ in range(2):
        assert same(whole_pass(*inputs, *ws), want)
    with pytest.raises(m.MrrError):
        whole_pass(*inputs, ws[0][:n - 256], ws[1])
    with pytest.raises(m.MrrError):
        whole_pass(*inputs, ws[0], ws[1][64:])
    with pytest.raises(ValueError):
        whole_pass(*inputs, ws[0].cpu(), ws[1])


# ----------------------------------------------------------------------------- refusals

def test_refusals():
    import torch

    x, idx, w = torch.ones((4, 16), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.ones(16, device="cuda")
    f = torch.ones((4, 2), device="cuda")
    rows, token = torch.ones((8, 16), device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    q = torch.zeros((4, 16), dtype=torch.int8, device="cuda")
    bad = [
        (ValueError, moe.moe_sort_tokens, (x.cpu(), idx, 2), {}),
        (ValueError, moe.moe_sort_tokens, (x, idx.cpu(), 2), {}),
        (ValueError, moe.moe_sort_tokens, (x.t(), idx, 2), {}),
        (ValueError, moe.moe_sort_tokens, (x[:1].expand(4, 16), idx, 2), {}),
        (ValueError, moe.moe_sort_tokens, (x, idx[:3], 2), {}),
        (ValueError, moe.moe_sort_tokens, (x, idx[:, :0], 2), {}),
        (ValueError, moe.moe_sort_tokens, (x, idx, 0), {}),
        (ValueError, moe.moe_sort_tokens, (x, idx, 4097), {}),
        (TypeError, moe.moe_sort_tokens, (x, idx.to(torch.int16), 2), {}),
        (TypeError, moe.moe_sort_tokens, (x, idx, 2), {"expert_topk_weight": f.double()}),
        (ValueError, moe.moe_sort_tokens, (x, idx, 2), {"expert_topk_weight": f[:, :1]}),
        (ValueError, moe.moe_sort_tokens, (x, idx, 2), {"per_token_scales": f[:3]}),
        (m.MrrError, moe.moe_sort_tokens, (x, idx, 2), {"expert_token_num_type": 2}),
        (ValueError, moe.moe_combine_tokens, (rows[:, ::2], idx), {}),
        (ValueError, moe.moe_combine_tokens, (rows, idx.long()), {}),
        (TypeError, moe.moe_combine_tokens, (rows.double(), idx), {}),
        (ValueError, moe.moe_combine_tokens, (rows, idx, f.t()), {}),
        (ValueError, moe.moe_combine_tokens_grad, (x, rows, idx, token[:7], f), {}),
        (TypeError, moe.moe_combine_tokens_grad, (x, rows.half(), idx, token, f), {}),
        (ValueError, moe.moe_combine_tokens_grad, (x[:3], rows, idx, token, f), {}),
        (TypeError, moe.moe_add_rms_norm, (x.half(), w.bfloat16()), {}),
        (ValueError, moe.moe_add_rms_norm, (x, w[:8]), {}),
        (ValueError, moe.moe_add_rms_norm, (x, w, x[:2]), {}),
        (ValueError, moe.moe_add_rms_norm, (x, w, x.half()), {}),
        (ValueError, moe.moe_add_rms_norm, (x, w), {"quant": "fp8"}),
        (ValueError, moe.moe_add_rms_norm, (x, w), {"eps": -1.0}),
        (ValueError, moe.moe_add_rms_norm, (x, w), {"return_y": False}),
        (ValueError, moe.moe_add_rms_norm, (x[:, :15], w[:15]), {"quant": "mxfp4"}),
        (m.MrrError, moe.moe_add_rms_norm, (torch.ones((1, 65537), device="cuda"), torch.ones(65537, device="cuda")), {}),
        (ValueError, moe.moe_add_rms_norm_grad, (x, x[:, :8], w[:8]), {}),
        (ValueError, moe.moe_add_rms_norm_grad, (x, x, w), {"grad_h": x.half()}),
        (ValueError, moe.moe_dequantize_rows, (q, f[:, :1].half()), {}),
        (ValueError, moe.moe_dequantize_rows, (q, f), {}),
        (TypeError, moe.moe_dequantize_rows, (q.view(torch.uint8), f[:, 0]), {}),
        (TypeError, moe.moe_gating_top_k_grad, (f.double(), x.double(), idx), {}),
        (ValueError, moe.moe_gating_top_k_grad, (f.half(), x, idx), {}),
        (ValueError, moe.moe_gating_top_k_grad, (f, x, idx.long()), {}),
        (ValueError, moe.moe_gating_top_k_grad, (f, x, idx), {"bias": w.half()}),
        (ValueError, moe.moe_gating_top_k_grad, (f, x, idx), {"grad_out": f}),
        (ValueError, moe.moe_gating_top_k_grad, (f, x, idx), {"additional_token_mask": idx[:, 0]}),
        (m.MrrError, moe.moe_gating_top_k_grad, (f, x, idx), {"norm_type": 3}),
    ]
    for error, call, args, kw in bad:
        with pytest.raises(error):
            call(*args, **kw)
