"""The expert operators on the GPU against the float64 oracle (oracle/experts.py).

MXFP4 codes, scales and values must be equal.  Products are held to the oracle's bound on float32
sums (see ``oracle.experts.sum_error``) plus the result's own rounding: a unit roundoff of 2^-8 for
bfloat16, 2^-11 for float16, 2^-24 for float32, and half of the least subnormal.  In the layer, h
is rounded once to 16 bits on the way, with the same unit roundoffs, or with up to 4 tokens goes on as
the sum of two 16-bit parts, with their squares (twice that allowed for); tokens whose experts a change
of the logits within their float32 error would change are left out (few are).
"""
import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from moe_expert_token_gb300 import experts as ex
from oracle import experts as ox

pytestmark = pytest.mark.gpu

UNIT = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
H_UNIT = {"float16": 2.0 ** -21, "bfloat16": 2.0 ** -15}
LEAST = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -150}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


def up(a, dt=None):
    """A device tensor of a numpy array, rounded to torch dtype name dt."""
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dt is None else t.to(torch.float32).to(getattr(torch, dt))).cuda()


def down(t):
    """float64 numpy values of a device tensor."""
    return t.detach().double().cpu().numpy()


def close(got, ref, bound, dt):
    """got (a tensor of dtype dt) within bound and its own rounding of ref; NaN and infinities alike."""
    g = down(got)
    fine = np.isfinite(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref))
    assert np.array_equal(g[~fine & ~np.isnan(ref)], ref[~fine & ~np.isnan(ref)])
    off = np.abs(g - ref)[fine]
    room = (bound * (1 + UNIT[dt]) + UNIT[dt] * np.abs(ref) + LEAST[dt])[fine]
    assert np.all(off <= room), f"{np.max(off / room)} times the bound"


def weights(rng, *shape):
    """MXFP4 weights of variance 1 / K: (codes, scales, float64 values)."""
    q, s = ox.mx_quantize((rng.standard_normal(shape) * shape[-1] ** -0.5).reshape(-1, shape[-1]))
    q, s = q.reshape(*shape[:-1], -1), s.reshape(*shape[:-1], -1, 2)
    return q, s, ox.mx_values(q, s)


# ----------------------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dt", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,K", [(1, 2), (1, 64), (3, 30), (5, 34), (2, 128), (7, 1026), (1, 7168), (33, 192)])
def test_quantize_and_back(dt, rows, K):
    import torch

    rng = np.random.default_rng(rows * 10000 + K)
    v = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-12, 12, (rows, K // 2)).repeat(2, 1))
    v[0, : K // 2] = 0
    v[-1, K // 2] = -0.0
    x = up(v, dt)
    q, s = moe.moe_mx_quantize(x)
    rq, rs = ox.mx_quantize(down(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    for out in ("float16", "bfloat16", "float32"):
        back = moe.moe_mx_dequantize(q, s, getattr(torch, out))
        want = torch.from_numpy(ox.mx_values(rq, rs)).to(getattr(torch, out))   # one rounding, to nearest
        assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("dt", ["float16", "bfloat16", "float32"])
def test_quantize_ties_and_extremes(dt):
    """Every tie at several scales, the type's largest and smallest values, and their blocks' scales."""
    import torch

    info = torch.finfo(getattr(torch, dt))
    rows = []
    for e in (0, -3, 6):
        v = np.zeros(64)
        v[:20] = np.array([7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 5.5, 6, -7, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5,
                           -5, -5.5, -6]) * 2.0 ** e
        v[32:36] = [4 * 2.0 ** e, 0.25 * 2.0 ** e, 0.5 * 2.0 ** e, -3 * 2.0 ** e]
        rows.append(v)
    v = np.zeros(64)
    v[:3] = [info.max, -info.max, info.max / 3]
    v[32:36] = [info.tiny, -info.tiny, info.smallest_normal / 4, info.tiny / 2]
    rows.append(v)
    x = up(np.array(rows), dt)
    q, s = moe.moe_mx_quantize(x)
    rq, rs = ox.mx_quantize(down(x))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def test_quantize_smallest_floats():
    """float32 subnormals: the scale stops at 2^-127."""
    v = np.zeros((1, 64))
    v[0, :4] = [2.0 ** -127, 2.0 ** -128, 2.0 ** -149, -(2.0 ** -126)]
    v[0, 32:34] = [2.0 ** -124, 2.0 ** -126]
    x = up(v, "float32")
    q, s = moe.moe_mx_quantize(x)
    rq, rs = ox.mx_quantize(v)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("K", [128, 70])
def test_quantize_nan_and_infinity_stay_in_their_block(K):
    rng = np.random.default_rng(K)
    v = rng.standard_normal((4, K))
    v[1, 3], v[2, 40], v[3, K - 1] = np.nan, np.inf, -np.inf
    x = up(v, "bfloat16")
    q, s = moe.moe_mx_quantize(x)
    rq, rs = ox.mx_quantize(down(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(np.isnan(down(moe.moe_mx_dequantize(q, s))), np.isnan(ox.mx_values(rq, rs)))
    ok = np.repeat(rs.reshape(4, -1) != 255, 16, axis=1)[:, :K // 2]
    assert np.array_equal(q.cpu().numpy()[ok], rq[ok])


def test_quantize_strided_unaligned_empty_and_3d():
    import torch

    rng = np.random.default_rng(3)
    big = up(rng.standard_normal((9, 400)), "bfloat16")
    for part in (big[:, 3:195], big[::2, :128], big[:, 16:80]):
        rq, rs = ox.mx_quantize(down(part))
        q, s = moe.moe_mx_quantize(part)
        assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    flat = big.reshape(-1)[1:1 + 6 * 128].view(2, 3, 128)               # 2-byte aligned only
    q, s = moe.moe_mx_quantize(flat)
    rq, rs = ox.mx_quantize(down(flat).reshape(6, 128))
    assert q.shape == (2, 3, 64) and s.shape == (2, 3, 2, 2)
    assert np.array_equal(q.cpu().numpy().reshape(6, -1), rq) and np.array_equal(s.cpu().numpy().reshape(6, 2, 2), rs)
    q, s = moe.moe_mx_quantize(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 32) and moe.moe_mx_dequantize(q, s).shape == (0, 64)
    q, s = moe.moe_mx_quantize(up(np.zeros((2, 2 ** 16)), "float32"))
    assert int(q.count_nonzero()) == 0 and int(s.count_nonzero()) == 0


def test_quantize_refuses():
    import torch

    x = torch.zeros(4, 64, device="cuda")
    for bad, err in ((x[:, :63], ValueError), (x.t(), ValueError), (x.int(), TypeError), (x.cpu(), ValueError),
                     (torch.zeros(2, 4, 64, device="cuda")[:, :, :32], ValueError)):
        with pytest.raises(err):
            moe.moe_mx_quantize(bad)
    q, s = moe.moe_mx_quantize(x)
    with pytest.raises(ValueError):
        moe.moe_mx_dequantize(q, s[:3])
    with pytest.raises(TypeError):
        moe.moe_mx_dequantize(q, s, torch.int32)


# ----------------------------------------------------------------------------- grouped product

def grouped_case(seed, counts, K, N, *, gate=False, out="bfloat16", i64=False, prefix=False, weighted=False,
                 x_edit=None, w_edit=None):
    import torch

    rng = np.random.default_rng(seed)
    counts = np.asarray(counts)
    A, E = int(counts.sum()), len(counts)
    q, s = ox.mx_quantize(rng.standard_normal((A, K))) if A else (np.zeros((0, K // 2), np.uint8),
                                                                   np.zeros((0, (K + 63) // 64, 2), np.uint8))
    wq, ws, _ = weights(rng, E, 2 * N if gate else N, K)
    for edit, a in ((x_edit, s), (w_edit, ws)):
        if edit is not None:
            edit(a)
    rw = rng.random(A) if weighted else None
    ref, bound = ox.grouped(ox.mx_values(q, s), counts, ox.mx_values(wq, ws), gate=gate,
                            row_weight=None if rw is None else rw.astype(np.float32).astype(np.float64))
    num = np.cumsum(counts) if prefix else counts
    got = moe.moe_mx_grouped_matmul(
        up(q), up(s), up(num.astype(np.int64 if i64 else np.int32)), up(wq), up(ws), gated=gate,
        out_dtype="mxfp4" if out == "mxfp4" else getattr(torch, out), expert_token_num_type=0 if prefix else 1,
        row_weight=None if rw is None else up(rw.astype(np.float32)), check_status=True)
    return got, ref, bound


COUNTS = [[1], [0, 1], [3, 0, 0, 5], [130, 1, 0, 64], [17, 15, 16, 33, 31, 2, 0, 1], [300, 129, 255]]


@pytest.mark.parametrize("counts", COUNTS, ids=[str(c) for c in COUNTS])
@pytest.mark.parametrize("K,N", [(32, 1), (64, 7), (96, 32), (256, 130), (544, 257), (1024, 96)])
@pytest.mark.parametrize("gate", [False, True])
def test_grouped(counts, K, N, gate):
    dt = ["bfloat16", "float16", "float32"][(K + N + len(counts)) % 3]
    got, ref, bound = grouped_case(K + N, counts, K, N, gate=gate, out=dt, i64=bool(K % 64), prefix=N % 2 == 0,
                                   weighted=N % 3 == 0)
    assert got.shape == ref.shape
    close(got, ref, bound, dt)


@pytest.mark.parametrize("counts,K,N", [([700, 900], 2048, 384), ([40] * 40, 1056, 200), ([1] * 100, 512, 129),
                                        ([2000], 320, 64)])
@pytest.mark.parametrize("gate", [False, True])
def test_grouped_more_rows(counts, K, N, gate):
    got, ref, bound = grouped_case(5, counts, K, N, gate=gate, weighted=gate)
    close(got, ref, bound, "bfloat16")


@pytest.mark.parametrize("counts", [[10] * 64, [70, 250, 3, 0, 128] * 12, [0] * 200 + [25] * 100], ids=["few", "many", "empty"])
@pytest.mark.parametrize("K,N", [(96, 512), (544, 480)])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_grouped_more_experts(counts, K, N, gate, dt):
    """Enough tiles for every block of the GPU, with few rows each and with many."""
    got, ref, bound = grouped_case(6, counts, K, N, gate=gate, out=dt, weighted=not gate)
    close(got, ref, bound, dt)


@pytest.mark.parametrize("counts,K,N", [([5, 0, 40], 256, 64), ([130, 200], 512, 160), ([1], 64, 32), ([16] * 9, 96, 96)])
@pytest.mark.parametrize("gate", [False, True])
def test_grouped_mxfp4_result(counts, K, N, gate):
    """The MXFP4 result stands for the float32 result, quantised: each value is within half a step of
    e2m1 of it (a step is at most a third of the block's largest magnitude) up to the sums' bound,
    and nearly all codes are those of the oracle's own quantisation."""
    (q, s), ref, bound = grouped_case(8, counts, K, N, gate=gate, out="mxfp4", weighted=True)
    rq, rs = ox.mx_quantize(ref)
    assert q.shape == rq.shape and s.shape == rs.shape
    if N % 64:
        assert np.all(s.cpu().numpy()[:, -1, 1] == 127)
    assert np.mean(q.cpu().numpy() != rq) < 0.01 and np.mean(s.cpu().numpy() != rs) < 0.01
    v = ox.mx_values(q.cpu().numpy(), s.cpu().numpy())
    top = np.abs(ref).reshape(len(ref), -1, 32).max(-1).repeat(32, 1)
    assert np.all(np.abs(v - ref) <= top / 4 + bound)    # saturation: 8 - 6 of at most 8


@pytest.mark.parametrize("counts", [[10] * 64, [70, 250, 3, 0, 128] * 12], ids=["few", "many"])
@pytest.mark.parametrize("gate", [False, True])
def test_grouped_mxfp4_result_more_experts(counts, gate):
    (q, s), ref, bound = grouped_case(12, counts, 160, 512, gate=gate, out="mxfp4")
    v = ox.mx_values(q.cpu().numpy(), s.cpu().numpy())
    top = np.abs(ref).reshape(len(ref), -1, 32).max(-1).repeat(32, 1)
    assert np.all(np.abs(v - ref) <= top / 4 + bound)    # saturation: 8 - 6 of at most 8


def test_grouped_nan_scales_stay_in_their_row():
    """A NaN scale in one token row or one weight row reaches that row or column only; scale bytes 0
    (2^-127) and 254 (2^127) are finite.  The rows next to an expert's own, and its neighbours'
    weights, are never mixed in."""
    def x_edit(s):
        s[4, 1, 0] = 255
        s[5] = 0
        s[70, :, 1] = 200
    def w_edit(s):
        s[1, 3, 0, 1] = 255
        s[2] = 0
    got, ref, bound = grouped_case(9, [5, 66, 3], 128, 48, out="float32", x_edit=x_edit, w_edit=w_edit)
    assert np.isnan(ref[4]).all() and np.isnan(ref[5:71, 3]).all() and np.isnan(ref).sum() == 48 + 66
    close(got, ref, bound, "float32")


def test_grouped_no_rows():
    got, ref, _ = grouped_case(1, [0, 0, 0], 64, 32)
    assert got.shape == (0, 32)


@pytest.mark.parametrize("num,code", [([3, 4], m.MRR_ERR_COUNT_SUM), ([9, 1], m.MRR_ERR_COUNT_SUM),
                                      ([-1, 9], m.MRR_ERR_COUNT_NONPOS), ([2 ** 40, 0], m.MRR_ERR_COUNT_SUM)])
def test_grouped_bad_counts_are_reported(num, code):
    import torch

    rng = np.random.default_rng(2)
    q, s = ox.mx_quantize(rng.standard_normal((8, 64)))
    wq, ws, _ = weights(rng, 2, 32, 64)
    with pytest.raises(m.MrrError) as err:
        moe.moe_mx_grouped_matmul(up(q), up(s), torch.tensor(num, dtype=torch.int64, device="cuda"), up(wq), up(ws),
                                  check_status=True)
    assert err.value.code == code
    good, ref, bound = grouped_case(2, [3, 5], 64, 32)     # and the next call is untouched by it
    close(good, ref, bound, "bfloat16")


def test_grouped_refuses():
    import torch

    q = torch.zeros(8, 32, dtype=torch.uint8, device="cuda")
    s = torch.zeros(8, 1, 2, dtype=torch.uint8, device="cuda")
    w = torch.zeros(2, 6, 32, dtype=torch.uint8, device="cuda")
    ws = torch.zeros(2, 6, 1, 2, dtype=torch.uint8, device="cuda")
    c = torch.tensor([4, 4], device="cuda")
    call = moe.moe_mx_grouped_matmul
    for args, kw, err in (
            ((q, s[:7], c, w, ws), {}, ValueError), ((q, s, c.float(), w, ws), {}, TypeError),
            ((q, s, c[:1], w, ws), {}, ValueError), ((q, s, c, w[:, :5], ws[:, :5]), {}, ValueError),
            ((q, s, c, w, ws), dict(out_dtype=torch.int32), TypeError),
            ((q, s, c, w, ws), dict(out_dtype="mxfp4"), ValueError),
            ((q, s, c, w, ws), dict(row_weight=torch.zeros(7, device="cuda")), ValueError),
            ((q.float(), s, c, w, ws), {}, TypeError), ((q.cpu(), s, c, w, ws), {}, ValueError),
            ((q[:, :16].contiguous(), s, c, w, ws), {}, ValueError)):
        with pytest.raises(err):
            call(*args, **kw)
    with pytest.raises(m.MrrError):                                      # K = 48 is no multiple of 32
        call(q[:, :24].contiguous(), s, c, w[..., :24].contiguous(), ws)


# ----------------------------------------------------------------------------- the layer

def layer_case(seed, T, E, k, H, I, dt="bfloat16", *, mx=False, bias=False, edit=None, scale=1.0, **kw):
    import torch

    rng = np.random.default_rng(seed)
    f = lambda a: torch.from_numpy(a).to(torch.float32).to(getattr(torch, dt))  # noqa: E731
    x, wr = f(rng.standard_normal((T, H)) * scale), f(rng.standard_normal((E, H)) * H ** -0.5 / scale)
    b = f(rng.random(E) * 0.1) if bias else None
    if edit is not None:
        edit(x)
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        w13, s13, w2, s2 = (up(a) for a in (w13, s13, w2, s2))
    else:
        w13, w2 = f(rng.standard_normal((E, 2 * I, H)) * H ** -0.5).cuda(), f(rng.standard_normal((E, H, I)) * I ** -0.5).cuda()
        s13, s2, v13, v2 = None, None, down(w13), down(w2)
    y, w, idx = moe.moe_few_token_layer(x.cuda(), wr.cuda(), w13, w2, k, bias=None if b is None else b.cuda(),
                                        w13_scales=s13, w2_scales=s2, return_routing=True, check_status=True, **kw)
    gate_kw = {n: v for n, v in kw.items()}
    if b is not None:
        gate_kw["bias"] = down(b).astype(np.float32)
    xv = down(x)
    ok = np.isfinite(xv).all(axis=1)
    xv = np.where(ok[:, None], xv, 0.0)
    rw, ridx, sure, logit_error = ox.routing(xv, down(wr), k, **gate_kw)
    sure &= ok
    assert sure.sum() >= 0.8 * ok.sum() - 1
    idx, w = idx.cpu().numpy(), down(w)
    assert idx.min() >= 0 and idx.max() < E and all(len(set(r)) == k for r in idx)
    assert np.array_equal(idx[sure], ridx[sure])
    # a logit error d moves a score, and the sum of scores, by a factor of at most 1 + d (+ float32 rounding)
    werr = 3 * logit_error + 1e-5
    assert np.all(np.abs(w - rw)[sure] <= (werr[:, None] * np.abs(rw) + 1e-9)[sure])
    unit = (H_UNIT if T <= 4 else UNIT)["float16" if mx else dt]
    ref, bound = ox.layer(xv, rw, ridx, werr, v13, v2, unit)
    close(y[torch.from_numpy(sure)], ref[sure], bound[sure], dt)
    return y, ok


ROUTING = [dict(), dict(norm_type=1), dict(norm_type=2, routed_scaling_factor=2.5),
           dict(norm_type=1, group_count=4, k_group=2, group_select_mode=1, routed_scaling_factor=2.5)]


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 33, 64])
@pytest.mark.parametrize("E,k,H,I", [(8, 2, 256, 128), (16, 4, 200, 72), (12, 3, 1031, 77), (64, 8, 512, 48)])
@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
def test_layer(T, E, k, H, I, dt):
    layer_case(T + E + H, T, E, k, H, I, dt, bias=T % 2 == 0, **ROUTING[(T + E // 4) % 4])


@pytest.mark.parametrize("T", [1, 3, 8, 17, 64])
@pytest.mark.parametrize("E,k,H,I", [(8, 2, 256, 128), (16, 4, 200, 72), (12, 3, 1030, 78), (64, 8, 512, 64)])
@pytest.mark.parametrize("dt", ["bfloat16", "float16"])
def test_layer_mxfp4(T, E, k, H, I, dt):
    layer_case(T + E + H, T, E, k, H, I, dt, mx=True, bias=T % 2 == 0, **ROUTING[(T + E // 4) % 4])


@pytest.mark.parametrize("E,k,H,I", [(1, 1, 64, 32), (5, 5, 40, 24), (3, 1, 1, 1), (2, 2, 2, 2), (1024, 64, 64, 16),
                                     (257, 3, 96, 8), (4, 1, 4096, 520)])
@pytest.mark.parametrize("mx", [False, True])
def test_layer_edges(E, k, H, I, mx):
    if mx and (H % 2 or I % 2):
        pytest.skip("MXFP4 rows hold an even number of elements")
    layer_case(E + H, 3, E, k, H, I, mx=mx)
    layer_case(E + H + 1, 1, E, k, H, I, "float16", mx=mx, norm_type=1)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 1024, 64, 64, 32), (8, 1024, 64, 64, 32), (64, 64, 64, 96, 40)])
def test_layer_most_assignments(T, E, k, H, I, mx):
    """The largest tables: every size of the routing at its limit, against the oracle on the GPU's routing."""
    import torch

    rng = np.random.default_rng(T + E)
    bf = lambda a: torch.from_numpy(a).to(torch.bfloat16).cuda()  # noqa: E731
    x, wr = bf(rng.standard_normal((T, H))), bf(rng.standard_normal((E, H)) * H ** -0.5)
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        w13, s13, w2, s2 = (up(a) for a in (w13, s13, w2, s2))
    else:
        w13, w2, s13, s2 = bf(rng.standard_normal((E, 2 * I, H)) * H ** -0.5), bf(rng.standard_normal((E, H, I)) * I ** -0.5), None, None
        v13, v2 = down(w13), down(w2)
    y, w, idx = moe.moe_few_token_layer(x, wr, w13, w2, k, w13_scales=s13, w2_scales=s2, norm_type=1,
                                        return_routing=True, check_status=True)
    idx, w = idx.cpu().numpy(), down(w)
    assert idx.min() >= 0 and idx.max() < E and all(len(set(r)) == k for r in idx)
    assert np.all(np.abs(w.sum(axis=1) - 1) < 1e-5) and np.all(np.diff(w, axis=1) <= 0)
    ref, bound = ox.layer(down(x), w, idx, np.full(T, 1e-6), v13, v2, UNIT["float16" if mx else "bfloat16"])
    close(y, ref, bound, "bfloat16")


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 1024, 64, 70, 38), (8, 1024, 64, 70, 38), (64, 64, 64, 102, 42)])
def test_layer_most_assignments_of_narrow_rows(T, E, k, H, I, mx):
    test_layer_most_assignments(T, E, k, H, I, mx)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(20, 40, 4, 96, 1040), (3, 24, 8, 30, 2050), (64, 9, 3, 1, 700), (8, 16, 8, 1216, 640)])
def test_layer_few_output_rows(T, E, k, H, I, mx):
    """Items of the down product that several blocks share: right, and bit for bit the same each time, whatever the
    workspace held before."""
    import torch

    H += mx and H % 2
    layer_case(T + H, T, E, k, H, I, "float16" if T == 20 else "bfloat16", mx=mx, norm_type=1)
    bf = lambda *s_: torch.randn(*s_, device="cuda").bfloat16()  # noqa: E731
    x, wr = bf(T, H), bf(E, H)
    w13, w2, kw = bf(E, 2 * I, H), bf(E, H, I), {}
    if mx:
        (w13, s13), (w2, s2) = moe.moe_mx_quantize(w13), moe.moe_mx_quantize(w2)
        kw = dict(w13_scales=s13, w2_scales=s2)
    n = moe.moe_few_token_layer_workspace(T, H, E, I, k)
    runs = [moe.moe_few_token_layer(x, wr, w13, w2, k, check_status=True, **kw,
                                    workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
            for fill in (0, 255, 1, 77)]
    assert all(torch.equal(runs[0], r) for r in runs[1:])


def test_layer_all_tokens_choose_the_same_experts():
    """A bias that decides the choice: one pair of experts takes all 64 tokens."""
    import torch

    rng = np.random.default_rng(4)
    T, E, H, I = 64, 32, 192, 80
    x = torch.from_numpy(rng.standard_normal((T, H))).to(torch.bfloat16)
    wr = torch.zeros(E, H, dtype=torch.bfloat16)
    bias = torch.zeros(E, dtype=torch.bfloat16)
    bias[5], bias[30] = 3.0, 1.0
    w13 = torch.from_numpy(rng.standard_normal((E, 2 * I, H)) * H ** -0.5).to(torch.bfloat16)
    w2 = torch.from_numpy(rng.standard_normal((E, H, I)) * I ** -0.5).to(torch.bfloat16)
    y, w, idx = moe.moe_few_token_layer(x.cuda(), wr.cuda(), w13.cuda(), w2.cuda(), 2, bias=bias.cuda(), norm_type=1,
                                        return_routing=True, check_status=True)
    assert idx.cpu().tolist() == [[5, 30]] * T
    rw = np.tile(np.array([3.5, 1.5]) / 5.0, (T, 1))
    ref, bound = ox.layer(down(x), rw, idx.cpu().numpy(), np.full(T, 1e-6), down(w13), down(w2), UNIT["bfloat16"])
    close(y, ref, bound, "bfloat16")


@pytest.mark.parametrize("mx", [False, True])
def test_layer_nan_and_infinity_stay_with_their_token(mx):
    def edit(x):
        x[2, 5] = float("nan")
        x[6, 0] = float("inf")
        x[9] = 0
    y, ok = layer_case(11, 12, 8, 2, 160, 64, mx=mx, edit=edit)
    assert not np.isfinite(down(y)[2]).any()
    assert np.isfinite(down(y)[ok]).all()


@pytest.mark.parametrize("dt", ["float16", "bfloat16"])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("scale", [2.0 ** -9, 2.0 ** 7])
def test_layer_small_and_large_inputs(dt, mx, scale):
    """Between the products h is as large as scale^2: far past float16's range at 2^7 times a wide weight."""
    layer_case(13, 5, 8, 2, 256, 128, dt, mx=mx, scale=scale)


def test_layer_unaligned_views():
    """Tensors that start 2 bytes past a 16-byte boundary."""
    import torch

    rng = np.random.default_rng(21)
    T, E, H, I, k = 3, 8, 128, 64, 2

    def off(shape, s):
        n = int(np.prod(shape))
        flat = torch.empty(n + 1, dtype=torch.bfloat16, device="cuda")
        flat[1:] = torch.from_numpy(rng.standard_normal(n) * s).to(torch.bfloat16).cuda()
        return flat[1:].view(*shape)
    x, wr, w13, w2 = off((T, H), 1.0), off((E, H), H ** -0.5), off((E, 2 * I, H), H ** -0.5), off((E, H, I), I ** -0.5)
    y = moe.moe_few_token_layer(x, wr, w13, w2, k, check_status=True)
    z = moe.moe_few_token_layer(x.clone(), wr.clone(), w13.clone(), w2.clone(), k, check_status=True)
    rw, ridx, sure, le = ox.routing(down(x), down(wr), k)
    ref, bound = ox.layer(down(x), rw, ridx, 3 * le + 1e-5, down(w13), down(w2), H_UNIT["bfloat16"])
    assert sure.all()
    close(y, ref, bound, "bfloat16")
    close(z, ref, bound, "bfloat16")


@pytest.mark.parametrize("T", [2, 20])
@pytest.mark.parametrize("H,I", [(334, 202), (648, 130), (1026, 516)])
@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("mx", [False, True])
def test_layer_rows_of_any_alignment(T, H, I, off, mx):
    """Rows that begin at any byte and end inside a word, with NaN right before and behind the experts
    that are chosen: nothing of a neighbour's row, expert or scales may reach them."""
    import torch

    rng = np.random.default_rng(H + off)
    E, k = 6, 2
    bf = lambda a: torch.from_numpy(a).to(torch.bfloat16)  # noqa: E731

    def view(a, n):   # the tensor, n elements past the start of an allocation
        flat = torch.zeros(a.numel() + n, dtype=a.dtype, device="cuda")
        flat[n:] = a.reshape(-1).cuda()
        return flat[n:].view(a.shape)
    x, wr = bf(rng.standard_normal((T, H))).cuda(), torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    bias = bf(np.array([0.0, 1.0, 0.0, 0.0, 3.0, 0.0])).cuda()
    if mx:
        (w13, s13, v13), (w2, s2, v2) = weights(rng, E, 2 * I, H), weights(rng, E, H, I)
        for e in (0, 2, 3, 5):
            s13[e], s2[e] = 255, 255
        w13, s13, w2, s2 = (view(torch.from_numpy(a), off) for a in (w13, s13, w2, s2))
    else:
        w13, w2 = bf(rng.standard_normal((E, 2 * I, H)) * H ** -0.5), bf(rng.standard_normal((E, H, I)) * I ** -0.5)
        v13, v2 = down(w13), down(w2)
        for e in (0, 2, 3, 5):
            w13[e], w2[e] = float("nan"), float("nan")
        w13, w2, s13, s2 = view(w13, off), view(w2, off), None, None
    y, w, idx = moe.moe_few_token_layer(x, wr, w13, w2, k, bias=bias, w13_scales=s13, w2_scales=s2, norm_type=1,
                                        return_routing=True, check_status=True)
    assert idx.cpu().tolist() == [[4, 1]] * T
    rw = np.tile(np.array([3.5, 1.5]) / 5.0, (T, 1))
    ref, bound = ox.layer(down(x), rw, idx.cpu().numpy(), np.full(T, 1e-6), v13, v2,
                          (H_UNIT if T <= 4 else UNIT)["float16" if mx else "bfloat16"])
    close(y, ref, bound, "bfloat16")


def test_layer_no_tokens_and_refusals():
    import torch

    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    wr = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w13 = torch.zeros(4, 64, 64, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(4, 64, 32, dtype=torch.bfloat16, device="cuda")
    call = moe.moe_few_token_layer
    assert call(x[:0], wr, w13, w2, 2, check_status=True).shape == (0, 64)
    many = torch.zeros(65, 64, dtype=torch.bfloat16, device="cuda")
    for args, err in (((many, wr, w13, w2, 2), m.MrrError), ((x, wr, w13, w2, 5), m.MrrError),
                      ((x.float(), wr, w13, w2, 2), TypeError), ((x, wr.half(), w13, w2, 2), ValueError),
                      ((x, wr, w13[:, :63], w2, 2), ValueError), ((x, wr, w13, w2.half(), 2), ValueError),
                      ((x, wr, w13, w2[:, :, ::2], 2), ValueError), ((x[:, ::2], wr, w13, w2, 2), ValueError)):
        with pytest.raises(err):
            call(*args)
    with pytest.raises(TypeError):
        call(x, wr, w13, w2, 2, w13_scales=torch.zeros(1, device="cuda"))


def test_layer_offsets_past_32_bits():
    """Weights of more than 2^32 elements: the last experts are read from the right place."""
    import torch

    E, I, H, T, k = 700, 64, 50000, 2, 2
    gen = torch.Generator(device="cuda").manual_seed(5)
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    assert w13.numel() > 2 ** 32
    for e in (1, E - 1):
        w13[e] = torch.randn(2 * I, H, generator=gen, device="cuda") * H ** -0.5
        w2[e] = torch.randn(H, I, generator=gen, device="cuda") * I ** -0.5
    x = torch.randn(T, H, generator=gen, device="cuda").to(torch.bfloat16)
    wr = torch.zeros(E, H, dtype=torch.bfloat16, device="cuda")
    bias = torch.zeros(E, dtype=torch.bfloat16, device="cuda")
    bias[E - 1], bias[1] = 3.0, 1.0
    y = moe.moe_few_token_layer(x, wr, w13, w2, k, bias=bias, norm_type=1, check_status=True)
    rw = np.tile(np.array([3.5, 1.5]) / 5.0, (T, 1))
    ref, bound = ox.layer(down(x), rw, np.tile([0, 1], (T, 1)), np.full(T, 1e-6), down(w13[[E - 1, 1]]),
                          down(w2[[E - 1, 1]]), H_UNIT["bfloat16"])
    close(y, ref, bound, "bfloat16")


# ----------------------------------------------------------------------------- streams, graphs, repeats

def test_results_repeat_and_do_not_depend_on_the_stream_or_a_graph():
    """The same call gives the same bits: again, on a second stream beside other work, and replayed
    from a CUDA graph; a used workspace, or one full of anything, changes nothing."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T, E, H, I, k = 6, 16, 512, 192, 4
    x, wr = rnd(T, H).bfloat16(), (rnd(E, H) * H ** -0.5).bfloat16()
    w13, s13 = moe.moe_mx_quantize(rnd(E, 2 * I, H) * H ** -0.5)
    w2, s2 = moe.moe_mx_quantize(rnd(E, H, I) * I ** -0.5)
    d13, d2 = moe.moe_mx_dequantize(w13, s13), moe.moe_mx_dequantize(w2, s2)
    rows = rnd(300, H).bfloat16()
    num = torch.full((E,), 300 // E, dtype=torch.int32, device="cuda")
    num[3] += 300 - int(num.sum())
    ws = torch.full((1 << 20,), 0xC3, dtype=torch.uint8, device="cuda")

    def everything(workspace=None):
        q, s = moe.moe_mx_quantize(rows)
        h = moe.moe_mx_grouped_matmul(q, s, num, w13, s13, gated=True, out_dtype="mxfp4", workspace=workspace)
        y = moe.moe_mx_grouped_matmul(*h, num, w2, s2, workspace=workspace)
        a = moe.moe_few_token_layer(x, wr, w13, w2, k, w13_scales=s13, w2_scales=s2, workspace=workspace)
        b = moe.moe_few_token_layer(x, wr, d13, d2, k, workspace=workspace)
        return [q, s, *h, y, a, b]

    want = everything()
    for again in (everything(), everything(ws), everything(ws)):
        assert all(torch.equal(p, q) for p, q in zip(want, again))
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        busy = [everything() for _ in range(3)]
    with torch.cuda.stream(side):
        again = everything()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, again))
    assert all(torch.equal(p, q) for p, q in zip(want, busy[-1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = everything(ws)
    for _ in range(3):
        for t in kept:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, kept))


def test_given_stream_is_used():
    """A call given a stream runs there: it is ordered behind what that stream does."""
    import torch

    side = torch.cuda.Stream()
    x = torch.zeros(64, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.fill_(3.0)
    q, s = moe.moe_mx_quantize(x, stream=side)
    v = moe.moe_mx_dequantize(q, s, stream=side)
    num = torch.tensor([64], dtype=torch.int32, device="cuda")
    y = moe.moe_mx_grouped_matmul(q, s, num, q[None], s[None], out_dtype=torch.float32, stream=side, check_status=True)
    side.synchronize()
    assert bool((v == 3.0).all()) and bool((y == 9.0 * 4096).all())


# ----------------------------------------------------------------------------- together

def test_example_block_end_to_end():
    """examples/moe_block.py: prefill (routing, quantisation, re-routing, products, inverse, sum) against
    the same steps in the oracle, given the GPU's own routing.  Each row's y is rounded to bfloat16 (2^-9
    of it at most, 2^-10 root mean square) and the sum once more; a float32 difference that moves a code
    of h is as rare as 2^-20 of them: the whole within 2^-8.  Decode on the same weights differs from it
    by the activations' quantisation only: two roundings to MXFP4 of about 10 % each, at random."""
    import importlib.util
    import os

    import torch

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")
    spec = importlib.util.spec_from_file_location("moe_block", path)
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    gen = torch.Generator(device="cuda").manual_seed(7)
    T, E, H, I, k = 256, 8, 256, 128, 4
    w = block.weights(E, H, I, gen)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    y = block.prefill(x, w, k, ranks=2)

    weight, expert, _ = moe.moe_gating_top_k(x @ w["router"].t(), k, bias=w["bias"], **block.ROUTING)
    weight, expert = down(weight), expert.cpu().numpy()
    xv = ox.mx_values(*ox.mx_quantize(down(x)))
    v13 = ox.mx_values(w["w13"].cpu().numpy(), w["s13"].cpu().numpy())
    v2 = ox.mx_values(w["w2"].cpu().numpy(), w["s2"].cpu().numpy())
    ref = np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(expert == e)
        h = ox.mx_values(*ox.mx_quantize(ox.gated(xv[t], v13[e], I)[0]))
        ref[t] += (h @ v2[e].T) * weight[t, j][:, None]
    assert np.linalg.norm(down(y) - ref) <= 2.0 ** -8 * np.linalg.norm(ref)
    z = block.decode(x[:8].contiguous(), w, k)
    assert np.linalg.norm(down(z) - ref[:8]) <= 0.3 * np.linalg.norm(ref[:8])
