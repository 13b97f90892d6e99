"""The operators around the experts where one of their forms ends and the next begins, and rows of many shared-memory
segments; tolerances are those of test_tokens_gpu.py."""
import numpy as np
import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from oracle import tokens as ox
from test_experts_gpu import down, up
from test_tokens_gpu import (check_quant, check_sort, close, combine_case, experts, ints, offset, ox_token, row_ops)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_token_gb300 import build

    build.build()
    m.load_library()


# ----------------------------------------------------------------------------- sort

@pytest.mark.parametrize("T,k", [(4096, 1), (4097, 1), (1365, 3), (1366, 3), (131072, 1), (131073, 1), (16384, 8), (16385, 8), (2049, 64)])
@pytest.mark.parametrize("E", [7, 1023, 1024])
def test_sort_where_forms_meet(T, k, E):
    """4096 slots are the most that one launch sorts, 131072 slots and 1023 experts the most that one cluster ranks."""
    rng = np.random.default_rng(T + E)
    idx = experts(rng, T, k, E, wrong=0.05)
    idx[-3:] = -1
    check_sort(up(rng.integers(0, 255, (T, 24)).astype(np.uint8)), idx, E, weight=up(rng.random((T, k)), "float16"), cumsum=E == 7)


@pytest.mark.parametrize("H", [8191, 8192, 8193, 16384, 20001])
@pytest.mark.parametrize("off", [0, 1, 6])
def test_sort_rows_of_several_segments(H, off):
    """Rows that shared memory holds in parts, from and to any byte."""
    import torch

    rng = np.random.default_rng(H)
    T, k = 2100, 2
    x = offset(torch.randint(0, 256, (T, H + 5), dtype=torch.uint8, device="cuda"), off)[:, 3:3 + H]
    check_sort(x, experts(rng, T, k, 9, wrong=0.3), 9)


@pytest.mark.parametrize("H", [1, 2, 3, 15, 16, 17, 31, 33])
@pytest.mark.parametrize("T", [9, 5000])
def test_sort_shortest_rows(H, T):
    import torch

    x = torch.randint(0, 256, (T, H), dtype=torch.uint8, device="cuda")
    check_sort(x, experts(np.random.default_rng(H), T, 3, 11, wrong=0.2), 11, scales=offset(x[:, :1].contiguous(), 1))


def test_sort_an_expert_parallel_share():
    """An eighth of the experts held here: most rows are zeros, of every output."""
    rng = np.random.default_rng(8)
    T, k, E = 4000, 8, 256
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    for H in (512, 517):
        check_sort(up(rng.standard_normal((T, H)), "bfloat16"), idx, 32, 64, scales=up(rng.random((T, 3)), "float32"),
                   weight=up(rng.random((T, k)), "bfloat16"), kind="int64")


# ----------------------------------------------------------------------------- combine

@pytest.mark.parametrize("k", [1, 2, 3, 4, 5, 8, 9, 17])
@pytest.mark.parametrize("H", [1000, 1001, 1002, 1004, 72])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_combine_many_tokens(k, H, dt):
    rng = np.random.default_rng(k * H)
    T = 700
    rows, row, w = combine_case(rng, T, k, T * k + 5, H, dt, "float32")
    y = moe.moe_combine_tokens(rows, ints(row, "int32"), w)
    ref, size = ox.combine(down(rows), row, down(w))
    close(y, ref, size, k + 2, dt)
    gy = up(rng.standard_normal((T, H)), dt)
    grows, gw = moe.moe_combine_tokens_grad(gy, rows, ints(row, "int32"), ints(ox_token(row, T * k + 5), "int32"), w)
    ref_rows, ref_w, size = ox.combine_grad(down(gy), down(rows), row, down(w))
    close(grows, ref_rows, np.abs(ref_rows), 2, dt)
    close(gw, ref_w, size, row_ops(H), "float32")


@pytest.mark.parametrize("k", [2, 3, 4, 5, 8])
@pytest.mark.parametrize("H", [2048, 1028, 2049, 1026])
@pytest.mark.parametrize("dt", ["float16", "float32"])
@pytest.mark.parametrize("T", [5, 640])
def test_combine_of_tokens_with_few_rows(k, H, dt, T):
    """Any number of a token's slots have rows; weights of the others are NaN, and rows of zeros fill the gradient."""
    rng = np.random.default_rng(k * H + T)
    rows, row, w = combine_case(rng, T, k, T * k, H, dt, "float32", wrong=0.0)
    row = np.where(rng.random((T, k)) < rng.random((T, 1)), row, -1)
    row[0], row[T // 2] = -1, np.arange(k)[::-1] % 3 - 1        # no row, and some rows more than once
    w[ints(row, "int64") < 0] = float("nan")
    ref, size = ox.combine(down(rows), row, down(w))
    close(moe.moe_combine_tokens(rows, ints(row, "int32"), w), ref, size, k + 2, dt)
    rows, row, w = combine_case(rng, T, k, T * k, H, dt, "float32", wrong=0.8)
    gy = up(rng.standard_normal((T, H)), dt)
    grows, gw = moe.moe_combine_tokens_grad(gy, rows, ints(row, "int32"), ints(ox_token(row, T * k), "int32"), w)
    ref_rows, ref_w, size = ox.combine_grad(down(gy), down(rows), row, down(w))
    close(grows, ref_rows, np.abs(ref_rows), 2, dt)
    close(gw, ref_w, size, row_ops(H), "float32")


@pytest.mark.parametrize("T", [303, 304, 607, 608, 609])
def test_combine_where_forms_meet(T):
    """Fewer than 608 blocks share a token's columns, fewer than 304 tokens have more threads each."""
    rng = np.random.default_rng(T)
    rows, row, w = combine_case(rng, T, 6, T * 6, 2064, "bfloat16", "bfloat16")
    idx = ints(row, "int32")
    ref, size = ox.combine(down(rows), row, down(w))
    close(moe.moe_combine_tokens(rows, idx, w), ref, size, 8, "bfloat16")
    gy = up(rng.standard_normal((T, 2064)), "bfloat16")
    grows, gw = moe.moe_combine_tokens_grad(gy, rows, idx, ints(ox_token(row, T * 6), "int32"), w)
    ref_rows, ref_w, size = ox.combine_grad(down(gy), down(rows), row, down(w))
    close(grows, ref_rows, np.abs(ref_rows), 2, "bfloat16")
    close(gw, ref_w, size, row_ops(2064), "bfloat16")


# ----------------------------------------------------------------------------- norm

@pytest.mark.parametrize("T", [303, 304, 305, 2431, 2433])
@pytest.mark.parametrize("H", [256, 257, 1024, 1032, 2048, 2056, 4100, 2050, 2049])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_norm_grad_where_forms_meet(T, H, dt):
    """Rows by warps and by blocks, of 1 and 2 chunks a thread, in pieces of 16, 8, 4 and 2 bytes; one block an SM or two."""
    rng = np.random.default_rng(T + H)
    h, gy, gh = (up(rng.standard_normal((T, H)), dt) for _ in range(3))
    w = up(1 + 0.2 * rng.standard_normal(H), dt)
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=gh)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w), down(gh))
    close(gx, rx, sx, row_ops(H), dt)
    close(gw, rw, sw, row_ops(H) + T / 64 + 60, dt)


@pytest.mark.parametrize("H", [64, 1000, 4096])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_norm_grad_of_rows_near_zero(H, dt):
    """Rows of zeros and of 2^-52 under a small eps: r is 2^50, and its third power no float32."""
    eps = 2.0 ** -100
    rng = np.random.default_rng(H)
    h, gy = rng.standard_normal((9, H)), up(rng.standard_normal((9, H)), dt)
    h[3:6] *= 2.0 ** -52
    h[6:] = 0.0
    h, w = up(h, dt), up(1 + 0.2 * rng.standard_normal(H), dt)
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, eps=eps)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w), None, eps)
    assert np.isfinite(rx).all()
    close(gx, rx, sx, row_ops(H), dt)
    close(gw, rw, sw, row_ops(H) + 60, dt)


@pytest.mark.parametrize("H", [7168, 7176, 16384, 16392, 32768, 32776])
@pytest.mark.parametrize("dt", ["float16", "float32"])
def test_norm_of_long_rows(H, dt):
    T = 400
    rng = np.random.default_rng(H)
    x, res, gy = (up(rng.standard_normal((T, H)), dt) for _ in range(3))
    w = up(1 + 0.2 * rng.standard_normal(H), "float32")
    y, h, q, s = moe.moe_add_rms_norm(x, w, res, quant="mxfp8")
    h32 = down(x.float() + res.float())
    ry = ox.add_rms_norm(h32, down(w))[0]
    close(y, ry, np.abs(ry), row_ops(H), dt)
    check_quant(q, s, ry, "mxfp8", row_ops(H) + 64)
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w))
    close(gx, rx, sx, row_ops(H), dt)
    close(gw, rw, sw, row_ops(H) + T / 64 + 60, "float32")


@pytest.mark.parametrize("quant", ["int8", "e4m3", "e4m3_128"])
@pytest.mark.parametrize("T,H", [(1, 7168), (64, 1000), (2000, 2048), (400, 513)])
def test_codes_are_of_the_rounded_quotient(quant, T, H):
    """y in float32 is what the codes are made of: each is that of y / s in float32, to the bit."""
    rng = np.random.default_rng(T + H)
    x, w = up(rng.standard_normal((T, H)), "float32"), up(1 + 0.2 * rng.standard_normal(H), "float32")
    y, _, q, s = moe.moe_add_rms_norm(x, w, quant=quant)
    y, s = down(y).astype(np.float32), down(s).astype(np.float32).reshape(T, -1)
    block = 128 if quant == "e4m3_128" else H
    top = np.maximum.reduceat(np.abs(y), np.arange(0, H, block), axis=1)
    assert np.array_equal(s, top / np.float32(127 if quant == "int8" else 448))
    v = y / np.repeat(s, block, axis=1)[:, :H]
    want = np.clip(np.rint(v), -127, 127) if quant == "int8" else ox.nearest(v.astype(np.float64), ox.E4M3)
    assert np.array_equal(down(q.float()), want)


@pytest.mark.parametrize("H", [7168, 7176, 9218, 12288, 12292, 14336, 14344, 20480, 20482, 20488])
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
def test_norm_grad_of_long_rows(H, dt):
    """grad_h beside rows that fit three, two or, without it, two times into shared memory, or not at all."""
    T = 320
    rng = np.random.default_rng(H)
    h, gy, gh = (up(rng.standard_normal((T, H)), dt) for _ in range(3))
    w = up(1 + 0.2 * rng.standard_normal(H), "float32")
    gx, gw = moe.moe_add_rms_norm_grad(gy, h, w, grad_h=gh)
    rx, sx, rw, sw = ox.add_rms_norm_grad(down(gy), down(h), down(w), down(gh))
    close(gx, rx, sx, row_ops(H), dt)
    close(gw, rw, sw, row_ops(H) + T / 64 + 60, "float32")


@pytest.mark.parametrize("quant", ["int8", "e4m3", "e4m3_128", "mxfp8"])
@pytest.mark.parametrize("H", [1, 3, 7, 8, 9, 31, 33, 127, 129, 130, 132, 136, 1000])
@pytest.mark.parametrize("off", [0, 1, 4])
def test_codes_of_rows_that_begin_anywhere(quant, H, off):
    """Codes are stored, and values read back, across rows that begin at any byte; T of many rows and of one."""
    import torch

    rng = np.random.default_rng(H)
    for T in (1, 77):
        x = up(rng.standard_normal((T, H)), "bfloat16")
        w = up(1 + 0.2 * rng.standard_normal(H), "bfloat16")
        y, _, q, s = moe.moe_add_rms_norm(x, w, quant=quant)
        codes, each = check_quant(q, s, ox.add_rms_norm(down(x), down(w))[0], quant, row_ops(H) + 64)
        want = torch.from_numpy(codes * each).float()
        for out in (torch.float32, torch.bfloat16):
            assert torch.equal(moe.moe_dequantize_rows(q, s, out).cpu(), want.to(out))
            moved = offset(q.view(torch.uint8), off).view(q.dtype)
            assert torch.equal(moe.moe_dequantize_rows(moved, s, out).cpu(), want.to(out))


# ----------------------------------------------------------------------------- the routing's gradient

@pytest.mark.parametrize("e", [1, 3, 4, 128, 129, 132, 256, 260, 512, 516, 1000, 1001])
@pytest.mark.parametrize("norm_type", [0, 1, 2])
@pytest.mark.parametrize("out", [False, True])
def test_gating_grad_where_forms_meet(e, norm_type, out):
    """Rows in groups of four elements and single ones, of each width; few tokens and many."""
    rng = np.random.default_rng(e)
    k = min(e, 9)
    for T, dt in ((5, "float32"), (330, "bfloat16")):
        x, gy = up(2 * rng.standard_normal((T, e)), dt), up(rng.standard_normal((T, k)), dt)
        go = up(rng.standard_normal((T, e)), "float32") if out else None
        bias = up(0.1 * rng.random(e), dt)
        idx = np.stack([rng.permutation(e)[:k] for _ in range(T)])
        ref = ox.gating_grad(down(gy), down(x), idx, bias=down(bias), grad_out=None if go is None else down(go), norm_type=norm_type)
        ops = 3 * (e / 32 + k / 32) + 120
        for shift in (0, 1):                                        # 1: addresses that are no multiple of four elements
            gx, gb, _ = moe.moe_gating_top_k_grad(offset(gy, shift), offset(x, shift), ints(idx, "int32"), bias=offset(bias, shift),
                                                  grad_out=None if go is None else offset(go, shift), norm_type=norm_type)
            close(gx, ref[0], ref[1], ops, dt)
            close(gb, ref[2], ref[3], ops + T / 64 + 60, dt)


# ----------------------------------------------------------------------------- graphs

@pytest.mark.parametrize("T,k,E", [(600, 7, 30), (20000, 7, 30), (900, 8, 2000)])
def test_sort_in_a_graph(T, k, E):
    """The launches of each form captured, and replayed on other experts; two graphs replayed at once, on two streams."""
    import torch

    rng = np.random.default_rng(T)
    x = [torch.randint(0, 256, (T, 40), dtype=torch.uint8, device="cuda") for _ in range(2)]
    held = [ints(experts(rng, T, k, E), "int32") for _ in range(2)]
    moe.moe_sort_tokens(x[0], held[0], E)
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(moe.moe_sort_tokens(x[i], held[i], E))
        graphs.append(g)
    for _ in range(3):
        idx = [experts(rng, T, k, E, wrong=0.2) for _ in range(2)]
        for i in range(2):
            held[i].copy_(ints(idx[i], "int32"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            row, token, counts = ox.sort_tokens_at_once(idx[i], E)
            rows, _, gt, gr, num, _ = outs[i]
            assert np.array_equal(gr.cpu().numpy(), row) and np.array_equal(gt.cpu().numpy(), token)
            assert np.array_equal(num.cpu().numpy(), counts)
            at = torch.from_numpy(token).cuda()
            want = x[i][at.clamp(min=0) // k] * (at >= 0)[:, None].to(torch.uint8)
            assert torch.equal(rows, want)
