"""Pins of the expert operators' CPU oracle, and the operators' refusals (no GPU needed)."""
import numpy as np
import pytest

from moe_expert_token_gb300 import build as mbuild
from moe_expert_token_gb300 import experts as x
import moe_expert_token_gb300.mrr_v2 as m
from oracle import experts as ox


def test_every_code_round_trips():
    """All 16 codes under a block maximum of 6 give themselves back, whatever the scale."""
    for e in (-100, -3, 0, 7, 90):
        v = np.tile(np.ldexp(ox.VALUES, e), 2)[None]
        q, s = ox.mx_quantize(v)
        assert s[0, 0, 0] == 127 + e and s[0, 0, 1] == 127
        assert q[0].tolist() == [(2 * i) % 16 | ((2 * i + 1) % 16) << 4 for i in range(16)]
        assert np.array_equal(ox.mx_values(q, s), v)


def test_rounding_by_hand():
    """Ties go to the even code, magnitudes above 6 to 6 (block maximum 7: scale 1)."""
    v = np.zeros((1, 32))
    v[0, :12] = [7, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 5.01, 0.2501, -0.24]
    q, s = ox.mx_quantize(v)
    assert s[0, 0, 0] == 127
    assert ox.mx_values(q, s)[0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4, 6, 0.5, 0]


def test_scales_by_hand():
    """2^(floor(log2 max) - 2): max 4 -> 1, max 3.99 -> 1/2, max 1 -> 1/4; zeros -> byte 0; not finite -> 255."""
    v = np.zeros((1, 32 * 6))
    v[0, 0], v[0, 32], v[0, 64], v[0, 128], v[0, 160] = 4, 3.99, -1, np.inf, np.nan
    _, s = ox.mx_quantize(v)
    assert s.reshape(-1).tolist() == [127, 126, 125, 0, 255, 255]


def test_grouped_by_hand():
    x_ = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    w = np.array([[[1.0, 0.0]], [[0.0, 1.0]], [[1.0, 1.0]]])
    assert ox.grouped(x_, [1, 0, 2], w, row_weight=np.array([1, 1, 0.5]))[0].ravel().tolist() == [1.0, 7.0, 5.5]
    w2 = np.array([[[1.0, 0.0], [0.0, 1.0]]])
    h = ox.grouped(x_, [3], w2, gate=True)[0].ravel()
    assert np.allclose(h, [2 / (1 + np.exp(-1)), 12 / (1 + np.exp(-3)), 30 / (1 + np.exp(-5))])


def test_layer_by_hand():
    """Two identity-like experts: y is the weighted sum of what each gives."""
    x_ = np.array([[1.0, -1.0]])
    w13 = np.array([[[1.0, 0.0], [2.0, 0.0]], [[0.0, -1.0], [0.0, 3.0]]])
    w2 = np.array([[[1.0], [0.0]], [[0.0], [2.0]]])
    y, _ = ox.layer(x_, np.array([[0.25, 0.75]]), np.array([[0, 1]]), np.zeros(1), w13, w2, 0.0)
    s = 1 / (1 + np.exp(-1))
    assert np.allclose(y, [[0.25 * s * 2, 0.75 * s * -3 * 2]])


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return m.load_library()


# stand-in addresses that are never dereferenced: every error below is found before any CUDA call
P = [0x10000 * i for i in range(1, 16)]


def test_quantize_refusals(lib):
    def q(**kw):
        a = dict(x=P[0], dt=x.MOE_BF16, rows=4, K=64, row_stride=64, codes=P[1], scales=P[2], stream=None)
        a.update(kw)
        return x.moe_mx_quantize_run(**a)

    assert q(dt=3) == m.MRR_ERR_DTYPE
    assert q(dt=-1) == m.MRR_ERR_DTYPE
    assert q(rows=-1) == m.MRR_ERR_SHAPE
    assert q(K=63, row_stride=63) == m.MRR_ERR_SHAPE
    assert q(K=0) == m.MRR_ERR_SHAPE
    assert q(row_stride=63) == m.MRR_ERR_SHAPE
    assert q(x=None) == q(codes=None) == q(scales=None) == m.MRR_ERR_NULL
    assert q(x=P[0] + 1) == m.MRR_ERR_ALIGN
    assert q(x=P[0] + 2, dt=x.MOE_F32) == m.MRR_ERR_ALIGN
    assert q(rows=0, x=None, codes=None, scales=None) == m.MRR_OK
    assert x.moe_mx_dequantize_run(P[0], P[1], 4, 64, 3, P[2], 64, None) == m.MRR_ERR_DTYPE
    assert x.moe_mx_dequantize_run(P[0], None, 4, 64, 0, P[2], 64, None) == m.MRR_ERR_NULL
    assert x.moe_mx_dequantize_run(P[0], P[1], 4, 62, 0, P[2], 60, None) == m.MRR_ERR_SHAPE


def test_grouped_refusals(lib):
    def g(**kw):
        a = dict(codes=P[0], scales=P[1], A=16, K=64, expert_num=P[2], expert_num_is_i64=0, expert_num_type=1, E=4,
                 w_codes=P[3], w_scales=P[4], N=32, gated=0, row_weight=None, out=P[5], out_dt=x.MOE_BF16,
                 out_scales=None, workspace=P[6], workspace_bytes=1 << 20, stream=None)
        a.update(kw)
        return m.load_library().moe_mx_grouped_run(*a.values())

    assert x.moe_mx_grouped_workspace(4) <= 1 << 20 and x.moe_mx_grouped_workspace(0) == 0
    assert g(out_dt=4) == m.MRR_ERR_DTYPE
    assert g(expert_num_is_i64=2) == m.MRR_ERR_DTYPE
    assert g(expert_num_type=2) == m.MRR_ERR_ATTR
    assert g(gated=2) == m.MRR_ERR_ATTR
    for kw in (dict(A=-1), dict(A=2 ** 31), dict(K=0), dict(K=48), dict(E=0), dict(E=4097), dict(N=0),
               dict(N=2 ** 20 + 1), dict(out_dt=x.MOE_MXFP4, out_scales=P[7], N=48)):
        assert g(**kw) == m.MRR_ERR_SHAPE, kw
    for name in ("codes", "scales", "expert_num", "w_codes", "w_scales", "out"):
        assert g(**{name: None}) == m.MRR_ERR_NULL, name
    assert g(out_dt=x.MOE_MXFP4) == m.MRR_ERR_NULL                 # no out_scales
    for kw in (dict(codes=P[0] + 8), dict(w_codes=P[3] + 8), dict(scales=P[1] + 1), dict(w_scales=P[4] + 1),
               dict(expert_num=P[2] + 2), dict(expert_num=P[2] + 4, expert_num_is_i64=1), dict(row_weight=P[7] + 2),
               dict(out=P[5] + 1)):
        assert g(**kw) == m.MRR_ERR_ALIGN, kw
    for kw in (dict(workspace=None), dict(workspace=P[6] + 16), dict(workspace_bytes=64)):
        assert g(**kw) == m.MRR_ERR_WORKSPACE, kw


def test_layer_refusals(lib):
    def f(**kw):
        a = dict(x=P[0], dt=x.MOE_BF16, T=2, H=64, w_router=P[1], E=8, bias=None, w13=P[2], w13_scales=None, w2=P[3],
                 w2_scales=None, w_dt=x.MOE_BF16, I=32, k=2, k_group=1, group_count=1, routed_scaling_factor=1.0,
                 eps=1e-20, group_select_mode=0, norm_type=0, y=P[4], topk_weight=None, expert_idx=None,
                 workspace=P[5], workspace_bytes=1 << 30, stream=None)
        a.update(kw)
        return x.moe_few_token_layer_run(**a)

    mx = dict(w_dt=x.MOE_MXFP4, w13_scales=P[6], w2_scales=P[7])
    assert f(dt=x.MOE_F32, w_dt=x.MOE_F32) == m.MRR_ERR_DTYPE
    assert f(w_dt=x.MOE_F16) == m.MRR_ERR_DTYPE                      # weights of another 16-bit type than x
    for kw in (dict(group_select_mode=2), dict(norm_type=3), dict(norm_type=-1)):
        assert f(**kw) == m.MRR_ERR_ATTR, kw
    for kw in (dict(T=-1), dict(T=65), dict(H=0), dict(H=65537), dict(I=0), dict(E=0), dict(E=1025), dict(k=0),
               dict(k=9), dict(k_group=2), dict(group_count=3), dict(group_count=4, k_group=1, k=3),
               dict(group_count=8, k_group=4, group_select_mode=1), dict(H=63, **mx), dict(I=31, **mx)):
        assert f(**kw) == m.MRR_ERR_SHAPE, kw
    for name in ("x", "w_router", "w13", "w2", "y"):
        assert f(**{name: None}) == m.MRR_ERR_NULL, name
    assert f(**dict(mx, w2_scales=None)) == m.MRR_ERR_NULL
    for kw in (dict(x=P[0] + 1), dict(w13=P[2] + 1), dict(bias=P[8] + 1), dict(topk_weight=P[8] + 2), dict(y=P[4] + 1)):
        assert f(**kw) == m.MRR_ERR_ALIGN, kw
    for kw in (dict(workspace=None), dict(workspace=P[5] + 8), dict(workspace_bytes=4096)):
        assert f(**kw) == m.MRR_ERR_WORKSPACE, kw
    assert x.moe_few_token_layer_workspace(65, 64, 8, 32, 2) == 0
    assert x.moe_few_token_layer_workspace(64, 64, 8, 32, 2) > 0


def test_header_functions_are_exported(lib):
    """Every moe_ function the two headers declare is in the library and bound."""
    import os
    import re

    names = set()
    for h in ("moe_mx.h", "moe_layer.h"):
        text = re.sub(r"/\*.*?\*/", "", open(os.path.join(mbuild.INCLUDE, h), encoding="utf-8").read(), flags=re.S)
        names |= set(re.findall(r"^(?:mrr_status|size_t)\s+(moe_\w+)\s*\(", text, flags=re.M))
    assert names == {"moe_mx_quantize_run", "moe_mx_dequantize_run", "moe_mx_grouped_workspace", "moe_mx_grouped_run",
                     "moe_few_token_layer_workspace", "moe_few_token_layer_run"}
    for n in names:
        assert hasattr(lib, n) and callable(getattr(x, n))
