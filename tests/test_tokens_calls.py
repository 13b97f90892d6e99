"""What the operators around the experts refuse before any CUDA call (no GPU needed): the C entries with stand-in
addresses and one argument wrong, and a stream of another device."""
from types import SimpleNamespace

import pytest

import moe_expert_token_gb300 as moe
import moe_expert_token_gb300.mrr_v2 as m
from moe_expert_token_gb300 import build as mbuild
from moe_expert_token_gb300 import tokens as tk

A, B, C, D, E, F, G, W = (0x10000 * i for i in range(1, 9))     # never touched
F16, BF16, F32 = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()


def check(run, base, cases):
    for kw, code in cases:
        got = run(*{**base, **kw, "stream": None}.values())
        assert got == code, (kw, m.mrr_status_str(got))


def test_sort_rejects():
    base = dict(expert_idx=A, idx_is_i64=0, T=1000, k=8, first_expert=0, E=16, x=B, row_bytes=256, row_stride=256, scales=C,
                scale_row_bytes=4, weight=D, weight_dt=F32, sorted_x=E, sorted_scales=F, sorted_weight=G, token_idx=A, row_idx=B,
                expert_num=C, expert_num_type=1, workspace=W, workspace_bytes=1 << 20, stream=None)
    check(moe.moe_sort_run, base, [
        (dict(weight_dt=3), m.MRR_ERR_DTYPE), (dict(expert_num_type=2), m.MRR_ERR_ATTR), (dict(T=-1), m.MRR_ERR_SHAPE),
        (dict(k=0), m.MRR_ERR_SHAPE), (dict(k=65), m.MRR_ERR_SHAPE), (dict(E=0), m.MRR_ERR_SHAPE), (dict(E=4097), m.MRR_ERR_SHAPE),
        (dict(T=2 ** 31 // 8), m.MRR_ERR_SHAPE), (dict(row_bytes=-1), m.MRR_ERR_SHAPE), (dict(row_bytes=2 ** 24 + 1, row_stride=2 ** 25), m.MRR_ERR_SHAPE),
        (dict(row_stride=255), m.MRR_ERR_SHAPE), (dict(scale_row_bytes=0), m.MRR_ERR_SHAPE), (dict(scale_row_bytes=2 ** 20 + 1), m.MRR_ERR_SHAPE),
        (dict(expert_idx=None), m.MRR_ERR_NULL), (dict(x=None), m.MRR_ERR_NULL), (dict(sorted_x=None), m.MRR_ERR_NULL),
        (dict(sorted_scales=None), m.MRR_ERR_NULL), (dict(sorted_weight=None), m.MRR_ERR_NULL), (dict(token_idx=None), m.MRR_ERR_NULL),
        (dict(row_idx=None), m.MRR_ERR_NULL), (dict(expert_num=None), m.MRR_ERR_NULL), (dict(expert_idx=A + 2), m.MRR_ERR_ALIGN),
        (dict(expert_idx=A + 4, idx_is_i64=1), m.MRR_ERR_ALIGN), (dict(expert_num=C + 4, idx_is_i64=1), m.MRR_ERR_ALIGN),
        (dict(weight=D + 2), m.MRR_ERR_ALIGN), (dict(weight=D + 1, weight_dt=F16), m.MRR_ERR_ALIGN), (dict(sorted_weight=G + 2), m.MRR_ERR_ALIGN),
        (dict(token_idx=A + 1), m.MRR_ERR_ALIGN), (dict(workspace=None), m.MRR_ERR_WORKSPACE), (dict(workspace=W + 128), m.MRR_ERR_WORKSPACE),
        (dict(workspace_bytes=moe.moe_sort_workspace(1000, 8, 16) - 1), m.MRR_ERR_WORKSPACE)])


def test_sort_workspace():
    """None for what one launch does; bounded by 608 rows of counts; 0 out of range."""
    assert moe.moe_sort_workspace(512, 8, 4096) == 0 and moe.moe_sort_workspace(0, 8, 16) == 0
    for T, k, E_ in ((513, 8, 1), (16384, 8, 256), (65, 64, 4096), (2 ** 31 - 1, 1, 4096), (2 ** 25, 63, 7)):
        assert 0 < moe.moe_sort_workspace(T, k, E_) <= 608 * (E_ + 1) * 4 + 255
    assert moe.moe_sort_workspace(2 ** 31, 1, 4) == moe.moe_sort_workspace(-1, 1, 4) == moe.moe_sort_workspace(9000, 65, 4) == 0


def test_combine_rejects():
    base = dict(rows=A, dt=BF16, R=100, H=64, row_idx=B, T=10, k=4, weight=C, weight_dt=F32, y=D, stream=None)
    check(moe.moe_combine_run, base, [
        (dict(dt=3), m.MRR_ERR_DTYPE), (dict(weight_dt=3), m.MRR_ERR_DTYPE), (dict(R=-1), m.MRR_ERR_SHAPE), (dict(R=2 ** 31), m.MRR_ERR_SHAPE),
        (dict(H=0), m.MRR_ERR_SHAPE), (dict(H=2 ** 20 + 1), m.MRR_ERR_SHAPE), (dict(T=-1), m.MRR_ERR_SHAPE), (dict(k=0), m.MRR_ERR_SHAPE),
        (dict(k=65), m.MRR_ERR_SHAPE), (dict(T=2 ** 31 - 1), m.MRR_ERR_SHAPE), (dict(rows=None), m.MRR_ERR_NULL),
        (dict(row_idx=None), m.MRR_ERR_NULL), (dict(y=None), m.MRR_ERR_NULL), (dict(rows=A + 1), m.MRR_ERR_ALIGN),
        (dict(y=D + 2, dt=F32), m.MRR_ERR_ALIGN), (dict(row_idx=B + 2), m.MRR_ERR_ALIGN), (dict(weight=C + 2), m.MRR_ERR_ALIGN)])
    base = dict(grad_y=A, rows=B, dt=BF16, R=100, H=64, row_idx=C, token_idx=D, T=10, k=4, weight=E, weight_dt=F16, grad_rows=F,
                grad_weight=G, stream=None)
    check(moe.moe_combine_grad_run, base, [
        (dict(dt=4), m.MRR_ERR_DTYPE), (dict(H=0), m.MRR_ERR_SHAPE), (dict(grad_y=None), m.MRR_ERR_NULL), (dict(rows=None), m.MRR_ERR_NULL),
        (dict(token_idx=None), m.MRR_ERR_NULL), (dict(grad_rows=None), m.MRR_ERR_NULL), (dict(weight=None), m.MRR_ERR_NULL),
        (dict(grad_y=A + 1), m.MRR_ERR_ALIGN), (dict(token_idx=D + 2), m.MRR_ERR_ALIGN), (dict(grad_weight=G + 1), m.MRR_ERR_ALIGN)])


def test_norm_rejects():
    base = dict(x=A, residual=B, dt=BF16, T=10, H=64, x_stride=64, residual_stride=64, weight=C, weight_dt=BF16, eps=1e-6, h=D, y=E,
                quant=tk.MOE_Q_INT8, q=F, scales=G, stream=None)
    check(moe.moe_add_rms_norm_run, base, [
        (dict(dt=3), m.MRR_ERR_DTYPE), (dict(weight_dt=F16), m.MRR_ERR_DTYPE), (dict(quant=6), m.MRR_ERR_ATTR), (dict(eps=-1.0), m.MRR_ERR_ATTR),
        (dict(eps=float("nan")), m.MRR_ERR_ATTR), (dict(T=-1), m.MRR_ERR_SHAPE), (dict(T=2 ** 31), m.MRR_ERR_SHAPE), (dict(H=0), m.MRR_ERR_SHAPE),
        (dict(H=65537, x_stride=65537, residual_stride=65537), m.MRR_ERR_SHAPE), (dict(x_stride=63), m.MRR_ERR_SHAPE),
        (dict(residual_stride=63), m.MRR_ERR_SHAPE), (dict(x_stride=2 ** 31 + 1), m.MRR_ERR_SHAPE), (dict(H=63, quant=tk.MOE_Q_MXFP4), m.MRR_ERR_SHAPE),
        (dict(x=None), m.MRR_ERR_NULL), (dict(weight=None), m.MRR_ERR_NULL), (dict(q=None), m.MRR_ERR_NULL), (dict(scales=None), m.MRR_ERR_NULL),
        (dict(h=None, y=None, quant=0), m.MRR_ERR_NULL), (dict(x=A + 1), m.MRR_ERR_ALIGN), (dict(residual=B + 1), m.MRR_ERR_ALIGN),
        (dict(scales=G + 2), m.MRR_ERR_ALIGN), (dict(y=E + 1), m.MRR_ERR_ALIGN), (dict(weight=C + 2, weight_dt=F32), m.MRR_ERR_ALIGN)])
    base = dict(grad_y=A, h=B, grad_h=None, dt=BF16, T=10, H=64, weight=C, weight_dt=F32, eps=1e-6, grad_x=D, grad_weight=E, workspace=W,
                workspace_bytes=1 << 20, stream=None)
    check(moe.moe_add_rms_norm_grad_run, base, [
        (dict(dt=3), m.MRR_ERR_DTYPE), (dict(eps=-1.0), m.MRR_ERR_ATTR), (dict(H=65537), m.MRR_ERR_SHAPE), (dict(grad_y=None), m.MRR_ERR_NULL),
        (dict(h=None), m.MRR_ERR_NULL), (dict(grad_x=None), m.MRR_ERR_NULL), (dict(grad_h=F + 1), m.MRR_ERR_ALIGN), (dict(workspace=None), m.MRR_ERR_WORKSPACE),
        (dict(workspace=W + 4), m.MRR_ERR_WORKSPACE), (dict(workspace_bytes=moe.moe_add_rms_norm_grad_workspace(10, 64) - 1), m.MRR_ERR_WORKSPACE)])
    assert moe.moe_add_rms_norm_grad_workspace(-1, 64) == moe.moe_add_rms_norm_grad_workspace(1, 65537) == 0


def test_dequantize_rejects():
    base = dict(q=A, scales=B, quant=tk.MOE_Q_E4M3, T=10, H=64, dt=BF16, x=C, stream=None)
    check(moe.moe_dequantize_rows_run, base, [
        (dict(dt=3), m.MRR_ERR_DTYPE), (dict(quant=0), m.MRR_ERR_ATTR), (dict(quant=tk.MOE_Q_MXFP4), m.MRR_ERR_ATTR), (dict(T=-1), m.MRR_ERR_SHAPE),
        (dict(H=0), m.MRR_ERR_SHAPE), (dict(H=2 ** 20 + 1), m.MRR_ERR_SHAPE), (dict(T=2 ** 31), m.MRR_ERR_SHAPE), (dict(q=None), m.MRR_ERR_NULL),
        (dict(x=C + 1), m.MRR_ERR_ALIGN), (dict(scales=B + 2), m.MRR_ERR_ALIGN)])


def test_gating_grad_rejects():
    base = dict(grad_y=A, x=B, dt=F32, T=10, e=16, k=4, expert_idx=C, bias=D, additional_bias=None, additional_token_mask=None,
                grad_norm_out=None, routed_scaling_factor=1.0, eps=1e-20, norm_type=1, grad_x=E, grad_bias=F, grad_additional_bias=None,
                workspace=W, workspace_bytes=1 << 20, stream=None)
    check(moe.moe_gating_topk_grad_run, base, [
        (dict(dt=3), m.MRR_ERR_DTYPE), (dict(norm_type=3), m.MRR_ERR_ATTR), (dict(T=-1), m.MRR_ERR_SHAPE), (dict(e=1025), m.MRR_ERR_SHAPE),
        (dict(k=17), m.MRR_ERR_SHAPE), (dict(k=0), m.MRR_ERR_SHAPE), (dict(grad_y=None), m.MRR_ERR_NULL), (dict(expert_idx=None), m.MRR_ERR_NULL),
        (dict(grad_x=None), m.MRR_ERR_NULL), (dict(x=B + 2), m.MRR_ERR_ALIGN), (dict(grad_norm_out=G + 2), m.MRR_ERR_ALIGN),
        (dict(workspace=None), m.MRR_ERR_WORKSPACE), (dict(workspace_bytes=moe.moe_gating_topk_grad_workspace(10, 16) - 1), m.MRR_ERR_WORKSPACE)])
    assert moe.moe_gating_topk_grad_workspace(10, 1025) == 0


def test_a_stream_of_another_device_is_refused():
    import torch

    x = SimpleNamespace(device=torch.device("cuda", 0))
    stream = SimpleNamespace(device=torch.device("cuda", 1))
    for call, n in ((moe.moe_sort_tokens, 3), (moe.moe_combine_tokens, 2), (moe.moe_sort_tokens_grad, 2), (moe.moe_combine_tokens_grad, 4),
                    (moe.moe_add_rms_norm, 2), (moe.moe_add_rms_norm_grad, 3), (moe.moe_dequantize_rows, 2), (moe.moe_gating_top_k_grad, 3)):
        with pytest.raises(ValueError, match="stream"):
            call(*(x,) * n, stream=stream)


def test_sort_rejects_experts_past_the_integers():
    """first_expert + E - 1 has to be an int64: past it the subtraction that makes a slot's key would wrap, and -2^63 count as
    an expert held here.  (No workspace: what the range allows goes no further.)"""
    base = dict(expert_idx=A, idx_is_i64=1, T=1000, k=8, first_expert=0, E=16, x=B, row_bytes=256, row_stride=256, scales=None,
                scale_row_bytes=0, weight=None, weight_dt=F32, sorted_x=E, sorted_scales=None, sorted_weight=None, token_idx=A, row_idx=B,
                expert_num=C, expert_num_type=1, workspace=None, workspace_bytes=0, stream=None)
    check(moe.moe_sort_run, base, [
        (dict(first_expert=2 ** 63 - 15), m.MRR_ERR_SHAPE), (dict(first_expert=2 ** 63 - 1), m.MRR_ERR_SHAPE),
        (dict(first_expert=2 ** 63 - 4095, E=4096), m.MRR_ERR_SHAPE), (dict(first_expert=2 ** 63 - 16), m.MRR_ERR_WORKSPACE),
        (dict(first_expert=2 ** 63 - 1, E=1), m.MRR_ERR_WORKSPACE), (dict(first_expert=-2 ** 63), m.MRR_ERR_WORKSPACE)])


def test_sort_workspace_is_the_table():
    """A row of E + 1 counts for each of 64 chunks and one word, in whole 256 bytes, whatever T and k."""
    for T, k, E_ in ((513, 8, 1), (16384, 8, 256), (65, 64, 4096), (2 ** 31 - 1, 1, 4096), (2 ** 25, 63, 7)):
        assert moe.moe_sort_workspace(T, k, E_) == -(-4 * (64 * (E_ + 1) + 1) // 256) * 256
