"""What stands around the experts on one rank: the norm in front of them, the tokens' way to expert order and
back, and the gradients of these and of the routing.  ctypes binding of include/moe_tokens.h, include/moe_norm.h and
include/moe_gating_grad.h (the ``*_run`` functions, integer device addresses) and the torch-level
calls on top of it.

``moe_add_rms_norm`` gives the router its input and the exchange its rows in 8 bits or MXFP4;
``moe_sort_tokens`` lays tokens out by their experts, as ``moe_re_routing`` and ``moe_mx_grouped_matmul`` take them;
``moe_combine_tokens`` brings the experts' rows back, weighted and summed.  Their gradients are calls of their own
(``*_grad``), with which a training loop builds its backward pass: results carry no gradient of torch's.
A call given a ``stream`` of the tensors' device runs and allocates there; its results are that stream's.
Calls may be captured in a CUDA graph.  Every step runs in the CUDA library; there is no other code path.
"""
from __future__ import annotations

from . import experts as _x
from . import mrr_v2 as _m
from .experts import _on, _ptr, _run, _space

MOE_Q_NONE, MOE_Q_INT8, MOE_Q_E4M3, MOE_Q_E4M3_128, MOE_Q_MXFP8, MOE_Q_MXFP4 = range(6)
QUANT_CODES = {None: MOE_Q_NONE, "int8": MOE_Q_INT8, "e4m3": MOE_Q_E4M3, "e4m3_128": MOE_Q_E4M3_128,
               "mxfp8": MOE_Q_MXFP8, "mxfp4": MOE_Q_MXFP4}


# ---------------------------------------------------------------------------- C functions, same names

def moe_sort_workspace(T, k, E) -> int:
    return _m.load_library().moe_sort_workspace(T, k, E)


def moe_sort_run(expert_idx, idx_is_i64, T, k, first_expert, E, x, row_bytes, row_stride, scales, scale_row_bytes, weight,
                 weight_dt, sorted_x, sorted_scales, sorted_weight, token_idx, row_idx, expert_num, expert_num_type,
                 workspace, workspace_bytes, stream) -> int:
    return _m.load_library().moe_sort_run(
        expert_idx, int(idx_is_i64), T, k, first_expert, E, x, row_bytes, row_stride, scales, scale_row_bytes, weight,
        weight_dt, sorted_x, sorted_scales, sorted_weight, token_idx, row_idx, expert_num, expert_num_type, workspace,
        workspace_bytes, stream)


def moe_combine_run(rows, dt, R, H, row_idx, T, k, weight, weight_dt, y, stream) -> int:
    return _m.load_library().moe_combine_run(rows, dt, R, H, row_idx, T, k, weight, weight_dt, y, stream)


def moe_combine_grad_run(grad_y, rows, dt, R, H, row_idx, token_idx, T, k, weight, weight_dt, grad_rows, grad_weight,
                         stream) -> int:
    return _m.load_library().moe_combine_grad_run(grad_y, rows, dt, R, H, row_idx, token_idx, T, k, weight, weight_dt,
                                                  grad_rows, grad_weight, stream)


def moe_add_rms_norm_run(x, residual, dt, T, H, x_stride, residual_stride, weight, weight_dt, eps, h, y, quant, q, scales,
                         stream) -> int:
    return _m.load_library().moe_add_rms_norm_run(x, residual, dt, T, H, x_stride, residual_stride, weight, weight_dt, eps,
                                                  h, y, quant, q, scales, stream)


def moe_add_rms_norm_grad_workspace(T, H) -> int:
    return _m.load_library().moe_add_rms_norm_grad_workspace(T, H)


def moe_add_rms_norm_grad_run(grad_y, h, grad_h, dt, T, H, weight, weight_dt, eps, grad_x, grad_weight, workspace,
                              workspace_bytes, stream) -> int:
    return _m.load_library().moe_add_rms_norm_grad_run(grad_y, h, grad_h, dt, T, H, weight, weight_dt, eps, grad_x,
                                                       grad_weight, workspace, workspace_bytes, stream)


def moe_dequantize_rows_run(q, scales, quant, T, H, dt, x, stream) -> int:
    return _m.load_library().moe_dequantize_rows_run(q, scales, quant, T, H, dt, x, stream)


def moe_gating_topk_grad_workspace(T, e) -> int:
    return _m.load_library().moe_gating_topk_grad_workspace(T, e)


def moe_gating_topk_grad_run(grad_y, x, dt, T, e, k, expert_idx, bias, additional_bias, additional_token_mask,
                             grad_norm_out, routed_scaling_factor, eps, norm_type, grad_x, grad_bias,
                             grad_additional_bias, workspace, workspace_bytes, stream) -> int:
    return _m.load_library().moe_gating_topk_grad_run(
        grad_y, x, dt, T, e, k, expert_idx, bias, additional_bias, additional_token_mask, grad_norm_out,
        routed_scaling_factor, eps, norm_type, grad_x, grad_bias, grad_additional_bias, workspace, workspace_bytes, stream)


# ---------------------------------------------------------------------------- torch-level calls

# As in experts.py, torch and the library are looked up once: what a call does on the host counts beside
# kernels of a few microseconds.
torch = None
_lib = None
_empty = _i32 = _i64 = _f32 = _u8 = None
_CODES = {}


def _load():
    global torch, _lib, _empty, _i32, _i64, _f32, _u8
    if _lib is None:
        lib = _x._load()
        torch = _x.torch
        _CODES.update(_x._CODES)
        _empty, _i32, _i64, _f32, _u8 = torch.empty, torch.int32, torch.int64, torch.float32, torch.uint8
        _lib = lib
    return _lib


def _stride_of(x, name):
    """The row stride, in elements, of x as [T, H] rows without gaps inside a row."""
    if not x.is_cuda or x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with rows of one element or more")
    T, H = x.shape
    if T < 2 or x.is_contiguous():
        if H > 1 and T and x.stride(1) != 1:
            raise ValueError(f"{name} must have contiguous rows")
        return H
    stride = x.stride(0)
    if (H > 1 and x.stride(1) != 1) or stride < H:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return stride


def _slots(t, dev, name):
    """The shape of an int32 index [T, k]."""
    shape = t.shape
    if t.dtype is not _i32 or len(shape) != 2 or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [T, k] on the tensors' device")
    return shape


def _weight(weight, shape, dev, name):
    """The code of a weight [T, k]."""
    code = _CODES.get(weight.dtype)
    if code is None:
        raise TypeError(f"{name} must be float16, bfloat16 or float32")
    if weight.shape != shape or weight.device != dev or not weight.is_contiguous():
        raise ValueError(f"{name} must be contiguous {list(shape)} on the tensors' device")
    return code


def _bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def moe_sort_tokens(x, expert_idx, num_experts: int, *, first_expert: int = 0, per_token_scales=None,
                    expert_topk_weight=None, expert_token_num_type: int = 1, workspace=None, stream=None):
    """Tokens laid out by the experts chosen for them.

    x [T, H] of any type (packed types by their bytes), rows without gaps inside, any row stride;
    expert_idx [T, k] int32 or int64: the experts of each token, as moe_gating_top_k gives them; the experts
    held here are first_expert .. first_expert + num_experts - 1, and any other value (-1 in a padded token)
    has no row.  per_token_scales [T, ...] of any type and expert_topk_weight [T, k] (float16, bfloat16 or
    float32) move with the rows.

    Returns (sorted_x [T k, H], sorted_scales [T k, ...] or None, token_idx [T k] int32, row_idx [T, k] int32,
    expert_token_num [num_experts] in expert_idx's type, sorted_weight [T k, 1] float32 or None): expert 0's rows in
    the tokens' order, then expert 1's, and behind the last one a row of zeros for each slot without a row;
    token_idx gives a row's slot t * k + j (-1 for zeros), row_idx a slot's row (-1 for none).
    expert_token_num_type 1: counts, 0: their inclusive prefix.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, x.device, moe_sort_tokens, x, expert_idx, num_experts, first_expert=first_expert,
                   per_token_scales=per_token_scales, expert_topk_weight=expert_topk_weight,
                   expert_token_num_type=expert_token_num_type, workspace=workspace)
    stride = _stride_of(x, "x")
    (T, H), dev, kind, slots = x.shape, x.device, expert_idx.dtype, expert_idx.shape
    if kind is not _i32 and kind is not _i64:
        raise TypeError("expert_idx must be int32 or int64")
    if len(slots) != 2 or slots[0] != T or expert_idx.device != dev or not expert_idx.is_contiguous():
        raise ValueError("expert_idx must be contiguous [T, k] on x's device")
    k = slots[1]
    if not 1 <= k <= 64 or not 1 <= num_experts <= 4096:
        raise ValueError("k must be in 1..64 and num_experts in 1..4096")
    if not -2 ** 63 <= first_expert < 2 ** 63 - 4096:
        raise ValueError("first_expert is out of range")
    scales, weight, n, size = per_token_scales, expert_topk_weight, T * k, x.element_size()
    sorted_scales = sorted_weight = None
    scale_bytes = weight_dt = 0
    if scales is not None:
        scale_shape = scales.shape
        if not scale_shape or scale_shape[0] != T or scales.device != dev or not scales.is_contiguous():
            raise ValueError("per_token_scales must be contiguous [T, ...] on x's device")
        scale_bytes = scales.element_size()
        for d in scale_shape[1:]:
            scale_bytes *= d
        if scale_bytes == 0:
            raise ValueError("per_token_scales' rows are empty")
        sorted_scales = _empty((n, *scale_shape[1:]), dtype=scales.dtype, device=dev)
    if weight is not None:
        weight_dt = _weight(weight, slots, dev, "expert_topk_weight")
        sorted_weight = _empty((n, 1), dtype=_f32, device=dev)
    sorted_x = _empty((n, H), dtype=x.dtype, device=dev)
    token_idx = _empty(n, dtype=_i32, device=dev)
    row_idx = _empty(slots, dtype=_i32, device=dev)
    num = _empty(num_experts, dtype=kind, device=dev)
    if n > 4096 or workspace is not None:   # (none is needed for fewer slots)
        workspace = _space(workspace, lib.moe_sort_workspace(T, k, num_experts), dev)
    _run(lib.moe_sort_run, "moe_sort_run",
         (expert_idx.data_ptr(), int(kind is _i64), T, k, first_expert, num_experts, x.data_ptr(), H * size,
          stride * size, _ptr(scales), scale_bytes, _ptr(weight), weight_dt, sorted_x.data_ptr(), _ptr(sorted_scales),
          _ptr(sorted_weight), token_idx.data_ptr(), row_idx.data_ptr(), num.data_ptr(), expert_token_num_type,
          _ptr(workspace), _bytes(workspace)), dev)
    return sorted_x, sorted_scales, token_idx, row_idx, num, sorted_weight


def moe_combine_tokens(rows, row_idx, weight=None, *, stream=None):
    """The experts' rows back to their tokens: y[t] = sum over j of weight[t, j] * rows[row_idx[t, j]].

    rows [R, H] float16, bfloat16 or float32, contiguous; row_idx [T, k] int32 as moe_sort_tokens returns it (an
    entry outside 0 .. R - 1 adds nothing); weight [T, k] float16, bfloat16 or float32, or None: each row counts
    once.  Sums are float32, in the order of j.  Returns [T, H] in rows' type.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, rows.device, moe_combine_tokens, rows, row_idx, weight)
    shape, dev = rows.shape, rows.device
    code = _CODES.get(rows.dtype)
    if code is None:
        raise TypeError("rows must be float16, bfloat16 or float32")
    if len(shape) != 2 or not shape[1] or not rows.is_cuda or not rows.is_contiguous():
        raise ValueError("rows must be a contiguous 2-D CUDA tensor")
    R, H = shape
    T, k = slots = _slots(row_idx, dev, "row_idx")
    weight_dt = 0 if weight is None else _weight(weight, slots, dev, "weight")
    y = _empty((T, H), dtype=rows.dtype, device=dev)
    _run(lib.moe_combine_run, "moe_combine_run",
         (rows.data_ptr(), code, R, H, row_idx.data_ptr(), T, k, _ptr(weight), weight_dt, y.data_ptr()), dev)
    return y


def moe_sort_tokens_grad(grad_sorted_x, row_idx, *, stream=None):
    """The gradient of moe_sort_tokens with respect to x [T, H]: each token's rows of grad_sorted_x [T k, H], summed.

    That of the weights it moves, [T, k] from grad_sorted_weight [T k, 1], is a combine with one slot a token:
    ``moe_combine_tokens(grad_sorted_weight, row_idx.view(-1, 1)).view(row_idx.shape)``, 0 for slots without a row.
    """
    return moe_combine_tokens(grad_sorted_x, row_idx, stream=stream)


def moe_combine_tokens_grad(grad_y, rows, row_idx, token_idx, weight=None, *, stream=None):
    """The gradient of moe_combine_tokens with respect to rows and weight.

    grad_y [T, H] and rows [R, H] in one type, contiguous; row_idx [T, k] and token_idx [R] of the moe_sort_tokens
    that made the order (no row is two slots').  Returns (grad_rows [R, H], grad_weight [T, k] in weight's type, or
    None without a weight); rows whose token_idx is negative get zeros, slots without a row 0.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, grad_y.device, moe_combine_tokens_grad, grad_y, rows, row_idx, token_idx, weight)
    shape, dev, dtype = grad_y.shape, grad_y.device, grad_y.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("grad_y must be float16, bfloat16 or float32")
    if rows.dtype is not dtype:
        raise TypeError("rows must have grad_y's type")
    if len(shape) != 2 or not shape[1] or not grad_y.is_cuda or not grad_y.is_contiguous():
        raise ValueError("grad_y must be a contiguous 2-D CUDA tensor")
    T, H = shape
    if rows.dim() != 2 or rows.shape[1] != H or rows.device != dev or not rows.is_contiguous():
        raise ValueError("rows must be contiguous [R, H] on grad_y's device")
    R = rows.shape[0]
    slots = _slots(row_idx, dev, "row_idx")
    if slots[0] != T:
        raise ValueError("row_idx must be [T, k]")
    if token_idx.dtype is not _i32 or token_idx.shape != (R,) or token_idx.device != dev or not token_idx.is_contiguous():
        raise ValueError("token_idx must be contiguous int32 [R] on the tensors' device")
    weight_dt, grad_weight = 0, None
    if weight is not None:
        weight_dt = _weight(weight, slots, dev, "weight")
        grad_weight = _empty(slots, dtype=weight.dtype, device=dev)
    grad_rows = _empty((R, H), dtype=dtype, device=dev)
    _run(lib.moe_combine_grad_run, "moe_combine_grad_run",
         (grad_y.data_ptr(), rows.data_ptr(), code, R, H, row_idx.data_ptr(), token_idx.data_ptr(), T, slots[1],
          _ptr(weight), weight_dt, grad_rows.data_ptr(), _ptr(grad_weight)), dev)
    return grad_rows, grad_weight


def _norm_weight(weight, dtype, H, dev):
    if weight.dtype is not dtype and weight.dtype is not _f32:
        raise TypeError("weight must be float32 or of the rows' type")
    if weight.shape != (H,) or weight.device != dev or not weight.is_contiguous():
        raise ValueError("weight must be contiguous [H] on the rows' device")
    return _CODES[weight.dtype]


def moe_add_rms_norm(x, weight, residual=None, *, eps: float = 1e-6, quant=None, return_y: bool = True, stream=None):
    """h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight, and y in 8 bits or MXFP4.

    x and residual [T, H] float16, bfloat16 or float32, rows without gaps inside, any row stride; weight [H] in their
    type or float32.  quant:
      "int8"      int8 rows, scales [T] float32
      "e4m3"      float8_e4m3fn rows, scales [T] float32
      "e4m3_128"  float8_e4m3fn rows, scales [T, ceil(H/128)] float32
      "mxfp8"     float8_e4m3fn rows, scales [T, ceil(H/64), 2] e8m0 bytes
      "mxfp4"     packed e2m1 codes [T, H/2], scales [T, ceil(H/64), 2] e8m0 bytes (H even)
    which are the rows and per_token_scales that moe_sort_tokens and moe_re_routing move, and the last ones what
    moe_mx_grouped_matmul takes.

    Returns (y, h, q, scales): y and h in x's type (y None without ``return_y``, h x itself without a residual), q and
    scales None without quant.  y is made of the float32 sum, the rows in 8 bits of the float32 y.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, x.device, moe_add_rms_norm, x, weight, residual, eps=eps, quant=quant, return_y=return_y)
    stride = _stride_of(x, "x")
    shape, dtype, dev = x.shape, x.dtype, x.device
    T, H = shape
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("x must be float16, bfloat16 or float32")
    kind = QUANT_CODES.get(quant)
    if kind is None:
        raise ValueError(f"quant must be one of {list(QUANT_CODES)}")
    if kind == MOE_Q_NONE and not return_y and residual is None:
        raise ValueError("nothing is asked for")
    if not eps >= 0.0:
        raise ValueError("eps must not be negative")
    weight_dt = _norm_weight(weight, dtype, H, dev)
    h, h_out, residual_stride = x, None, 0
    if residual is not None:
        residual_stride = _stride_of(residual, "residual")
        if residual.dtype is not dtype or residual.shape != shape or residual.device != dev:
            raise ValueError("residual must be like x")
        h = _empty(shape, dtype=dtype, device=dev)
        h_out = h.data_ptr()
    y = _empty(shape, dtype=dtype, device=dev) if return_y else None
    q = scales = None
    if kind == MOE_Q_MXFP4:
        if H % 2:
            raise ValueError("mxfp4 rows need an even H")
        q = _empty((T, H // 2), dtype=_u8, device=dev)
    elif kind != MOE_Q_NONE:
        q = _empty(shape, dtype=torch.int8 if kind == MOE_Q_INT8 else torch.float8_e4m3fn, device=dev)
    if kind == MOE_Q_MXFP8 or kind == MOE_Q_MXFP4:
        scales = _empty((T, (H + 63) // 64, 2), dtype=_u8, device=dev)
    elif kind != MOE_Q_NONE:
        scales = _empty((T, (H + 127) // 128) if kind == MOE_Q_E4M3_128 else (T,), dtype=_f32, device=dev)
    _run(lib.moe_add_rms_norm_run, "moe_add_rms_norm_run",
         (x.data_ptr(), _ptr(residual), code, T, H, stride, residual_stride, weight.data_ptr(), weight_dt, eps, h_out,
          _ptr(y), kind, _ptr(q), _ptr(scales)), dev)
    return y, h, q, scales


def moe_add_rms_norm_grad(grad_y, h, weight, *, grad_h=None, eps: float = 1e-6, workspace=None, stream=None):
    """The gradient of moe_add_rms_norm's y (and, with grad_h, of its h) with respect to x, which is the residual's too,
    and to weight.  grad_y, h and grad_h [T, H] in one type, contiguous; h as moe_add_rms_norm returned it (without a residual
    that is x itself: a contiguous copy of one with gaps between its rows).
    Returns (grad_x [T, H], grad_weight [H] in weight's type)."""
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, h.device, moe_add_rms_norm_grad, grad_y, h, weight, grad_h=grad_h, eps=eps, workspace=workspace)
    shape, dtype, dev = h.shape, h.dtype, h.device
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("h must be float16, bfloat16 or float32")
    if len(shape) != 2 or not shape[1] or not h.is_cuda:
        raise ValueError("h must be a 2-D CUDA tensor with rows of one element or more")
    for t in (grad_y, h) if grad_h is None else (grad_y, h, grad_h):
        if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
            raise ValueError("grad_y, h and grad_h must be contiguous [T, H] of one type and device")
    if not eps >= 0.0:
        raise ValueError("eps must not be negative")
    T, H = shape
    weight_dt = _norm_weight(weight, dtype, H, dev)
    grad_x = _empty(shape, dtype=dtype, device=dev)
    grad_weight = _empty(H, dtype=weight.dtype, device=dev)
    workspace = _space(workspace, lib.moe_add_rms_norm_grad_workspace(T, H), dev)
    _run(lib.moe_add_rms_norm_grad_run, "moe_add_rms_norm_grad_run",
         (grad_y.data_ptr(), h.data_ptr(), _ptr(grad_h), code, T, H, weight.data_ptr(), weight_dt, eps,
          grad_x.data_ptr(), grad_weight.data_ptr(), workspace.data_ptr(), _bytes(workspace)), dev)
    return grad_x, grad_weight


def moe_dequantize_rows(q, scales, dtype=None, *, stream=None):
    """The values [T, H] of rows in 8 bits, as moe_add_rms_norm makes them and the re-routing moves them, in ``dtype``
    (float16, bfloat16, the default, or float32): int8 with float32 scales [T], or float8_e4m3fn with float32 scales [T] or
    [T, ceil(H/128)], or with e8m0 bytes [T, ceil(H/64), 2].  (MXFP4 rows: moe_mx_dequantize.)"""
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, q.device, moe_dequantize_rows, q, scales, dtype)
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("dtype must be float16, bfloat16 or float32")
    is_int8, shape, dev = q.dtype is torch.int8, q.shape, q.device
    if not is_int8 and q.dtype is not torch.float8_e4m3fn:
        raise TypeError("q must be int8 or float8_e4m3fn")
    if len(shape) != 2 or not shape[1] or not q.is_cuda or not q.is_contiguous():
        raise ValueError("q must be a contiguous 2-D CUDA tensor")
    if scales.device != dev or not scales.is_contiguous():
        raise ValueError("scales must be contiguous and on q's device")
    T, H = shape
    of, is_f32 = scales.shape, scales.dtype is _f32
    if is_f32 and (of == (T,) or is_int8 and of == (T, 1)):
        kind = MOE_Q_INT8 if is_int8 else MOE_Q_E4M3
    elif is_f32 and not is_int8 and of == (T, (H + 127) // 128):
        kind = MOE_Q_E4M3_128
    elif not is_int8 and scales.element_size() == 1 and of == (T, (H + 63) // 64, 2):
        kind = MOE_Q_MXFP8
    else:
        raise ValueError("scales must be float32 [T] (int8 also [T, 1], e4m3 also [T, ceil(H/128)]), or with e4m3 rows "
                         "e8m0 bytes [T, ceil(H/64), 2]")
    x = _empty(shape, dtype=dtype, device=dev)
    _run(lib.moe_dequantize_rows_run, "moe_dequantize_rows_run",
         (q.data_ptr(), scales.data_ptr(), kind, T, H, code, x.data_ptr()), dev)
    return x


def moe_gating_top_k_grad(grad_y, x, expert_idx, *, bias=None, additional_bias=None, additional_token_mask=None,
                          grad_out=None, routed_scaling_factor: float = 1.0, eps: float = 1e-20, norm_type: int = 0,
                          workspace=None, stream=None):
    """The gradient of moe_gating_top_k's weights y (and, with grad_out, of its normalised scores) with respect to the
    logits x and the biases, for the experts that were chosen.

    grad_y and expert_idx [T, k] (or [b, s, k]) and x [T, e] (or [b, s, e]), grad_y in x's type, expert_idx int32;
    bias, additional_bias, additional_token_mask, routed_scaling_factor, eps and norm_type as the call had them;
    grad_out float32 like x.  Returns (grad_x like x, grad_bias [e] or None, grad_additional_bias [e] or None), in x's
    type; the choice of experts itself has no gradient.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, x.device, moe_gating_top_k_grad, grad_y, x, expert_idx, bias=bias,
                   additional_bias=additional_bias, additional_token_mask=additional_token_mask, grad_out=grad_out,
                   routed_scaling_factor=routed_scaling_factor, eps=eps, norm_type=norm_type, workspace=workspace)
    if not x.is_cuda or not x.is_contiguous() or x.dim() not in (2, 3):
        raise ValueError("x must be a contiguous 2-D or 3-D CUDA tensor")
    dtype, dev = x.dtype, x.device
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("x must be float16, bfloat16 or float32")
    shape, of = x.shape, expert_idx.shape
    e, k = shape[-1], of[-1]
    if expert_idx.dtype is not _i32 or of[:-1] != shape[:-1] or expert_idx.device != dev or not expert_idx.is_contiguous():
        raise ValueError("expert_idx must be contiguous int32 [..., k] on x's device")
    if grad_y.dtype is not dtype or grad_y.shape != of or grad_y.device != dev or not grad_y.is_contiguous():
        raise ValueError("grad_y must be contiguous [..., k] in x's type on x's device")
    if grad_out is not None and (grad_out.dtype is not _f32 or grad_out.shape != shape
                                 or grad_out.device != dev or not grad_out.is_contiguous()):
        raise ValueError("grad_out must be contiguous float32 like x")
    T = 1
    for d in shape[:-1]:
        T *= d
    for b in (bias, additional_bias):
        if b is not None and (b.dtype is not dtype or b.numel() != e or b.device != dev or not b.is_contiguous()):
            raise ValueError("bias / additional_bias must be contiguous [e] in x's dtype on x's device")
    mask = additional_token_mask
    if mask is not None:
        if mask.dtype is not torch.bool or mask.numel() != T or mask.device != dev or not mask.is_contiguous():
            raise ValueError("additional_token_mask must be contiguous [T] bool on x's device")
    grad_x = _empty(shape, dtype=dtype, device=dev)
    grad_bias = None if bias is None else _empty(e, dtype=dtype, device=dev)
    grad_extra = None if additional_bias is None else _empty(e, dtype=dtype, device=dev)
    if bias is not None or additional_bias is not None or workspace is not None:
        workspace = _space(workspace, lib.moe_gating_topk_grad_workspace(T, e), dev)
    _run(lib.moe_gating_topk_grad_run, "moe_gating_topk_grad_run",
         (grad_y.data_ptr(), x.data_ptr(), code, T, e, k, expert_idx.data_ptr(), _ptr(bias), _ptr(additional_bias),
          _ptr(mask), _ptr(grad_out), routed_scaling_factor, eps, norm_type, grad_x.data_ptr(), _ptr(grad_bias),
          _ptr(grad_extra), _ptr(workspace), _bytes(workspace)), dev)
    return grad_x, grad_bias, grad_extra
