"""The experts' side of the re-routing: MXFP4 rows, the experts' products, and a whole layer for a
few tokens.  ctypes binding of include/moe_mx.h and include/moe_layer.h (the ``*_run`` functions,
integer device addresses) and the torch-level calls on top of it.

``moe_mx_quantize`` makes the packed float4_e2m1 rows and e8m0 scales that ``moe_re_routing`` moves;
``moe_mx_grouped_matmul`` takes what it returns, with its expert_token_num;
``moe_few_token_layer`` runs router, top-k, experts and the weighted sum of a decode step at once.
A call given a ``stream`` of the tensors' device runs and allocates there; its results are that stream's.
Results have no gradient, whatever the inputs ask for: the operators are for inference.
Every step runs in the CUDA library; there is no other code path.
"""
from __future__ import annotations

from . import mrr_v2 as _m
from .mrr_v2 import MRR_OK, MrrError

MOE_F16, MOE_BF16, MOE_F32, MOE_MXFP4 = range(4)
MOE_LAYER_MAX_TOKENS = 64


# ---------------------------------------------------------------------------- C functions, same names

def moe_mx_quantize_run(x, dt, rows, K, row_stride, codes, scales, stream) -> int:
    return _m.load_library().moe_mx_quantize_run(x, dt, rows, K, row_stride, codes, scales, stream)


def moe_mx_dequantize_run(codes, scales, rows, K, dt, x, row_stride, stream) -> int:
    return _m.load_library().moe_mx_dequantize_run(codes, scales, rows, K, dt, x, row_stride, stream)


def moe_mx_grouped_workspace(E) -> int:
    return _m.load_library().moe_mx_grouped_workspace(E)


def moe_mx_grouped_run(codes, scales, A, K, expert_num, expert_num_is_i64, expert_num_type, E, w_codes, w_scales, N,
                       gated, row_weight, out, out_dt, out_scales, workspace, workspace_bytes, stream) -> int:
    return _m.load_library().moe_mx_grouped_run(
        codes, scales, A, K, expert_num, int(expert_num_is_i64), expert_num_type, E, w_codes, w_scales, N, int(gated),
        row_weight, out, out_dt, out_scales, workspace, workspace_bytes, stream)


def moe_few_token_layer_workspace(T, H, E, I, k) -> int:
    return _m.load_library().moe_few_token_layer_workspace(T, H, E, I, k)


def moe_few_token_layer_run(x, dt, T, H, w_router, E, bias, w13, w13_scales, w2, w2_scales, w_dt, I, k, k_group,
                            group_count, routed_scaling_factor, eps, group_select_mode, norm_type, y, topk_weight,
                            expert_idx, workspace, workspace_bytes, stream) -> int:
    return _m.load_library().moe_few_token_layer_run(
        x, dt, T, H, w_router, E, bias, w13, w13_scales, w2, w2_scales, w_dt, I, k, k_group, group_count,
        routed_scaling_factor, eps, group_select_mode, norm_type, y, topk_weight, expert_idx, workspace,
        workspace_bytes, stream)


# ---------------------------------------------------------------------------- torch-level calls

# A decode step makes a few of these calls for each layer, on kernels of a few microseconds: what a
# call does on the host counts.  So torch and the library are looked up once, and each call reads a
# tensor's properties once.
torch = None
_lib = None
_raw_stream = None     # a device's current stream as an integer, without a Stream object around it
_CODES = {}


def _load():
    """The library, with torch imported beside it."""
    global torch, _lib, _raw_stream
    if _lib is None:
        import torch as torch_

        torch = torch_
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _CODES.update({torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32})
        _lib = _m.load_library()
    return _lib


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(stream, dev, call, *args, **kw):
    """``call`` on tensors of ``dev`` with ``stream`` current: what it allocates belongs to that stream too."""
    if stream.device != dev:
        raise ValueError("stream must be one of the tensors' device")
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def _space(workspace, nbytes, dev):
    """The caller's workspace, which must be memory of the tensors' device, or a new one."""
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on the tensors' device")
    return workspace


def _run(function, name, args, dev, workspace=None, check_status=False):
    """Call ``function(*args, stream)`` on dev's current stream, with ``dev`` current."""
    handle = _raw_stream(dev.index)
    if dev.index == torch.cuda.current_device():
        st = function(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = function(*args, handle)
    if st != MRR_OK:
        raise MrrError(st, name)
    if check_status:
        with torch.cuda.device(dev):
            st = _m.mrr_v2_read_status(workspace.data_ptr(), workspace.numel(), handle)
        if st != MRR_OK:
            raise MrrError(st, "device")


def _check_mx(codes, scales, name):
    """Contiguous codes [..., K/2] and scales [..., ceil(K/64), 2] of one device; returns K."""
    if codes.dtype != torch.uint8 and codes.dtype != getattr(torch, "float4_e2m1fn_x2", None):
        raise TypeError(f"{name} must be packed float4_e2m1 bytes (uint8)")
    if scales is None or scales.element_size() != 1:
        raise TypeError(f"{name}'s scales must be e8m0 bytes")
    shape = codes.shape
    K = 2 * shape[-1]
    if scales.shape != (*shape[:-1], (K + 63) // 64, 2):
        raise ValueError(f"{name}'s scales must be [..., ceil(K/64), 2] for codes [..., K/2]")
    if not codes.is_cuda or scales.device != codes.device or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{name} and its scales must be contiguous CUDA tensors of one device")
    return K


def moe_mx_quantize(x, *, stream=None):
    """MXFP4 codes and scales of x's rows: x is [..., K] float16, bfloat16 or float32, K even, rows
    without gaps except that a 2-D x may have any row stride.  Returns (codes [..., K/2] uint8,
    scales [..., ceil(K/64), 2] uint8): the float4_e2m1 rows and e8m0 scales moe_re_routing takes.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, x.device, moe_mx_quantize, x)
    shape = x.shape
    if not x.is_cuda or not shape:
        raise ValueError("x must be a CUDA tensor of at least one dimension")
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError("x must be float16, bfloat16 or float32")
    K = stride = shape[-1]
    if K < 2 or K % 2:
        raise ValueError("x's last dimension must be even")
    if not x.is_contiguous():
        if len(shape) != 2 or x.stride(1) != 1 or x.stride(0) < K:
            raise ValueError("x must be contiguous, or 2-D with contiguous rows")
        stride = x.stride(0)
    lead, dev = shape[:-1], x.device
    codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((*lead, (K + 63) // 64, 2), dtype=torch.uint8, device=dev)
    _run(lib.moe_mx_quantize_run, "moe_mx_quantize_run",
         (x.data_ptr(), code, x.numel() // K, K, stride, codes.data_ptr(), scales.data_ptr()), dev)
    return codes, scales


def moe_mx_dequantize(codes, scales, dtype=None, *, stream=None):
    """The values [..., K] of MXFP4 codes [..., K/2] and scales [..., ceil(K/64), 2], in ``dtype``
    (float16, bfloat16, the default, or float32)."""
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, codes.device, moe_mx_dequantize, codes, scales, dtype)
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError("dtype must be float16, bfloat16 or float32")
    K = _check_mx(codes, scales, "codes")
    if K < 2:
        raise ValueError("codes' rows are empty")
    dev = codes.device
    x = torch.empty((*codes.shape[:-1], K), dtype=dtype, device=dev)
    _run(lib.moe_mx_dequantize_run, "moe_mx_dequantize_run",
         (codes.data_ptr(), scales.data_ptr(), x.numel() // K, K, code, x.data_ptr(), K), dev)
    return x


def moe_mx_grouped_matmul(tokens, scales, expert_token_num, weight, weight_scales, *, gated: bool = False,
                          out_dtype=None, row_weight=None, expert_token_num_type: int = 1, workspace=None,
                          stream=None, check_status: bool = False):
    """Each expert's product on its rows of expert-major MXFP4 tokens.

    tokens [A, K/2] and scales [A, ceil(K/64), 2]: MXFP4 rows, expert 0's first (moe_re_routing's
    permuted tokens and scales); expert_token_num [E] int32 or int64: its count (or, with
    expert_token_num_type 0, cumsum) output; weight [E, N, K/2] and weight_scales [E, N,
    ceil(K/64), 2]; with ``gated`` weight holds N/2 gate rows and then N/2 up rows for each expert
    and the result is silu(gate) * up.  row_weight ([A] or [A, 1] float32) scales the rows.

    Returns [A, N] (gated: [A, N/2]) in out_dtype (float16, bfloat16, the default, or float32), or
    for out_dtype "mxfp4" the pair (codes, scales).  Sums are float32 throughout.
    ``check_status=True`` synchronises and raises on counts that do not sum to A.
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, tokens.device, moe_mx_grouped_matmul, tokens, scales, expert_token_num, weight, weight_scales,
                   gated=gated, out_dtype=out_dtype, row_weight=row_weight,
                   expert_token_num_type=expert_token_num_type, workspace=workspace, check_status=check_status)
    K = _check_mx(tokens, scales, "tokens")
    if tokens.dim() != 2 or weight.dim() != 3:
        raise ValueError("tokens must be 2-D and weight 3-D")
    if _check_mx(weight, weight_scales, "weight") != K:
        raise ValueError("tokens and weight differ in K")
    A, dev, c = tokens.shape[0], tokens.device, expert_token_num
    E, N, _ = weight.shape
    if gated:
        if N % 2:
            raise ValueError("a gated weight has as many gate rows as up rows")
        N //= 2
    if c.dtype not in (torch.int32, torch.int64):
        raise TypeError("expert_token_num must be int32 or int64")
    if c.shape != (E,) or not c.is_contiguous() or c.device != dev or weight.device != dev:
        raise ValueError("expert_token_num must be contiguous [E] on the tokens' device, and weight be there too")
    if row_weight is not None and (row_weight.dtype != torch.float32 or row_weight.device != dev
                                   or tuple(row_weight.shape) not in ((A,), (A, 1)) or not row_weight.is_contiguous()):
        raise ValueError("row_weight must be contiguous float32 [A] or [A, 1] on the tokens' device")
    out_scales = None
    if isinstance(out_dtype, str) and out_dtype == "mxfp4":
        if N % 32:
            raise ValueError("an mxfp4 result needs a multiple of 32 columns")
        code = MOE_MXFP4
        out = torch.empty((A, N // 2), dtype=torch.uint8, device=dev)
        out_scales = torch.empty((A, (N + 63) // 64, 2), dtype=torch.uint8, device=dev)
    else:
        out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
        code = _CODES.get(out_dtype)
        if code is None:
            raise TypeError("out_dtype must be float16, bfloat16, float32 or 'mxfp4'")
        out = torch.empty((A, N), dtype=out_dtype, device=dev)
    workspace = _space(workspace, lib.moe_mx_grouped_workspace(E), dev)
    _run(lib.moe_mx_grouped_run, "moe_mx_grouped_run",
         (tokens.data_ptr(), scales.data_ptr(), A, K, c.data_ptr(), int(c.dtype == torch.int64), expert_token_num_type,
          E, weight.data_ptr(), weight_scales.data_ptr(), N, int(gated), _ptr(row_weight), out.data_ptr(), code,
          _ptr(out_scales), workspace.data_ptr(), workspace.numel()), dev, workspace, check_status)
    return out if out_scales is None else (out, out_scales)


def moe_few_token_layer(x, w_router, w13, w2, k: int, *, bias=None, w13_scales=None, w2_scales=None,
                        k_group: int = 1, group_count: int = 1, routed_scaling_factor: float = 1.0,
                        eps: float = 1e-20, group_select_mode: int = 0, norm_type: int = 0,
                        return_routing: bool = False, workspace=None, stream=None, check_status: bool = False):
    """A whole mixture-of-experts layer for up to 64 tokens (a decode step).

    x [T, H] float16 or bfloat16; w_router [E, H] and bias [E] in x's dtype; the experts' weights
    w13 [E, 2 I, H] (I gate rows, then I up rows) and w2 [E, H, I] in x's dtype, or MXFP4: uint8
    codes [E, 2 I, H/2] and [E, H, I/2] with w13_scales [E, 2 I, ceil(H/64), 2] and w2_scales.
    The gating arguments are moe_gating_top_k's; router logits and weights stay in float32.

    Returns y [T, H] in x's dtype, or with ``return_routing`` (y, weights [T, k] float32, experts
    [T, k] int32).
    """
    lib = _lib or _load()
    if stream is not None:
        return _on(stream, x.device, moe_few_token_layer, x, w_router, w13, w2, k, bias=bias, w13_scales=w13_scales,
                   w2_scales=w2_scales, k_group=k_group, group_count=group_count,
                   routed_scaling_factor=routed_scaling_factor, eps=eps, group_select_mode=group_select_mode,
                   norm_type=norm_type, return_routing=return_routing, workspace=workspace, check_status=check_status)
    if not x.is_cuda or x.dim() != 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D CUDA tensor")
    dtype, dev = x.dtype, x.device
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError("x must be float16 or bfloat16")
    dt = w_dt = _CODES[dtype]
    T, H = x.shape
    if w_router.dim() != 2 or w13.dim() != 3 or w2.dim() != 3:
        raise ValueError("w_router must be 2-D, w13 and w2 3-D")
    E, I = w_router.shape[0], w2.shape[2]
    if w13_scales is not None or w2_scales is not None:
        if _check_mx(w13, w13_scales, "w13") != H:
            raise ValueError("w13 must be [E, 2 I, H/2]")
        I = _check_mx(w2, w2_scales, "w2")
        w_dt = MOE_MXFP4
    elif w13.dtype is not dtype or w2.dtype is not dtype or w13.shape[2] != H:
        raise ValueError("w13 must be [E, 2 I, H] and w2 [E, H, I], in x's dtype")
    if w_router.dtype is not dtype or w_router.shape[1] != H or w13.shape[:2] != (E, 2 * I) or w2.shape[:2] != (E, H):
        raise ValueError("w_router must be [E, H] in x's dtype, w13 [E, 2 I, H] and w2 [E, H, I]")
    if bias is not None and (bias.dtype is not dtype or bias.shape != (E,) or not bias.is_contiguous()
                             or bias.device != dev):
        raise ValueError("bias must be contiguous [E] in x's dtype on x's device")
    for w in (w_router, w13, w2):
        if w.device != dev or not w.is_contiguous():
            raise ValueError("weights must be contiguous and on x's device")
    y = torch.empty_like(x)
    weight = idx = None
    if return_routing:
        weight = torch.empty((T, k), dtype=torch.float32, device=dev)
        idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    workspace = _space(workspace, lib.moe_few_token_layer_workspace(T, H, E, I, k), dev)
    _run(lib.moe_few_token_layer_run, "moe_few_token_layer_run",
         (x.data_ptr(), dt, T, H, w_router.data_ptr(), E, _ptr(bias), w13.data_ptr(), _ptr(w13_scales), w2.data_ptr(),
          _ptr(w2_scales), w_dt, I, k, k_group, group_count, routed_scaling_factor, eps, group_select_mode, norm_type,
          y.data_ptr(), _ptr(weight), _ptr(idx), workspace.data_ptr(), workspace.numel()), dev, workspace, check_status)
    return (y, weight, idx) if return_routing else y
