"""ctypes binding of the operators around the expert layer
(include/ops/moe_ops.h), with the C ABI's own names.

As in ``_lib``: argument marshalling only, and no fallback.  Every tensor is
a torch device tensor of the current device; results go to tensors the
caller passes.  Element types, shapes and strides are checked here (the
pointers handed over then mean what the header says) and again by the
library.  ``stream`` defaults to torch's current stream; with another one the
caller orders it against the tensors' own, as for any torch tensor.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import MOE_DT_BF16, MOE_DT_F32, MOE_DT_U8, _check, _ptr, _stream

MOE_EPI_NONE = 0
MOE_EPI_SILU = 1
MOE_EPI_GELU = 2
MOE_EPI_SILU_MUL = 3

OPS_EXPORTED = ("moe_rmsnorm", "moe_mxfp8_linear", "moe_mxfp8_linear_workspace", "moe_dispatch",
                "moe_dispatch_workspace", "moe_dispatch_backward", "moe_combine", "moe_combine_backward")

_i32, _i64, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class moe_rmsnorm_args(ctypes.Structure):
    _fields_ = [("x", _vp), ("x_stride", _i64), ("x_dtype", _i32), ("residual_dtype", _i32),
                ("residual", _vp), ("residual_stride", _i64), ("residual_out", _vp),
                ("residual_out_stride", _i64), ("weight", _vp), ("weight_dtype", _i32), ("reserved", _i32),
                ("eps", ctypes.c_double), ("y", _vp), ("y_stride", _i64), ("codes", _vp), ("scales", _vp),
                ("num_tokens", _i64), ("hidden", _i64)]


class moe_mxfp8_linear_args(ctypes.Structure):
    _fields_ = [("x_codes", _vp), ("x_scales", _vp), ("w_tiles", _vp), ("w_scales", _vp), ("bias", _vp),
                ("residual", _vp), ("residual_stride", _i64), ("out", _vp), ("out_stride", _i64),
                ("out_codes", _vp), ("out_scales", _vp), ("workspace", _vp), ("workspace_bytes", _i64),
                ("num_tokens", _i64), ("rows", _i64), ("inner", _i64), ("activation", _i32),
                ("reserved", _i32)]


class moe_dispatch_args(ctypes.Structure):
    _fields_ = [("ids", _vp), ("x", _vp), ("x_stride", _i64), ("x_scales", _vp), ("counts", _vp),
                ("offsets", _vp), ("sorted", _vp), ("pos", _vp), ("rows", _vp), ("row_scales", _vp),
                ("workspace", _vp), ("workspace_bytes", _i64), ("num_tokens", _i64),
                ("num_experts", _i64), ("hidden", _i64), ("top_k", _i32), ("dtype", _i32)]


class moe_combine_args(ctypes.Structure):
    _fields_ = [("rows", _vp), ("rows_stride", _i64), ("weights", _vp), ("pos", _vp), ("out", _vp),
                ("out_stride", _i64), ("dout", _vp), ("dout_stride", _i64), ("drows", _vp),
                ("drows_stride", _i64), ("dweights", _vp), ("num_tokens", _i64), ("num_rows", _i64),
                ("hidden", _i64), ("top_k", _i32), ("rows_dtype", _i32), ("out_dtype", _i32),
                ("reserved", _i32)]


_ready = None


def ops_lib() -> ctypes.CDLL:
    """The HIP library with the operators' signatures set."""
    global _ready
    L = _lib.lib()
    if _ready is not L:
        for name, args in (("moe_rmsnorm", moe_rmsnorm_args), ("moe_mxfp8_linear", moe_mxfp8_linear_args),
                           ("moe_dispatch", moe_dispatch_args), ("moe_combine", moe_combine_args),
                           ("moe_combine_backward", moe_combine_args),
                           ("moe_dispatch_backward", moe_combine_args)):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = ctypes.c_int, [ctypes.POINTER(args), _vp]
        L.moe_mxfp8_linear_workspace.restype = _i64
        L.moe_mxfp8_linear_workspace.argtypes = [_i64, _i64, _i64, _i32]
        L.moe_dispatch_workspace.restype = _i64
        L.moe_dispatch_workspace.argtypes = [_i64, _i64, _i32]
        _ready = L
    return L


def _want(t, name, dtypes, shape, strided=False):
    """t is a tensor of the current device with one of the element types and
    the shape, contiguous or (``strided``, two dimensions) with contiguous
    rows.  Returns the distance between its rows in elements."""
    import torch
    if t.dtype not in dtypes or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: expected a tensor of the current device, got {t.device}")
    if t.is_contiguous():
        return t.shape[-1] if t.dim() == 2 else 0
    if not strided or (t.shape[1] > 1 and t.stride(1) != 1) or t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: expected contiguous {'rows' if strided else 'memory'}, got strides {t.stride()}")
    return t.stride(0)


def _dt(t):
    import torch
    return {torch.bfloat16: MOE_DT_BF16, torch.float32: MOE_DT_F32, torch.uint8: MOE_DT_U8}[t.dtype]


def _floats():
    import torch
    return (torch.bfloat16, torch.float32)


def moe_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, y=None, codes=None, scales=None,
                stream=None, check: bool = True) -> int:
    """n = s * weight / sqrt(mean(s^2) + eps), s = x + residual.

    x [T, H] and residual [T, H] bfloat16 or float32, weight [H] bfloat16 or
    float32.  Writes those given of residual_out [T, H] (s, the residual's
    type; may be ``residual`` itself), y [T, H] bfloat16, and codes [T, H] with
    scales [T, H/32] uint8 (MXFP8).  Rows of x, residual, residual_out and y
    may be strided."""
    import torch
    if x.dim() != 2:
        raise ValueError(f"x: expected [tokens, hidden], got {tuple(x.shape)}")
    T, H = x.shape
    a = moe_rmsnorm_args(num_tokens=T, hidden=H, eps=eps, x=_ptr(x), weight=_ptr(weight))
    a.x_stride = _want(x, "x", _floats(), (T, H), strided=True)
    a.x_dtype = _dt(x)
    _want(weight, "weight", _floats(), (H,))
    a.weight_dtype = _dt(weight)
    if residual is not None:
        a.residual, a.residual_stride = _ptr(residual), _want(residual, "residual", _floats(), (T, H), strided=True)
        a.residual_dtype = _dt(residual)
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out: given without residual")
        a.residual_out = _ptr(residual_out)
        a.residual_out_stride = _want(residual_out, "residual_out", (residual.dtype,), (T, H), strided=True)
    if y is not None:
        a.y, a.y_stride = _ptr(y), _want(y, "y", (torch.bfloat16,), (T, H), strided=True)
    if codes is not None:
        _want(codes, "codes", (torch.uint8,), (T, H))
        a.codes = _ptr(codes)
    if scales is not None:
        _want(scales, "scales", (torch.uint8,), (T, H // 32))
        a.scales = _ptr(scales)
    rc = ops_lib().moe_rmsnorm(ctypes.byref(a), _stream(stream))
    return _check(rc, "moe_rmsnorm") if check else rc


def moe_mxfp8_linear_workspace(num_tokens: int, rows: int, inner: int, activation: int = MOE_EPI_NONE) -> int:
    """Bytes of workspace of a moe_mxfp8_linear call of these sizes."""
    n = ops_lib().moe_mxfp8_linear_workspace(num_tokens, rows, inner, activation)
    return n if n >= 0 else _check(n, "moe_mxfp8_linear_workspace")


def moe_mxfp8_linear(x_codes, x_scales, w_tiles, w_scales, out=None, out_codes=None, out_scales=None,
                     bias=None, activation: int = MOE_EPI_NONE, residual=None, workspace=None, stream=None,
                     check: bool = True) -> int:
    """act(x W^T + bias) + residual.

    x_codes [T, K], x_scales [T, K/32]; w_tiles [rows, K], w_scales
    [rows, K/32] as written by moe_mxfp8_prepack (gate_up_pairs for
    MOE_EPI_SILU_MUL), all uint8; bias [rows] float32; residual and out
    [T, cols] bfloat16 (rows may be strided; ``residual`` may be ``out``), or
    out_codes [T, cols] and out_scales [T, cols/32] uint8, where cols is rows,
    or rows / 2 for MOE_EPI_SILU_MUL.  workspace: a uint8 tensor of at least
    moe_mxfp8_linear_workspace(...) bytes, or None if that is 0."""
    import torch
    u8 = (torch.uint8,)
    if x_codes.dim() != 2 or w_tiles.dim() != 2:
        raise ValueError(f"expected x_codes [tokens, inner] and w_tiles [rows, inner], got {tuple(x_codes.shape)} "
                         f"and {tuple(w_tiles.shape)}")
    T, K = x_codes.shape
    rows = w_tiles.shape[0]
    cols = rows // 2 if activation == MOE_EPI_SILU_MUL else rows
    _want(x_codes, "x_codes", u8, (T, K))
    _want(x_scales, "x_scales", u8, (T, K // 32))
    _want(w_tiles, "w_tiles", u8, (rows, K))
    _want(w_scales, "w_scales", u8, (rows, K // 32))
    a = moe_mxfp8_linear_args(x_codes=_ptr(x_codes), x_scales=_ptr(x_scales), w_tiles=_ptr(w_tiles),
                              w_scales=_ptr(w_scales), num_tokens=T, rows=rows, inner=K, activation=activation)
    if bias is not None:
        _want(bias, "bias", (torch.float32,), (rows,))
        a.bias = _ptr(bias)
    if residual is not None:
        a.residual = _ptr(residual)
        a.residual_stride = _want(residual, "residual", (torch.bfloat16,), (T, cols), strided=True)
    if out is not None:
        a.out, a.out_stride = _ptr(out), _want(out, "out", (torch.bfloat16,), (T, cols), strided=True)
    if out_codes is not None:
        _want(out_codes, "out_codes", u8, (T, cols))
        a.out_codes = _ptr(out_codes)
    if out_scales is not None:
        _want(out_scales, "out_scales", u8, (T, cols // 32))
        a.out_scales = _ptr(out_scales)
    if workspace is not None:
        _want(workspace, "workspace", u8, workspace.shape)
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    rc = ops_lib().moe_mxfp8_linear(ctypes.byref(a), _stream(stream))
    return _check(rc, "moe_mxfp8_linear") if check else rc


def moe_dispatch_workspace(num_tokens: int, num_experts: int, top_k: int) -> int:
    """Bytes of workspace of a moe_dispatch call of these sizes."""
    n = ops_lib().moe_dispatch_workspace(num_tokens, num_experts, top_k)
    return n if n >= 0 else _check(n, "moe_dispatch_workspace")


def moe_dispatch(x, ids, num_experts: int, offsets, sorted, pos, rows, workspace=None, x_scales=None,
                 row_scales=None, counts=None, stream=None, check: bool = True) -> int:
    """The slots of ids [T, k] int32 sorted by expert, and the rows of x.

    Writes offsets [E + 1], sorted [T * k] (may be None), pos [T, k], counts
    [E] (optional), all int32, and rows [T * k, H] (x and rows None: the order
    alone).  x [T, H] bfloat16 or float32 (rows may be strided), or uint8 with
    x_scales [T, H/32] and row_scales [T * k, H/32] uint8 (MXFP8).  A slot
    whose id is outside 0 .. num_experts-1 gets pos -1 and no row; sorted and
    rows behind offsets[E] are left as they were.  workspace: a uint8 tensor
    of at least moe_dispatch_workspace(...) bytes, or None if that is 0."""
    import torch
    i32, u8 = (torch.int32,), (torch.uint8,)
    if ids.dim() != 2:
        raise ValueError(f"ids: expected [tokens, top_k], got {tuple(ids.shape)}")
    T, k = ids.shape
    _want(ids, "ids", i32, (T, k))
    _want(offsets, "offsets", i32, (num_experts + 1,))
    _want(pos, "pos", i32, (T, k))
    a = moe_dispatch_args(ids=_ptr(ids), offsets=_ptr(offsets), pos=_ptr(pos), num_tokens=T,
                          num_experts=num_experts, top_k=k)
    if sorted is not None:
        _want(sorted, "sorted", i32, (T * k,))
        a.sorted = _ptr(sorted)
    if counts is not None:
        _want(counts, "counts", i32, (num_experts,))
        a.counts = _ptr(counts)
    if (x is None) != (rows is None):
        raise ValueError("x and rows: both or neither")
    if x is not None:
        if x.dim() != 2:
            raise ValueError(f"x: expected [tokens, hidden], got {tuple(x.shape)}")
        H = x.shape[1]
        mx = x.dtype == torch.uint8
        a.hidden, a.x, a.rows = H, _ptr(x), _ptr(rows)
        a.x_stride = _want(x, "x", (*_floats(), torch.uint8), (T, H), strided=True)
        a.dtype = _dt(x)
        _want(rows, "rows", (x.dtype,), (T * k, H))
        if mx != (x_scales is not None) or mx != (row_scales is not None):
            raise ValueError("x_scales and row_scales: with uint8 rows (MXFP8), and only with them")
        if mx:
            _want(x_scales, "x_scales", u8, (T, H // 32))
            _want(row_scales, "row_scales", u8, (T * k, H // 32))
            a.x_scales, a.row_scales = _ptr(x_scales), _ptr(row_scales)
    if workspace is not None:
        _want(workspace, "workspace", u8, workspace.shape)
        a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    rc = ops_lib().moe_dispatch(ctypes.byref(a), _stream(stream))
    return _check(rc, "moe_dispatch") if check else rc


def _slots(pos, weights, top):
    import torch
    if pos.dim() != 2:
        raise ValueError(f"pos: expected [tokens, top_k], got {tuple(pos.shape)}")
    _want(pos, "pos", (torch.int32,), pos.shape)
    if weights is not None:
        _want(weights, "weights", (torch.float32,), pos.shape)
    if top.dim() != 2 or top.shape[0] != pos.shape[0]:
        raise ValueError(f"expected [{pos.shape[0]}, hidden] token rows, got {tuple(top.shape)}")
    return moe_combine_args(pos=_ptr(pos), weights=_ptr(weights), num_tokens=pos.shape[0], top_k=pos.shape[1],
                            hidden=top.shape[1], out_dtype=_dt(top) if top.dtype in _floats() else 0)


def _combine(name, rows, weights, pos, out, stream, check):
    a = _slots(pos, weights, out)
    n = rows.shape[0]
    a.rows_stride = _want(rows, "rows", _floats(), (n, out.shape[1]), strided=True)
    a.rows, a.num_rows, a.rows_dtype = _ptr(rows), n, _dt(rows)
    a.out, a.out_stride = _ptr(out), _want(out, "out", _floats(), tuple(out.shape), strided=True)
    rc = getattr(ops_lib(), name)(ctypes.byref(a), _stream(stream))
    return _check(rc, name) if check else rc


def moe_combine(rows, weights, pos, out, stream=None, check: bool = True) -> int:
    """out[t] = sum_j weights[t, j] * rows[pos[t, j]], over the slots with
    pos >= 0.  rows [R, H] and out [T, H] bfloat16 or float32 (rows may be
    strided), weights [T, k] float32 or None (weight 1), pos [T, k] int32."""
    return _combine("moe_combine", rows, weights, pos, out, stream, check)


def moe_dispatch_backward(drows, pos, dx, stream=None, check: bool = True) -> int:
    """dx[t] = sum_j drows[pos[t, j]]: the gradient of moe_dispatch's rows."""
    return _combine("moe_dispatch_backward", drows, None, pos, dx, stream, check)


def moe_combine_backward(dout, rows, weights, pos, drows=None, dweights=None, stream=None,
                         check: bool = True) -> int:
    """The gradients of moe_combine: drows[pos[t, j]] = weights[t, j] * dout[t]
    (rows without a slot are left as they were) and dweights[t, j] =
    <dout[t], rows[pos[t, j]]>.  Either may be None; rows [R, H] gives the
    rows' type and is read for dweights only.  ``drows`` may be ``rows``."""
    import torch
    a = _slots(pos, weights, dout)
    n, H = rows.shape[0], dout.shape[1]
    a.rows_stride = _want(rows, "rows", _floats(), (n, H), strided=True)
    a.rows, a.num_rows, a.rows_dtype = _ptr(rows), n, _dt(rows)
    a.dout, a.dout_stride = _ptr(dout), _want(dout, "dout", _floats(), tuple(dout.shape), strided=True)
    if drows is not None:
        a.drows, a.drows_stride = _ptr(drows), _want(drows, "drows", (rows.dtype,), (n, H), strided=True)
    if dweights is not None:
        _want(dweights, "dweights", (torch.float32,), pos.shape)
        a.dweights = _ptr(dweights)
    rc = ops_lib().moe_combine_backward(ctypes.byref(a), _stream(stream))
    return _check(rc, "moe_combine_backward") if check else rc
