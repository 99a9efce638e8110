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
import struct

import torch

from . import _lib
from ._lib import MOE_DT_BF16, MOE_DT_F32, MOE_DT_U8, _check

MOE_EPI_NONE = 0
MOE_EPI_SILU = 1
MOE_EPI_GELU = 2
MOE_EPI_SILU_MUL = 3

OPS_EXPORTED = ("moe_rmsnorm", "moe_mxfp8_linear", "moe_mxfp8_linear_workspace", "moe_dispatch",
                "moe_dispatch_workspace", "moe_dispatch_backward", "moe_combine", "moe_combine_backward",
                "moe_mxfp4_forward_mx8")

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


_FORMAT = {_vp: "Q", _i64: "q", _i32: "i", ctypes.c_double: "d"}


def _packer(struct_type):
    """The pack function of an argument structure: its fields in order, with
    the compiler's own alignment.  A call hands the library the packed bytes
    (building a ctypes structure field by field costs several microseconds,
    as much as the smallest operators' GPU time)."""
    s = struct.Struct("@" + "".join(_FORMAT[t] for _, t in struct_type._fields_))
    assert s.size == ctypes.sizeof(struct_type)
    return s.pack


_pack_rmsnorm = _packer(moe_rmsnorm_args)
_pack_linear = _packer(moe_mxfp8_linear_args)
_pack_dispatch = _packer(moe_dispatch_args)
_pack_combine = _packer(moe_combine_args)

_ready = None
_entry = {}


def ops_lib() -> ctypes.CDLL:
    """The HIP library with the operators' signatures set."""
    global _ready
    L = _lib.lib()
    if _ready is not L:
        for name in OPS_EXPORTED:
            if name.endswith("_workspace") or name == "moe_mxfp4_forward_mx8":
                continue
            getattr(L, name).restype, getattr(L, name).argtypes = ctypes.c_int, [_vp, _vp]
            _entry[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, _vp)((name, L))
        L.moe_mxfp8_linear_workspace.restype = _i64
        L.moe_mxfp8_linear_workspace.argtypes = [_i64, _i64, _i64, _i32]
        L.moe_dispatch_workspace.restype = _i64
        L.moe_dispatch_workspace.argtypes = [_i64, _i64, _i32]
        L.moe_mxfp4_forward_mx8.restype = ctypes.c_int
        L.moe_mxfp4_forward_mx8.argtypes = [_vp, _vp, _vp, _i64, _i32, _vp, _vp, ctypes.POINTER(_lib.moe_mxfp4_scales),
                                            _vp, _vp, ctypes.POINTER(_lib.moe_mxfp4_options)]
        _ready = L
    return L


# the current stream's handle without the Stream object around it, and the
# current device without a check of the initialisation that a device tensor
# has made (torch's own generated code asks this way; 0.1 us against 3 us and
# 0.3)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: _lib._stream(None))
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, packed, dev, stream, check):
    if _ready is None:
        ops_lib()
    rc = _entry[name](packed, _current_stream(dev) if stream is None else _lib._stream(stream))
    return _check(rc, name) if check and rc else rc


def _want(t, name, dtypes, shape, dev, strided=False):
    """t is a tensor of device `dev` with one of the element types and the
    shape, contiguous or (``strided``, two dimensions) with contiguous rows.
    Returns its address."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == dev and (t.is_contiguous() or (
            strided and (shape[1] <= 1 or t.stride(1) == 1) and t.stride(0) >= shape[1])):
        return t.data_ptr()
    if t.dtype not in dtypes or t.shape != shape:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor of the current device, got {t.device}")
    raise ValueError(f"{name}: expected contiguous {'rows' if strided else 'memory'}, got strides {t.stride()}")


def _row(t):
    """The distance between t's rows (any, where it has one row at most)."""
    return t.stride(0) if t.shape[0] > 1 else 0


_BF16, _F32, _U8, _I32 = (torch.bfloat16,), (torch.float32,), (torch.uint8,), (torch.int32,)
_FLOATS = _BF16 + _F32
_ROWS = _FLOATS + _U8
_DT = {torch.bfloat16: MOE_DT_BF16, torch.float32: MOE_DT_F32, torch.uint8: MOE_DT_U8}


def _dev(t):
    """The current device, if t is a device tensor (no context is made for a
    host tensor, which then fails its check)."""
    return _device() if t.is_cuda else 0


def _matrix(t, name, what):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected {what}, got {tuple(t.shape)}")
    return t.shape


def moe_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, y=None, codes=None, scales=None,
                stream=None, check: bool = True) -> int:
    """n = s * weight / sqrt(mean(s^2) + eps), s = x + residual.

    x [T, H] and residual [T, H] bfloat16 or float32, weight [H] bfloat16 or
    float32.  Writes those given of residual_out [T, H] (s, the residual's
    type; may be ``residual`` itself), y [T, H] bfloat16, and codes [T, H] with
    scales [T, H/32] uint8 (MXFP8).  Rows of x, residual, residual_out and y
    may be strided."""
    shape = T, H = _matrix(x, "x", "[tokens, hidden]")
    dev = _dev(x)
    px, pw = _want(x, "x", _FLOATS, shape, dev, True), _want(weight, "weight", _FLOATS, (H,), dev)
    pr = ld_r = po = ld_o = py = ld_y = dt_r = 0
    if residual is not None:
        pr, ld_r, dt_r = _want(residual, "residual", _FLOATS, shape, dev, True), _row(residual), _DT[residual.dtype]
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out: given without residual")
        po, ld_o = _want(residual_out, "residual_out", (residual.dtype,), shape, dev, True), _row(residual_out)
    if y is not None:
        py, ld_y = _want(y, "y", _BF16, shape, dev, True), _row(y)
    pc = 0 if codes is None else _want(codes, "codes", _U8, shape, dev)
    ps = 0 if scales is None else _want(scales, "scales", _U8, (T, H // 32), dev)
    return _call("moe_rmsnorm", _pack_rmsnorm(px, _row(x), _DT[x.dtype], dt_r, pr, ld_r, po, ld_o, pw,
                                              _DT[weight.dtype], 0, eps, py, ld_y, pc, ps, T, H), dev, stream, check)


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
    T, K = _matrix(x_codes, "x_codes", "[tokens, inner]")
    rows = _matrix(w_tiles, "w_tiles", "[rows, inner]")[0]
    cols = rows // 2 if activation == MOE_EPI_SILU_MUL else rows
    dev = _dev(x_codes)
    px, pxs = _want(x_codes, "x_codes", _U8, (T, K), dev), _want(x_scales, "x_scales", _U8, (T, K // 32), dev)
    pw, pws = _want(w_tiles, "w_tiles", _U8, (rows, K), dev), _want(w_scales, "w_scales", _U8, (rows, K // 32), dev)
    pr = ld_r = po = ld_o = nw = 0
    pb = 0 if bias is None else _want(bias, "bias", _F32, (rows,), dev)
    if residual is not None:
        pr, ld_r = _want(residual, "residual", _BF16, (T, cols), dev, True), _row(residual)
    if out is not None:
        po, ld_o = _want(out, "out", _BF16, (T, cols), dev, True), _row(out)
    pc = 0 if out_codes is None else _want(out_codes, "out_codes", _U8, (T, cols), dev)
    ps = 0 if out_scales is None else _want(out_scales, "out_scales", _U8, (T, cols // 32), dev)
    pk = 0
    if workspace is not None:
        pk, nw = _want(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel()
    return _call("moe_mxfp8_linear", _pack_linear(px, pxs, pw, pws, pb, pr, ld_r, po, ld_o, pc, ps, pk, nw, T, rows,
                                                  K, activation, 0), dev, stream, check)


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
    T, k = _matrix(ids, "ids", "[tokens, top_k]")
    dev = _dev(ids)
    pi = _want(ids, "ids", _I32, (T, k), dev)
    pf = _want(offsets, "offsets", _I32, (num_experts + 1,), dev)
    pp = _want(pos, "pos", _I32, (T, k), dev)
    pt = 0 if sorted is None else _want(sorted, "sorted", _I32, (T * k,), dev)
    pn = 0 if counts is None else _want(counts, "counts", _I32, (num_experts,), dev)
    px = ld_x = pxs = pr = prs = pk = nw = H = dt = 0
    if (x is None) != (rows is None):
        raise ValueError("x and rows: both or neither")
    if x is not None:
        H = _matrix(x, "x", "[tokens, hidden]")[1]
        px, ld_x, dt = _want(x, "x", _ROWS, (T, H), dev, True), _row(x), _DT[x.dtype]
        pr = _want(rows, "rows", (x.dtype,), (T * k, H), dev)
        mx = dt == MOE_DT_U8
        if mx != (x_scales is not None) or mx != (row_scales is not None):
            raise ValueError("x_scales and row_scales: with uint8 rows (MXFP8), and only with them")
        if mx:
            pxs = _want(x_scales, "x_scales", _U8, (T, H // 32), dev)
            prs = _want(row_scales, "row_scales", _U8, (T * k, H // 32), dev)
    if workspace is not None:
        pk, nw = _want(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel()
    return _call("moe_dispatch", _pack_dispatch(pi, px, ld_x, pxs, pn, pf, pt, pp, pr, prs, pk, nw, T, num_experts, H,
                                                k, dt), dev, stream, check)


def _combine(name, rows, weights, pos, out, stream, check):
    slots = T, k = _matrix(pos, "pos", "[tokens, top_k]")
    shape = _matrix(out, "out", "[tokens, hidden]")
    H, n, dev = shape[1], _matrix(rows, "rows", "[rows, hidden]")[0], _dev(pos)
    pp = _want(pos, "pos", _I32, slots, dev)
    pw = 0 if weights is None else _want(weights, "weights", _F32, slots, dev)
    pr, po = _want(rows, "rows", _FLOATS, (n, H), dev, True), _want(out, "out", _FLOATS, (T, H), dev, True)
    return _call(name, _pack_combine(pr, _row(rows), pw, pp, po, _row(out), 0, 0, 0, 0, 0, T, n, H, k,
                                     _DT[rows.dtype], _DT[out.dtype], 0), dev, stream, check)


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
    slots = T, k = _matrix(pos, "pos", "[tokens, top_k]")
    H, n, dev = _matrix(dout, "dout", "[tokens, hidden]")[1], _matrix(rows, "rows", "[rows, hidden]")[0], _dev(pos)
    pp = _want(pos, "pos", _I32, slots, dev)
    pw = 0 if weights is None else _want(weights, "weights", _F32, slots, dev)
    pr, pg = _want(rows, "rows", _FLOATS, (n, H), dev, True), _want(dout, "dout", _FLOATS, (T, H), dev, True)
    pd = ld_d = 0
    if drows is not None:
        pd, ld_d = _want(drows, "drows", (rows.dtype,), (n, H), dev, True), _row(drows)
    pdw = 0 if dweights is None else _want(dweights, "dweights", _F32, slots, dev)
    return _call("moe_combine_backward",
                 _pack_combine(pr, _row(rows), pw, pp, 0, 0, pg, _row(dout), pd, ld_d, pdw, T, n, H, k,
                               _DT[rows.dtype], _DT[dout.dtype], 0), dev, stream, check)


def moe_mxfp4_forward_mx8(x_codes, x_scales, router_logits, top_k: int, W_gate_up, W_down, scales, out,
                          shared=None, stream=None, check: bool = True) -> int:
    """The expert layer on MXFP8 activations: moe_mxfp4_forward_ex with
    MOE_ACT_MXFP8 on x_codes [T, H] and x_scales [T, H/32] uint8 in place of x.
    router_logits [T, E] float32, out [T, H] bfloat16; W_gate_up, W_down and
    scales in the tile layout (moe_mxfp4_prepack); shared as there."""
    T, H = _matrix(x_codes, "x_codes", "[tokens, hidden]")
    E, dev = _matrix(router_logits, "router_logits", "[tokens, experts]")[1], _dev(x_codes)
    pc, ps = _want(x_codes, "x_codes", _U8, (T, H), dev), _want(x_scales, "x_scales", _U8, (T, H // 32), dev)
    pl, po = _want(router_logits, "router_logits", _F32, (T, E), dev), _want(out, "out", _BF16, (T, H), dev)
    inter2 = W_gate_up.numel() * 2 // (E * H)  # 2 I, from the byte count
    weights = [(W_gate_up, E * inter2 * H // 2, "W_gate_up"), (W_down, E * H * inter2 // 4, "W_down"),
               (scales[0], E * inter2 * H // 32, "scales[0]"), (scales[1], E * H * inter2 // 64, "scales[1]")]
    if shared is not None:
        weights += [(t, n, f"shared[{i}]") for i, (t, n) in enumerate(zip(
            shared, (inter2 * H, inter2 * H // 32, H * inter2 // 2, H * inter2 // 64)))]
    ptrs = []
    for t, n, name in weights:
        if t.numel() != n:
            raise ValueError(f"{name}: expected {n} bytes, got {tuple(t.shape)}")
        ptrs.append(_want(t, name, _U8, t.shape, dev))
    opt = _lib.moe_mxfp4_options(act_format=_lib.MOE_ACT_MXFP8, weight_layout=_lib.MOE_LAYOUT_TILES)
    if shared is not None:
        opt.shared_gate_up, opt.shared_gate_up_scales, opt.shared_down, opt.shared_down_scales = ptrs[4:]
    sc = _lib.moe_mxfp4_scales(ptrs[2], ptrs[3])
    rc = ops_lib().moe_mxfp4_forward_mx8(pc, ps, pl, T, top_k, ptrs[0], ptrs[1], ctypes.byref(sc), po,
                                         _current_stream(dev) if stream is None else _lib._stream(stream),
                                         ctypes.byref(opt))
    return _check(rc, "moe_mxfp4_forward_mx8") if check else rc
