"""ctypes binding of the key/value cache and the attention over it
(include/ops/moe_attention.h), with the C ABI's own names and the manner of
``_ops``: argument marshalling only, no fallback, torch device tensors of the
current device, results into tensors that the caller passes.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib, _ops
from ._lib import _check
from ._ops import _DT, _FLOATS, _FORMAT, _I32, _U8, _dev, _matrix, _row, _want

ATTENTION_EXPORTED = ("moe_kv_write", "moe_kv_read", "moe_tree_attention", "moe_tree_attention_workspace")

_i32, _i64, _vp, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class moe_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_scales", _vp), ("v_codes", _vp), ("v_scales", _vp),
                ("codes_page_stride", _i64), ("scales_page_stride", _i64), ("num_pages", _i64),
                ("page_size", _i32), ("kv_heads", _i32), ("head_dim", _i32), ("reserved", _i32)]


class moe_kv_rows_args(ctypes.Structure):
    _fields_ = [("cache", moe_kv_cache), ("k", _vp), ("v", _vp), ("k_stride", _i64), ("v_stride", _i64),
                ("slots", _vp), ("num_tokens", _i64), ("dtype", _i32), ("reserved", _i32)]


class moe_tree_attention_args(ctypes.Structure):
    _fields_ = [("cache", moe_kv_cache), ("q", _vp), ("q_stride", _i64), ("out", _vp), ("out_stride", _i64),
                ("block_table", _vp), ("block_table_stride", _i64), ("context_lens", _vp),
                ("token_offsets", _vp), ("mask", _vp), ("mask_words", _i64), ("workspace", _vp),
                ("workspace_bytes", _i64), ("num_tokens", _i64), ("num_seqs", _i64), ("max_pages", _i64),
                ("num_heads", _i32), ("scale", _f32)]


def _format(struct_type):
    return "".join(_format(t) if issubclass(t, ctypes.Structure) else "f" if t is _f32 else _FORMAT[t]
                   for _, t in struct_type._fields_)


def _packer(struct_type):
    """As in ``_ops``; the cache's fields come first, in order."""
    s = struct.Struct("@" + _format(struct_type))
    assert s.size == ctypes.sizeof(struct_type)
    return s.pack


_I64 = (torch.int64,)
_pack_rows = _packer(moe_kv_rows_args)
_pack_attention = _packer(moe_tree_attention_args)

_ready = None
_entry = {}


def attention_lib() -> ctypes.CDLL:
    """The HIP library with these operators' signatures set."""
    global _ready
    L = _lib.lib()
    if _ready is not L:
        for name in ATTENTION_EXPORTED[:3]:
            getattr(L, name).restype, getattr(L, name).argtypes = ctypes.c_int, [_vp, _vp]
            _entry[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, _vp)((name, L))
        L.moe_tree_attention_workspace.restype = _i64
        L.moe_tree_attention_workspace.argtypes = [_i64, _i64, _i32, _i32, _i32]
        _ready = L
    return L


def _call(name, packed, dev, stream, check):
    if _ready is None:
        attention_lib()
    rc = _entry[name](packed, _ops._current_stream(dev) if stream is None else _lib._stream(stream))
    return _check(rc, name) if check and rc else rc


_u8 = torch.uint8


def _cache(kc, ks, vc, vs, dev):
    """The cache's fields, and its [pages, kv_heads, page_size, head_dim].
    Pages may lie apart (keys' and values' alike); a page is contiguous."""
    shape, scales = kc.shape, ks.shape
    if len(shape) != 4:
        raise ValueError(f"k_codes: expected [pages, kv_heads, page_size, head_dim], got {tuple(shape)}")
    pages, kv, size, D = shape
    if (vc.shape != shape or vs.shape != scales or scales != (pages, kv, size, D // 32) or not (
            kc.dtype is ks.dtype is vc.dtype is vs.dtype is _u8) or not (
            kc.get_device() == ks.get_device() == vc.get_device() == vs.get_device() == dev)):
        for t, name, s in ((kc, "k_codes", shape), (ks, "k_scales", (pages, kv, size, D // 32)),
                           (vc, "v_codes", shape), (vs, "v_scales", (pages, kv, size, D // 32))):
            if t.dtype != _u8 or t.shape != s:
                raise ValueError(f"{name}: expected torch.uint8 {tuple(s)}, got {t.dtype} {tuple(t.shape)}")
            if t.get_device() != dev:
                raise ValueError(f"{name}: expected a tensor of the current device, got {t.device}")
    n = kv * size * D
    ld_c, ld_s = n, n // 32
    if not (kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        for t, name, d, row in ((kc, "k_codes", D, n), (ks, "k_scales", D // 32, ld_s), (vc, "v_codes", D, n),
                                (vs, "v_scales", D // 32, ld_s)):
            if not t.is_contiguous() and (t.stride()[1:] != (size * d, d, 1) or t.stride(0) < row):
                raise ValueError(f"{name}: expected contiguous pages, got strides {t.stride()}")
        if pages > 1:
            ld_c, ld_s = kc.stride(0), ks.stride(0)
            if vc.stride(0) != ld_c or vs.stride(0) != ld_s:
                raise ValueError("expected keys' and values' pages equally far apart, got strides "
                                 f"{kc.stride()}, {vc.stride()}, {ks.stride()}, {vs.stride()}")
    return kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), ld_c, ld_s, pages, size, kv, D, 0


def _heads(t, name, dtype, shape, n, dev):
    """t is [tokens, heads, head_dim], tokens any distance apart, n the
    elements of one: its address and that distance."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        if t.dtype != dtype or t.shape != shape:
            raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
        raise ValueError(f"{name}: expected a tensor of the current device, got {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), n
    if t.stride()[1:] != (shape[2], 1) or (shape[0] > 1 and t.stride(0) < n):
        raise ValueError(f"{name}: expected contiguous heads, got strides {t.stride()}")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else n


def _rows(name, k, v, slots, kc, ks, vc, vs, stream, check):
    dev = _dev(k)
    c = _cache(kc, ks, vc, vs, dev)
    kv, D, dtype = c[8], c[9], k.dtype
    if dtype not in _FLOATS:
        raise ValueError(f"k: expected {' or '.join(map(str, _FLOATS))}, got {dtype}")
    if slots.dim() != 1:
        raise ValueError(f"slots: expected [tokens], got {tuple(slots.shape)}")
    T = slots.shape[0]
    shape = (T, kv, D)
    pk, ld_k = _heads(k, "k", dtype, shape, kv * D, dev)
    pv, ld_v = _heads(v, "v", dtype, shape, kv * D, dev)
    return _call(name, _pack_rows(*c, pk, pv, ld_k, ld_v, _want(slots, "slots", _I64, (T,), dev), T, _DT[dtype], 0),
                 dev, stream, check)


def moe_kv_write(k, v, slots, k_codes, k_scales, v_codes, v_scales, stream=None, check: bool = True) -> int:
    """Keys and values of new tokens into the cache, as MXFP8.

    k and v [T, kv_heads, head_dim] bfloat16 or float32 (tokens may be strided:
    parts of a joined projection's output), slots [T] int64: page * page_size +
    position; a token whose slot is outside the cache (-1) is not written, and
    two tokens may not share one.  k_codes and v_codes [pages, kv_heads,
    page_size, head_dim], k_scales and v_scales [.., head_dim / 32] uint8 (pages
    may be strided, keys and values alike).  head_dim is a multiple of 32 up to
    512; moe_tree_attention takes 64, 128 and 256."""
    return _rows("moe_kv_write", k, v, slots, k_codes, k_scales, v_codes, v_scales, stream, check)


def moe_kv_read(k_codes, k_scales, v_codes, v_scales, slots, k, v, stream=None, check: bool = True) -> int:
    """k[t] and v[t] = the keys and values at slots[t] (tensors as for
    moe_kv_write); zeros for a slot outside the cache."""
    return _rows("moe_kv_read", k, v, slots, k_codes, k_scales, v_codes, v_scales, stream, check)


def moe_tree_attention_workspace(num_tokens: int, num_seqs: int, num_heads: int, kv_heads: int,
                                 head_dim: int) -> int:
    """Bytes of workspace of a moe_tree_attention call of these sizes."""
    n = attention_lib().moe_tree_attention_workspace(num_tokens, num_seqs, num_heads, kv_heads, head_dim)
    return n if n >= 0 else _check(n, "moe_tree_attention_workspace")


def moe_tree_attention(q, k_codes, k_scales, v_codes, v_scales, block_table, context_lens, token_offsets, out,
                       scale: float, mask=None, workspace=None, stream=None, check: bool = True) -> int:
    """Attention of drafted tokens over the cache.

    q and out [T, heads, head_dim] bfloat16 (tokens may be strided); sequence b
    has tokens token_offsets[b] .. token_offsets[b + 1] - 1, its positions in
    the pages block_table[b] (rows may be strided), context_lens[b] of them
    committed, its drafted tokens' keys and values at the positions behind
    them.  A drafted token sees the committed positions and of the drafted ones
    those whose bit is set in its row of mask [T, words] int64 (bit j % 64 of
    word j / 64), or without a mask those up to its own.  block_table [B, pages],
    context_lens [B] and token_offsets [B + 1] int32.  Tokens of no sequence are
    left as they were in ``out``, one that sees nothing gets zeros.  head_dim is
    64, 128 or 256.  workspace: a uint8 tensor of at least
    moe_tree_attention_workspace(...) bytes for the call's own sizes."""
    dev = _dev(q)
    c = _cache(k_codes, k_scales, v_codes, v_scales, dev)
    shape, D = q.shape, c[9]
    if len(shape) != 3 or shape[2] != D:
        raise ValueError(f"q: expected [tokens, heads, {D}], got {tuple(shape)}")
    T, heads, _ = shape
    pq, ld_q = _heads(q, "q", torch.bfloat16, shape, heads * D, dev)
    po, ld_o = _heads(out, "out", torch.bfloat16, shape, heads * D, dev)
    B, pages = _matrix(block_table, "block_table", "[sequences, pages]")
    pt = _want(block_table, "block_table", _I32, (B, pages), dev, True)
    pc = _want(context_lens, "context_lens", _I32, (B,), dev)
    pf = _want(token_offsets, "token_offsets", _I32, (B + 1,), dev)
    pm = words = pw = nw = 0
    if mask is not None:
        words = _matrix(mask, "mask", "[tokens, words]")[1]
        if words < 1:  # an empty tensor has no address: not to be taken for no mask
            raise ValueError(f"mask: expected a word a token at least, got {tuple(mask.shape)}")
        pm = _want(mask, "mask", _I64, (T, words), dev)
    if workspace is not None:
        pw, nw = _want(workspace, "workspace", _U8, workspace.shape, dev), workspace.numel()
    return _call("moe_tree_attention", _pack_attention(*c, pq, ld_q, po, ld_o, pt, _row(block_table), pc, pf, pm,
                                                       words, pw, nw, T, B, pages, heads, scale), dev, stream, check)
