"""The cache's and the attention's entry points without a GPU: what their
header declares is exported and bound, and every refused call returns its
status before any HIP call (nothing here dereferences a pointer)."""
import ctypes
import os
import re

import pytest

from tests.conftest import ROOT, gpu_available

HEADER = os.path.join(ROOT, "include", "ops", "moe_attention.h")


@pytest.fixture(scope="module")
def A():
    from mxfp4_moe_expert_02_amd import _attention, _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libmoe_mxfp4.so is not built (run __graft_entry__.build())")
    _attention.attention_lib()
    return _attention


def test_declared_exported_and_bound(A):
    import mxfp4_moe_expert_02_amd as M
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\w+ (moe_\w+)\(", text, re.M))
    assert names == set(A.ATTENTION_EXPORTED)
    for n in names:
        assert hasattr(A.attention_lib(), n) and callable(getattr(M, n)) and n in M.__all__
    for struct in ("moe_kv_cache", "moe_kv_rows_args", "moe_tree_attention_args"):
        body = re.search(r"typedef struct %s \{(.*?)\}" % struct, text, re.S).group(1)
        fields = re.findall(r"(\w+);", body)
        assert fields == [f for f, _ in getattr(A, struct)._fields_], struct


def _cache(A, **over):
    a = dict(k_codes=0x1000, k_scales=0x2000, v_codes=0x3000, v_scales=0x4000, num_pages=4, page_size=64, kv_heads=8,
             head_dim=128)
    a.update({k: v for k, v in over.items() if k in dict(A.moe_kv_cache._fields_)})
    return A.moe_kv_cache(**a)


def _rows(A, name, **over):
    from mxfp4_moe_expert_02_amd import MOE_DT_BF16
    fields = dict(A.moe_kv_rows_args._fields_)
    a = dict(k=0x5000, v=0x6000, slots=0x7000, num_tokens=9, dtype=MOE_DT_BF16)
    a.update({k: v for k, v in over.items() if k in fields})
    assert all(k in fields or k in dict(A.moe_kv_cache._fields_) for k in over)
    return getattr(A.attention_lib(), name)(ctypes.byref(A.moe_kv_rows_args(cache=_cache(A, **over), **a)), None)


CACHE_SHAPES = [dict(num_pages=0), dict(num_pages=-1), dict(num_pages=1 << 31), dict(page_size=8), dict(page_size=48),
                dict(page_size=2048), dict(kv_heads=0), dict(kv_heads=1025), dict(codes_page_stride=65535),
                dict(codes_page_stride=-16), dict(scales_page_stride=16)]
CACHE_NULLS = [dict(k_codes=0), dict(k_scales=0), dict(v_codes=0), dict(v_scales=0)]
CACHE_ALIGNS = [dict(k_codes=0x1008), dict(k_scales=0x2004), dict(v_codes=0x3001), dict(v_scales=0x4008),
                dict(codes_page_stride=65544), dict(scales_page_stride=2056)]


@pytest.mark.parametrize("name", ["moe_kv_write", "moe_kv_read"])
def test_rows_refusals(A, name):
    from mxfp4_moe_expert_02_amd import (MOE_DT_F32, MOE_DT_U8, MOE_E_ALIGN, MOE_E_DTYPE, MOE_E_HIP, MOE_E_NULL,
                                         MOE_E_OPTION, MOE_E_SHAPE, MOE_OK)
    assert getattr(A.attention_lib(), name)(None, None) == MOE_E_NULL
    for kw in CACHE_SHAPES + [dict(head_dim=0), dict(head_dim=48), dict(head_dim=544), dict(num_tokens=-1),
                              dict(num_tokens=(1 << 20) + 1), dict(k_stride=1023), dict(v_stride=-8)]:
        assert _rows(A, name, **kw) == MOE_E_SHAPE, kw
    for kw in CACHE_NULLS + [dict(k=0), dict(v=0), dict(slots=0)]:
        assert _rows(A, name, **kw) == MOE_E_NULL, kw
    for kw in CACHE_ALIGNS + [dict(k=0x5008), dict(v=0x6002), dict(slots=0x7004), dict(k_stride=1028),
                              dict(v_stride=1026, dtype=MOE_DT_F32)]:
        assert _rows(A, name, **kw) == MOE_E_ALIGN, kw
    for kw in (dict(dtype=0), dict(dtype=MOE_DT_U8)):
        assert _rows(A, name, **kw) == MOE_E_DTYPE, kw
    assert _rows(A, name, reserved=1) == MOE_E_OPTION   # the cache's, and the call's
    assert _rows(A, name, num_tokens=0, k=0, slots=0) == MOE_OK
    if not gpu_available():   # nothing to refuse: on to the launch, which finds no device
        assert _rows(A, name) == MOE_E_HIP
        assert _rows(A, name, dtype=MOE_DT_F32, head_dim=96, k_stride=1 << 20) == MOE_E_HIP


def _attend(A, **over):
    fields = dict(A.moe_tree_attention_args._fields_)
    a = dict(q=0x5000, out=0x6000, block_table=0x7000, context_lens=0x8000, token_offsets=0x9000, mask=0xa000,
             mask_words=1, workspace=0x10000, workspace_bytes=1 << 40, num_tokens=18, num_seqs=2, max_pages=32,
             num_heads=48, scale=0.125)
    a.update({k: v for k, v in over.items() if k in fields})
    assert all(k in fields or k in dict(A.moe_kv_cache._fields_) for k in over)
    args = A.moe_tree_attention_args(cache=_cache(A, **over), **a)
    return A.attention_lib().moe_tree_attention(ctypes.byref(args), None)


def test_attention_refusals(A):
    from mxfp4_moe_expert_02_amd import (MOE_E_ALIGN, MOE_E_HIP, MOE_E_LIMIT, MOE_E_NULL, MOE_E_OPTION, MOE_E_SHAPE,
                                         MOE_OK)
    L = A.attention_lib()
    assert L.moe_tree_attention(None, None) == MOE_E_NULL
    for kw in CACHE_SHAPES + [dict(head_dim=32), dict(head_dim=96), dict(head_dim=192), dict(head_dim=512),
                              dict(num_tokens=-1), dict(num_tokens=(1 << 20) + 1), dict(num_seqs=-1),
                              dict(num_seqs=(1 << 16) + 1), dict(num_heads=0), dict(num_heads=49),
                              dict(num_heads=1032), dict(mask_words=0), dict(mask_words=65), dict(mask=0),
                              dict(q_stride=6143), dict(out_stride=-8), dict(max_pages=0), dict(max_pages=-1),
                              dict(max_pages=(1 << 24) + 1), dict(block_table_stride=31)]:
        assert _attend(A, **kw) == MOE_E_SHAPE, kw
    for kw in CACHE_NULLS + [dict(q=0), dict(out=0), dict(block_table=0), dict(context_lens=0), dict(token_offsets=0),
                             dict(workspace=0)]:
        assert _attend(A, **kw) == MOE_E_NULL, kw
    for kw in CACHE_ALIGNS + [dict(q=0x5008), dict(out=0x6002), dict(block_table=0x7002), dict(context_lens=0x8001),
                              dict(token_offsets=0x9002), dict(mask=0xa004), dict(workspace=0x10008),
                              dict(q_stride=6148), dict(out_stride=6146)]:
        assert _attend(A, **kw) == MOE_E_ALIGN, kw
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(scale=1e-40), dict(scale=3e38), dict(reserved=1)):
        assert _attend(A, **kw) == MOE_E_OPTION, kw
    # more units than a call can count
    assert _attend(A, max_pages=1 << 24, num_tokens=1 << 20, num_seqs=1 << 16) == MOE_E_LIMIT
    for kw in (dict(num_tokens=0), dict(num_seqs=0)):
        assert _attend(A, q=0, block_table=0, workspace=0, workspace_bytes=0, **kw) == MOE_OK
    need = L.moe_tree_attention_workspace(18, 2, 48, 8, 128)
    assert need > 0
    assert _attend(A, workspace_bytes=need - 1) == MOE_E_LIMIT
    if not gpu_available():
        assert _attend(A, workspace_bytes=need) == MOE_E_HIP
        assert _attend(A, mask=0, mask_words=0) == MOE_E_HIP


def test_workspace_sizes(A):
    from mxfp4_moe_expert_02_amd import MOE_E_SHAPE
    f = A.attention_lib().moe_tree_attention_workspace
    assert f(0, 4, 48, 8, 128) == 0 and f(9, 0, 48, 8, 128) == 0
    for args in ((-1, 1, 48, 8, 128), (9, 1 << 17, 48, 8, 128), (9, 1, 48, 7, 128), (9, 1, 48, 8, 96),
                 (1 << 21, 1, 8, 8, 64)):
        assert f(*args) == MOE_E_SHAPE, args
    for T in (1, 9, 288, 4096, 1 << 20):
        for B in (1, 32, 1 << 16):
            for heads, kv in ((1, 1), (48, 8), (56, 8), (1024, 1)):
                for D in (64, 128, 256):
                    # within 1024 results of 80 rows, whatever the lengths
                    assert 0 < f(T, B, heads, kv, D) <= 1024 * 80 * 4 * (D + 4), (T, B, heads, kv, D)


@pytest.mark.parametrize("name", ["moe_kv_write", "moe_kv_read", "moe_tree_attention"])
def test_far_strides(A, name):
    """Pages, and tokens of queries, may lie 2^31 apart and no further."""
    from mxfp4_moe_expert_02_amd import MOE_E_HIP, MOE_E_SHAPE
    call = (lambda **kw: _attend(A, **kw)) if name == "moe_tree_attention" else (lambda **kw: _rows(A, name, **kw))
    over = ["codes_page_stride", "scales_page_stride"] + ["q_stride", "out_stride"] * (name == "moe_tree_attention")
    for field in over:
        assert call(**{field: (1 << 31) + 16}) == MOE_E_SHAPE, field
        if not gpu_available():
            assert call(**{field: 1 << 31}) == MOE_E_HIP, field


def test_nothing_to_do_with_a_mask(A):
    """No tokens, or no sequences: an empty mask has no address, and the words
    of its rows are no reason to refuse."""
    from mxfp4_moe_expert_02_amd import MOE_E_SHAPE, MOE_OK
    for empty in (dict(num_tokens=0), dict(num_seqs=0)):
        for words in (0, 1, 2, 64):
            for mask in (0, 0xa000):
                assert _attend(A, q=0, out=0, workspace=0, workspace_bytes=0, mask=mask, mask_words=words,
                               **empty) == MOE_OK, (empty, mask, words)
        for words in (-1, 65):
            assert _attend(A, mask=0, mask_words=words, **empty) == MOE_E_SHAPE
