"""GPU: keys and values into the MXFP8 cache and out of it, bit for bit
against the encoder and the decoder of the oracle."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.attention_reference import Cache
from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def _inputs(rng, T, kv, D, dtype):
    """Ordinary rows, and blocks of zeros, of the largest and smallest
    magnitudes, of ties, and with values that are no numbers."""
    v = rng.standard_normal((T, kv, D)) * np.exp2(rng.integers(-20, 20, (T, kv, 1)))
    b = v.reshape(-1, 32)
    kinds = rng.integers(0, 12, len(b))
    b[kinds == 0] = 0.0
    b[kinds == 1] *= 0.0
    b[kinds == 1, 3] = -1.5 * 2.0 ** -126
    b[kinds == 2] *= 1e38 / np.abs(b[kinds == 2]).max(initial=1.0)
    b[kinds == 3, 5] = 3.3895e38
    b[kinds == 4] = rng.integers(-64, 65, b[kinds == 4].shape) * 4.0      # halfway between codes
    b[kinds == 4, 0] = 256.0
    b[kinds == 5, 7] = np.inf
    b[kinds == 6, 31] = np.nan
    b[kinds == 7] = rng.integers(-3, 4, b[kinds == 7].shape) * 2.0 ** -133  # below float32's normal range
    b[kinds == 8, 0] = 1.9990234375 * np.abs(b[kinds == 8]).max(initial=1.0)
    return R.tensor(b.reshape(v.shape), dtype)


def _encoded(x):
    """codes [n, kv, D], scales [n, kv, D/32] of a tensor, by the oracle."""
    import oracle
    v = R.values(x)
    codes, scales = oracle.quantize_mxfp8(np.ascontiguousarray(v.reshape(-1, v.shape[-1])))
    return codes.reshape(v.shape), scales.reshape(*v.shape[:2], v.shape[2] // 32)


def _same_codes(got, want):
    """equal, a zero of either sign for the other (-0 is its own code)"""
    return np.array_equal(got, want) or np.array_equal(np.where(got == 0x80, 0, got), np.where(want == 0x80, 0, want))


def _written(cache, slots):
    return [t[slots // cache.page, :, slots % cache.page].cpu().numpy() for t in cache.tensors]


SIZES = [  # tokens, kv heads, head_dim, page size, pages
    (1, 1, 32, 16, 1), (1, 8, 128, 64, 4), (9, 8, 128, 64, 4), (7, 3, 96, 16, 3), (33, 2, 256, 32, 5),
    (100, 5, 64, 128, 2), (17, 16, 512, 16, 4), (300, 1, 64, 1024, 2), (65, 7, 160, 64, 3), (1000, 8, 128, 16, 80)]


@pytest.mark.parametrize("T,kv,D,page,pages", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("strided", [False, True])
def test_write_then_read(M, T, kv, D, page, pages, dtype, strided):
    import torch
    say(f"kv write and read T={T} kv={kv} D={D} page={page} {dtype} strided={strided}")
    rng = np.random.default_rng(T * 131 + D)
    n = min(T, pages * page)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots = np.concatenate([slots, np.full(T - n, -1)]).astype(np.int64)
    if T > 4:   # padding of every kind
        slots[2], slots[-1] = -1, pages * page
        slots[1] = 1 << 40
    held = (slots >= 0) & (slots < pages * page)
    k, v = _inputs(rng, T, kv, D, dtype), _inputs(rng, T, kv, D, dtype)
    if strided:   # parts of a joined projection's output
        joined = torch.cat([torch.zeros_like(k), k, v, torch.zeros_like(k)], 1)
        k, v = joined[:, kv:2 * kv], joined[:, 2 * kv:3 * kv]
    cache = Cache(pages, kv, page, D, apart=strided, seed=T)
    before = [t.clone() for t in cache.tensors]
    M.moe_kv_write(k, v, torch.from_numpy(slots).cuda(), *cache.tensors)
    torch.cuda.synchronize()
    at = torch.from_numpy(slots[held]).cuda()
    got = _written(cache, at)
    for x, codes, scales in ((k, got[0], got[1]), (v, got[2], got[3])):
        want_c, want_s = _encoded(x)
        assert np.array_equal(scales, want_s[held])
        assert _same_codes(codes, want_c[held])
    # and nothing else was
    for t, b in zip(cache.tensors, before):
        t = t.clone()
        t[at // page, :, at % page] = b[at // page, :, at % page]
        assert torch.equal(t, b)
    # back, rows outside the cache as zeros
    shape = (T, 4 * kv, D) if strided else (T, kv, D)
    full_k, full_v = (torch.full(shape, 7.0, dtype=k.dtype, device="cuda") for _ in range(2))
    rk, rv = (full_k[:, kv:2 * kv], full_v[:, 2 * kv:3 * kv]) if strided else (full_k, full_v)
    M.moe_kv_read(*cache.tensors, torch.from_numpy(slots).cuda(), rk, rv)
    torch.cuda.synchronize()
    rnd = R.bf16_rne if dtype == "bf16" else lambda x: x
    for out, codes, scales in ((rk, got[0], got[1]), (rv, got[2], got[3])):
        want = np.zeros((T, kv, D))
        want[held] = rnd(R.mx8_values(codes, scales))
        assert np.array_equal(R.values(out), want, equal_nan=True)
    if strided:
        assert (full_k[:, :kv] == 7).all() and (full_k[:, 2 * kv:] == 7).all() and (full_v[:, :2 * kv] == 7).all()
    # written again to other slots: the same codes and scales (accepted tokens moved to their places)
    other = Cache(pages, kv, page, D, seed=T + 1)
    moved = torch.from_numpy(np.where(held, (slots + 5) % (pages * page), -1)).cuda()
    M.moe_kv_write(rk, rv, moved, *other.tensors)
    for a, b in zip(got, _written(other, moved[torch.from_numpy(held).cuda()])):
        assert _same_codes(b, a)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_read_every_code_and_scale(M, dtype):
    """All 256 codes at all 256 scales, rounded to nearest even where the type
    does not hold the value."""
    import torch
    say(f"kv read of every code and scale {dtype}")
    codes = np.broadcast_to(np.arange(256, dtype=np.uint8), (256, 1, 256)).copy()
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8)[:, None, None], (256, 1, 8)).copy()
    cache = Cache(16, 1, 16, 256)
    cache.put("k", np.arange(256), codes, scales)
    cache.put("v", np.arange(256), codes[:, :, ::-1].copy(), scales)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v = (torch.empty(256, 1, 256, dtype=dt, device="cuda") for _ in range(2))
    M.moe_kv_read(*cache.tensors, torch.arange(256, device="cuda"), k, v)
    want = R.mx8_values(codes, scales)
    with np.errstate(over="ignore"):
        want = R.bf16_rne(want) if dtype == "bf16" else want.astype(np.float32).astype(np.float64)
    assert np.array_equal(R.values(k), want, equal_nan=True)
    assert np.array_equal(R.values(v), want[:, :, ::-1], equal_nan=True)


def test_slots_may_repeat_when_read(M):
    import torch
    say("kv read of repeated slots")
    cache = Cache(4, 2, 16, 64, seed=3)
    slots = torch.tensor([5, 5, 63, 0, 5, 63], device="cuda")
    k, v = (torch.empty(6, 2, 64, device="cuda") for _ in range(2))
    M.moe_kv_read(*cache.tensors, slots, k, v)
    kc, ks = cache.kc.cpu().numpy(), cache.ks.cpu().numpy()
    for i, s in enumerate(slots.tolist()):
        with np.errstate(over="ignore"):
            want = R.mx8_values(kc[s // 16, :, s % 16], ks[s // 16, :, s % 16]).astype(np.float32)
        assert np.array_equal(k[i].cpu().numpy(), want, equal_nan=True)


def test_far_pages(M):
    """Pages beyond 4 GiB of codes."""
    import torch
    say("kv write and read beyond 32 bits")
    kv, page, D = 8, 64, 128
    pages = (1 << 32) // (kv * page * D) + 3
    cache = Cache(pages, kv, page, D, fill=0)
    rng = np.random.default_rng(5)
    k, v = (R.tensor(rng.standard_normal((4, kv, D)), "bf16") for _ in range(2))
    slots = torch.tensor([(pages - 1) * page + 63, (pages - 2) * page, (1 << 31) // (kv * D) + 1, 0], device="cuda")
    M.moe_kv_write(k, v, slots, *cache.tensors)
    got = _written(cache, slots)
    for x, c, s in ((k, got[0], got[1]), (v, got[2], got[3])):
        want_c, want_s = _encoded(x)
        assert np.array_equal(s, want_s) and _same_codes(c, want_c)
    assert int((cache.kc != 0).sum()) <= 4 * kv * D
    rk, rv = torch.empty_like(k), torch.empty_like(v)
    M.moe_kv_read(*cache.tensors, slots, rk, rv)
    assert np.array_equal(R.values(rk), R.mx8_values(got[0], got[1]))
    assert np.array_equal(R.values(rv), R.mx8_values(got[2], got[3]))


def test_graph_and_stream(M):
    """Captured and replayed on new slots and rows, and on a stream of the
    caller's."""
    import torch
    say("kv write and read in a graph")
    rng = np.random.default_rng(6)
    cache = Cache(8, 4, 16, 128, seed=1)
    k, v = (R.tensor(rng.standard_normal((9, 4, 128)), "bf16") for _ in range(2))
    slots = torch.arange(9, device="cuda")
    rk, rv = torch.empty_like(k), torch.empty_like(v)

    def both(stream=None):
        M.moe_kv_write(k, v, slots, *cache.tensors, stream=stream)
        M.moe_kv_read(*cache.tensors, slots, rk, rv, stream=stream)

    both()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for rnd in range(3):
        k.copy_(R.tensor(rng.standard_normal((9, 4, 128)), "bf16"))
        v.copy_(R.tensor(rng.standard_normal((9, 4, 128)), "bf16"))
        slots.copy_(torch.from_numpy(rng.permutation(128)[:9]))
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in (*cache.tensors, rk, rv)]
        rk.zero_(), rv.zero_(), cache.kc.zero_()
        both()   # the whole cache as after one call on this state
        eager = [t.clone() for t in (*cache.tensors, rk, rv)]
        rk.zero_(), rv.zero_(), cache.kc.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (*cache.tensors, rk, rv)):
            assert torch.equal(a, b)
        assert torch.equal(want[4], rk) and torch.equal(want[5], rv)
        s = torch.cuda.Stream()
        rk.zero_(), rv.zero_()
        torch.cuda.synchronize()
        both(stream=s)
        s.synchronize()
        assert torch.equal(want[4], rk) and torch.equal(want[5], rv)


def test_binding_refuses(M):
    import torch
    cache = Cache(4, 2, 16, 64)
    k, v = (torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    bad = [(k[:2], v, slots, *cache.tensors), (k, v.float(), slots, *cache.tensors), (k, v, slots.int(), *cache.tensors),
           (k.half(), v.half(), slots, *cache.tensors), (k.transpose(1, 2).contiguous().transpose(1, 2), v, slots, *cache.tensors),
           (k, v, slots, cache.kc, cache.ks[:, :, :, :1], cache.vc, cache.vs),
           (k, v, slots, cache.kc.transpose(1, 2), cache.ks, cache.vc, cache.vs),
           (k, v, slots, cache.kc.view(torch.int8), cache.ks, cache.vc, cache.vs),
           (k, v, slots.cpu(), *cache.tensors), (k.cpu(), v.cpu(), slots, *cache.tensors),
           (k, v, slots, cache.kc[::2], cache.ks[::2], cache.vc[:2], cache.vs[:2])]
    for args in bad:
        with pytest.raises((ValueError, M.MoeError)):
            M.moe_kv_write(*args)
    empty = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert M.moe_kv_write(empty, empty, slots[:0], *cache.tensors) == M.MOE_OK
    assert M.moe_kv_read(*cache.tensors, slots[:0], empty, empty) == M.MOE_OK
