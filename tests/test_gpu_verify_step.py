"""GPU: the attention block of verify steps, as a model runs them: norm ->
joined projection -> keys and values into the cache -> attention of the
drafted trees -> output projection -> the accepted path moved to its places,
and the next step on what the cache then holds.  Every stage is compared in 64
bits on the inputs the GPU gave it; each step runs from a graph as well."""
import numpy as np
import pytest

from tests import attention_reference as A
from tests import ops_reference as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

HEADS, KV, D, H, PAGE = 6, 2, 128, 512, 16


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def _weights(M, rng, rows, inner):
    import oracle
    c, s = oracle.quantize_mxfp8(rng.standard_normal((rows, inner)) / np.sqrt(inner))
    return (c, s), R.prepacked(M, c, s, False)


def _random_tree(rng, n):
    """parents (-1: none) and the mask's words"""
    parent = [-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, n)]
    bits = []
    for i, p in enumerate(parent):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return parent, np.array(bits, np.uint64)[:, None]


def _positions(cache, table, n):
    """Values of a sequence's first n positions, [n, KV, D] twice."""
    import torch
    pos = np.arange(n)
    page, at = torch.from_numpy(table[pos // PAGE].astype(np.int64)).cuda(), torch.from_numpy(pos % PAGE).cuda()
    get = lambda c, s: R.mx8_values(c[page, :, at].cpu().numpy(), s[page, :, at].cpu().numpy())
    return get(cache.kc, cache.ks), get(cache.vc, cache.vs)


def test_verify_steps(M):
    import torch
    say("verify steps")
    rng = np.random.default_rng(21)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    i32 = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
    counts, lens = [9, 5, 9], [0, 77, 250]
    off = np.cumsum([0] + counts)
    T, B, max_pages = int(off[-1]) + 2, len(counts), 20   # two tokens of padding
    cache = A.Cache(B * max_pages, KV, PAGE, D, apart=True, seed=3)
    table = rng.permutation(B * max_pages).reshape(B, max_pages)
    (qkv_c, qkv_s), (qkv_t, qkv_ts) = _weights(M, rng, (HEADS + 2 * KV) * D, H)
    (o_c, o_s), (o_t, o_ts) = _weights(M, rng, H, HEADS * D)
    w = R.tensor(1 + 0.1 * rng.standard_normal(H), "bf16")
    res = R.tensor(rng.standard_normal((T, H)), "bf16")
    codes, scales, qkv = u8(T, H), u8(T, H // 32), bf(T, HEADS + 2 * KV, D)
    attn, attn_c, attn_s, out = bf(T, HEADS, D), u8(T, HEADS * D), u8(T, HEADS * D // 32), bf(T, H)
    attn32 = torch.zeros(T, HEADS * D, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    mask = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    lens_t, table_t, off_t = i32(lens), i32(table), i32(off)
    work = lambda n: u8(n) if n else None
    ws_qkv = work(M.moe_mxfp8_linear_workspace(T, (HEADS + 2 * KV) * D, H))
    ws_o = work(M.moe_mxfp8_linear_workspace(T, H, HEADS * D))
    ws_a = work(M.moe_tree_attention_workspace(T, B, HEADS, KV, D))
    q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]

    # what the committed positions hold before the first step
    for b in range(B):
        n = lens[b]
        at = torch.from_numpy(table[b, np.arange(n) // PAGE] * PAGE + np.arange(n) % PAGE).cuda()
        M.moe_kv_write(R.tensor(rng.standard_normal((n, KV, D)), "bf16"), R.tensor(rng.standard_normal((n, KV, D)), "f32")
                       .to(torch.bfloat16), at, *cache.tensors)

    def step():
        M.moe_rmsnorm(res, w, 1e-5, codes=codes, scales=scales)
        M.moe_mxfp8_linear(codes, scales, qkv_t, qkv_ts, out=qkv.view(T, -1), workspace=ws_qkv)
        M.moe_kv_write(k, v, slots, *cache.tensors)
        M.moe_tree_attention(q, *cache.tensors, table_t, lens_t, off_t, attn, D ** -0.5, mask=mask, workspace=ws_a)
        attn32.copy_(attn.view(T, -1))
        M.moe_mxfp8_quantize(attn32, attn_c, attn_s)
        M.moe_mxfp8_linear(attn_c, attn_s, o_t, o_ts, out=out, residual=res, workspace=ws_o)

    step()     # padding alone is written nowhere
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rnd in range(4):
        trees = [_random_tree(rng, n) for n in counts]
        where = np.full(T, -1, np.int64)
        for b, L in enumerate(lens):
            pos = np.arange(L, L + counts[b])
            where[off[b]:off[b + 1]] = table[b, pos // PAGE] * PAGE + pos % PAGE
            mask[off[b]:off[b + 1]] = torch.from_numpy(trees[b][1].view(np.int64)).cuda()
        slots.copy_(torch.from_numpy(where))
        lens_t.copy_(i32(lens))
        res.copy_(R.tensor(rng.standard_normal((T, H)), "bf16"))
        attn.fill_(5)
        before = [t.clone() for t in cache.tensors]
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (codes, scales, qkv, attn, out, *cache.tensors)]
        for t, was in zip(cache.tensors, before):
            t.copy_(was)
        for t in (codes, scales, qkv, out):
            t.zero_()
        attn.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (codes, scales, qkv, attn, out, *cache.tensors)):
            assert torch.equal(a, b), rnd

        cpu = lambda t: t.cpu().numpy()
        _, n = R.rmsnorm(R.values(res), None, R.values(w), 1e-5)
        R.assert_mx8_of(cpu(codes), cpu(scales), n, np.abs(n) * (H + 8) * 2.0 ** -53, "norm")
        x, dx = R.linear(cpu(codes), cpu(scales), qkv_c, qkv_s)
        R.assert_between(R.values(qkv.view(T, -1)), R.bf16_rne(x - dx), R.bf16_rne(x + dx), "projection")
        for b, L in enumerate(lens):
            rows = slice(int(off[b]), int(off[b + 1]))
            kb, vb = _positions(cache, table[b], L + counts[b])
            for got, x in ((kb, k), (vb, v)):     # the drafted tokens' are their own, encoded
                import oracle
                c, s = oracle.quantize_mxfp8(np.ascontiguousarray(R.values(x[rows]).reshape(-1, D)))
                assert np.array_equal(got[L:], R.mx8_values(c, s).reshape(-1, KV, D))
            ref = A.attention(R.values(q[rows]), kb, vb, trees[b][1], L, np.float64(np.float32(D ** -0.5)))
            A.check(R.values(attn[rows]), *ref, f"attention of sequence {b}, step {rnd}")
        assert (attn[int(off[-1]):] == 5).all()
        x, dx = R.linear(cpu(attn_c), cpu(attn_s), o_c, o_s, res=R.values(res))
        R.assert_between(R.values(out), R.bf16_rne(x - dx), R.bf16_rne(x + dx), "output")

        # a path of each tree is accepted; its keys and values move to the places
        # behind the committed ones
        src, dst, paths = [], [], []
        for b, L in enumerate(lens):
            path, at = [], int(rng.integers(0, counts[b]))
            while at >= 0:
                path.append(at)
                at = trees[b][0][at]
            path = path[::-1]
            paths.append(path)
            slot = lambda p: table[b, p // PAGE] * PAGE + p % PAGE
            src += [slot(L + a) for a in path]
            dst += [slot(L + i) for i in range(len(path))]
        held = [_positions(cache, table[b], lens[b] + counts[b]) for b in range(B)]
        tk, tv = bf(len(src), KV, D), bf(len(src), KV, D)
        M.moe_kv_read(*cache.tensors, torch.tensor(src, device="cuda"), tk, tv)
        M.moe_kv_write(tk, tv, torch.tensor(dst, device="cuda"), *cache.tensors)
        for b, path in enumerate(paths):
            L = lens[b]
            for got, was in zip(_positions(cache, table[b], L + len(path)), held[b]):
                assert np.array_equal(got, np.concatenate([was[:L], was[[L + a for a in path]]]))
            lens[b] = L + len(path)
