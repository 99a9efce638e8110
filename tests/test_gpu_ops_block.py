"""The operators and the layer used together, as a block of a model uses them:
every stage is compared in 64 bits on the inputs the GPU gave it, so that an
error belongs to the stage that made it."""
import ctypes

import numpy as np
import pytest

from tests import ops_reference as R
from tests.gpu_common import get_layer, get_shared, say
from workloads import Config

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def _dev(*shape, dtype):
    import torch
    return torch.full(shape, 1, dtype=dtype, device="cuda")


def _encode(v):
    import oracle
    return oracle.quantize_mxfp8(np.ascontiguousarray(v, np.float64))


def _norm(M, x, residual, w, eps=1e-5):
    """residual in place, y, codes, scales; checked."""
    import torch
    T, H = x.shape
    xv, rv, wv = R.values(x), R.values(residual), R.values(w)
    y = _dev(T, H, dtype=torch.bfloat16)
    codes, scales = _dev(T, H, dtype=torch.uint8), _dev(T, H // 32, dtype=torch.uint8)
    M.moe_rmsnorm(x, w, eps, residual=residual, residual_out=residual, y=y, codes=codes, scales=scales)
    s, n = R.rmsnorm(xv, rv, wv, eps)
    err = np.abs(n) * (H + 8) * 2.0 ** -53
    want = R.bf16_rne(s) if residual.dtype == torch.bfloat16 else s.astype(np.float32).astype(np.float64)
    assert np.array_equal(R.values(residual), want)
    R.assert_between(R.values(y), R.bf16_rne(n - err), R.bf16_rne(n + err), "y")
    R.assert_mx8_of(codes.cpu().numpy(), scales.cpu().numpy(), n, err, "norm")
    return y, codes, scales


def _workspace(n):
    import torch
    return torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") if n else None


@pytest.mark.parametrize("T", [1, 9, 150, 400])
def test_experts_in_8_bits(M, T):
    """norm -> dispatch of MXFP8 rows -> gate/up product with SiLU-mul into
    MXFP8 and down product, per expert -> combine -> its gradients -> gradient
    of the dispatch.  Experts with no token, and tokens with none."""
    import torch
    say(f"8-bit expert block T={T}")
    H, I, E, k = 512, 256, 6, 3
    rng = np.random.default_rng(T)
    x = R.tensor(rng.standard_normal((T, H)), "bf16")
    res = R.tensor(3 * rng.standard_normal((T, H)), "f32")
    w = R.tensor(1 + 0.1 * rng.standard_normal(H), "bf16")
    y, codes, scales = _norm(M, x, res, w)
    ids = rng.integers(-1, E - 1, size=(T, k)).astype(np.int32)   # expert E-1 gets none
    if T > 2:
        ids[1] = -1
    counts, off, srt, pos = R.order(ids, E)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    o = dict(offsets=i32(E + 1), sorted=i32(T * k), pos=i32(T, k))
    xr, xrs = _dev(T * k, H, dtype=torch.uint8), _dev(T * k, H // 32, dtype=torch.uint8)
    M.moe_dispatch(codes, torch.from_numpy(ids).cuda(), E, o["offsets"], o["sorted"], o["pos"], xr,
                   _workspace(M.moe_dispatch_workspace(T, E, k)), x_scales=scales, row_scales=xrs)
    n = int(off[-1])
    assert np.array_equal(o["offsets"].cpu().numpy(), off) and np.array_equal(o["pos"].cpu().numpy(), pos)
    tok = torch.from_numpy(srt // k).cuda()
    assert torch.equal(xr[:n], codes[tok]) and torch.equal(xrs[:n], scales[tok])
    h, hs = _dev(T * k, I, dtype=torch.uint8), _dev(T * k, I // 32, dtype=torch.uint8)
    out_rows = torch.full((T * k, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    for e in range(E):
        a, b = int(off[e]), int(off[e + 1])
        gc, gs = _encode(rng.standard_normal((2 * I, H)) / np.sqrt(H))
        dc, ds = _encode(rng.standard_normal((H, I)) / np.sqrt(I))
        gt, gts = R.prepacked(M, gc, gs, True)
        dt, dts = R.prepacked(M, dc, ds, False)
        ws = _workspace(max(M.moe_mxfp8_linear_workspace(b - a, 2 * I, H, M.MOE_EPI_SILU_MUL),
                            M.moe_mxfp8_linear_workspace(b - a, H, I)))
        M.moe_mxfp8_linear(xr[a:b], xrs[a:b], gt, gts, out_codes=h[a:b], out_scales=hs[a:b],
                           activation=M.MOE_EPI_SILU_MUL, workspace=ws)
        M.moe_mxfp8_linear(h[a:b], hs[a:b], dt, dts, out=out_rows[a:b], workspace=ws)
        if b > a:
            cpu = lambda t: t[a:b].cpu().numpy()
            v, dv = R.linear(cpu(xr), cpu(xrs), gc, gs, "silu_mul")
            R.assert_mx8_of(cpu(h), cpu(hs), v, dv, f"h of expert {e}")
            v, dv = R.linear(cpu(h), cpu(hs), dc, ds)
            R.assert_between(R.values(out_rows[a:b]), R.bf16_rne(v - dv), R.bf16_rne(v + dv), f"expert {e}")
    assert torch.isnan(out_rows[n:]).all()
    wts = R.tensor(rng.random((T, k)), "f32")
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_combine(out_rows, wts, o["pos"], out)
    r = np.nan_to_num(R.values(out_rows))
    g = r[np.maximum(pos, 0)] * (R.values(wts) * (pos >= 0))[..., None]
    err = (k + 1) * R.U32 * np.abs(g).sum(1)
    R.assert_between(R.values(out), R.bf16_rne(g.sum(1) - err), R.bf16_rne(g.sum(1) + err), "out")
    dout = R.tensor(rng.standard_normal((T, H)), "bf16")
    drows, dw = torch.zeros_like(out_rows), torch.zeros_like(wts)
    M.moe_combine_backward(dout, out_rows, wts, o["pos"], drows, dw)
    terms = R.values(dout)[:, None] * r[np.maximum(pos, 0)] * (pos >= 0)[..., None]
    err = (H + 8) * R.U32 * np.abs(terms).sum(-1)
    R.assert_between(R.values(dw), terms.sum(-1) - err, terms.sum(-1) + err, "dweights")
    dx = torch.full((T, H), float("nan"), device="cuda")
    M.moe_dispatch_backward(drows, o["pos"], dx)
    d = np.nan_to_num(R.values(drows))[np.maximum(pos, 0)] * (pos >= 0)[..., None]
    err = (k + 1) * R.U32 * np.abs(d).sum(1)
    R.assert_between(R.values(dx), d.sum(1) - err, d.sum(1) + err, "dx")


@pytest.mark.parametrize("T,E,H,I,k", [(9, 8, 256, 128, 2), (130, 16, 512, 256, 4), (1, 4, 384, 128, 1)])
@pytest.mark.parametrize("shared", [False, True])
def test_layer_reads_the_norms_codes(M, T, E, H, I, k, shared):
    """The expert layer on the norm's codes gives the bits of
    moe_mxfp4_forward_ex on the values they stand for (which bf16 holds
    exactly and whose encoding they are), captured in a graph as well."""
    import torch
    say(f"layer on MXFP8 rows T={T} E={E} H={H} shared={shared}")
    cfg = Config("mx8_rows", f"mx8_rows_t{T}_e{E}_h{H}_i{I}_k{k}", T, E, H, I, k, "normal", "mxfp8", 4001)
    layer = get_layer(cfg)
    sh = get_shared(cfg).tiles if shared else None
    M.moe_mxfp4_init(T, E, H, I, k)
    wgu, wdn, sc = layer.weights(M.MOE_LAYOUT_TILES)
    rng = np.random.default_rng(T)
    res = R.tensor(rng.standard_normal((T, H)), "bf16")
    _, codes, scales = _norm(M, layer.x.clone(), res, R.tensor(np.ones(H), "f32"))
    x = R.tensor(R.mx8_values(codes.cpu().numpy(), scales.cpu().numpy()), "bf16")
    want, xq, xs = torch.empty_like(layer.out), torch.empty_like(codes), torch.empty_like(scales)
    M.moe_mxfp4_forward_ex(x, layer.logits, k, wgu, wdn, sc, want, act_format=M.MOE_ACT_MXFP8,
                           weight_layout=M.MOE_LAYOUT_TILES, shared=sh, x_codes=xq, x_scales=xs)
    assert torch.equal(xq, codes) and torch.equal(xs, scales)
    got = torch.full_like(want, float("nan"))
    M.moe_mxfp4_forward_mx8(codes, scales, layer.logits, k, wgu, wdn, sc, got, shared=sh)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # norm, layer and the next norm in one graph, replayed on new inputs
    g = torch.cuda.CUDAGraph()
    xin, rin, w = layer.x.clone(), res.clone(), R.tensor(np.ones(H), "f32")
    y2, c2, s2 = torch.empty_like(want), torch.empty_like(codes), torch.empty_like(scales)

    def block():
        M.moe_rmsnorm(xin, w, 1e-5, residual=rin, residual_out=rin, codes=codes, scales=scales)
        M.moe_mxfp4_forward_mx8(codes, scales, layer.logits, k, wgu, wdn, sc, got, shared=sh)
        M.moe_rmsnorm(got, w, 1e-5, residual=rin, residual_out=rin, y=y2, codes=c2, scales=s2)

    block()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        block()
    for rnd in range(3):
        xin.copy_(R.tensor(rng.standard_normal((T, H)), "bf16"))
        start = R.tensor(rng.standard_normal((T, H)), "bf16")
        rin.copy_(start)
        block()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (got, rin, y2, c2, s2)]
        rin.copy_(start)
        for t in (got, y2, c2, s2):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (got, rin, y2, c2, s2)):
            assert torch.equal(a, b)


def test_forward_mx8_refusals(M):
    """With a workspace, what forward_ex refuses; out is left as it was."""
    import torch

    from mxfp4_moe_expert_02_amd import _lib, _ops
    T, E, H, I, k = 9, 8, 256, 128, 2
    cfg = Config("mx8_refuse", "mx8_refuse_t9", T, E, H, I, k, "normal", "mxfp8", 4002)
    layer = get_layer(cfg)
    M.moe_mxfp4_init(T, E, H, I, k)
    wgu, wdn, (s1, s2) = layer.weights(M.MOE_LAYOUT_TILES)
    codes, scales = _dev(T + 1, H, dtype=torch.uint8), _dev(T + 1, H // 32, dtype=torch.uint8)
    layer.out.fill_(3)

    def call(c=codes.data_ptr(), s=scales.data_ptr(), n=T, top=k, opt=None):
        sc = _lib.moe_mxfp4_scales(s1.data_ptr(), s2.data_ptr())
        return _ops.ops_lib().moe_mxfp4_forward_mx8(c, s, layer.logits.data_ptr(), n, top, wgu.data_ptr(),
                                                    wdn.data_ptr(), ctypes.byref(sc), layer.out.data_ptr(), None, opt)

    assert call(c=None) == M.MOE_E_NULL and call(s=None) == M.MOE_E_NULL
    assert call(c=codes.data_ptr() + 8) == M.MOE_E_ALIGN and call(s=scales.data_ptr() + 4) == M.MOE_E_ALIGN
    assert call(n=T + 1) == M.MOE_E_TOKENS and call(top=k + 1) == M.MOE_E_TOPK and call(n=-1) == M.MOE_E_SHAPE
    for o in (_lib.moe_mxfp4_options(M.MOE_ACT_BF16, 0), _lib.moe_mxfp4_options(M.MOE_ACT_MXFP8, 0)):
        assert call(opt=ctypes.byref(o)) == M.MOE_E_OPTION        # bf16 rows, row-major weights
    o = _lib.moe_mxfp4_options(M.MOE_ACT_MXFP8, 0)
    o.weight_layout, o.router_weight = M.MOE_LAYOUT_TILES, codes.data_ptr()
    assert call(opt=ctypes.byref(o)) == M.MOE_E_OPTION
    torch.cuda.synchronize()
    assert (layer.out == 3).all()
    assert call(n=0) == M.MOE_OK and call() == M.MOE_OK
    torch.cuda.synchronize()
