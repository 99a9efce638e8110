"""moe_mxfp8_linear against the product in 64 bits; the bounds are derived in
ops_reference.linear."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def encode(v):
    import oracle
    return oracle.quantize_mxfp8(np.ascontiguousarray(v, np.float64))


class Case:
    def __init__(self, M, T, rows, K, act="none", bias=False, residual=False, out="bf16", seed=0):
        import torch
        rng = np.random.default_rng([seed, T, rows, K])
        self.T, self.rows, self.K, self.act, self.out = T, rows, K, act, out
        self.cols = rows // 2 if act == "silu_mul" else rows
        self.xc, self.xs = encode(rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1))))
        self.wc, self.ws = encode(rng.standard_normal((rows, K)) / np.sqrt(K))
        self.bias = rng.standard_normal(rows).astype(np.float32).astype(np.float64) if bias else None
        self.res = R.bf16_rne(rng.standard_normal((T, self.cols))) if residual else None
        self.dev = dict(x_codes=torch.from_numpy(self.xc).cuda(), x_scales=torch.from_numpy(self.xs).cuda())
        self.upload_weights(M)
        self.kw = dict(activation={"none": M.MOE_EPI_NONE, "silu": M.MOE_EPI_SILU, "gelu": M.MOE_EPI_GELU,
                                   "silu_mul": M.MOE_EPI_SILU_MUL}[act])
        self.kw["bias"] = None if self.bias is None else R.tensor(self.bias, "f32")
        self.kw["residual"] = None if self.res is None else R.tensor(self.res, "bf16")
        n = M.moe_mxfp8_linear_workspace(T, rows, K, self.kw["activation"])
        self.kw["workspace"] = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") if n else None

    def upload_weights(self, M):
        t, ts = R.prepacked(M, self.wc, self.ws, self.act == "silu_mul")
        self.dev.update(w_tiles=t, w_scales=ts)

    def outputs(self):
        import torch
        if self.out == "bf16":
            return dict(out=torch.full((self.T, self.cols), float("nan"), dtype=torch.bfloat16, device="cuda"))
        return dict(out_codes=torch.full((self.T, self.cols), 0x7f, dtype=torch.uint8, device="cuda"),
                    out_scales=torch.full((self.T, self.cols // 32), 77, dtype=torch.uint8, device="cuda"))

    def run(self, M, **over):
        import torch
        o = self.outputs()
        M.moe_mxfp8_linear(**self.dev, **{**self.kw, **o, **over})
        torch.cuda.synchronize()
        return o

    def check(self, o, rows=None):
        """All tokens, or those of `rows`."""
        at = np.arange(self.T) if rows is None else np.asarray(rows)
        v, dv = R.linear(self.xc[at], self.xs[at], self.wc, self.ws, self.act, self.bias,
                         None if self.res is None else self.res[at], tokens=self.T)
        o = {k: t[at.tolist()] for k, t in o.items()}
        if self.out == "bf16":
            R.assert_between(R.values(o["out"]), R.bf16_rne(v - dv), R.bf16_rne(v + dv), "out")
        else:
            R.assert_mx8_of(o["out_codes"].cpu().numpy(), o["out_scales"].cpu().numpy(), v, dv, "out")


@pytest.mark.parametrize("T", [1, 2, 9, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 127, 128, 129, 200, 255, 257, 300,
                               513, 1025, 1040, 1055, 1057, 1151, 1279, 1281])
@pytest.mark.parametrize("rows,K", [(64, 128), (192, 384), (512, 1152)])
def test_every_token_count(M, T, rows, K):
    say(f"linear T={T} rows={rows} K={K}")
    c = Case(M, T, rows, K, residual=True, bias=True)
    c.check(c.run(M))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "silu_mul"])
@pytest.mark.parametrize("out", ["bf16", "mxfp8"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T", [3, 40, 150, 1060])
def test_every_epilogue(M, act, out, bias, residual, T):
    say(f"linear act={act} out={out} bias={bias} residual={residual} T={T}")
    c = Case(M, T, 320, 640, act, bias, residual, out, seed=1)
    c.check(c.run(M))


@pytest.mark.parametrize("T,rows,K", [(1, 64, 7168), (16, 64, 65536), (9, 6144, 2048), (72, 4096, 7168), (72, 64, 7168),
                                      (288, 512, 6144), (400, 6144, 256), (1001, 2048, 512), (2050, 512, 256), (5, 16384, 128),
                                      (130, 8192, 256)])
def test_real_shapes(M, T, rows, K):
    say(f"linear T={T} rows={rows} K={K}")
    for act, out in (("none", "bf16"), ("silu_mul", "mxfp8")):
        c = Case(M, T, rows, K, act, out=out, seed=2)
        c.check(c.run(M))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "silu_mul"])
@pytest.mark.parametrize("out", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T", [9, 100, 150, 1100])
def test_epilogues_of_a_split_sum(M, act, out, T):
    """An inner axis long enough to be split over workgroups."""
    say(f"linear split act={act} out={out} T={T}")
    c = Case(M, T, 192, 2176, act, True, True, out, seed=12)
    c.check(c.run(M))


@pytest.mark.parametrize("T,rows,K", [(12301, 1088, 256), (2050, 2176, 384), (49200, 256, 128)])
@pytest.mark.parametrize("act,out", [("none", "bf16"), ("silu_mul", "mxfp8"), ("gelu", "mxfp8"), ("silu_mul", "bf16")])
def test_large_grids(M, T, rows, K, act, out):
    """Enough tiles for the largest tile shape, and for several rounds of the
    smaller one; tokens around the tile borders and some between."""
    import torch
    say(f"linear T={T} rows={rows} K={K} act={act} out={out}")
    c = Case(M, T, rows, K, act, True, out == "bf16", out, seed=13)
    o = c.run(M)
    if out == "bf16":
        assert not torch.isnan(o["out"]).any()
    else:  # the marks that outputs() left: no finite code, no scale that occurs here
        assert not (o["out_codes"] == 0x7f).any() and not (o["out_scales"] == 77).any()
    edges = {0, 1, T - 2, T - 1} | {t + d for t in range(128, T, T // 9 // 128 * 128) for d in (-1, 0, 31, 32)}
    c.check(o, sorted(e for e in edges if e < T))


@pytest.mark.parametrize("T", [9, 50, 1100])
def test_strided_rows_and_in_place(M, T):
    import torch
    say(f"linear strided T={T}")
    c = Case(M, T, 192, 256, bias=True, residual=True, seed=3)
    wide = torch.full((T + 1, 400), 3.0, dtype=torch.bfloat16, device="cuda")
    part = wide[:T, 200:392]
    part.copy_(c.kw["residual"])
    c.run(M, residual=part, out=part)
    c.check(dict(out=part.clone()))
    assert (wide[:, :200] == 3).all() and (wide[:, 392:] == 3).all() and (wide[T] == 3).all()


@pytest.mark.parametrize("T", [4, 70, 300, 1100])
@pytest.mark.parametrize("out", ["bf16", "mxfp8"])
def test_nan_blocks_stay_where_they_are(M, T, out):
    """A NaN block of one weight row reaches its column alone, one of a token
    its row alone; infinite sums become infinities (bf16) or NaN blocks."""
    say(f"linear NaN T={T} {out}")
    c = Case(M, T, 256, 384, out=out, seed=4)
    c.ws[37, 5] = 255
    c.wc[37, 160:192] = 0
    c.xs[2, 1] = 255
    c.xc[2, 32:64] = 0
    import torch
    c.dev["x_scales"], c.dev["x_codes"] = torch.from_numpy(c.xs).cuda(), torch.from_numpy(c.xc).cuda()
    c.upload_weights(M)
    c.check(c.run(M))


@pytest.mark.parametrize("T", [4, 70, 300, 1100])
def test_wide_range_of_scales(M, T):
    """Blocks of very different scales in one row, far from 1 (products down
    to 2^-80 and up to 2^80)."""
    say(f"linear scales T={T}")
    c = Case(M, T, 128, 512, seed=5)
    rng = np.random.default_rng(6)
    c.xs = (127 + rng.integers(-45, 30, size=c.xs.shape)).astype(np.uint8)
    c.ws = (127 + rng.integers(-45, 30, size=c.ws.shape)).astype(np.uint8)
    import torch
    c.dev["x_scales"] = torch.from_numpy(c.xs).cuda()
    c.upload_weights(M)
    c.check(c.run(M))


@pytest.mark.parametrize("T", [64, 200, 1100])
def test_small_products_beside_large_ones(M, T):
    """One large product in each group of 8 consecutive k and small ones at
    every distance below it: up to 128 tokens all of them count, beyond it
    the FP8 matrix cores may drop what the bound allows and no more."""
    say(f"linear small products T={T}")
    import torch
    c = Case(M, T, 64, 256, seed=11)
    x, w = np.full((T, 256), 1.0), np.zeros((64, 256))
    for n in range(64):
        w[n] = 2.0 ** -(4 + n % 14)        # within E4M3's range at one block scale
        w[n, n % 8::8] = 256.0 if n % 2 else 0.0
    c.xc, c.xs = encode(x)
    c.wc, c.ws = encode(w)
    c.dev["x_codes"], c.dev["x_scales"] = torch.from_numpy(c.xc).cuda(), torch.from_numpy(c.xs).cuda()
    c.upload_weights(M)
    c.check(c.run(M))


def test_exact_small_integers(M):
    """Sums of small integers are exact in float32 (and on the FP8 matrix cores:
    products up to 9 need no bits below 2^-13 of the largest): the output is,
    whatever the order of the sum."""
    say("linear integers")
    rng = np.random.default_rng(7)
    for T in (7, 90, 310, 1050):
        c = Case(M, T, 256, 1024, seed=8)
        x, w = rng.integers(-3, 4, size=(T, 1024)), rng.integers(-3, 4, size=(256, 1024))
        c.xc, c.xs = encode(x)
        c.wc, c.ws = encode(w)
        import torch
        c.dev["x_codes"], c.dev["x_scales"] = torch.from_numpy(c.xc).cuda(), torch.from_numpy(c.xs).cuda()
        c.upload_weights(M)
        got = R.values(c.run(M)["out"])
        assert np.array_equal(got, R.bf16_rne((x @ w.T).astype(np.float64)))


def test_no_tokens_and_determinism(M):
    import torch
    c = Case(M, 1, 64, 128)
    e = lambda n: torch.empty(0, n, dtype=torch.uint8, device="cuda")
    assert M.moe_mxfp8_linear(e(128), e(4), c.dev["w_tiles"], c.dev["w_scales"],
                              out=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")) == M.MOE_OK
    for T in (9, 72, 300, 600, 1100):
        c = Case(M, T, 1024, 2048, seed=9)
        a, b = c.run(M), c.run(M)
        assert torch.equal(a["out"], b["out"])


@pytest.mark.parametrize("T,rows", [(9, 1024), (72, 1024), (600, 1024), (1100, 256)])
def test_streams_and_graphs(M, T, rows):
    """A call on a stream of its own; two captured calls with workspaces of
    their own replayed side by side on changed inputs give the eager bits."""
    import torch
    say(f"linear graphs T={T} rows={rows}")
    cs = [Case(M, T, rows, 2048, "silu", True, True, seed=10 + i) for i in range(2)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    cs[0].check(cs[0].run(M, stream=st))
    outs, graphs = [c.outputs() for c in cs], []
    for c, o in zip(cs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.moe_mxfp8_linear(**c.dev, **c.kw, **o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rnd in range(3):
        for i, (c, o) in enumerate(zip(cs, outs)):
            n = Case(M, T, rows, 2048, "silu", True, True, seed=30 + 2 * rnd + i)
            for name in ("x_codes", "x_scales"):
                c.dev[name].copy_(n.dev[name])
            o["out"].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            assert torch.equal(c.run(M)["out"], o["out"])
