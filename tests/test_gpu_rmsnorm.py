"""moe_rmsnorm against the formula in 64 bits.

The kernel forms the sum, its statistic and n in 64 bits; between its n and
numpy's lie a few roundings of 2^-53 and the order of the row's sum (at most
H of them, all terms positive): relative (H + 8) * 2^-53.  codes, y and
residual_out have to be the roundings of a value that close."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def _case(T, H, x, residual, weight, seed):
    rng = np.random.default_rng(seed)
    col = np.exp(0.5 * rng.standard_normal(H))
    t = dict(x=R.tensor(rng.standard_normal((T, H)) * col, x),
             w=R.tensor(1 + 0.1 * rng.standard_normal(H), weight),
             r=None if residual is None else R.tensor(4 * rng.standard_normal((T, H)) * col, residual))
    return t


def _outputs(T, H, r, y=True, codes=True):
    import torch
    full = lambda *s, dtype, v: torch.full(s, v, dtype=dtype, device="cuda")
    return dict(residual_out=None if r is None else full(T, H, dtype=r.dtype, v=float("nan")),
                y=full(T, H, dtype=torch.bfloat16, v=float("nan")) if y else None,
                codes=full(T, H, dtype=torch.uint8, v=0x7f) if codes else None,
                scales=full(T, H // 32, dtype=torch.uint8, v=77) if codes else None)


def _check(t, o, eps):
    r = None if t["r"] is None else R.values(t["r"])
    s, n = R.rmsnorm(R.values(t["x"]), r, R.values(t["w"]), eps)
    H = n.shape[1]
    err = np.abs(n) * (H + 8) * 2.0 ** -53
    if o["residual_out"] is not None:
        want = R.bf16_rne(s) if "bfloat16" in str(o["residual_out"].dtype) else s.astype(np.float32).astype(np.float64)
        got = R.values(o["residual_out"])
        assert np.array_equal(got, want, equal_nan=True), "residual_out"
    if o["y"] is not None:
        R.assert_between(R.values(o["y"]), R.bf16_rne(n - err), R.bf16_rne(n + err), "y")
    if o["codes"] is not None:
        R.assert_mx8_of(o["codes"].cpu().numpy(), o["scales"].cpu().numpy(), n, err, "mxfp8")


@pytest.mark.parametrize("H", [32, 64, 96, 480, 512, 544, 2048, 2080, 4096, 4128, 6144, 7168, 8192, 8224, 16384])
@pytest.mark.parametrize("T", [1, 5])
def test_every_row_length(M, T, H):
    say(f"rmsnorm T={T} H={H}")
    t = _case(T, H, "bf16", "bf16", "bf16", 1000 + H)
    o = _outputs(T, H, t["r"])
    M.moe_rmsnorm(t["x"], t["w"], 1e-5, residual=t["r"], **o)
    _check(t, o, 1e-5)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [None, "bf16", "f32"])
@pytest.mark.parametrize("weight", ["bf16", "f32"])
@pytest.mark.parametrize("outputs", ["y", "codes", "both"])
def test_every_type(M, x, residual, weight, outputs):
    say(f"rmsnorm x={x} residual={residual} weight={weight} outputs={outputs}")
    t = _case(9, 1440, x, residual, weight, 7)
    o = _outputs(9, 1440, t["r"], y=outputs != "codes", codes=outputs != "y")
    M.moe_rmsnorm(t["x"], t["w"], 1e-6, residual=t["r"], **o)
    _check(t, o, 1e-6)


@pytest.mark.parametrize("T", [2, 63, 64, 257, 1025])
def test_many_rows(M, T):
    say(f"rmsnorm T={T}")
    t = _case(T, 352, "bf16", "f32", "f32", T)
    o = _outputs(T, 352, t["r"])
    M.moe_rmsnorm(t["x"], t["w"], 1e-5, residual=t["r"], **o)
    _check(t, o, 1e-5)


def test_strided_rows_and_in_place(M):
    import torch
    say("rmsnorm strided rows, residual in place, y over x")
    T, H = 6, 288
    t = _case(T, H, "bf16", "bf16", "f32", 3)
    wide = torch.full((T, 3 * H), float("nan"), dtype=torch.bfloat16, device="cuda")
    x, r = wide[:, :H], wide[:, H:2 * H]
    x.copy_(t["x"])
    r.copy_(t["r"])
    o = _outputs(T, H, t["r"])
    o["residual_out"], o["y"] = r, x
    M.moe_rmsnorm(x, t["w"], 1e-5, residual=r, **o)
    _check(t, dict(o, residual_out=r.clone(), y=x.clone()), 1e-5)
    assert torch.isnan(wide[:, 2 * H:]).all(), "columns beside the rows were written"
    # the sum over x itself
    x.copy_(t["x"])
    o = dict(_outputs(T, H, t["r"]), residual_out=x)
    M.moe_rmsnorm(x, t["w"], 1e-5, residual=t["r"], **o)
    _check(t, dict(o, residual_out=x.clone()), 1e-5)


def test_rows_far_apart(M):
    """Row offsets past 2^31 elements."""
    import torch
    say("rmsnorm rows 2^31 elements apart")
    H, stride = 64, (1 << 31) + 64
    t = _case(2, H, "bf16", "bf16", "f32", 4)
    big = torch.empty(stride + H, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, H), (stride, 1))
    x.copy_(t["x"])
    o = _outputs(2, H, t["r"])
    M.moe_rmsnorm(x, t["w"], 1e-5, residual=t["r"], **o)
    _check(t, o, 1e-5)


def test_rows_of_zeros_infinities_and_nan(M):
    """A zero row gives zeros (scale code 0), with eps = 0 NaN as the formula
    does; an infinity or a NaN reaches what the formula says it reaches and
    no other row."""
    import torch
    say("rmsnorm special rows")
    T, H = 7, 128
    t = _case(T, H, "f32", None, "f32", 5)
    t["x"][1] = 0
    t["x"][2, 40] = float("inf")
    t["x"][3, 100] = float("nan")
    t["x"][4] = 1e30
    t["x"][5] = 1e-30
    t["x"][6, ::2] = 0
    for eps in (1e-5, 0.0):
        o = _outputs(T, H, None)
        M.moe_rmsnorm(t["x"], t["w"], eps, **o)
        _check(t, o, eps)
    o = _outputs(T, H, None)
    M.moe_rmsnorm(t["x"], t["w"], 1e-5, **o)
    assert not o["codes"][1].any() and not o["scales"][1].any()
    assert (o["scales"][3] == 255).all() and torch.isnan(o["y"][3]).all()
    assert (o["scales"][2] == 255).sum() == 1


def test_block_scales_at_the_ends_of_their_range(M):
    """n from far below to far above what a block scale can hold: clamped
    scales, saturated codes, as the encoder's rule says."""
    say("rmsnorm scale range")
    H = 32 * 12
    t = _case(3, H, "f32", None, "f32", 6)
    for b in range(12):
        t["w"][32 * b:32 * b + 32] = 2.0 ** (-148 + 25 * b)
    o = _outputs(3, H, None, y=False)
    M.moe_rmsnorm(t["x"], t["w"], 1e-5, **o)
    _check(t, o, 1e-5)


def test_no_tokens(M):
    import torch
    t = _case(1, 64, "bf16", "bf16", "f32", 8)
    e = t["x"][:0]
    assert M.moe_rmsnorm(e, t["w"], 1e-5, residual=e, residual_out=e, y=e,
                         codes=torch.empty(0, 64, dtype=torch.uint8, device="cuda"),
                         scales=torch.empty(0, 2, dtype=torch.uint8, device="cuda")) == M.MOE_OK


def test_another_stream_and_a_graph(M):
    """Work goes to the stream given; a captured call replayed on new inputs
    gives the eager bits, with eager calls between the replays."""
    import torch
    say("rmsnorm stream and graph")
    T, H = 33, 2048
    t = _case(T, H, "bf16", "bf16", "f32", 9)
    o = _outputs(T, H, t["r"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.moe_rmsnorm(t["x"], t["w"], 1e-5, residual=t["r"], stream=s, **o)
    s.synchronize()
    _check(t, o, 1e-5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_rmsnorm(t["x"], t["w"], 1e-5, residual=t["r"], **o)
    for seed in range(3):
        n = _case(T, H, "bf16", "bf16", "f32", 20 + seed)
        t["x"].copy_(n["x"])
        e = _outputs(T, H, t["r"])
        M.moe_rmsnorm(t["x"], t["w"], 1e-5, residual=t["r"], **e)
        for v in o.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], e[k]), k
