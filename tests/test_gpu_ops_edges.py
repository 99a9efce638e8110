"""Calls at the ends of the operators' ranges."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.gpu_common import say
from tests.test_gpu_dispatch_combine import _dispatch, _ids, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


@pytest.mark.parametrize("H", [512, 2048, 16384])
def test_norm_results_below_the_normal_range_are_rounded_once(M, H):
    """y just beside the middle of two of bf16's subnormals (steps of 2^-133), by
    less than float32's subnormals can tell (2^-149): the nearer one, not the
    even one.  x = 1/2 (1 + d) in every column and eps = 1 - x^2 make the norm's
    factor 1 to 2^-51; n = w (1 + d) / 2."""
    import torch
    say(f"rmsnorm subnormal y H={H}")
    for d in (2.0 ** -22, -2.0 ** -22, 0.0):
        x = 0.5 * (1 + d)
        k = np.arange(H) % 200
        w = (2 * k + 1) * 2.0 ** -133 * np.where(np.arange(H) % 3 == 0, -1.0, 1.0)   # n = (k + 1/2) steps
        xt, wt = R.tensor(np.full((3, H), x), "f32"), R.tensor(w, "f32")
        assert np.array_equal(R.values(wt), w) and np.array_equal(R.values(xt), np.full((3, H), x))
        y = torch.full((3, H), 7.0, dtype=torch.bfloat16, device="cuda")
        M.moe_rmsnorm(xt, wt, 1.0 - x * x, y=y)
        _, n = R.rmsnorm(R.values(xt), None, w, 1.0 - x * x)
        if d:
            assert np.array_equal(R.values(y), R.bf16_rne(n))
        else:  # on the middle itself, or 2^-51 beside it
            err = np.abs(n) * (H + 8) * 2.0 ** -53
            R.assert_between(R.values(y), R.bf16_rne(n - err), R.bf16_rne(n + err), "y")


def test_combine_gradient_without_rows(M):
    """No row is held here: every position is elsewhere, and there is nothing to
    write but zeros for the weights."""
    import torch
    say("combine backward without rows")
    T, k, H = 5, 3, 64
    dout, w = torch.randn(T, H, device="cuda"), torch.rand(T, k, device="cuda")
    pos = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    pos[2, 1] = 4                                # past the rows
    for dt in (torch.float32, torch.bfloat16):
        rows, drows = torch.empty(0, H, dtype=dt, device="cuda"), torch.empty(0, H, dtype=dt, device="cuda")
        assert M.moe_combine_backward(dout, rows, w, pos, drows, None) == M.MOE_OK
        dw = torch.full((T, k), 3.0, device="cuda")
        M.moe_combine_backward(dout, rows, w, pos, drows, dw)
        out = torch.full((T, H), 3.0, device="cuda")
        M.moe_combine(rows, w, pos, out)
        torch.cuda.synchronize()
        assert not dw.any() and not out.any()


@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("act", ["silu", "silu_mul"])
def test_silu_of_large_arguments(M, T, act):
    """SiLU over the whole range where its result is a float32, through the bias
    (W is zero): v / (1 + exp(-v)) is normal down to v = -91.8, where exp(-v)
    has left float32's range."""
    import torch
    say(f"linear {act} of large arguments T={T}")
    rows, K = 1024, 128
    n = rows // 2 if act == "silu_mul" else rows
    v = np.concatenate([np.linspace(-103.9, 104, n - 6), [-91.5, -88.75, -88.5, -87.4, -1e4, 1e4]]).astype(np.float32)
    v = v.astype(np.float64)
    u = np.full(n, 1.0)
    bias = np.concatenate([v, u]) if act == "silu_mul" else v
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")
    out = torch.full((T, n), 3.0, dtype=torch.bfloat16, device="cuda")
    M.moe_mxfp8_linear(z(T, K), z(T, K // 32), z(rows, K), z(rows, K // 32), out=out, bias=R.tensor(bias, "f32"),
                       activation=M.MOE_EPI_SILU if act == "silu" else M.MOE_EPI_SILU_MUL)
    a = R.silu(v)
    err = (8 + np.abs(v)) * R.STEP * np.abs(a) + 2.0 ** -149
    lo, hi = R.bf16_rne(a - err), R.bf16_rne(a + err)
    R.assert_between(R.values(out), np.broadcast_to(lo, (T, n)), np.broadcast_to(hi, (T, n)), "silu")


@pytest.mark.parametrize("T,k,E", [(4096, 8, 128), (4224, 8, 128), (4096, 8, 129), (8192, 8, 1024), (16384, 1, 128),
                                   (16385, 1, 128), (2048, 32, 64), (70_000, 1, 7), (20_000, 4, 1024)])
def test_dispatch_on_both_sides_of_its_choice(M, T, k, E):
    """Counts summed by each workgroup, and scanned in a launch of their own."""
    say(f"dispatch T={T} k={k} E={E}")
    _dispatch(M, _x(T, 8, "bf16", T), _ids(T, k, E, T + k), E)
