"""moe_mxfp8_linear's sums over the inner axis are float32's at every number of
tokens.

Planted sums: products and partial sums that float32 holds whatever the order
of the additions (whole multiples of 2^-8, those of one sign together below
2^16), where large products that cancel stand beside small ones in every
eight consecutive k: a sum in fewer bits loses the small ones, which are the
result.  Random sums: the residual is minus the rounded result, so that the
output holds what a bf16 result hides.

FORMS: sizes of each form the call has (test_linear_plan_cpu.py holds them to
it): the few-token kernel, 128 x 128 tiles with up to one workgroup per CU and
with more, split sums, and 256 x 256 tiles, each with more chunks of 128 k
than twice those in LDS, odd and even counts."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.gpu_common import say
from tests.test_gpu_mxfp8_linear import Case, encode

pytestmark = pytest.mark.gpu

# name: (form, (tokens, rows, inner))
FORMS = {"few tokens": ("rows", (100, 256, 1152)), "small product": ("rows", (300, 512, 1152)),
         "narrow, a few": ("narrow", (1100, 256, 1152)), "narrow, whole tiles": ("narrow", (1152, 384, 1024)),
         "narrow, two per CU": ("narrow", (1300, 3328, 1152)), "narrow, even": ("narrow", (1409, 3200, 1024)),
         "split": ("narrow split", (1100, 192, 2176)), "wide": ("wide", (2600, 4096, 640)),
         "wide, even": ("wide", (2561, 4160, 1024))}


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def planted(T, rows, K, seed):
    """x and W: in each eight consecutive k of W one element of
    magnitude 256, of alternating sign and at the same x, the others up to
    3 * 2^-8."""
    rng = np.random.default_rng(seed)
    x = rng.choice([-2.0, -1.0, 1.0, 2.0], size=(T, K))
    w = rng.integers(-3, 4, size=(rows, K)) * 2.0 ** -8
    for n in range(rows):
        w[n, n % 8::8] = 256.0
        w[n, n % 8 + 8::16] = -256.0
    # x has the same value in each pair of eights that a large pair meets
    x.reshape(T, -1, 16)[:, :, 8:] = x.reshape(T, -1, 16)[:, :, :8]
    return x, w


def upload(c, M, x, w):
    import torch
    c.xc, c.xs = encode(x)
    c.wc, c.ws = encode(w)
    c.dev["x_codes"], c.dev["x_scales"] = torch.from_numpy(c.xc).cuda(), torch.from_numpy(c.xs).cuda()
    c.upload_weights(M)
    assert np.array_equal(R.mx8_values(c.xc, c.xs), x) and np.array_equal(R.mx8_values(c.wc, c.ws), w)


@pytest.mark.parametrize("form", FORMS)
def test_small_products_survive_large_ones(M, form):
    T, rows, K = FORMS[form][1]
    say(f"linear exact sums {form}: T={T} rows={rows} K={K}")
    x, w = planted(T, rows, K, T)
    assert ((np.abs(x) @ np.abs(w).T).max() + np.abs(x @ w.T).max()) / 2 < 2.0 ** 16
    v = x @ w.T
    c = Case(M, T, rows, K)
    upload(c, M, x, w)
    assert np.array_equal(R.values(c.run(M)["out"]), R.bf16_rne(v))
    # gated into MXFP8: the sums are exact, SiLU(g) * u is float32's
    c = Case(M, T, rows, K, "silu_mul", out="mxfp8")
    upload(c, M, x, w)
    o = c.run(M)
    g, u = v[:, :rows // 2], v[:, rows // 2:]
    a = R.silu(g)
    err = np.abs(u) * (8 + np.abs(g)) * R.STEP * np.abs(a) + R.STEP * np.abs(a * u)
    R.assert_mx8_of(o["out_codes"].cpu().numpy(), o["out_scales"].cpu().numpy(), a * u, err, form)


@pytest.mark.parametrize("form", FORMS)
def test_error_of_random_sums(M, form):
    """rms error against 64 bits, relative to the sum's rms.  d = v - r is even
    over half a step of bf16, 2^-8 |v| at most: rms 2^-8 / sqrt 3 of it; d's own
    rounding to bf16 as much again of d: 2^-16 / 3.  K float32 additions of
    at most half a step of the running sum each, independent: sqrt(K) 2^-24 at
    most.  (The subtraction is exact.)"""
    T, rows, K = FORMS[form][1]
    say(f"linear error {form}: T={T} rows={rows} K={K}")
    c = Case(M, T, rows, K, seed=21)
    v = R.mx8_values(c.xc, c.xs) @ R.mx8_values(c.wc, c.ws).T
    r = R.bf16_rne(v)
    got = R.values(c.run(M, residual=R.tensor(-r, "bf16"))["out"])
    scale = np.sqrt((v * v).mean(1, keepdims=True))  # tokens differ in size
    rms = np.sqrt((((got - (v - r)) / scale) ** 2).mean())
    print(f"rms error {rms:.2e}")
    assert rms <= 2.0 ** -16 / 3 + np.sqrt(K) * 2.0 ** -24


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("act,out", [("none", "bf16"), ("silu_mul", "mxfp8"), ("gelu", "mxfp8")])
def test_float32_bound_everywhere(M, form, act, out):
    """The bound of a float32 sum (ops_reference.linear at few tokens), with
    bias and residual, for each form's steady loop."""
    T, rows, K = FORMS[form][1]
    say(f"linear float32 bound {form} {act}: T={T} rows={rows} K={K}")
    c = Case(M, T, rows, K, act, True, True, out, seed=22)
    o = c.run(M)
    at = np.unique(np.concatenate([np.arange(0, T, max(1, T // 40)), [127, 128, 255, 256, T - 1]]) % T)
    v, dv = R.linear(c.xc[at], c.xs[at], c.wc, c.ws, act, c.bias, c.res[at], tokens=1)
    o = {k: t[at.tolist()] for k, t in o.items()}
    if out == "bf16":
        R.assert_between(R.values(o["out"]), R.bf16_rne(v - dv), R.bf16_rne(v + dv), form)
    else:
        R.assert_mx8_of(o["out_codes"].cpu().numpy(), o["out_scales"].cpu().numpy(), v, dv, form)
