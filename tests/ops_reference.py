"""The operators around the expert layer in 64 bits (numpy), for their tests:
written from the formulas in include/ops/moe_ops.h.

``between`` is how a rounded result is compared: with lo <= exact <= hi the
bounds of what the kernel may have rounded, the result must be a rounding of
some value in there, i.e. lie between the roundings of lo and hi (roundings
are monotone)."""
from __future__ import annotations

import math

import numpy as np

from oracle import brute

U32 = 2.0 ** -24  # half a step of float32, relative


def bf16_rne(v: np.ndarray) -> np.ndarray:
    """float64 -> the nearest bf16 (ties to even), as float64."""
    v = np.asarray(v, np.float64)
    e = np.maximum(np.frexp(np.where(np.isfinite(v), v, 0.0))[1] - 1, -126)
    step = np.ldexp(1.0, e - 7)
    with np.errstate(invalid="ignore"):
        r = np.where(np.isfinite(v), np.round(v / step) * step, v)
    return np.where(np.abs(r) > 3.3895313892515355e38, np.sign(r) * np.inf, r)


def tensor(v: np.ndarray, dtype: str, device="cuda"):
    """float64 -> a device tensor ("bf16" or "f32"); values are rounded there."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(v, np.float64))
    return t.to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(device)


def values(t) -> np.ndarray:
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def mx8_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """MXFP8 codes [.., n] and scales [.., n/32] as float64."""
    v = brute.e4m3_decode(codes)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def assert_between(got, lo, hi, what: str):
    ok = ((got >= lo) & (got <= hi)) | (np.isnan(got) & np.isnan(lo) & np.isnan(hi))
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.size} outside their bounds, first at {at}: "
                             f"got {got[at]!r}, bounds {lo[at]!r} .. {hi[at]!r}")


def assert_mx8_of(codes, scales, ref, err, what: str):
    """codes [T, n], scales [T, n/32] are the MXFP8 encoding of some values
    within err of ref: each block's scale is that of its largest magnitude
    there (one of two neighbours where the bounds straddle a power of two),
    each element, at that scale, a rounding of a value within the bounds."""
    T, n = ref.shape
    b, e = ref.reshape(T, -1, 32), np.broadcast_to(err, ref.shape).reshape(T, -1, 32)
    finite = np.isfinite(b).all(-1)
    assert np.array_equal(scales == 255, ~finite), f"{what}: NaN blocks"
    assert not codes.reshape(b.shape)[~finite].any(), f"{what}: a NaN block's codes are zero"
    b, e = np.where(finite[..., None], b, 0.0), np.where(finite[..., None], e, 0.0)

    def scale_exp(amax):
        x = np.where(amax > 0, np.frexp(amax)[1] - 1 - 8, -127)
        return np.clip(x, -127, 127)

    lo_s = scale_exp(np.maximum(np.abs(b) - e, 0.0).max(-1))
    hi_s = scale_exp((np.abs(b) + e).max(-1))
    s = scales.astype(np.int64) - 127
    assert (((s >= lo_s) & (s <= hi_s)) | ~finite).all(), f"{what}: block scales"
    x = np.ldexp(1.0, np.where(finite, s, 0))[..., None]
    got = brute.e4m3_decode(codes).reshape(b.shape)
    lo = brute._round_to_format((b - e) / x, 3, -6, 448.0)
    hi = brute._round_to_format((b + e) / x, 3, -6, 448.0)
    assert_between(got[finite], lo[finite], hi[finite], f"{what}: codes")


def rmsnorm(x, r, w, eps):
    s = x if r is None else x + r
    with np.errstate(all="ignore"):
        return s, s * w / np.sqrt((s * s).mean(1, keepdims=True) + eps)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def gelu(v):
    erfc = np.vectorize(math.erfc, otypes=[float])
    return 0.5 * v * erfc(-v / math.sqrt(2.0))


def order(ids, E):
    """(counts, offsets, sorted, pos) of the slots of ids [T, k] by counting."""
    flat = ids.reshape(-1)
    held = (flat >= 0) & (flat < E)
    counts = np.bincount(flat[held], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    at, pos, srt = offsets[:-1].copy(), np.full(flat.size, -1), np.full(int(offsets[-1]), -1)
    for s in np.nonzero(held)[0]:
        p = at[flat[s]]
        pos[s], srt[p] = p, s
        at[flat[s]] += 1
    return counts, offsets, srt, pos.reshape(ids.shape)


STEP = 2.0 ** -23  # a float32 step, relative


def linear(xc, xs, wc, ws, act="none", bias=None, res=None, tokens=None):
    """act(x W^T + bias) + res of MXFP8 operands, before the output's rounding,
    and how far a float32 evaluation of it may be off.

    x and W are exact in MXFP8, and so is each product in float32 (two
    four-bit significands).  The sum over K of them:
      the bf16 matrix cores (up to 128 tokens) and the additions between
      products: each partial sum is off by at most one float32 step of the
      sum of magnitudes, (K + 1) * 2^-23 * (sum |x w| + |bias|) in all;
      the FP8 matrix cores (more tokens): they add the 8 products of
      consecutive k first, and drop what lies below 2^-13 of the largest one's
      leading bit: each of the 8 is off by less than 2^-13 of the group's
      largest magnitude, 8 * 2^-13 * (sum over groups of max |x w|) in all
      (the typical error is far smaller: 1.4e-5 of the sum's rms).
    The activation:
      SiLU   moves by at most 1.1 dv, its own evaluation by (8 + |v|) * 2^-23 of
             it (an exponential of an argument rounded at 2^-24 |v|, a
             reciprocal, two products)
      GELU   moves by at most 1.13 dv, its evaluation by (16 + 2 v^2) * 2^-23 of
             it (erfc to a few steps, its argument rounded: relative
             2 a^2 * 2^-23 for a = v / sqrt 2)"""
    x, w = mx8_values(xc, xs), mx8_values(wc, ws)
    T, K = x.shape
    with np.errstate(invalid="ignore"):
        v, mag = x @ w.T, np.abs(x) @ np.abs(w).T
        if bias is not None:
            v, mag = v + bias, mag + np.abs(bias)
        dv = (K + 1) * STEP * mag
        if (tokens or T) > 128:  # tokens: of the call, where x holds some of them
            top = np.zeros_like(v)
            for k in range(0, K, 8):
                top += np.abs(x[:, None, k:k + 8] * w[None, :, k:k + 8]).max(-1)
            dv = dv + 8 * 2.0 ** -13 * top
        if act == "silu":
            a = silu(v)
            v, dv = a, 1.1 * dv + (8 + np.abs(v)) * STEP * np.abs(a)
        elif act == "gelu":
            a = gelu(v)
            v, dv = a, 1.13 * dv + (16 + 2 * v * v) * STEP * np.abs(a)
        elif act == "silu_mul":
            h = v.shape[1] // 2
            g, u, dg, du = v[:, :h], v[:, h:], dv[:, :h], dv[:, h:]
            a = silu(g)
            da = 1.1 * dg + (8 + np.abs(g)) * STEP * np.abs(a)
            v, dv = a * u, np.abs(u) * da + np.abs(a) * du + da * du + STEP * np.abs(a * u)
        if res is not None:
            v = v + res
            dv = dv + STEP * np.abs(v)
    return v, dv + 2.0 ** -149


def prepacked(M, codes: np.ndarray, scales: np.ndarray, pairs: bool):
    """Row-major MXFP8 weights on the device in the tile layout."""
    import torch
    c, s = torch.from_numpy(np.ascontiguousarray(codes)).cuda(), torch.from_numpy(np.ascontiguousarray(scales)).cuda()
    t, ts = torch.empty_like(c), torch.empty_like(s)
    M.moe_mxfp8_prepack(c.view(1, *c.shape), s.view(1, *s.shape), t, ts, gate_up_pairs=pairs)
    return t, ts
