"""The cache and the attention over it in 64 bits (numpy), for their tests:
written from the formulas in include/ops/moe_attention.h."""
from __future__ import annotations

import numpy as np

from tests import ops_reference as R

BF16 = 2.0 ** -8   # half a step of bf16, relative


class Cache:
    """A device cache; pages may lie apart, as parts of one allocation."""

    def __init__(self, pages, kv, page, D, apart=False, seed=0, fill=None):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def random(*shape):
            if fill is not None:
                return torch.full(shape, fill, dtype=torch.uint8, device="cuda")
            return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)

        if apart:
            codes, scales = random(pages, 2, kv, page, D), random(pages, 2, kv, page, D // 32)
            self.kc, self.vc, self.ks, self.vs = codes[:, 0], codes[:, 1], scales[:, 0], scales[:, 1]
        else:
            self.kc, self.vc = random(pages, kv, page, D), random(pages, kv, page, D)
            self.ks, self.vs = random(pages, kv, page, D // 32), random(pages, kv, page, D // 32)
        self.page = page

    @property
    def tensors(self):
        return self.kc, self.ks, self.vc, self.vs

    def put(self, which, slots, codes, scales):
        """codes [n, kv, D], scales [n, kv, D/32] (numpy) into the slots, by torch."""
        import torch
        c, s = (self.kc, self.ks) if which == "k" else (self.vc, self.vs)
        at = torch.as_tensor(np.asarray(slots, np.int64), device="cuda")
        c[at // self.page, :, at % self.page] = torch.from_numpy(codes).cuda()
        s[at // self.page, :, at % self.page] = torch.from_numpy(scales).cuda()


def seen(L, n, mask, i):
    """The positions that drafted token i of n sees behind L committed ones;
    mask: the token's words (uint64), or None."""
    if mask is None:
        drafted = [j for j in range(n) if j <= i]
    else:
        drafted = [j for j in range(min(n, 64 * len(mask))) if int(mask[j // 64]) >> (j % 64) & 1]
    return np.array(list(range(L)) + [L + j for j in drafted], np.int64)


def attend(q, k, v, scale):
    """q [D], k and v [n, D]: the result, the bound of its error from all but
    the last rounding, and the mean square of the error that independent
    roundings of the weights leave.

    A score is a float32 sum of D exact products: off by at most D 2^-24 of the
    sum of their magnitudes, twice that for adders that do not round to
    nearest.  The exponent c s - c m takes one rounding of c (2^-23 with log2
    e's), two of its own; the exponential 2^-22, the weight's rounding 2^-8.
    With weights w_p (1 + e_p) the quotient is off by sum w_p e_p (v_p - o) /
    sum w_p (1 + e_p).  The sums over the n positions and their joins add
    (n + 64) 2^-23 of sum w |v|."""
    if len(k) == 0:
        z = np.zeros(v.shape[1])
        return z, z, z
    s = k @ q * scale
    w = np.exp(s - s.max())
    w /= w.sum()
    o = w @ v
    D = len(q)
    ds = scale * (D * 2.0 ** -23) * (np.abs(k) @ np.abs(q))
    e = BF16 + 2.0 ** -22 + ds + 2.0 ** -22 * (np.abs(s) + np.abs(s).max())
    away = np.abs(v - o)
    err = (w * e) @ away / (1 - e.max()) + (len(k) + 64) * 2.0 ** -23 * (w @ np.abs(v))
    return o, err, (w * w) @ (away * away) * BF16 ** 2 / 3


def attention(q, k, v, mask, L, scale):
    """All drafted tokens of a sequence.  q [n, H, D], k and v [len, kv, D] in
    float64 (len <= L + n where the table ends), mask [n, words] uint64 or None."""
    n, H, D = q.shape
    kv = k.shape[1]
    out = [np.zeros((n, H, D)) for _ in range(3)]
    for i in range(n):
        at = seen(L, n, None if mask is None else mask[i], i)
        at = at[at < len(k)]
        for h in range(H):
            g = h // (H // kv)
            for x, y in zip(out, attend(q[i, h], k[at, g], v[at, g], scale)):
                x[i, h] = y
    return out


def check(got, ref, err, square, what):
    """Each element within its bound's roundings, and the whole's error no
    more than 1.3 times what independent roundings leave (of the weights, and
    of the result: uniform within half a step)."""
    R.assert_between(got, R.bf16_rne(ref - err), R.bf16_rne(ref + err), what)
    want = np.sqrt((square + (ref * BF16) ** 2 / 3).sum())
    off = np.sqrt(((got - ref) ** 2).sum())
    assert off <= 1.3 * want + 1e-30 or got.size < 2048, (what, off, want)
