"""GPU: the attention over cached values that are no numbers, in every shape of
workgroup: what sees such a value becomes one, whichever tile of 32 positions
it lies in, and every other element keeps its bits."""
import numpy as np
import pytest

from tests import attention_reference as A
from tests import ops_reference as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

PAGE, CONTEXT = 32, 4112   # half a page of the committed positions is a sequence's own


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


class Shared:
    """Sequences that share the pages of their first positions; lost: pages
    that a sequence's table names outside the cache.  As many of them as give
    each workgroup a run of several tiles."""

    def __init__(self, M, D, kv, G, counts, lost=None, empty=0.1, seed=0):
        import torch
        self.M, self.D, self.kv, self.G, self.counts, self.lost = M, D, kv, G, counts, lost or {}
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B, held = len(counts), CONTEXT // PAGE
        own = -(-(CONTEXT % PAGE + max(counts)) // PAGE)
        self.pages = held + B * own
        self.cache = A.Cache(self.pages, kv, PAGE, D, fill=0)
        for start in range(0, self.pages * PAGE, 4096):
            slots = torch.arange(start, min(self.pages * PAGE, start + 4096), device="cuda")
            k, v = (torch.randn(len(slots), kv, D, device="cuda", generator=gen) for _ in range(2))
            M.moe_kv_write(k, v, slots, *self.cache.tensors)
        self.table = np.concatenate([np.broadcast_to(np.arange(held), (B, held)),
                                     held + np.arange(B * own).reshape(B, own)], 1).astype(np.int32)
        for b, pages in self.lost.items():
            self.table[b, pages] = self.pages + np.arange(len(pages))
        self.offsets = np.cumsum([0] + list(counts))
        self.T, self.words = int(self.offsets[-1]), -(-max(counts) // 64)
        bits = []
        for n in counts:
            for i in range(n):
                up = bits[-1] if i and rng.random() < 0.6 else 0
                bits.append(0 if rng.random() < empty else up | 1 << i)
        self.mask = np.array([[b >> 64 * w & (1 << 64) - 1 for w in range(self.words)] for b in bits], np.uint64)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        self.q = torch.randn(self.T, kv * G, D, device="cuda", generator=gen).bfloat16()
        self.out = torch.empty_like(self.q)
        self.table_t, self.ctx_t, self.off_t = i32(self.table), i32([CONTEXT] * B), i32(self.offsets)
        self.mask_t = torch.from_numpy(self.mask.view(np.int64)).cuda()
        self.ws = torch.empty(M.moe_tree_attention_workspace(self.T, B, kv * G, kv, D), dtype=torch.uint8,
                              device="cuda")

    def call(self):
        """The result [tokens, key/value heads, heads of one, D]."""
        import torch
        self.out.fill_(9)
        self.M.moe_tree_attention(self.q, *self.cache.tensors, self.table_t, self.ctx_t, self.off_t, self.out,
                                  self.D ** -0.5, mask=self.mask_t, workspace=self.ws)
        torch.cuda.synchronize()
        return R.values(self.out).reshape(self.T, self.kv, self.G, self.D)

    def place(self, b, position):
        return int(self.table[b, position // PAGE]), position % PAGE

    def seers(self, b, position):
        """The tokens that see a position of sequence b's table."""
        first, n = self.offsets[b], self.counts[b]
        if not 0 <= self.table[b, position // PAGE] < self.pages:
            return []
        if position < CONTEXT:
            return list(range(first, first + n))
        j = position - CONTEXT
        return [t for t in range(first, first + n) if int(self.mask[t, j // 64]) >> (j % 64) & 1]

    def spots(self):
        """(sequence or None, position) to put a value at: shared positions at
        the start, all over the first tiles, in every unit of 128 positions at
        a place of its own, behind the pages that are none; of a few sequences
        the last committed position and drafted ones."""
        shared = [0, 5, 31, 32, 77, 96, 127] + [128 * u + 37 * u % 128 for u in range(1, CONTEXT // 128)] + [
            128, 1024, 3 * PAGE + 40, 20 * PAGE + 16, 22 * PAGE, 40 * PAGE + 65, 40 * PAGE + 130]
        own = []
        for b in (0, 1, len(self.counts) - 1):
            own += [(b, CONTEXT - 1), (b, CONTEXT), (b, CONTEXT + self.counts[b] - 1)]
        return [(None, p) for p in dict.fromkeys(shared)] + list(dict.fromkeys(own))

    def put(self, spots, codes):
        """Code i of the last head at spot i, in an element of its own; what then
        sees element d of that head and which code it sees, as [(tokens, d, code)]."""
        at = []
        for i, ((b, position), code) in enumerate(zip(spots, codes)):
            d = (11 * i + 2) % self.D
            page, offset = self.place(b or 0, position)
            assert 0 <= page < self.pages
            self.cache.vc[page, self.kv - 1, offset, d] = code
            at.append((sum((self.seers(s, position) for s in (range(len(self.counts)) if b is None else [b])), []), d,
                       code))
        return at


LOST = {1: [3], 2: [0, 20, 21], 3: [40], 5: [127]}
SHAPES = [  # head_dim, query heads of a key/value head, drafted tokens: row tiles full, partly filled, of waves without rows
    (64, 7, [1] * 16), (64, 7, [4] * 16), (64, 7, [9] * 16), (64, 7, [16, 2] * 8),
    (128, 8, [2] * 16), (128, 7, [4] * 16), (128, 8, [4] * 16), (128, 7, [9] * 16), (128, 7, [15, 2] * 8),
    (128, 7, [64, 61, 20, 3] * 2), (256, 7, [1] * 16), (256, 7, [4] * 16), (256, 7, [7, 1] * 8), (256, 7, [9] * 16),
    (256, 7, [15, 2] * 8), (256, 7, [64, 61, 20, 3] * 2)]


@pytest.mark.parametrize("D,G,counts", SHAPES, ids=str)
def test_nan_in_any_tile(M, D, G, counts):
    """A value's NaN, wherever in the committed positions and the drafted ones
    it lies, reaches what sees it."""
    say(f"attention with NaN in committed values D={D} G={G} counts={counts}")
    s = Shared(M, D, 2, G, counts, {b: p for b, p in LOST.items() if b < len(counts)}, seed=D + sum(counts))
    plain = s.call()
    assert np.isfinite(plain).all()
    spots = s.spots()
    assert len(spots) <= D
    want = plain.copy()
    for tokens, d, _ in s.put(spots, [0x7f, 0xff] * len(spots)):
        want[tokens, -1, :, d] = np.nan
    np.testing.assert_array_equal(s.call(), want)


@pytest.mark.parametrize("D,G,counts", SHAPES, ids=str)
def test_block_without_a_scale(M, D, G, counts):
    """What moe_kv_write makes of an infinite input (a block of scale 255) in a
    position of whole tiles reaches all that sees it, and its block alone."""
    say(f"attention with a written infinity D={D} G={G} counts={counts}")
    import torch
    s = Shared(M, D, 2, G, counts, {b: p for b, p in LOST.items() if b < len(counts)}, seed=D)
    plain = s.call()
    for position in (3, 128 * 5 + 64, 24 * PAGE + 7, 30 * 128 + 33):
        page, offset = s.place(0, position)
        keep = [t[page].clone() for t in s.cache.tensors]
        slots = torch.tensor([page * PAGE + offset], device="cuda")
        k, v = (torch.empty(1, s.kv, D, device="cuda") for _ in range(2))
        M.moe_kv_read(*s.cache.tensors, slots, k, v)
        v[0, 0, 40] = float("inf")
        M.moe_kv_write(k, v, slots, *s.cache.tensors)
        want = plain.copy()
        for b in range(len(counts)):
            want[s.seers(b, position), 0, :, 32:64] = np.nan
        np.testing.assert_array_equal(s.call(), want, err_msg=str(position))
        # a scale that is none makes NaN of every code, not infinities
        s.cache.vc[page, 0, offset, 32:64] = torch.arange(32, device="cuda").byte() * 8 + 4
        np.testing.assert_array_equal(s.call(), want, err_msg=f"codes at {position}")
        for t, was in zip(s.cache.tensors, keep):
            t[page] = was


@pytest.mark.parametrize("D,G,counts", SHAPES, ids=str)
def test_infinite_values_in_any_tile(M, D, G, counts):
    """A value beyond float32's range is an infinity of its sign for what sees
    it, whether its tile holds committed positions alone, drafted ones or a page
    that is none; two of different signs, or one beside a NaN, make a NaN."""
    say(f"attention with infinite cached values D={D} G={G} counts={counts}")
    s = Shared(M, D, 2, G, counts, {b: p for b, p in LOST.items() if b < len(counts)}, seed=D + len(counts))
    spots = s.spots()
    # their blocks: zeros under the largest scale, 448 2^127 being no float32
    for b, position in spots:
        page, offset = s.place(b or 0, position)
        s.cache.vc[page, s.kv - 1, offset] = 0
        s.cache.vs[page, s.kv - 1, offset] = 254
    plain = s.call()
    assert np.isfinite(plain).all()
    keep = s.cache.vc.clone()
    # one infinity an element
    want = plain.copy()
    for tokens, d, code in s.put(spots, [0x7e, 0xfe, 0xfe, 0x7e, 0x7e] * len(spots)):
        want[tokens, -1, :, d] = -np.inf if code & 0x80 else np.inf
    np.testing.assert_array_equal(s.call(), want)
    # several in one element: of one sign, of both, beside a NaN
    for n, codes in ((5, [0x7e] * 5), (5, [0xfe] * 5), (6, [0x7e] * 5 + [0xfe]), (4, [0x7f, 0x7e, 0x7e, 0x7e]),
                     (len(spots), [0xfe] * (len(spots) - 1) + [0x7e])):
        s.cache.vc.copy_(keep)
        some = spots[-n:]
        seen = np.zeros((2, s.T), bool)     # tokens that see a value above, below zero (a NaN: both)
        for (b, position), code in zip(some, codes):
            page, offset = s.place(b or 0, position)
            s.cache.vc[page, s.kv - 1, offset, 17] = code
            tokens = sum((s.seers(q, position) for q in (range(len(counts)) if b is None else [b])), [])
            seen[0, tokens] |= code in (0x7e, 0x7f)
            seen[1, tokens] |= code in (0xfe, 0x7f)
        want = plain.copy()
        for above, below, value in ((True, False, np.inf), (False, True, -np.inf), (True, True, np.nan)):
            want[(seen[0] == above) & (seen[1] == below), -1, :, 17] = value
        np.testing.assert_array_equal(s.call(), want, err_msg=str(codes))


@pytest.mark.parametrize("D,G,counts", [s for s in SHAPES if max(s[2]) > 1], ids=str)
def test_rows_do_not_touch_each_other(M, D, G, counts):
    """A token's result keeps its bits whatever its siblings ask for, and
    whatever the drafted keys and values that it does not see are: over several
    tiles a wave, with scores that rise again and again."""
    say(f"attention with siblings changed D={D} G={G} counts={counts}")
    s = Shared(M, D, 2, G, counts, {b: p for b, p in LOST.items() if b < len(counts)}, seed=2 * D + sum(counts))
    s.q.mul_(3)
    plain = s.call()
    query, mask = s.q.clone(), s.mask.copy()
    # the second token of each sequence asks for something else, louder and louder
    odd = s.offsets[:-1][np.array(counts) > 1] + 1
    others = np.setdiff1d(np.arange(s.T), odd)
    for factor in (-1, 0.01, 4, 30):
        s.q.copy_(query)
        s.q[odd] *= factor
        got = s.call()
        assert np.array_equal(got[others], plain[others]), factor
        assert not np.array_equal(got[odd], plain[odd])
    # a head alone, beside the other heads of its rows
    s.q.copy_(query)
    s.q[:, G] *= 20
    got = s.call()
    assert np.array_equal(np.delete(got, 0, 2)[:, 1], np.delete(plain, 0, 2)[:, 1])
    assert np.array_equal(got[:, 0], plain[:, 0])
    s.q.copy_(query)
    # drafted keys and values as large as any, of which each only its own token sees
    changed = False
    for b, n in enumerate(counts):
        for j in range(n):
            if s.seers(b, CONTEXT + j) not in ([], [s.offsets[b] + j]):
                continue
            page, offset = s.place(b, CONTEXT + j)
            for t in (s.cache.ks, s.cache.vs):
                t[page, :, offset] = 140
            got = s.call()
            others = np.setdiff1d(np.arange(s.T), s.seers(b, CONTEXT + j))
            assert np.array_equal(got[others], plain[others]), (b, j)
            plain[s.seers(b, CONTEXT + j)] = got[s.seers(b, CONTEXT + j)]
            changed = True
    assert changed
