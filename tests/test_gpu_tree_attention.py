"""GPU: attention of drafted tokens over the MXFP8 cache, against 64 bits."""
import numpy as np
import pytest

from tests import attention_reference as A
from tests import ops_reference as R
from tests.gpu_common import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import mxfp4_moe_expert_02_amd as M
    return M


def _encode(v):
    import oracle
    c, s = oracle.quantize_mxfp8(np.ascontiguousarray(v.reshape(-1, v.shape[-1])))
    return c.reshape(v.shape), s.reshape(*v.shape[:-1], v.shape[-1] // 32)


def _tree(rng, n, words, empty=0.1):
    """A random tree's masks [n, words] uint64; some rows without a bit."""
    bits = []
    for i in range(n):
        up = bits[rng.integers(max(0, i - 5), i)] if i and rng.random() < 0.8 else 0
        bits.append(0 if rng.random() < empty else up | 1 << i)
    return np.array([[b >> (64 * w) & (1 << 64) - 1 for w in range(words)] for b in bits], np.uint64).reshape(n, words)


class Batch:
    """seqs: (committed, drafted) of each sequence.  The cache's other slots,
    the tables' ends and the tokens of no sequence hold anything."""

    def __init__(self, M, seqs, heads, kv, D, page, tree=False, words=None, strided=False, pad=0, lead=0, seed=0,
                 spread=1.0, extra=2):
        import torch
        rng = np.random.default_rng(seed)
        self.M, self.seqs, self.kv, self.D, self.heads = M, seqs, kv, D, heads
        self.scale = spread / np.sqrt(D)
        self.T = lead + sum(n for _, n in seqs) + pad
        B = len(seqs)
        held = [-(-(L + n) // page) for L, n in seqs]
        self.max_pages = max(held) + extra
        pages = sum(held) + 3
        self.cache = A.Cache(pages, kv, page, D, apart=strided, seed=seed)
        order = rng.permutation(pages)
        # behind a sequence's pages its table names anything, other sequences' pages among it
        self.table = rng.choice([-1, -(1 << 31), pages, (1 << 31) - 1, 0, 1], size=(B, self.max_pages)).astype(np.int32)
        at, self.k, self.v = 0, [], []
        for b, (L, n) in enumerate(seqs):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
            pos = np.arange(L + n)
            slots = self.table[b, pos // page].astype(np.int64) * page + pos % page
            for which, store in (("k", self.k), ("v", self.v)):
                x = rng.standard_normal((L + n, kv, D)) * np.exp(0.5 * rng.standard_normal((1, kv, D)))
                codes, scales = _encode(x)
                self.cache.put(which, slots, codes, scales)
                store.append(R.mx8_values(codes, scales))
        self.offsets = lead + np.cumsum([0] + [n for _, n in seqs])
        words = words or max(1, -(-max([n for _, n in seqs] + [1]) // 64))
        self.mask = None
        if tree:
            self.mask = rng.integers(0, 1 << 63, (self.T, words)).astype(np.uint64)
            for b, (L, n) in enumerate(seqs):
                # bits past the sequence's tokens mean nothing
                junk = rng.integers(0, 1 << 63, (n, words)).astype(np.uint64)
                keep = np.array([sum(1 << j for j in range(64 * w, min(n, 64 * w + 64))) >> 64 * w for w in range(words)],
                                np.uint64)
                self.mask[self.offsets[b]:self.offsets[b + 1]] = (_tree(rng, n, words) & keep) | (junk & ~keep)
        q = rng.standard_normal((self.T, heads, D))
        self.qt = R.tensor(q, "bf16")
        if strided:
            wide = torch.zeros(self.T, heads + 2 * kv, D, dtype=torch.bfloat16, device="cuda")
            wide[:, :heads] = self.qt
            self.qt = wide[:, :heads]
        self.q = R.values(self.qt)
        self.out_wide = torch.full((self.T, heads + (3 if strided else 0), D), 9.0, dtype=torch.bfloat16, device="cuda")
        self.out = self.out_wide[:, :heads]
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
        self.table_t = i32(self.table)
        if strided:
            t = torch.full((B, self.max_pages + 3), -7, dtype=torch.int32, device="cuda")
            t[:, :self.max_pages] = self.table_t
            self.table_t = t[:, :self.max_pages]
        self.ctx_t, self.off_t = i32([L for L, _ in seqs]), i32(self.offsets)
        self.mask_t = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        need = M.moe_tree_attention_workspace(self.T, B, heads, kv, D)
        # no more than is asked for, and holding anything
        self.ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")

    def call(self, **kw):
        args = dict(mask=self.mask_t, workspace=self.ws)
        args.update(kw)
        return self.M.moe_tree_attention(self.qt, *self.cache.tensors, self.table_t, self.ctx_t, self.off_t, self.out,
                                         self.scale, **args)

    def reference(self):
        out = [np.zeros((self.T, self.heads, self.D)) for _ in range(3)]
        for b, (L, n) in enumerate(self.seqs):
            a, e = self.offsets[b], self.offsets[b + 1]
            m = None if self.mask is None else self.mask[a:e]
            for x, y in zip(out, A.attention(self.q[a:e], self.k[b], self.v[b], m, L, self.scale)):
                x[a:e] = y
        return out

    def check(self, what):
        import torch
        torch.cuda.synchronize()
        got = R.values(self.out)
        a, e = self.offsets[0], self.offsets[-1]
        assert (got[:a] == 9).all() and (got[e:] == 9).all(), f"{what}: tokens of no sequence"
        assert (self.out_wide[:, self.heads:] == 9).all(), f"{what}: beside the rows"
        ref, err, square = self.reference()
        A.check(got[a:e], ref[a:e], err[a:e], square[a:e], what)


SHAPES = [  # heads, kv heads, head_dim, page size
    (8, 8, 64, 16), (6, 2, 64, 64), (48, 8, 128, 64), (7, 1, 128, 16), (12, 12, 128, 128), (16, 1, 128, 32),
    (56, 8, 128, 64), (4, 2, 256, 16), (8, 1, 256, 64), (40, 2, 64, 1024), (3, 3, 256, 256)]
LENGTHS = [
    [(0, 1)], [(1, 1)], [(15, 1), (16, 1), (17, 1)], [(127, 1), (128, 2), (129, 3)], [(1000, 1)],
    [(0, 9)], [(5, 9), (0, 0), (300, 4), (31, 1)], [(64, 9), (23, 9), (500, 9)], [(0, 40), (97, 33)], [(250, 64)]]


@pytest.mark.parametrize("heads,kv,D,page", SHAPES)
@pytest.mark.parametrize("seqs", LENGTHS, ids=str)
@pytest.mark.parametrize("tree", [False, True])
def test_against_64_bits(M, heads, kv, D, page, seqs, tree):
    say(f"attention heads={heads} kv={kv} D={D} page={page} seqs={seqs} tree={tree}")
    b = Batch(M, seqs, heads, kv, D, page, tree=tree, strided=(heads + len(seqs)) % 2 == 0, pad=len(seqs) % 3,
              lead=len(seqs) % 2, seed=heads + D)
    assert b.call() == M.MOE_OK
    b.check("out")


@pytest.mark.parametrize("heads,kv,D,page,seqs,tree", [
    (56, 8, 128, 64, [(5003, 9)], True), (8, 2, 128, 16, [(9000, 1), (17, 1), (4097, 1)], False),
    (16, 2, 64, 32, [(3000, 7), (2000, 2)], True), (4, 1, 256, 64, [(2500, 9)], False),
    (8, 8, 128, 64, [(1500, 61)], True), (64, 4, 64, 16, [(700, 5)] * 9, True)])
def test_long(M, heads, kv, D, page, seqs, tree):
    say(f"attention over long sequences heads={heads} kv={kv} D={D} seqs={seqs}")
    b = Batch(M, seqs, heads, kv, D, page, tree=tree, pad=2, seed=11)
    b.call()
    b.check("out")


def test_many_sequences(M):
    """More than a wave's lanes, lengths of every kind, some without tokens."""
    say("attention of 150 sequences")
    rng = np.random.default_rng(2)
    seqs = [(int(rng.integers(0, 200)), int(rng.integers(0, 4))) for _ in range(150)]
    for tree in (False, True):
        b = Batch(M, seqs, 6, 2, 64, 16, tree=tree, pad=3, lead=2, seed=5)
        b.call()
        b.check("out")


@pytest.mark.parametrize("words,n", [(1, 64), (1, 70), (2, 70), (2, 128), (3, 130), (4, 100)])
def test_mask_words(M, words, n):
    """Trees of more than a word's tokens; tokens past the mask's words are
    seen by none."""
    say(f"attention with {words} mask words, {n} tokens")
    for L in (0, 33, 100):
        b = Batch(M, [(L, n), (7, 3)], 4, 2, 64, 32, tree=True, words=words, seed=n + L)
        b.call()
        b.check("out")


def test_chunk_of_a_prompt(M):
    """Without a mask any number of tokens: a chunk of a prompt."""
    say("attention of a prompt's chunk")
    for L, n in ((0, 300), (200, 190)):
        b = Batch(M, [(L, n)], 4, 1, 128, 64, seed=L)
        b.call()
        b.check("out")


@pytest.mark.parametrize("spread", [1e-3, 8.0, 60.0])
def test_scores_of_every_spread(M, spread):
    """Nearly equal weights, and scores that run up over hundreds of powers of
    two, in rising order, so that the reference is moved again and again."""
    say(f"attention with scores of spread {spread}")
    b = Batch(M, [(700, 9)], 8, 2, 128, 64, tree=True, seed=3, spread=spread)
    b.call()
    b.check("out")
    order = np.argsort(b.k[0][:, 0] @ b.q[0, 0])     # rising for the first row
    for which, store in (("k", b.k), ("v", b.v)):
        store[0] = store[0][order]
        pos = np.arange(709)
        b.cache.put(which, b.table[0, pos // 64].astype(np.int64) * 64 + pos % 64, *_encode(store[0]))
    b.call()
    b.check("rising")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L,n", [(0, 9), (45, 9), (100, 40)])
def test_no_numbers_where_nothing_sees_them(M, D, L, n):
    """Drafted keys and values that are no numbers reach the tokens that see
    them and no other; one in a committed position reaches all."""
    import torch
    say(f"attention with NaN in drafted tokens D={D} L={L} n={n}")
    b = Batch(M, [(L, n), (60, 2)], 6, 2, D, 16, tree=True, seed=D + L)
    a = b.offsets[0]
    plain = None
    for which, at in (("v", 0), ("k", 0), ("v", n - 1)):
        b.call()
        torch.cuda.synchronize()
        plain = R.values(b.out)
        for code, scale in ((0x7f, 127), (0xff, 100), (0, 255)):
            c, s = (b.cache.kc, b.cache.ks) if which == "k" else (b.cache.vc, b.cache.vs)
            p = L + at
            where = (int(b.table[0, p // 16]), 1, p % 16)
            keep = c[where].clone(), s[where].clone()
            c[where][33], s[where][1] = code, scale
            b.out.fill_(9)
            b.call()
            torch.cuda.synchronize()
            c[where], s[where] = keep
            got = R.values(b.out)
            for i in range(n):
                sees = p in A.seen(L, n, b.mask[a + i], i)
                nan = np.isnan(got[a + i])
                if not sees:
                    assert np.array_equal(got[a + i], plain[a + i]), (which, at, i)
                    continue
                assert not nan[:3].any()                 # heads of the other key/value head
                if which == "k":
                    assert nan[3:].all()
                elif scale == 255:
                    assert nan[3:, 32:64].all() and not nan[3:, :32].any() and not nan[3:, 64:].any()
                else:
                    assert nan[3:, 33].all() and nan[3:].sum() == 3
            assert np.array_equal(got[a + n:], plain[a + n:])
    if L:
        where = (int(b.table[0, (L - 1) // 16]), 0, (L - 1) % 16)
        b.cache.vc[where][5] = 0x7f
        b.call()
        got = R.values(b.out)
        rows = got[a:a + n]
        assert np.isnan(rows[:, :3, 5]).all() and np.isnan(rows).sum() == 3 * n


def test_infinite_query_in_one_row(M):
    """A row that is no number leaves the others of its tile alone."""
    import torch
    say("attention with a NaN query")
    b = Batch(M, [(200, 9)], 14, 2, 128, 64, seed=1)
    b.call()
    torch.cuda.synchronize()
    plain = R.values(b.out)
    b.qt[4, 3, 17] = float("nan")
    b.qt[6, 13] = float("inf")
    b.call()
    torch.cuda.synchronize()
    got = R.values(b.out)
    assert np.isnan(got[4, 3]).all() and np.isnan(got[6, 13]).all()
    got[4, 3], got[6, 13] = plain[4, 3], plain[6, 13]
    assert np.array_equal(got, plain)


def test_pages_that_are_none(M):
    """A page number outside the cache: its positions are not seen, whichever
    they are; lengths beyond the table end with it."""
    import torch
    say("attention with page numbers out of range")
    for bad in (-1, 1 << 20, -(1 << 31)):
        for page_at in (0, 2, 4):
            b = Batch(M, [(70, 6), (40, 3)], 6, 2, 128, 16, tree=True, seed=page_at)
            b.table_t[0, page_at] = bad
            b.call()
            torch.cuda.synchronize()
            got = R.values(b.out)
            gone = np.arange(16 * page_at, min(76, 16 * page_at + 16))
            for i in range(6):
                at = np.setdiff1d(A.seen(70, 6, b.mask[b.offsets[0] + i], i), gone)
                for h in range(6):
                    o, err, _ = A.attend(b.q[b.offsets[0] + i, h], b.k[0][at, h // 3], b.v[0][at, h // 3], b.scale)
                    R.assert_between(got[b.offsets[0] + i, h], R.bf16_rne(o - err), R.bf16_rne(o + err), f"token {i}")
    # all of them: nothing is seen
    b.table_t.fill_(-1)
    b.call()
    assert (b.out[int(b.offsets[0]):int(b.offsets[-1])] == 0).all()


def test_lengths_out_of_range(M):
    import torch
    say("attention with lengths out of range")
    # a negative length counts as none committed: the drafted tokens start at 0
    b = Batch(M, [(0, 5), (30, 2)], 4, 2, 64, 16, seed=8)
    b.ctx_t[0] = -5
    b.call()
    b.check("negative")
    # a table that ends before the drafted tokens: they are not there
    b = Batch(M, [(48, 5)], 4, 2, 64, 16, seed=9, extra=0)
    short = b.table_t[:, :3].contiguous()
    b.table_t, b.k[0], b.v[0] = short, b.k[0][:48], b.v[0][:48]
    b.call()
    b.check("cut table")
    b.ctx_t.fill_((1 << 31) - 1)
    b.out.fill_(9)
    b.call()
    b.check("longer than its table")
    # offsets that do not ascend, or leave the tokens: no result at all
    for off in ([0, 5, 4], [-1, 3, 7], [0, 3, 8], [2, 1, 7], [0, 1 << 30, 7], [-(1 << 31), 0, (1 << 31) - 1]):
        b = Batch(M, [(20, 4), (30, 3)], 4, 2, 64, 16, seed=8)
        b.off_t.copy_(torch.tensor(off, dtype=torch.int32))
        b.call()
        torch.cuda.synchronize()
        assert (b.out == 9).all(), off


def test_far_pages(M):
    """Pages beyond 4 GiB of codes."""
    import torch
    say("attention beyond 32 bits")
    b = Batch(M, [(200, 9)], 16, 8, 128, 64, tree=True, seed=4)
    b.call()
    torch.cuda.synchronize()
    want = b.out.clone()
    pages = (1 << 32) // (8 * 64 * 128) + 20
    far = A.Cache(pages, 8, 64, 128, fill=0)
    move = torch.arange(b.cache.kc.shape[0], device="cuda") * 3 + pages - 3 * b.cache.kc.shape[0]
    for dst, src in zip(far.tensors, b.cache.tensors):
        dst[move] = src
    b.cache = far
    held = -(-209 // 64)
    b.table_t[0, :held] = move[b.table_t[0, :held].long()].int()
    b.out.fill_(9)
    b.call()
    torch.cuda.synchronize()
    assert torch.equal(b.out, want)


def test_same_bits_again(M):
    """The same inputs give the same bits, whatever the workspace held, with a
    workspace larger than asked for, and on another stream; two calls at once
    with a workspace each."""
    import torch
    say("attention again, on streams")
    b = Batch(M, [(3000, 9), (100, 9), (800, 9)], 56, 8, 128, 64, tree=True, seed=6)
    b.call()
    torch.cuda.synchronize()
    want = b.out.clone()
    for fill in (0, 255):
        b.ws.fill_(fill)
        b.out.fill_(9)
        b.call(workspace=torch.full((b.ws.numel() + 4096,), fill, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(b.out, want)
    c = Batch(M, [(3000, 9), (100, 9), (800, 9)], 56, 8, 128, 64, tree=True, seed=6)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        b.out.fill_(9), c.out.fill_(9)
        torch.cuda.synchronize()
        b.call(stream=s1)
        c.call(stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(b.out, want) and torch.equal(c.out, want)


def test_graph(M):
    """A step captured once and replayed on sequences that have grown, in a
    batch padded to the captured size; another graph with its own workspace."""
    import torch
    say("write and attention in a graph")
    page, kv, D, heads, n = 16, 2, 128, 12, 9
    rng = np.random.default_rng(7)
    big = Batch(M, [(400, n), (333, n), (250, n)], heads, kv, D, page, tree=True, seed=7, pad=4)
    kt, vt = (R.tensor(rng.standard_normal((big.T, kv, D)), "bf16") for _ in range(2))
    slots = torch.full((big.T,), -1, dtype=torch.int64, device="cuda")

    def step():
        M.moe_kv_write(kt, vt, slots, *big.cache.tensors)
        big.call()

    step()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        step()
    ws = big.ws
    big.ws = torch.empty_like(ws)
    with torch.cuda.graph(g2):
        step()
    big.ws = ws
    lens = [390, 200, 0]
    for rnd in range(4):
        counts = [n, n, n] if rnd % 2 else [n, 0, 4]
        off = np.cumsum([0] + counts)
        s = np.full(big.T, -1, np.int64)
        big.seqs, big.offsets = list(zip(lens, counts)), off
        for b, (L, k) in enumerate(big.seqs):
            pos = np.arange(L, L + k)
            s[off[b]:off[b + 1]] = big.table[b, pos // page].astype(np.int64) * page + pos % page
        kt.copy_(R.tensor(rng.standard_normal((big.T, kv, D)), "bf16"))
        vt.copy_(R.tensor(rng.standard_normal((big.T, kv, D)), "bf16"))
        slots.copy_(torch.from_numpy(s))
        big.ctx_t.copy_(torch.tensor(lens, dtype=torch.int32))
        big.off_t.copy_(torch.from_numpy(off.astype(np.int32)))
        big.out.fill_(9)
        step()
        torch.cuda.synchronize()
        eager = big.out.clone()
        for g in (g1, g2, g1):
            big.out.fill_(9)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(big.out, eager), rnd
        # what the cache holds now
        for store, codes, scales in ((big.k, big.cache.kc, big.cache.ks), (big.v, big.cache.vc, big.cache.vs)):
            for b, (L, k) in enumerate(big.seqs):
                pos = np.arange(L + k)
                at = torch.from_numpy(big.table[b, pos // page].astype(np.int64)).cuda()
                i = torch.from_numpy(pos % page).cuda()
                store[b] = R.mx8_values(codes[at, :, i].cpu().numpy(), scales[at, :, i].cpu().numpy())
        mask, big.mask = big.mask, big.mask.copy()
        big.check(f"replay {rnd}")
        big.mask = mask
        lens = [min(400, lens[0] + 3), lens[1] + 9, lens[2] + 4]


@pytest.mark.parametrize("heads,kv,D,page,seqs", [
    (56, 8, 128, 64, [(300, 30), (700, 31), (20, 20)]), (7, 1, 128, 16, [(200, 60), (330, 60)] * 5),
    (13, 1, 64, 32, [(600, 200), (100, 150)]), (6, 2, 256, 16, [(260, 40)] * 18), (64, 4, 64, 16, [(500, 5)] * 14)])
def test_parts_of_many_rows(M, heads, kv, D, page, seqs):
    """Rows enough that a wave joins the parts of several heads, numbers of
    heads that are not a multiple of those."""
    say(f"attention of many rows heads={heads} kv={kv} D={D} seqs={seqs[:2]}")
    b = Batch(M, seqs, heads, kv, D, page, pad=1, seed=heads)
    assert b.T * heads >= 4096
    b.call()
    b.check("out")


@pytest.mark.parametrize("heads,kv,D,n", [
    (8, 8, 128, 1), (12, 4, 64, 1), (4, 4, 256, 1), (16, 4, 128, 7), (16, 4, 64, 7), (16, 4, 256, 7), (14, 2, 128, 9),
    (14, 2, 64, 9), (14, 2, 256, 9), (14, 2, 128, 12), (14, 2, 256, 12)])
def test_long_runs_of_a_shared_prefix(M, heads, kv, D, n):
    """Sequences whose tables name the same pages up to their drafted tokens,
    and so many of them that a workgroup goes through long runs of positions,
    over the ends of sequences and over a page that is none.  Every eleventh
    sequence is compared."""
    import torch
    say(f"attention behind a shared prefix heads={heads} kv={kv} D={D} n={n}")
    rng = np.random.default_rng(D + n)
    page, B, L = 32, 64, 8032
    own = 1 if n <= page else 2
    held = L // page
    cache = A.Cache(held + B * own, kv, page, D, seed=n)
    draw = lambda m: rng.standard_normal((m, kv, D)).astype(np.float32).astype(np.float64)
    prefix = []
    for which in "kv":
        codes, scales = _encode(draw(L))
        cache.put(which, np.arange(L), codes, scales)
        prefix.append(R.mx8_values(codes, scales))
    table = np.concatenate([np.broadcast_to(np.arange(held), (B, held)),
                            held + np.arange(B * own).reshape(B, own)], 1).astype(np.int32)
    drafted = {"k": {}, "v": {}}
    for b in range(B):
        for which in "kv":
            codes, scales = _encode(draw(n))
            pos = np.arange(L, L + n)
            cache.put(which, table[b, pos // page].astype(np.int64) * page + pos % page, codes, scales)
            drafted[which][b] = R.mx8_values(codes, scales)
    lost = {11: held - 2, 33: 150, 55: 0}           # a page of these sequences is none
    for b, at in lost.items():
        table[b, at] = held + B * own + at
    mask = _tree(rng, n, 1, empty=0.0)
    q = R.tensor(rng.standard_normal((B * n, heads, D)), "bf16")
    out = torch.full_like(q, 9)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    ws = torch.randint(0, 256, (M.moe_tree_attention_workspace(B * n, B, heads, kv, D),), dtype=torch.uint8,
                       device="cuda")
    scale = 1.0 / np.sqrt(D)
    M.moe_tree_attention(q, *cache.tensors, i32(table), i32([L] * B), i32(np.arange(B + 1) * n), out, scale,
                         mask=torch.from_numpy(np.tile(mask, (B, 1)).view(np.int64)).cuda(), workspace=ws)
    torch.cuda.synchronize()
    got, qv = R.values(out), R.values(q)
    for b in range(0, B, 11):
        k, v = (np.concatenate([p, drafted[w][b]]) for p, w in zip(prefix, "kv"))
        gone = np.arange(lost[b] * page, lost[b] * page + page) if b in lost else []
        for i in (0, n - 1):
            at = np.setdiff1d(A.seen(L, n, mask[i], i), gone)
            for h in range(heads):
                g = h // (heads // kv)
                o, err, _ = A.attend(qv[b * n + i, h], k[at, g], v[at, g], scale)
                R.assert_between(got[b * n + i, h], R.bf16_rne(o - err), R.bf16_rne(o + err), f"sequence {b}, {i}")


@pytest.mark.parametrize("count", [63, 64, 65, 129])
@pytest.mark.parametrize("heads,kv,D", [(7, 1, 128), (4, 2, 256)])
def test_numbers_of_sequences(M, count, heads, kv, D):
    """As many sequences as a wave's lanes, fewer and more, the first and the
    last of them without tokens."""
    say(f"attention of {count} sequences D={D}")
    rng = np.random.default_rng(count)
    seqs = [(int(rng.integers(0, 150)), int(rng.integers(0, 3)) * int(0 < i < count - 1)) for i in range(count)]
    b = Batch(M, seqs, heads, kv, D, 16, tree=count % 2 == 0, pad=2, lead=1, seed=count)
    b.call()
    b.check("out")


def test_binding_refuses(M):
    import torch
    b = Batch(M, [(20, 4), (30, 3)], 4, 2, 64, 16, tree=True)
    kw = dict(mask=b.mask_t, workspace=b.ws)
    good = [b.qt, *b.cache.tensors, b.table_t, b.ctx_t, b.off_t, b.out, b.scale]
    for at, bad in ((0, b.qt.float()), (0, b.qt[:, :3]), (0, b.qt.cpu()), (0, b.qt[..., :32]), (5, b.table_t.long()),
                    (5, b.table_t[0]), (5, b.table_t.t()), (6, b.ctx_t[:1]), (7, b.off_t[:2]), (8, b.out.float()),
                    (8, b.out[:-1]), (9, 0.0), (9, float("nan"))):
        args = list(good)
        args[at] = bad
        with pytest.raises((ValueError, M.MoeError)):
            M.moe_tree_attention(*args, **kw)
    for bad in (dict(kw, mask=b.mask_t[:-1]), dict(kw, mask=b.mask_t.int()), dict(kw, workspace=None),
                dict(kw, workspace=b.ws[:-16]), dict(kw, workspace=b.ws.float()), dict(kw, mask=b.mask_t[:, :0])):
        with pytest.raises((ValueError, M.MoeError)):
            M.moe_tree_attention(*good, **bad)
    assert (b.out == 9).all()
    assert M.moe_tree_attention(b.qt[:0], *b.cache.tensors, b.table_t, b.ctx_t, b.off_t, b.out[:0], 1.0) == M.MOE_OK


def test_empty_batch(M):
    """A call without tokens, or without sequences, is one that does nothing,
    with a mask and without."""
    import torch
    b = Batch(M, [(20, 4), (30, 3)], 4, 2, 64, 16, tree=True)
    for mask in (b.mask_t, None):
        kw = dict(mask=None if mask is None else mask[:0], workspace=b.ws)
        none = torch.zeros_like(b.off_t)
        assert M.moe_tree_attention(b.qt[:0], *b.cache.tensors, b.table_t, b.ctx_t, none, b.out[:0], 1.0, **kw) == M.MOE_OK
        assert M.moe_tree_attention(b.qt, *b.cache.tensors, b.table_t[:0], b.ctx_t[:0], none[:1], b.out, 1.0, mask=mask,
                                    workspace=b.ws[:0]) == M.MOE_OK
    torch.cuda.synchronize()
    assert (b.out == 9).all()


def test_rows_beyond_one_grid(M):
    """2^28 rows of queries (more threads than a grid's dimension holds, and far
    past 32 bits of elements), nearly all of no sequence."""
    import torch
    say("attention of 2^28 rows of queries")
    heads, D, T = 1024, 64, 1 << 18
    b = Batch(M, [(300, 5)], heads, 1, D, 16, tree=True, seed=12)
    b.call()
    b.check("small")
    q = torch.empty(T, heads, D, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 9)
    q[T - 7:T - 2] = b.qt
    mask = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    mask[T - 7:T - 2] = b.mask_t
    ws = torch.empty(M.moe_tree_attention_workspace(T, 1, heads, 1, D), dtype=torch.uint8, device="cuda")
    assert M.moe_tree_attention(q, *b.cache.tensors, b.table_t, b.ctx_t, b.off_t + (T - 7), out, b.scale, mask=mask,
                                workspace=ws) == M.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(out[T - 7:T - 2], b.out)
    for rest in (out[:100], out[T // 2:T // 2 + 100], out[T - 100:T - 7], out[T - 2:]):
        assert (rest == 9).all()
    del q, out, rest
    torch.cuda.empty_cache()
