"""The attention of a verify step over an 8-bit cache, as it is measured.

Three operators stand next to the expert layer's other neighbours.  The cache
holds keys and values in MXFP8 (E4M3 elements, one E8M0 scale per 32 along the
head), in pages of ``page`` positions: codes [pages, kv_heads, page, head_dim]
and scales [pages, kv_heads, page, head_dim / 32].  A slot is page * page_size
+ position in the page.

  write   the keys and values of new tokens, encoded into their slots
  read    keys and values of given slots, decoded
  attend  attention of drafted tokens over the cache: a sequence's committed
          positions are seen by each of its drafted tokens, and of the drafted
          ones (which lie in the cache behind them) those that a token's mask
          names: its ancestors in the tree and itself; without a mask a chain

``listed`` and ``draw`` give cases, ``prepare`` the inputs of one, ``run`` one
pass (plain torch operations, or with ``own`` the library's entry points),
``exact`` the same outputs in 64 bits, ``work`` what a pass cannot do without.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
F8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # the 9 tokens of one verify step into the cache: latency alone
        dict(name="write_t9_kv8_d128", op="write", tokens=9, kv_heads=8, head_dim=128, page=64, slots=8192, rows="bf16",
             pad=0),
        # 32 sequences' verify steps, in a batch padded to a captured graph's size
        dict(name="write_t288_kv8_d128", op="write", tokens=288, kv_heads=8, head_dim=128, page=16, slots=16384,
             rows="bf16", pad=31),
        # a prefill chunk
        dict(name="write_t4096_kv8_d128", op="write", tokens=4096, kv_heads=8, head_dim=128, page=64, slots=16384,
             rows="bf16", pad=0),
        # an accepted path of drafted tokens taken out of the cache: latency alone
        dict(name="read_n7_kv8_d128", op="read", tokens=7, kv_heads=8, head_dim=128, page=64, slots=8192, rows="bf16",
             pad=0),
        # a prompt's keys and values for a consumer that reads them in bf16
        dict(name="read_n16001_kv8_d128", op="read", tokens=16001, kv_heads=8, head_dim=128, page=64, slots=32768,
             rows="bf16", pad=0),
        # one new token of a short sequence: latency alone
        dict(name="attend_b1_n1_c1000", op="attend", batch=1, nodes=1, tree=False, ragged=False, context=1000, heads=48,
             kv_heads=8, head_dim=128, page=64, pad=0, layout=1),
        # 8 drafts + 1 as a chain, one sequence
        dict(name="attend_b1_n9_c8192", op="attend", batch=1, nodes=9, tree=False, ragged=False, context=8192, heads=48,
             kv_heads=8, head_dim=128, page=64, pad=0, layout=2),
        # a tree of drafts over a long sequence
        dict(name="attend_b1_n61_c30001_tree", op="attend", batch=1, nodes=61, tree=True, ragged=False, context=30001,
             heads=56, kv_heads=8, head_dim=128, page=64, pad=0, layout=3),
        # new tokens of many sequences, small heads, small pages
        dict(name="attend_b64_n1_c8000_d64", op="attend", batch=64, nodes=1, tree=False, ragged=False, context=8000,
             heads=64, kv_heads=8, head_dim=64, page=16, pad=0, layout=4),
        # a batch of verify steps, 8 sequences x 9 tokens, each a tree
        dict(name="attend_b8_n9_c4096_tree", op="attend", batch=8, nodes=9, tree=True, ragged=False, context=4096,
             heads=56, kv_heads=8, head_dim=128, page=64, pad=0, layout=5),
        # 32 sequences x 9 tokens, the largest batch of verify steps, over long sequences
        dict(name="attend_b32_n9_c16384", op="attend", batch=32, nodes=9, tree=False, ragged=False, context=16384,
             heads=56, kv_heads=8, head_dim=128, page=64, pad=0, layout=6),
        # wide trees of several sequences, not all of one size: the products bound it
        dict(name="attend_b8_n64_c16001_tree", op="attend", batch=8, nodes=64, tree=True, ragged=True, context=16001,
             heads=56, kv_heads=8, head_dim=128, page=64, pad=5, layout=7),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number from lo to hi, spread over its logarithm, on multiples of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, round(v / step) * step))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "attend"))
    D, kv, page = rng.choice((64, 128, 128, 256)), rng.choice((1, 2, 3, 4, 8, 8, 16)), rng.choice((16, 32, 64, 128))
    if op != "attend":
        tokens = _spread(rng, 1, min(4096 if op == "write" else 16000, 4096 * 1024 // (kv * D)))
        slots = -(-2 * tokens // page) * page + page * rng.randrange(1, 9)
        return dict(op=op, tokens=tokens, kv_heads=kv, head_dim=D, page=page, slots=slots,
                    rows=rng.choice(("bf16", "bf16", "f32")) if tokens <= 2048 else "bf16",
                    pad=rng.choice((0, 0, rng.randrange(8))))
    group = rng.choice((1, 2, 3, 4, 6, 7, 8, 12, 16))
    nodes, batch = rng.choice((1, 9, _spread(rng, 1, 64), _spread(rng, 2, 100))), _spread(rng, 1, 64)
    # no more rows, keys and products than the largest listed cases
    nodes = min(nodes, max(1, (1 << 24) // (batch * group * kv * D)))
    most = min(32 * 8192 * 1024 // (batch * kv * D), 8 * 40 * 10000 * 56 * 128 // (batch * nodes * group * kv * D))
    return dict(op=op, batch=batch, nodes=nodes, tree=nodes > 1 and rng.random() < 0.6, ragged=rng.random() < 0.4,
                context=_spread(rng, 1, max(1, min(32768, most))) - 1, heads=group * kv, kv_heads=kv, head_dim=D,
                page=page, pad=rng.choice((0, 0, rng.randrange(8))), layout=rng.randrange(1 << 30))


def _layout(c):
    """What the host knows of an attend case: committed positions and drafted
    tokens of each sequence, and each token's mask as a number (bit j: it sees
    the sequence's drafted token j).  A tree's token hangs on the committed
    positions or on an earlier token; a few are padding that no mask names and
    whose own is empty."""
    rng = random.Random(c["layout"])
    ctx = [c["context"]] + [int(c["context"] * rng.uniform(0.25, 1)) for _ in range(c["batch"] - 1)]
    n = [c["nodes"]] + [rng.randrange(c["nodes"] + 1) if c["ragged"] else c["nodes"] for _ in range(c["batch"] - 1)]
    masks = []
    for k in n:
        own_masks = []
        for i in range(k):
            if not c["tree"]:
                own_masks.append((2 << i) - 1)
            elif i and rng.random() < 1 / 16:
                own_masks.append(0)
            else:
                up = own_masks[rng.randrange(max(0, i - 6), i)] if i and rng.random() < 0.9 else 0
                own_masks.append(up | 1 << i)
        masks.append(own_masks)
    return ctx, n, masks


def work(case):
    c = case
    D, kv = c["head_dim"], c["kv_heads"]
    if c["op"] != "attend":
        held = c["tokens"] - c["pad"] if c["tokens"] > c["pad"] else c["tokens"]
        rows = 2 * held * kv * D * SIZE[c["rows"]]
        return {"bytes": rows + 2 * held * kv * D * 33 // 32 + 8 * c["tokens"], "flops": 0}
    ctx, n, masks = _layout(c)
    keys = sum(L + k for L, k in zip(ctx, n) if k)
    seen = sum(L * k + sum(m.bit_count() if hasattr(m, "bit_count") else bin(m).count("1") for m in ms)
               for L, k, ms in zip(ctx, n, masks))
    T = sum(n)
    words = -(-c["nodes"] // 64) if c["tree"] else 0
    return {"bytes": 2 * keys * kv * D * 33 // 32 + 4 * T * c["heads"] * D + 4 * (keys // c["page"]) + 8 * T * words,
            "flops": 4 * c["heads"] * D * seen}


# --------------------------------------------------------------- the inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV)


def _encode(v):
    """The MXFP8 encoding of float32 v along its last axis: codes (E4M3) and
    scales (E8M0), the scale 2^(floor(log2 amax) - 8), elements rounded to the
    nearest (ties to even, saturating), a block with a non-finite element NaN.
    Every step is exact in float32 but the rounding (a power of two is applied
    in two halves, so that neither is out of range)."""
    b = v.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    se = (torch.frexp(amax).exponent - 9).clamp(-127, 127)
    se = torch.where(amax == 0, -127, se)
    bad = ~torch.isfinite(amax)
    half = torch.div(-se, 2, rounding_mode="floor")
    q = torch.ldexp(torch.ldexp(b, half.unsqueeze(-1)), (-se - half).unsqueeze(-1))
    step = torch.ldexp(torch.ones_like(q), (torch.frexp(q).exponent - 1).clamp(min=-6) - 3)
    q = (torch.round(q / step) * step).clamp(-448, 448)
    q = torch.where(bad.unsqueeze(-1), 0.0, q)
    return q.flatten(-2).to(F8), torch.where(bad, 255, se + 127).to(torch.uint8).view(E8M0)


def _pages(gen, pages, c):
    """Codes and scales of a cache whose every slot was written: keys or
    values of uneven columns, as a trained model's are."""
    D = c["head_dim"]
    col = torch.exp(0.5 * _normal(gen, c["kv_heads"], 1, D))
    # random values in float32 one part of the pages after the other: a large cache need not be held twice
    codes = torch.empty(pages, c["kv_heads"], c["page"], D, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, c["kv_heads"], c["page"], D // 32, dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 26) // (c["kv_heads"] * c["page"] * D))
    for at in range(0, pages, part):
        end = min(pages, at + part)
        x, s = _encode(_normal(gen, end - at, c["kv_heads"], c["page"], D) * col)
        codes[at:end], scales[at:end] = x.view(torch.uint8), s.view(torch.uint8)
    return codes, scales


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed)
    st = {"case": c}
    D, kv, page = c["head_dim"], c["kv_heads"], c["page"]
    if c["op"] != "attend":
        T, pages = c["tokens"], c["slots"] // page
        st["kc"], st["ks"] = _pages(gen, pages, c)
        st["vc"], st["vs"] = _pages(gen, pages, c)
        # consecutive positions of a sequence whose pages lie anywhere; the last tokens are the batch's padding
        order = rng.sample(range(pages), pages)
        at = rng.randrange(c["slots"] - T + 1)
        slots = [order[(at + t) // page] * page + (at + t) % page for t in range(T)]
        if c["pad"] < T:
            slots[T - c["pad"]:] = [-1] * c["pad"]
        st["slots"] = torch.tensor(slots, dtype=torch.int64, device=DEV)
        if c["op"] == "write":
            col = torch.exp(0.5 * _normal(gen, kv, D))
            st["k"] = (_normal(gen, T, kv, D) * col).to(DT[c["rows"]])
            st["v"] = _normal(gen, T, kv, D).to(DT[c["rows"]])
        else:
            st["k"] = torch.zeros(T, kv, D, dtype=DT[c["rows"]], device=DEV)
            st["v"] = torch.zeros(T, kv, D, dtype=DT[c["rows"]], device=DEV)
        return st
    ctx, n, masks = _layout(c)
    B, T = c["batch"], sum(n) + c["pad"]
    # each sequence's table names the pages it has; entries behind them are as an allocator leaves them
    held = [-(-(L + k) // page) for L, k in zip(ctx, n)]
    pages = sum(held) + 1
    order = rng.sample(range(pages), pages)
    table, at = [], 0
    for h in held:
        table.append(order[at:at + h] + [-1] * (max(held) + 1 - h))
        at += h
    st["kc"], st["ks"] = _pages(gen, pages, c)
    st["vc"], st["vs"] = _pages(gen, pages, c)
    st["q"] = _normal(gen, T, c["heads"], D).to(torch.bfloat16)
    st["out"] = torch.zeros(T, c["heads"], D, dtype=torch.bfloat16, device=DEV)
    st["table"] = torch.tensor(table, dtype=torch.int32, device=DEV)
    st["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=DEV)
    offsets = [0]
    for k in n:
        offsets.append(offsets[-1] + k)
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    st["mask"] = None
    if c["tree"]:
        words = -(-c["nodes"] // 64)
        flat = [m for ms in masks for m in ms] + [0] * c["pad"]
        signed = [[w - (1 << 64) if w >> 63 else w for w in ((m >> (64 * i)) & (1 << 64) - 1 for i in range(words))]
                  for m in flat]
        st["mask"] = torch.tensor(signed, dtype=torch.int64, device=DEV)
    st["scale"] = 1 / math.sqrt(D)
    st["scratch"] = _scratch(c, T)
    return st


def _scratch(c, T):
    """Scratch memory that a program keeps for its calls of these sizes: the
    partial results of a long axis split over 1024 workgroups, 80 rows each in
    float32 with their statistics."""
    return torch.zeros(1024 * 80 * 4 * (c["head_dim"] + 4) + (1 << 16), dtype=torch.uint8, device=DEV)


# ----------------------------------------------------------- the plain form

def _values(codes, scales):
    """MXFP8 codes and scales as float32."""
    v = codes.view(F8).float().unflatten(-1, (-1, 32)) * scales.view(E8M0).float().unsqueeze(-1)
    return v.flatten(-2)


def _places(s):
    """The tokens whose slot is in the cache, and that slot's page and place."""
    page = s["case"]["page"]
    slots, held = s["slots"], (s["slots"] >= 0) & (s["slots"] < s["kc"].shape[0] * page)
    at = held.nonzero().squeeze(1)
    slot = slots[at]
    return at, slot // page, slot % page


def _plain_write(s):
    at, page, place = _places(s)
    for x, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        c, e = _encode(s[x][at].float())
        s[codes][page, :, place] = c.view(torch.uint8)
        s[scales][page, :, place] = e.view(torch.uint8)
    return _cache(s)


def _cache(s):
    return {"k": s["kc"].view(F8), "k_scales": s["ks"].view(E8M0), "v": s["vc"].view(F8),
            "v_scales": s["vs"].view(E8M0)}


def _plain_read(s):
    at, page, place = _places(s)
    out = {}
    for x, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
        out[x] = torch.zeros_like(s[x])
        out[x][at] = _values(s[codes][page, :, place], s[scales][page, :, place]).to(s[x].dtype)
    return out


def _plain_attend(s):
    c, table = s["case"], s["table"]
    B, P = table.shape
    kv, D, G, N = c["kv_heads"], c["head_dim"], c["heads"] // c["kv_heads"], c["nodes"]
    keys = P * c["page"]
    pages = table.clamp(min=0).long()

    def gathered(codes, scales):   # [B, kv, keys, D]
        return _values(codes[pages], scales[pages]).transpose(1, 2).reshape(B, kv, keys, D)

    start, end, ctx = s["offsets"][:-1].long(), s["offsets"][1:].long(), s["ctx"].long()
    node = torch.arange(N, device=table.device)
    tokens = start.unsqueeze(1) + node                                   # [B, N]
    real = tokens < end.unsqueeze(1)
    row = tokens.clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(B, N, kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, kv, N * G, D)
    # position p is seen if it is committed, or a drafted token that the mask names
    p = torch.arange(keys, device=table.device)
    j = p - ctx.unsqueeze(1)                                             # [B, keys]: the drafted token there
    if s["mask"] is None:
        named = j.unsqueeze(1) <= node.unsqueeze(1)
    else:
        word = (j.clamp(0, 64 * s["mask"].shape[1] - 1) // 64).unsqueeze(1).expand(B, N, keys)
        named = (s["mask"][row].gather(2, word) >> (j.clamp(min=0) % 64).unsqueeze(1)) & 1 == 1
    seen = ((j < 0).unsqueeze(1) | named) & (j < (end - start).unsqueeze(1)).unsqueeze(1)  # [B, N, keys]
    seen = seen.view(B, 1, N, 1, keys).expand(B, 1, N, G, keys).reshape(B, 1, N * G, keys)
    scores = q @ gathered(s["kc"], s["ks"]).transpose(2, 3).contiguous() * s["scale"]
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    o = e @ gathered(s["vc"], s["vs"]) / torch.where(total == 0, 1.0, total)
    o = o.view(B, kv, N, G, D).permute(0, 2, 1, 3, 4).reshape(B, N, c["heads"], D).to(torch.bfloat16)
    out = s["out"].clone()
    out[tokens[real]] = o[real]
    return {"out": out}


# ------------------------------------------------------- the library's calls

def _own(s):
    import mxfp4_moe_expert_02_amd as M
    op = s["case"]["op"]
    cache = (s["kc"], s["ks"], s["vc"], s["vs"])
    if op == "write":
        M.moe_kv_write(s["k"], s["v"], s["slots"], *cache)
        return _cache(s)
    if op == "read":
        M.moe_kv_read(*cache, s["slots"], s["k"], s["v"])
        return {"k": s["k"], "v": s["v"]}
    M.moe_tree_attention(s["q"], *cache, s["table"], s["ctx"], s["offsets"], s["out"], s["scale"], mask=s["mask"],
                         workspace=s["scratch"])
    return {"out": s["out"]}


PLAIN = {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------- the definition

def _exact_mx8(v):
    """MXFP8 of v in 64 bits by the format's own table: the scale from the
    exponent bits of the block's largest magnitude, each element the nearest
    of the 127 finite magnitudes, a tie to the even one."""
    b = v.reshape(-1, 32)
    top = b.abs().max(1).values
    se = ((top.view(torch.int64) >> 52) - 1023 - 8).clamp(-127, 127)
    table = torch.arange(127, dtype=torch.uint8, device=v.device).view(F8).double()
    mid = (table[1:] + table[:-1]) / 2                       # between code i and i + 1
    q = b * torch.exp2(-se.double()).unsqueeze(1)
    low = torch.bucketize(q.abs(), mid)                      # midpoints below |q|: its code, a tie downward
    tie = (low < 126) & (q.abs() == mid[low.clamp(max=125)])
    low = torch.where(tie & (low % 2 == 1), low + 1, low)
    val = table[low] * torch.where(torch.signbit(q), -1.0, 1.0)
    return val.reshape(v.shape), torch.exp2(se.double()).view(*v.shape[:-1], -1)


def _exact_values(codes, scales):
    return codes.view(F8).double() * scales.view(E8M0).double().repeat_interleave(32, dim=-1)


def exact(case, seed):
    s = prepare(case, seed)
    c, page = s["case"], case["page"]
    if c["op"] != "attend":
        slots = s["slots"].tolist()
        held = [t for t, slot in enumerate(slots) if slot >= 0]
        where = torch.tensor([slots[t] for t in held], dtype=torch.long, device=DEV)
        out = {}
        for x, codes, scales in (("k", "kc", "ks"), ("v", "vc", "vs")):
            if c["op"] == "write":
                # slots first, heads second, as the rows lie
                flat = s[codes].view(F8).double().transpose(1, 2).flatten(0, 1)
                flat_s = s[scales].view(E8M0).double().transpose(1, 2).flatten(0, 1)
                flat[where], flat_s[where] = _exact_mx8(s[x][held].double())
                out[x] = flat.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
                out[x + "_scales"] = flat_s.unflatten(0, (-1, page)).transpose(1, 2).contiguous()
            else:
                out[x] = torch.zeros(s[x].shape, dtype=torch.float64, device=DEV)
                rows = [s[t].transpose(1, 2).flatten(0, 1)[where] for t in (codes, scales)]
                out[x][held] = _exact_values(*rows)
        return out
    ctx, n, masks = _layout(c)
    kv, G, D = c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (L, k, ms) in enumerate(zip(ctx, n, masks)):
        if not k:
            continue
        pos = torch.arange(L + k, device=DEV)
        pages, place = s["table"][b].long()[pos // page], pos % page
        key = _exact_values(s["kc"][pages, :, place], s["ks"][pages, :, place])            # [L + k, kv, D]
        val = _exact_values(s["vc"][pages, :, place], s["vs"][pages, :, place])
        hidden = torch.tensor([[not m >> j & 1 for j in range(k)] for m in ms], device=DEV)
        empty = torch.tensor([L == 0 and m == 0 for m in ms], device=DEV)
        for h in range(kv):
            q = s["q"][at:at + k, h * G:(h + 1) * G].double().reshape(k * G, D)
            t = (torch.mm(q, key[:, h].t().contiguous()) * s["scale"]).view(k, G, L + k)
            t[:, :, L:].masked_fill_(hidden.unsqueeze(1), -math.inf)
            t[empty] = 0.0
            o = torch.mm(torch.softmax(t, -1).view(k * G, L + k), val[:, h].contiguous()).view(k, G, D)
            o[empty] = 0.0
            out[at:at + k, h * G:(h + 1) * G] = o
        at += k
    return {"out": out}
