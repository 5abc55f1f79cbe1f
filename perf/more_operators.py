"""Workloads of the operators around the paged 8-bit cache that come before and beside its attention: the rotation
of queries and keys by their positions (with a norm of every head), attention of a batch whose sequences share a long
prefix, and attention over blocks that a cheap score selects (the blocks' bounds, the selection, the attention).

listed() and draw() give cases, prepare() the inputs a program holds before the call, run() one pass, exact() the same
results in 64 bits. With `own` false, run() computes the operators from elementary torch operations; with it true,
run() calls the package.

The cache: pages of 64 tokens. Per page and head, K and V are int8 codes with one fp32 scale s each; a code c stands
for c * (s / 127). Codes are stored as 256-byte tiles of 16 rows x 16 bytes:
  K of a page and head: [token % 4][dim / 16][token / 4][dim % 16]
  V of a page and head: [dim / 16][token / 16][dim % 16][token % 16]
Bounds: per page and head the largest and the smallest K code of every dim, int8 [pages][heads][2][d].
"""
import math

import torch

own = False

BLOCK = 64
SMALLEST = 1e-30  # the smallest of what a row of queries is quantized by
EPS = 1e-5

# The largest of what draw() makes: rotated elements; cached tokens x kv heads x head width of a shared prefix's rows
# and logits; scored block bounds; selected tokens x kv heads x head width.
MOST_ROTATED = 8192 * 40 * 128
MOST_LOGITS = 64 * 32 * 17000
MOST_BOUNDS = 64 * 512 * 8 * 128
MOST_SELECTED = 40 * 32 * 64 * 8 * 128
MOST_HELD = 40 * 15000 * 8 * 128


def listed():
    """Twelve cases: head layouts of the 2B-class layer (20 query and 5 kv heads of 128) and of the 8B-class one (32
    and 8)."""
    return [
        # one user's next token, queries and keys normed
        {"name": "rotate_one", "kind": "rotate", "lens": "1", "begin": "1023", "hq": 20, "hkv": 5, "d": 128, "dtype": "bf16", "rot": 128,
         "interleaved": False, "norm": True, "factor": 1.0},
        # four tokens checked at once for each of a batch, far positions scaled, half of the head rotated, fp32 as the projection leaves it
        {"name": "rotate_verify_fp32", "kind": "rotate", "lens": ",".join(["4"] * 48), "begin": ",".join(str(997 * i * i % 900000) for i in range(48)),
         "hq": 20, "hkv": 5, "d": 128, "dtype": "f32", "rot": 64, "interleaved": True, "norm": False, "factor": 8.0},
        # packed prompts
        {"name": "rotate_prompts", "kind": "rotate", "lens": "4096,33,1500,700,1,911,64,887", "begin": "0,0,5000,0,77,0,131,0", "hq": 32, "hkv": 8,
         "d": 128, "dtype": "bf16", "rot": 128, "interleaved": False, "norm": True, "factor": 4.0},
        # a few users behind one instruction text, their next tokens
        {"name": "shared_2b_few", "kind": "shared", "prefix": 2000, "lens": "17,96,1,64,130,45,0,77", "new": 1, "hq": 20, "hkv": 5, "d": 128,
         "dtype": "bf16"},
        # a full batch behind a long document
        {"name": "shared_8b_batch", "kind": "shared", "prefix": 16384, "lens": ",".join(str(700 - 7 * i * i % 650) for i in range(64)), "new": 1,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
        # several continuations of one text, four tokens of each checked at once, fp32
        {"name": "shared_2b_verify", "kind": "shared", "prefix": 6001, "lens": "130,399,62,207,640,250,1,333,447,808,95,160", "new": 4, "hq": 20,
         "hkv": 5, "d": 128, "dtype": "f32"},
        # the blocks that a batch's next tokens went to
        {"name": "bounds_decode", "kind": "bounds", "lens": ",".join(str(97 * i % 2000) for i in range(32)), "new": "1", "hkv": 5, "d": 128},
        # all blocks of prompts just appended, one of them going on inside a block
        {"name": "bounds_prompt", "kind": "bounds", "lens": "0,1000,0", "new": "40960,2000,12099", "hkv": 8, "d": 128},
        # blocks for one user's next token after a very long context
        {"name": "select_8b_long", "kind": "select", "lens": "131070", "new": 1, "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "keep": 64,
         "first": 1, "recent": 2},
        # and for a batch, two tokens each, fp32
        {"name": "select_2b_batch", "kind": "select", "lens": ",".join(str(32000 - 61 * i * i % 24000) for i in range(64)), "new": 2, "hq": 20,
         "hkv": 5, "d": 128, "dtype": "f32", "keep": 32, "first": 1, "recent": 2},
        # one user's next token over 64 of the long context's 2048 blocks
        {"name": "selected_8b_long", "kind": "selected", "lens": "131070", "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16", "keep": 64},
        # a batch's next tokens over 32 blocks of each one's context, fp32
        {"name": "selected_8b_batch", "kind": "selected", "lens": ",".join(str(15000 - 29 * i * i % 13000) for i in range(40)), "hq": 32, "hkv": 8,
         "d": 128, "dtype": "f32", "keep": 32},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def _lens(rng, seqs, longest):
    lens = [longest] + [_log_int(rng, 1, longest) for _ in range(seqs - 1)]
    rng.shuffle(lens)
    return ",".join(map(str, lens))


def draw(rng):
    kind = rng.choice(["rotate", "rotate", "shared", "shared", "bounds", "select", "selected", "selected"])
    hq, hkv = rng.choice([(20, 5), (32, 8), (8, 8), (16, 2), (12, 4), (7, 1), (6, 2)])
    d, dtype = rng.choice([128, 128, 64]), rng.choice(["bf16", "f32"])
    heads = {"hq": hq, "hkv": hkv, "d": d, "dtype": dtype}
    if kind == "rotate":
        seqs = _log_int(rng, 1, 64)
        longest = _log_int(rng, 1, max(1, min(8192, MOST_ROTATED // (2 * seqs * (hq + hkv) * d))))
        lens = _lens(rng, seqs, longest) if rng.random() < 0.7 else ",".join(["1"] * seqs)
        return {"kind": kind, "lens": lens, "begin": ",".join(str(_log_int(rng, 1, 1 << 20) - 1) for _ in range(seqs)), **heads,
                "rot": rng.choice([d, d, d // 2, d // 4]), "interleaved": rng.random() < 0.5, "norm": rng.random() < 0.5,
                "factor": rng.choice([1.0, 4.0, 8.0, 32.0])}
    if kind == "shared":
        seqs, new = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        prefix = _log_int(rng, 60, min(32768, MOST_LOGITS // (seqs * new * hq)))
        own_lens = _lens(rng, seqs, _log_int(rng, 1, max(2, min(1500, MOST_LOGITS // (seqs * new * hq) - prefix))))
        return {"kind": kind, "prefix": prefix, "lens": own_lens, "new": new, **heads}
    if kind == "bounds":
        seqs = _log_int(rng, 1, 48)
        new = [_log_int(rng, 1, max(2, 32768 // seqs)) for _ in range(seqs)] if rng.random() < 0.6 else [1] * seqs
        return {"kind": kind, "lens": ",".join(str(rng.randrange(0, 1500)) for _ in new), "new": ",".join(map(str, new)), "hkv": hkv, "d": d}
    if kind == "select":
        seqs = _log_int(rng, 1, 64)
        blocks = _log_int(rng, 40, min(2048, MOST_BOUNDS // (seqs * hkv * d)))
        first, recent = rng.randrange(0, 3), rng.randrange(1, 4)
        return {"kind": kind, "lens": _lens(rng, seqs, blocks * BLOCK - 9), "new": rng.choice([1, 1, 1, 2, 4]), **heads,
                "keep": first + recent + _log_int(rng, 8, min(blocks // 2, 256)), "first": first, "recent": recent}
    seqs = _log_int(rng, 1, 40)
    keep = _log_int(rng, 1, min(128, MOST_SELECTED // (seqs * BLOCK * hkv * d)))
    return {"kind": kind, "lens": _lens(rng, seqs, _log_int(rng, 40, min(131072, MOST_HELD // (seqs * hkv * d)) - 8)), **heads, "keep": keep}


# ---------------------------------------------------------------- inputs

def _ints(text):
    return [int(t) for t in str(text).split(",")]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(lens):
    return torch.tensor([0] + list(lens), device="cuda").cumsum(0).to(torch.int32)


def _projected(rows, heads, d, gen):
    """Rows as a projection leaves them: normal, with channels of their own size and 1 % of them large."""
    width = heads * d
    size = torch.exp(0.3 * torch.randn(width, generator=gen, device="cuda"))
    size[torch.randperm(width, generator=gen, device="cuda")[: max(1, width // 100)]] *= 4.0
    return torch.randn(rows, width, generator=gen, device="cuda") * size


def _tables(nblocks, gen, more=0):
    """A block table of pages in no order, as a server's free list deals them, `more` pages besides, and the number
    of pages."""
    wide, pages = max(nblocks), sum(nblocks) + more + 3
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    count = torch.tensor(nblocks, device="cuda")
    at = torch.arange(wide, device="cuda")[None, :]
    flat = (count.cumsum(0) - count)[:, None] + at
    table = torch.where(at < count[:, None], order[flat.clamp(max=pages - 1)], torch.zeros((), dtype=torch.int32, device="cuda"))
    return table, order[sum(nblocks):sum(nblocks) + more].contiguous(), pages


def _codes(pages, hkv, d, gen):
    c = torch.empty((pages, hkv, BLOCK * d), dtype=torch.int8, device="cuda")
    step = max(1, (1 << 27) // (hkv * BLOCK * d))
    for i in range(0, pages, step):
        c[i:i + step] = (torch.randn(c[i:i + step].shape, generator=gen, device="cuda") * 34).round_().clamp_(-127, 127).to(torch.int8)
    return c


def _scales(pages, hkv, gen):
    return 2.5 + 2.5 * torch.rand((pages, hkv), generator=gen, device="cuda")


def _cache(pages, hkv, d, gen):
    """A cache in use: codes of normal values whose largest takes the whole range."""
    return {"k": _codes(pages, hkv, d, gen), "v": _codes(pages, hkv, d, gen), "ks": _scales(pages, hkv, gen), "vs": _scales(pages, hkv, gen)}


def _queries(rows, case, gen):
    return _projected(rows, case["hq"], case["d"], gen).to(_dtype(case)).unflatten(1, (case["hq"], case["d"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, hkv, d, lens = case["kind"], case["hkv"], case["d"], _ints(case["lens"])
    s = {"kind": kind}
    if kind == "rotate":
        hq, rot = case["hq"], case["rot"]
        qkv = _projected(sum(lens), hq + 2 * hkv, d, gen).to(_dtype(case))  # the fused projection's output
        # the angle per position of every pair; a longer context squeezes the slow ones
        freq = 500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        turns = 8192 * freq / (2 * math.pi)
        part = ((turns - 1) / 31).clamp(0, 1)
        freq = freq * (part + (1 - part) / case["factor"])
        s |= {"q": qkv[:, : hq * d].unflatten(1, (hq, d)), "k": qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)), "freq": freq.float(),
              "begin": _i32(_ints(case["begin"])), "starts": None if max(lens) == min(lens) == 1 else _starts(lens),
              "interleaved": case["interleaved"], "magnitude": 0.1 * math.log(case["factor"]) + 1}
        gains = [1 + 0.3 * torch.randn(d, generator=gen, device="cuda") for _ in range(2)]
        s["gq"], s["gk"] = gains if case["norm"] else (None, None)
        return s
    if kind == "bounds":
        new = _ints(case["new"])
        new = new * len(lens) if len(new) == 1 else new
        s["table"], _, pages = _tables([-(-(a + b) // BLOCK) for a, b in zip(lens, new)], gen)
        s |= {"k": _codes(pages, hkv, d, gen), "ks": _scales(pages, hkv, gen), "lens": _i32(lens), "m": sum(new),
              "starts": None if max(new) == 1 else _starts(new), "spans": max(b // BLOCK + 2 for b in new)}
        s["v"], s["vs"] = s["k"], s["ks"]  # the cache's other half is not looked at
        s["bounds"] = torch.zeros((pages, hkv, 2, d), dtype=torch.int8, device="cuda")
        return s
    new = case.get("new", 1)
    held = [-(-(n + new) // BLOCK) for n in lens]
    s |= {"q": _queries(len(lens) * new, case, gen), "lens": _i32(lens), "starts": None if new == 1 else _starts([new] * len(lens))}
    if kind == "select":
        s["table"], _, pages = _tables(held, gen)
        wide = (torch.randn((pages, hkv, 2, d), generator=gen, device="cuda") * 18 + 80).round_().clamp_(1, 127)
        s |= {"bounds": (wide * torch.tensor([1.0, -1.0], device="cuda")[:, None]).to(torch.int8), "ks": _scales(pages, hkv, gen),
              "keep": case["keep"], "first": case["first"], "recent": case["recent"]}
        return s
    if kind == "shared":
        s["table"], s["prefix"], pages = _tables(held, gen, -(-case["prefix"] // BLOCK))
        s["prefix_len"] = _i32([case["prefix"]])
        return s | _cache(pages, hkv, d, gen)
    s["table"], _, pages = _tables(held, gen)
    s |= _cache(pages, hkv, d, gen)
    # every row and head its own blocks, the last one among them
    chance = torch.rand((len(lens), hkv, max(held)), generator=gen, device="cuda")
    used = torch.tensor(held, device="cuda")[:, None, None]
    at = torch.arange(max(held), device="cuda")
    chance = torch.where(at == used - 1, 2.0, chance).masked_fill(at >= used, -1.0)
    best = torch.nn.functional.pad(chance, (0, max(0, case["keep"] - max(held))), value=-1.0).topk(case["keep"], dim=2)
    far = 1 << 30
    order = torch.where(best.values >= 0, best.indices, far).sort(dim=2).values
    s["selected"] = torch.where(order == far, -1, order).to(torch.int32)
    return s


# ---------------------------------------------------------------- plain forms

def _natural_k(codes, d):
    """[..., 64 * d] stored K codes -> [..., 64, d]"""
    x = codes.unflatten(-1, (4, d // 16, 16, 16))  # token % 4, dim / 16, token / 4, dim % 16
    return x.movedim(-2, -4).flatten(-4, -3).flatten(-2, -1)


def _natural_v(codes, d):
    """[..., 64 * d] stored V codes -> [..., 64, d]"""
    x = codes.unflatten(-1, (d // 16, 4, 16, 16))  # dim / 16, token / 16, dim % 16, token % 16
    return x.movedim((-3, -1), (-4, -3)).flatten(-4, -3).flatten(-2, -1)


def _sequence_of(starts, count, device):
    """Sequence and place in it of every row of a packed batch (starts None: one row each)."""
    rows = torch.arange(count, device=device)
    if starts is None:
        return rows, torch.zeros_like(rows)
    seq = torch.searchsorted(starts[1:].long(), rows, right=True)
    return seq, rows - starts.long()[seq]


def _plain_rotate(s):
    seq, place = _sequence_of(s["starts"], s["q"].shape[0], s["q"].device)
    angle = (s["begin"].long()[seq] + place).double()[:, None] * s["freq"].double()
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    rot = 2 * s["freq"].shape[0]

    def turned(x, gain):
        y = x.float()
        if gain is not None:
            y = y * ((y * y).mean(-1, keepdim=True) + EPS).rsqrt() * gain
        a, b = (y[..., :rot:2], y[..., 1:rot:2]) if s["interleaved"] else (y[..., : rot // 2], y[..., rot // 2:rot])
        u, v = a * cos - b * sin, b * cos + a * sin
        return torch.cat((torch.stack((u, v), -1).flatten(-2) if s["interleaved"] else torch.cat((u, v), -1), y[..., rot:]), -1).to(x.dtype)
    return turned(s["q"], s["gq"]), turned(s["k"], s["gk"])


def _values(s, table, hkv, d):
    """K and V of a table's blocks, [..., blocks] -> [..., heads, blocks * 64, d]"""
    ks, vs = (s[n][table].div(127.0)[..., None, None] for n in ("ks", "vs"))
    k, v = _natural_k(s["k"][table], d) * ks, _natural_v(s["v"][table], d) * vs
    return k.movedim(-3, -4).flatten(-3, -2), v.movedim(-3, -4).flatten(-3, -2)


def _plain_shared(s):
    q, table = s["q"], s["table"].long()
    seqs, hkv, (m, hq, d) = table.shape[0], s["k"].shape[1], q.shape
    new, group = m // seqs, hq // hkv
    rows = q.view(seqs, new, hkv, group, d).permute(2, 0, 3, 1, 4).float().mul(1 / math.sqrt(d))  # [hkv][seqs][group][new][d]
    kp, vp = _values(s, s["prefix"].long(), hkv, d)  # once for all
    before = rows.reshape(hkv, -1, d) @ kp.transpose(1, 2).contiguous()
    before.masked_fill_(torch.arange(kp.shape[1], device=q.device) >= s["prefix_len"], -math.inf)
    k, v = _values(s, table, hkv, d)
    after = (rows.transpose(0, 1).reshape(seqs, hkv, group * new, d) @ k.transpose(2, 3).contiguous()).view(seqs, hkv, group, new, -1)
    last = s["lens"][:, None] + torch.arange(new, device=q.device)[None, :]
    seen = torch.arange(k.shape[2], device=q.device)[None, None, :] <= last[:, :, None]
    after.masked_fill_(~seen[:, None, None], -math.inf)
    top = torch.maximum(before.amax(-1).view(hkv, seqs, group, new), after.amax(-1).transpose(0, 1))
    before = before.view(hkv, seqs, group, new, -1).sub_(top[..., None]).exp_()
    after = after.sub_(top.transpose(0, 1)[..., None]).exp_()
    total = before.sum(-1) + after.sum(-1).transpose(0, 1)
    out = (before.view(hkv, -1, kp.shape[1]) @ vp).view(hkv, seqs, group, new, d)
    out = out + (after.view(seqs, hkv, group * new, -1) @ v).view(seqs, hkv, group, new, d).transpose(0, 1)
    return (out / total[..., None]).permute(1, 3, 0, 2, 4).reshape(m, hq * d).to(q.dtype)


def _plain_bounds(s):
    lens, table, d = s["lens"].long(), s["table"].long(), s["bounds"].shape[3]
    rows = torch.ones_like(lens) if s["starts"] is None else (s["starts"][1:] - s["starts"][:-1]).long()
    end = lens + rows
    block = (lens // BLOCK)[:, None] + torch.arange(s["spans"], device=lens.device)
    seq, nth = torch.nonzero((block * BLOCK < end[:, None]) & (rows > 0)[:, None], as_tuple=True)
    block = block[seq, nth]
    page = table[seq, block]
    codes = _natural_k(s["k"][page], d)
    there = (torch.arange(BLOCK, device=lens.device)[None, :] < (end[seq] - block * BLOCK)[:, None])[:, None, :, None]
    s["bounds"][page, :, 0] = codes.masked_fill(~there, -128).amax(2)
    s["bounds"][page, :, 1] = codes.masked_fill(~there, 127).amin(2)
    return s["bounds"]


def _plain_select(s):
    q, table, keep = s["q"].float(), s["table"].long(), s["keep"]
    seqs, wide, hkv, (m, hq, d) = *s["table"].shape, s["bounds"].shape[1], s["q"].shape
    x = q.view(m, hkv, hq // hkv, d)
    # every row's queries of a kv head as integers of one scale, and the sums of their positive and negative parts
    c = (x * torch.full((), 127.0, device=q.device).div(x.abs().amax((2, 3), keepdim=True).clamp(min=SMALLEST))).round()
    parts = torch.cat((c.clamp(min=0).sum(2), c.clamp(max=0).sum(2)), -1).double()  # [m][hkv][2 * d]
    seq, place = _sequence_of(s["starts"], m, q.device)
    # no key of the block has a larger sum of products (whole numbers: exact in 64 bits)
    bounds = s["bounds"].flatten(2)[table].transpose(1, 2).double()  # [seqs][hkv][wide][2 * d]
    most = (bounds @ parts.view(seqs, -1, hkv, 2 * d).permute(0, 2, 3, 1).contiguous()).permute(0, 3, 1, 2).flatten(0, 1)
    score = most.float() * s["ks"][table].transpose(1, 2)[seq]
    used = ((s["lens"][seq] + place + BLOCK) // BLOCK)[:, None, None]
    at = torch.arange(wide, device=q.device)
    score = torch.where((at < s["first"]) | (at >= used - s["recent"]), math.inf, score).masked_fill(at >= used, -math.inf)
    order = score.argsort(dim=2, descending=True, stable=True)[..., :keep]  # of equal scores the lower block stays
    order = torch.where(order < used, order, wide).sort(dim=2).values
    order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=wide)
    return torch.where(order < wide, order, -1).to(torch.int32)


def _plain_selected(s):
    q, chosen = s["q"], s["selected"].long()
    (m, hkv, keep), (_, hq, d) = chosen.shape, q.shape
    block = chosen.clamp(min=0)
    page = s["table"].long()[torch.arange(m, device=q.device)[:, None, None], block]
    head = torch.arange(hkv, device=q.device)[None, :, None]
    ks, vs = (s[n][page, head].div(127.0)[..., None, None] for n in ("ks", "vs"))
    k = (_natural_k(s["k"][page, head], d) * ks).flatten(2, 3)  # [m][hkv][keep * 64][d]
    v = (_natural_v(s["v"][page, head], d) * vs).flatten(2, 3)
    token = block[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)
    seen = ((token <= s["lens"][:, None, None, None]) & (chosen >= 0)[..., None]).flatten(2)[:, :, None]
    logits = (q.view(m, hkv, hq // hkv, d).float() @ k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(d)).masked_fill_(~seen, -math.inf)
    p = (logits - logits.amax(-1, keepdim=True)).exp_()
    return (p @ v).div_(p.sum(-1, keepdim=True)).reshape(m, hq * d).to(q.dtype)


def _own(s):
    import bit_ternary_weight_bitlinear_amd as bl
    if s["kind"] == "rotate":
        return bl.rotate(s["q"], s["k"], s["freq"], s["begin"], s["starts"], interleaved=s["interleaved"], magnitude=s["magnitude"],
                         q_gain=s["gq"], k_gain=s["gk"], eps=EPS)
    if s["kind"] == "select":
        return bl.block_select(s["q"], s["bounds"], s["ks"], s["table"], s["lens"], s["keep"], s["starts"], first=s["first"], recent=s["recent"])
    cache = bl.KVCache(s["k"], s["v"], s["ks"], s["vs"])
    if s["kind"] == "bounds":
        bl.cache_bounds(cache, s["bounds"], s["table"], s["lens"], s["starts"], s["m"])
        return s["bounds"]
    if s["kind"] == "shared":
        return bl.attention_shared(s["q"], cache, s["prefix"], s["prefix_len"], s["table"], s["lens"], s["starts"])
    return bl.attention_selected(s["q"], cache, s["table"], s["lens"], s["selected"])


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "shared": _plain_shared, "bounds": _plain_bounds, "select": _plain_select,
            "selected": _plain_selected}[state["kind"]](state)


# ---------------------------------------------------------------- work

def work(case):
    kind, hkv, d, lens = case["kind"], case["hkv"], case["d"], _ints(case["lens"])
    if kind == "bounds":
        new = _ints(case["new"])
        new = new * len(lens) if len(new) == 1 else new
        blocks = sum(-(-(a + b) // BLOCK) - a // BLOCK for a, b in zip(lens, new))
        tokens = sum(a + b - a // BLOCK * BLOCK for a, b in zip(lens, new))
        return {"bytes": hkv * d * (tokens + 2 * blocks) + 4 * blocks, "flops": 2 * tokens * hkv * d}
    size, hq, new = (2 if case["dtype"] == "bf16" else 4), case["hq"], case.get("new", 1)
    if kind == "rotate":
        n = sum(lens) * (hq + hkv) * d
        return {"bytes": 2 * n * size + 4 * len(lens), "flops": (10 if case["norm"] else 6) * n}
    rows = len(lens) * new
    both = 2 * rows * hq * d * size  # q and out
    held = [-(-(n + new) // BLOCK) for n in lens]
    if kind == "shared":
        blocks = sum(held) + -(-case["prefix"] // BLOCK)
        pairs = rows * case["prefix"] + sum(new * n + new * (new + 1) // 2 for n in lens)
        return {"bytes": 2 * hkv * ((sum(lens) + rows + case["prefix"]) * d + 4 * blocks) + 4 * blocks + both, "flops": 4 * pairs * hq * d}
    if kind == "select":
        return {"bytes": sum(held) * (hkv * (2 * d + 4) + 4) + both // 2 + 4 * rows * hkv * case["keep"], "flops": 4 * new * sum(held) * hkv * d}
    taken = sum(min(case["keep"], n) for n in held)  # per kv head
    tokens = sum(min(case["keep"] * BLOCK, n + 1) for n in lens)
    return {"bytes": 2 * hkv * (tokens * d + 4 * taken) + 4 * rows * hkv * case["keep"] + 4 * taken + both, "flops": 4 * tokens * hq * d}


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "shared": _exact_shared, "bounds": _exact_bounds, "select": _exact_select,
            "selected": _exact_selected}[s["kind"]](s)


def _exact_rotate(s):
    """Every pair as a complex number times magnitude * exp(i * position * frequency)."""
    starts = range(s["q"].shape[0] + 1) if s["starts"] is None else s["starts"].tolist()
    at = torch.cat([torch.arange(p, p + b - a) for p, a, b in zip(s["begin"].tolist(), starts[:-1], starts[1:])]).to("cuda").double()
    turn = torch.polar(torch.full((len(at), len(s["freq"])), float(s["magnitude"]), dtype=torch.float64, device="cuda"), torch.outer(at, s["freq"].double()))
    outs = []
    for x, gain in ((s["q"].double(), s["gq"]), (s["k"].double(), s["gk"])):
        if gain is not None:
            x = gain.double() * x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)
        n = len(s["freq"])
        first = torch.arange(n, device="cuda") * (2 if s["interleaved"] else 1)
        second = first + (1 if s["interleaved"] else n)
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _places(d):
    """Byte of every (token, dim) inside a page and head, for K and V."""
    token, dim = torch.arange(BLOCK, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    return (token % 4 * (d // 16) + dim // 16) * 256 + token // 4 * 16 + dim % 16, (dim // 16 * 4 + token // 16) * 256 + dim % 16 * 16 + token % 16


def _tokens(s, pages, head, d):
    """K and V of the tokens of `pages`, one head, in 64 bits: [pages * 64][d]"""
    return tuple((s[n][pages, head][:, place].double() * (s[n + "s"][pages, head].double() / 127)[:, None, None]).flatten(0, 1)
                 for n, place in zip("kv", _places(d)))


def _softmax_rows(logits, seen):
    """Softmax of the entries of each row that are seen, in place of the others 0."""
    p = torch.where(seen, torch.exp(logits - torch.where(seen, logits, -math.inf).max(1, keepdim=True).values), 0.0)
    return p / p.sum(1, keepdim=True)


def _exact_shared(s):
    q, lens, length = s["q"].double(), s["lens"].tolist(), int(s["prefix_len"])
    (m, hq, d), hkv = q.shape, s["k"].shape[1]
    new, group = m // len(lens), hq // hkv
    out = torch.zeros_like(q)
    for g in range(hkv):
        kp, vp = (x[:length] for x in _tokens(s, s["prefix"].long(), g, d))
        for n, have in enumerate(lens):
            k, v = _tokens(s, s["table"][n, : -(-(have + new) // BLOCK)].long(), g, d)
            k, v = torch.cat((kp, k)), torch.cat((vp, v))
            rows = q[n * new:(n + 1) * new, g * group:(g + 1) * group].reshape(-1, d)
            when = length + have + torch.arange(new, device=q.device).repeat_interleave(group)
            p = _softmax_rows(rows @ k.T.contiguous() / math.sqrt(d), torch.arange(len(k), device=q.device)[None] <= when[:, None])
            out[n * new:(n + 1) * new, g * group:(g + 1) * group] = (p @ v).view(new, group, d)
    return out.flatten(1)


def _exact_bounds(s):
    lens, table, d = s["lens"].tolist(), s["table"].tolist(), s["bounds"].shape[3]
    starts = list(range(len(lens) + 1)) if s["starts"] is None else s["starts"].tolist()
    bounds, place = s["bounds"].clone(), _places(d)[0]
    for n, have in enumerate(lens):
        end = have + starts[n + 1] - starts[n]
        for b in range(have // BLOCK, -(-end // BLOCK)):
            codes = s["k"][table[n][b]][:, place[: min(BLOCK, end - b * BLOCK)]]
            bounds[table[n][b]] = torch.stack((codes.max(1).values, codes.min(1).values), 1)
    return bounds


def _fp32(x):
    """Rounded to fp32, held in 64 bits: where the operator's definition rounds."""
    return x.float().double()


def _exact_select(s):
    """The definition rounds 127 / s, the products that are rounded to integers, the bound and its product with the
    block's scale to fp32; the sums are whole numbers."""
    q, lens, hkv, keep = s["q"].double(), s["lens"].tolist(), s["bounds"].shape[1], s["keep"]
    new, group = q.shape[0] // len(lens), q.shape[1] // hkv
    out = torch.full((q.shape[0], hkv, keep), -1, dtype=torch.int32)
    for r in range(q.shape[0]):
        used = (lens[r // new] + r % new) // BLOCK + 1
        pages = s["table"][r // new, :used].long()
        for g in range(hkv):
            x = q[r, g * group:(g + 1) * group]
            c = torch.round(_fp32(x * _fp32(127 / x.abs().max().clamp(min=SMALLEST))))
            high, low = s["bounds"][pages, g].double().unbind(1)
            bound = torch.maximum(high[:, None] * c, low[:, None] * c).sum((1, 2))
            score = _fp32(_fp32(bound) * s["ks"][pages, g].double()).tolist()
            held = [b for b in range(used) if b < s["first"] or b >= used - s["recent"]]
            rest = sorted(range(s["first"], used - s["recent"]), key=lambda b: (-score[b], b))
            stays = sorted(held + rest[: keep - len(held)])
            out[r, g, : len(stays)] = torch.tensor(stays, dtype=torch.int32)
    return out


def _exact_selected(s):
    q, lens, hkv = s["q"].double(), s["lens"].tolist(), s["k"].shape[1]
    d, group = q.shape[2], q.shape[1] // hkv
    out = torch.zeros_like(q)
    for r, have in enumerate(lens):
        for g in range(hkv):
            blocks = s["selected"][r, g]
            blocks = blocks[blocks >= 0].long()
            k, v = _tokens(s, s["table"][r].long()[blocks], g, d)
            seen = (blocks[:, None] * BLOCK + torch.arange(BLOCK, device=q.device)).flatten()[None] <= have
            out[r, g * group:(g + 1) * group] = _softmax_rows(q[r, g * group:(g + 1) * group] @ k.T.contiguous() / math.sqrt(d), seen) @ v
    return out.flatten(1)
