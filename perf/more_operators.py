"""Measured cases of a serving step over the paged MXFP4 cache: the append with the
position rotation on the way, attention of sequences that share a prefix, the
selection of cache blocks by a cheap score, and attention over the selected blocks.

Each operator has a plain form (elementary torch operations) and the library's call
(own = True); `exact` is its definition in 64 bits.  The cache is
`fp4_kv_append_mx`'s: a row holds one token's kv_heads * head_dim values as E2M1
codes (two to a byte) with a UE8M0 scale per 32; row page * page_size + i is token i
of a page.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
THETA = 1e6
GRID = [0, 0.5, 1, 1.5, 2, 3, 4, 6]


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: 64 rows of 64 + 8 + 8 heads, where the launch counts
        {"name": "append_decode", "op": "append", "tokens": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "interleaved": False, "page": 64, "pad": 0},
        # a prompt of 8192 tokens, whole heads rotated
        {"name": "append_prompt", "op": "append", "tokens": 8192, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "interleaved": False, "page": 64, "pad": 0},
        # an odd number of tokens and some padding, heads of 96 of which 64 values turn in neighbouring pairs
        {"name": "append_odd", "op": "append", "tokens": 4097, "q_heads": 20, "kv_heads": 4, "head_dim": 96,
         "rot_dim": 64, "interleaved": True, "page": 48, "pad": 13},
        # four samples of one short prompt, a token each: latency
        {"name": "shared_few", "op": "shared", "groups": 1, "members": 4, "prefix_low": 1500, "prefix_high": 1500,
         "own_low": 1, "own_high": 90, "drafts": 1, "page": 64, "q_heads": 32, "kv_heads": 8, "head_dim": 128},
        # 64 samples of a long document, each some way into its answer
        {"name": "shared_samples", "op": "shared", "groups": 1, "members": 64, "prefix_low": 16384, "prefix_high": 16384,
         "own_low": 0, "own_high": 1024, "drafts": 1, "page": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128},
        # six system prompts, sessions of each with drafted tokens, odd lengths
        {"name": "shared_sessions", "op": "shared", "groups": 6, "members": 9, "prefix_low": 1000, "prefix_high": 9000,
         "own_low": 0, "own_high": 700, "drafts": 3, "page": 48, "q_heads": 20, "kv_heads": 4, "head_dim": 64},
        # one user, one token, a long context: latency
        {"name": "select_one", "op": "select", "batch": 1, "drafts": 1, "low": 100003, "high": 100003, "page": 64,
         "lists": 1, "dim": 128, "select": 32, "first": 1, "recent": 1},
        # a serving step of 64 long contexts, four drafted tokens each
        {"name": "select_batch", "op": "select", "batch": 64, "drafts": 4, "low": 20000, "high": 131072, "page": 64,
         "lists": 1, "dim": 128, "select": 64, "first": 0, "recent": 0},
        # a selection for every key/value head, small blocks
        {"name": "select_heads", "op": "select", "batch": 12, "drafts": 1, "low": 0, "high": 65536, "page": 32,
         "lists": 8, "dim": 64, "select": 48, "first": 1, "recent": 2},
        # one user, one token: 32 blocks of a long context
        {"name": "blocks_one", "op": "blocks", "batch": 1, "drafts": 1, "low": 100003, "high": 100003, "page": 64,
         "lists": 1, "select": 32, "q_heads": 64, "kv_heads": 8, "head_dim": 128},
        # a decode step of 64 contexts, 64 blocks each
        {"name": "blocks_batch", "op": "blocks", "batch": 64, "drafts": 1, "low": 5000, "high": 12000, "page": 64,
         "lists": 1, "select": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128},
        # drafted tokens with a list for every key/value head, small blocks, contexts that have fewer
        {"name": "blocks_heads", "op": "blocks", "batch": 16, "drafts": 4, "low": 100, "high": 9000, "page": 32,
         "lists": 4, "select": 40, "q_heads": 20, "kv_heads": 4, "head_dim": 64},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "shared", "select", "blocks"])
    page = rng.choice([16, 32, 48, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "append":
        d = rng.choice([32, 64, 96, 128, 192, 256])
        kv = max(kv, 32 // d)
        return {"op": op, "tokens": _log(rng, 1, 8192), "q_heads": kv * rng.choice([0, 1, 2, 4, 5, 8]), "kv_heads": kv,
                "head_dim": d, "rot_dim": 16 * rng.randint(0, d // 16), "interleaved": rng.random() < 0.5, "page": page,
                "pad": rng.choice([0, 0, 5])}
    d = rng.choice([64, 64, 128, 128, 128, 256])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "select":
        batch, drafts = _log(rng, 1, 64), rng.choice([1, 1, 2, 5, 8])
        lists = rng.choice([1, 1, kv])
        high = _log(rng, page, min(131072, 8388608 * page // 64 // batch // lists // drafts * 4))
        return {"op": op, "batch": batch, "drafts": drafts, "low": rng.randint(0, high), "high": high, "page": page,
                "lists": lists, "dim": rng.choice([32, 64, 96, 128, 256]), "select": _log(rng, 1, 128),
                "first": rng.choice([0, 0, 1]), "recent": rng.choice([0, 0, 1, 3])}
    drafts = rng.choice([1, 1, 1, 2, 4, 7])
    if op == "shared":
        members = _log(rng, 1, 64)
        groups = _log(rng, 1, max(1, 64 // members))
        high = _log(rng, 1, min(16384, 900000 // (groups * members * drafts) // max(1, kv * d // 1024)))
        return {"op": op, "groups": groups, "members": members, "prefix_low": rng.randint(1, high), "prefix_high": high,
                "own_low": 0, "own_high": _log(rng, 1, 1024 // drafts), "drafts": drafts, "page": page,
                "q_heads": kv * group, "kv_heads": kv, "head_dim": d}
    batch = _log(rng, 1, 64)
    most = min(4096, 4096 * 64 // (batch * drafts)) // max(1, kv * d // 1024)         # tokens of a list
    select = _log(rng, 1, max(1, most // page))
    high = _log(rng, 1, 12000)
    return {"op": op, "batch": batch, "drafts": drafts, "low": rng.randint(0, high), "high": high, "page": page,
            "lists": rng.choice([1, kv]), "select": select, "q_heads": kv * group, "kv_heads": kv, "head_dim": d}


def _spread(low, high, n, salt):
    """n lengths between low and high, the same for every seed."""
    r = random.Random(f"{low}-{high}-{n}-{salt}")
    return [r.randint(low, high) for _ in range(n)]


def _shared_lens(case):
    """Lengths of the groups' prefixes (whole pages) and of the sequences' own tokens."""
    page = case["page"]
    prefix = [max(1, n // page) * page for n in _spread(case["prefix_low"], case["prefix_high"], case["groups"], "prefix")]
    return prefix, _spread(case["own_low"], case["own_high"], case["groups"] * case["members"], "own")


# ----------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _mx_quantize(x):
    """[rows, d] to E2M1 codes and UE8M0 scale bytes: E = floor(log2 amax) - 2 of
    each 32 values, codes rounded to nearest, ties to the even code, at most 6."""
    rows, d = x.shape
    blocks = x.float().reshape(rows, d // 32, 32)
    amax = blocks.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(-127, 127)
    a = torch.ldexp(blocks.abs(), -e)
    idx = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    idx = (idx | (torch.signbit(blocks).byte() << 3)).reshape(rows, d // 2, 2)
    return idx[..., 0] | (idx[..., 1] << 4), (e + 127).byte().reshape(rows, d // 32)


def _cache(g, rows, d):
    """Codes and scales of `rows` normal vectors, a tenth of them larger."""
    codes = torch.empty(rows, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(rows, d // 32, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 28) // d)
    for r in range(0, rows, step):
        x = _normal(g, min(step, rows - r), d)
        x *= 1 + 2 * (torch.rand(x.shape[0], 1, generator=g, device=DEV) < 0.1)
        codes[r:r + step], scales[r:r + step] = _mx_quantize(x)
    return codes, scales


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _table(g, counts, columns, spare=3):
    """Page table of sequences that hold `counts` pages of their own, over shuffled pages."""
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((len(counts), max(1, columns)), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(table.shape[1], device=DEV) < _i32(counts)[:, None]] = order[:sum(counts)]
    return table, pages


def _tree_masks(seed, batch, drafts):
    """For each drafted token the bits of the tokens that it follows in its tree, and its own."""
    r = random.Random(seed)
    masks = np.zeros((batch, drafts), np.uint64)
    for b in range(batch):
        for i in range(drafts):
            up = masks[b, r.randint(max(0, i - 4), i - 1)] if i else np.uint64(0)
            masks[b, i] = up | np.uint64(1 << i)
    return torch.from_numpy(masks.view(np.int64)).to(DEV)


def prepare(case, seed):
    g, op, page = _gen(seed), case["op"], case["page"]
    r = random.Random(seed + 1)
    if op == "append":
        n, hq, hk, d, rot = (case[k] for k in ("tokens", "q_heads", "kv_heads", "head_dim", "rot_dim"))
        qkv = (_normal(g, n, hq + 2 * hk, d) * (0.5 + 2 * torch.rand(1, hq + 2 * hk, 1, generator=g, device=DEV))).bfloat16()
        places = 131072 if n <= 256 else 2 * n
        turns = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / max(rot, 1))
        angles = torch.arange(places, dtype=torch.float64, device=DEV)[:, None] * turns
        # a decode step's sequences stand anywhere, a prompt's tokens one after another
        positions = torch.randint(0, places, (n,), generator=g, device=DEV)
        if n > 256:
            positions = positions[:1] % n + torch.arange(n, device=DEV)
        pages = -(-n // page) + 3
        order = torch.randperm(pages, generator=g, device=DEV)
        slots = (order[:, None] * page + torch.arange(page, device=DEV)).flatten()[:n].int()
        slots[n - min(case["pad"], n - 1):] = -1
        cache = [torch.randint(0, 256, (pages * page, hk * d // w), generator=g, device=DEV, dtype=torch.uint8)
                 for w in (2, 32, 2, 32)]
        return {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:], "slots": slots,
                "cos_sin": torch.cat([angles.cos(), angles.sin()], 1).float(), "positions": positions.int(),
                "q_out": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), "cache": cache}
    if op == "select":
        batch, shape = case["batch"], (case["batch"], case["drafts"], case["lists"], case["dim"])
        lens = _spread(case["low"], case["high"], batch, "lens")
        table, pages = _table(g, [-(-n // page) for n in lens], -(-case["high"] // page))
        codes, scales = _cache(g, pages, case["lists"] * case["dim"])
        ids = (*shape[:3], case["select"])
        return {"case": case, "q": _normal(g, *shape).bfloat16(), "codes": codes, "scales": scales, "table": table,
                "lens": _i32(lens), "ids": torch.zeros(ids, dtype=torch.int32, device=DEV),
                "scores": torch.zeros(ids, dtype=torch.float32, device=DEV)}
    hq, hk, hd, drafts = (case[k] for k in ("q_heads", "kv_heads", "head_dim", "drafts"))
    if op == "shared":
        groups, members = case["groups"], case["members"]
        prefix, more = _shared_lens(case)
        base = [n for n in prefix for _ in range(members)]
        lens = [a + b for a, b in zip(base, more)]
        columns = -(-(max(lens) + drafts) // page)
        mine = [-(-(n + drafts) // page) for n in more]
        table, pages = _table(g, [n // page for n in prefix] + mine, columns)
        held, own_pages = table[:groups].repeat_interleave(members, 0), table[groups:]
        # a sequence's own pages stand behind those that it shares
        at = torch.arange(columns, device=DEV) - _i32(base)[:, None] // page
        table = torch.where(at < 0, held, own_pages.gather(1, at.clamp(0, columns - 1).long()))
        batch = groups * members
        extra = {"groups": _i32([members * i for i in range(groups + 1)]), "prefix": _i32(prefix)}
    else:
        batch = case["batch"]
        lens = _spread(case["low"], case["high"], batch, "lens")
        table, pages = _table(g, [-(-(n + drafts) // page) for n in lens], -(-(case["high"] + drafts) // page))
        # of each sequence's complete blocks some, in order, for every drafted token and list
        score = torch.rand(batch, drafts, case["lists"], case["high"] // page + 1, generator=g, device=DEV)
        score.masked_fill_(torch.arange(score.shape[-1], device=DEV) >= _i32(lens)[:, None, None, None] // page, 2.0)
        n = case["select"]
        score = torch.nn.functional.pad(score, (0, max(0, n - score.shape[-1])), value=2.0)
        top, at = score.sort(dim=-1)
        ids = torch.where(top < 1.5, at, 1 << 30)[..., :n].sort(dim=-1).values
        extra = {"ids": torch.where(ids < 1 << 30, ids, -1).int()}
    kc, ks = _cache(g, pages * page, hk * hd)
    vc, vs = _cache(g, pages * page, hk * hd)
    shape = (batch, drafts, hq, hd)
    return {"case": case, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": table, "lens": _i32(lens), "most": max(lens) + drafts,
            "q": _normal(g, *shape).bfloat16(), "masks": _tree_masks(seed, batch, drafts),
            "drafted": _i32([r.randint(1, drafts) for _ in lens]),
            "out": torch.zeros(shape, dtype=torch.bfloat16, device=DEV), **extra}


# ------------------------------------------------------------------ plain forms

def _turned(x, row, rot, interleaved):
    """The first rot values of every head turned by the angles of `row` (cosines, then
    sines).  A turned value is rounded to 32 bits as one product and one fused
    multiply-add are (64 bits hold the inner one), since values next to a border between
    two codes are what it goes into."""
    cos, sin = row[:, None, :rot // 2], row[:, None, rot // 2:]
    turned, rest = x[..., :rot].float(), x[..., rot:].float()
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :rot // 2], turned[..., rot // 2:])
    both = [(a.double() * cos.double() - (b * sin).double()).float(), (b.double() * cos.double() + (a * sin).double()).float()]
    turned = torch.stack(both, -1).flatten(-2) if interleaved else torch.cat(both, -1)
    return torch.cat([turned, rest], -1).bfloat16()


def _append(s):
    rot, inter = s["case"]["rot_dim"], s["case"]["interleaved"]
    row = s["cos_sin"][s["positions"].long()]
    used = s["slots"] >= 0
    slots = s["slots"].long()[used]
    kc, ks, vc, vs = s["cache"]
    s["q_out"].copy_(_turned(s["q"], row, rot, inter))
    kc[slots], ks[slots] = _mx_quantize(_turned(s["k"], row, rot, inter).flatten(1)[used])
    vc[slots], vs[slots] = _mx_quantize(s["v"].flatten(1)[used])
    return [s["q_out"], *s["cache"]]


def _values(codes, scales):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    x = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1)
    x = x.reshape(*scales.shape, 32)
    return torch.ldexp(x, scales.int().unsqueeze(-1) - 127).flatten(-2)


def _softmax_product(scores, hidden, v):
    """Rows of softmax(scores) v over what is not hidden; zero where all is."""
    scores = scores.masked_fill(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(scores - top)
    return (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _drafted_seen(s, rank):
    """Whether each drafted token sees the one of this rank ([batch, n]; negative: a committed one)."""
    seen = (s["masks"][:, :, None] >> rank.clamp(0, 63)[:, None]) & 1 == 1
    return (rank[:, None] < 0) | (seen & (rank < s["drafted"][:, None])[:, None])


def _used(s, out):
    used = torch.arange(out.shape[1], device=DEV) < s["drafted"][:, None]
    return torch.where(used[:, :, None, None], out, 0.0).bfloat16()


def _shared(s):
    case = s["case"]
    page, hq, hk, d = case["page"], case["q_heads"], case["kv_heads"], case["head_dim"]
    batch, drafts = s["q"].shape[:2]
    at = torch.arange(s["most"], device=DEV)
    rows = s["table"][:, at // page].long().clamp_min(0) * page + at % page
    k, v = (_values(c[rows], e[rows]).reshape(batch, at.numel(), hk, d).transpose(1, 2)
            for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    q = s["q"].float().reshape(batch, drafts, hk, hq // hk, d).transpose(1, 2).reshape(batch, hk, -1, d)
    seen = _drafted_seen(s, at - s["lens"][:, None])
    hidden = ~seen[:, None, :, None].expand(batch, 1, drafts, hq // hk, at.numel()).reshape(batch, 1, -1, at.numel())
    out = _softmax_product(q @ k.transpose(-1, -2) * d ** -0.5, hidden, v)
    return _used(s, out.reshape(batch, hk, drafts, hq // hk, d).transpose(1, 2).reshape(batch, drafts, hq, d))


def _select(s):
    case = s["case"]
    page, n, lists, dim = case["page"], case["select"], case["lists"], case["dim"]
    batch, drafts = s["q"].shape[:2]
    complete = (s["lens"] // page)[:, None, None, None]
    table = torch.nn.functional.pad(s["table"], (0, max(0, n - s["table"].shape[1])), value=-1)
    at = torch.arange(table.shape[1], device=DEV)
    entries = _values(s["codes"], s["scales"])[table.clamp_min(0).long()].reshape(batch, -1, lists, dim)
    q = _values(*_mx_quantize(s["q"].reshape(-1, dim))).reshape(s["q"].shape)
    scores = (q.transpose(1, 2) @ entries.permute(0, 2, 3, 1).contiguous()).transpose(1, 2)
    there = (at < complete) & (table >= 0)[:, None, None]
    forced = there & ((at < case["first"]) | (at >= complete - case["recent"]))
    rank = scores.masked_fill(forced, math.inf).double().masked_fill(~there, -math.inf)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :n]
    best = torch.where(there.expand(rank.shape).gather(-1, best), best, 1 << 30).sort(dim=-1).values
    chosen = best < 1 << 30
    picked = scores.gather(-1, best.clamp_max(table.shape[1] - 1)).masked_fill(~chosen, -math.inf)
    return [torch.where(chosen, best, -1).int(), picked]


def _blocks(s):
    case = s["case"]
    page, hq, hk, d = case["page"], case["q_heads"], case["kv_heads"], case["head_dim"]
    batch, drafts = s["q"].shape[:2]
    ids = s["ids"].expand(batch, drafts, hk, -1)
    i = torch.arange(page, device=DEV)
    listed_at = (ids.clamp_min(0)[..., None] * page + i).flatten(3)
    start = (s["lens"] // page * page)[:, None]
    tail_at = start + torch.arange(page + drafts, device=DEV)
    at = torch.cat([listed_at, tail_at[:, None, None].expand(batch, drafts, hk, -1)], -1)
    pages = s["table"].gather(1, (at // page).clamp_max(s["table"].shape[1] - 1).reshape(batch, -1).long())
    rows = pages.reshape(at.shape).long().clamp_min(0) * page + at % page
    head = torch.arange(hk, device=DEV)[:, None]
    k, v = (_values(c.reshape(-1, hk, d // 2)[rows, head], e.reshape(-1, hk, d // 32)[rows, head])
            for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    q = s["q"].float().reshape(batch, drafts, hk, hq // hk, d)
    in_list = (ids >= 0)[..., None].expand(*ids.shape, page).flatten(3)
    in_tail = _drafted_seen(s, tail_at - s["lens"][:, None])[:, :, None].expand(batch, drafts, hk, -1)
    hidden = ~torch.cat([in_list, in_tail], -1)[:, :, :, None]
    out = _softmax_product(q @ k.transpose(-1, -2) * d ** -0.5, hidden, v)
    return _used(s, out.reshape(batch, drafts, hq, d))


# ------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"append": _append, "shared": _shared, "select": _select, "blocks": _blocks}[s["case"]["op"]](s)


def _run_own(s):
    import block_scaled_fp4_mx_amd as F

    case, op = s["case"], s["case"]["op"]
    page = case["page"]
    if op == "append":
        F.fp4_kv_append_rope_mx(s["q"], s["k"], s["v"], F.KvCache(*s["cache"], page), s["slots"], s["q_out"], s["positions"],
                                s["cos_sin"], interleaved=case["interleaved"])
        return [s["q_out"], *s["cache"]]
    if op == "select":
        if "ws" not in s:
            s["ws"] = torch.empty(F.fp4_kv_select_workspace_bytes(*s["q"].shape[:3], s["table"].shape[1]),
                                  dtype=torch.uint8, device=DEV)
        F.fp4_kv_select_mx(s["q"], s["codes"], s["scales"], s["table"], s["lens"], page, s["ids"], s["ws"],
                           scores=s["scores"], n_first=case["first"], n_recent=case["recent"])
        return [s["ids"], s["scores"]]
    cache = F.KvCache(s["kc"], s["ks"], s["vc"], s["vs"], page)
    if op == "shared":
        if "ws" not in s:
            s["ws"] = torch.empty(F.fp4_attn_shared_workspace_bytes(*s["q"].shape, case["kv_heads"], case["groups"]),
                                  dtype=torch.uint8, device=DEV)
        F.fp4_attn_shared_mx(s["q"], cache, s["table"], s["lens"], s["groups"], s["prefix"], s["out"], s["ws"],
                             draft_lens=s["drafted"], tree_mask=s["masks"])
    else:
        if "ws" not in s:
            s["ws"] = torch.empty(F.fp4_attn_blocks_workspace_bytes(*s["q"].shape, case["kv_heads"]),
                                  dtype=torch.uint8, device=DEV)
        F.fp4_attn_blocks_mx(s["q"], cache, s["table"], s["lens"], s["ids"], s["out"], s["ws"], draft_lens=s["drafted"],
                             tree_mask=s["masks"])
    return s["out"]


# ------------------------------------------------------------------------- work

def work(case):
    op, page = case["op"], case["page"]
    if op == "append":
        n, d, rot = case["tokens"], case["head_dim"], case["rot_dim"]
        heads = case["q_heads"] + case["kv_heads"]
        row = 2 * (case["kv_heads"] * d * 17 // 32)
        return {"bytes": n * (4 * case["q_heads"] * d + 4 * case["kv_heads"] * d + row + 4 * rot + 8),
                "flops": n * (3 * heads * rot + 8 * case["kv_heads"] * d)}
    if op == "select":
        blocks = sum(n // page for n in _spread(case["low"], case["high"], case["batch"], "lens"))
        rows = case["batch"] * case["drafts"] * case["lists"]
        return {"bytes": blocks * (case["lists"] * case["dim"] * 17 // 32 + 4) + rows * (2 * case["dim"] + 8 * case["select"]),
                "flops": 2 * blocks * case["drafts"] * case["lists"] * case["dim"]}
    hq, d, drafts = case["q_heads"], case["head_dim"], case["drafts"]
    row = 2 * (case["kv_heads"] * d * 17 // 32)                        # a token's keys and values
    if op == "shared":
        prefix, more = _shared_lens(case)
        batch = len(more)
        once = sum(prefix) + sum(more) + batch * drafts
        seen = sum(prefix) * case["members"] + sum(more) + batch * drafts
        return {"bytes": row * once + 4 * batch * drafts * hq * d + 4 * once // page,
                "flops": 4 * drafts * hq * d * seen}
    lens = _spread(case["low"], case["high"], case["batch"], "lens")
    # every drafted token's list; those of a sequence may name the same blocks, at most all of them
    listed_tokens = [min(case["select"], n // page) * page for n in lens]
    seen = sum(drafts * t + drafts * (n % page + drafts) for t, n in zip(listed_tokens, lens))
    once = sum(min(drafts * t, n) + n % page + drafts for t, n in zip(listed_tokens, lens))
    return {"bytes": row * once + len(lens) * drafts * (4 * hq * d + 4 * case["lists"] * case["select"]),
            "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------------ exact

def _decoded(codes, scales):
    value = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64, device=DEV)
    two = torch.stack([value[(codes % 16).long()], value[(codes // 16).long()]], -1).flatten(-2)
    return two * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)


def _attend(q, k, v, seen):
    """q [m, d] of one key/value head, k and v [n, d], seen [m, n], in 64 bits."""
    logits = torch.mm(q, k.t().contiguous()) / math.sqrt(q.shape[1])
    p = torch.nan_to_num(torch.softmax(logits.masked_fill(~seen, -math.inf), 1))
    return p @ v


def exact(case, seed):
    op = case["op"]
    if op == "append":
        s = prepare(case, seed)
        half, y = case["rot_dim"] // 2, s["q"].double()
        row = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(row[:, :half], row[:, half:])[:, None]
        first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return [y, None, None, None, None]
    if op == "select":
        s = prepare(case, seed)
        page, n, dim = case["page"], case["select"], case["dim"]
        chosen = np.full((case["batch"], case["drafts"], case["lists"], n), -np.inf)
        table, lens = s["table"].tolist(), s["lens"].tolist()
        grid = np.array(GRID)
        x = s["q"].float().cpu().numpy().astype(np.float64).reshape(*chosen.shape[:3], dim // 32, 32)
        amax = np.abs(x).max(-1, keepdims=True)
        unit = np.exp2(np.floor(np.log2(np.maximum(amax, 2.0 ** -120))) - 2)
        ratio = np.abs(x) / unit
        # the nearest grid value, of two the one with the even code
        near = np.abs(ratio[..., None] - grid) + np.array([0, 1e-9] * 4)
        q = np.sign(x) * grid[near.argmin(-1)] * unit
        q = torch.tensor(q.reshape(*chosen.shape[:3], dim), device=DEV)
        for b, length in enumerate(lens):
            complete = length // page
            if not complete:
                continue
            pages = torch.tensor(table[b][:complete], device=DEV)
            entries = _decoded(s["codes"][pages], s["scales"][pages]).reshape(complete, case["lists"], dim)
            for g in range(case["lists"]):
                scores = torch.mm(q[b, :, g], entries[:, g].t().contiguous()).cpu().numpy()
                forced = [m for m in range(complete) if m < case["first"] or m >= complete - case["recent"]]
                for i in range(case["drafts"]):
                    order = sorted(range(complete), key=lambda m: (-scores[i, m], m))
                    kept = [*forced, *(m for m in order if m not in set(forced))][:n] if forced else order[:n]
                    chosen[b, i, g, :len(kept)] = scores[i, sorted(kept)]
        return [None, torch.tensor(chosen, device=DEV)]
    s = prepare(case, seed)
    page, hq, hk, d, drafts = case["page"], case["q_heads"], case["kv_heads"], case["head_dim"], case["drafts"]
    per = hq // hk
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    masks, drafted, lens = (s[x].cpu().tolist() for x in ("masks", "drafted", "lens"))
    ids = s["ids"].cpu().tolist() if op == "blocks" else None
    for b, n in enumerate(lens):
        t = drafted[b]
        bits = torch.tensor([[(masks[b][i] >> j) & 1 == 1 for j in range(t)] for i in range(t)], device=DEV)
        if op == "shared":
            at = torch.arange(n + t, device=DEV)
            rows = s["table"][b].long()[at // page] * page + at % page
            k, v = _decoded(s["kc"][rows], s["ks"][rows]), _decoded(s["vc"][rows], s["vs"][rows])
            seen = torch.cat([torch.ones(t, n, dtype=torch.bool, device=DEV), bits], 1).repeat_interleave(per, 0)
            for h in range(hk):
                q = s["q"][b, :t, h * per:(h + 1) * per].double().reshape(t * per, d)
                o = _attend(q, k[:, h * d:(h + 1) * d], v[:, h * d:(h + 1) * d], seen)
                out[b, :t, h * per:(h + 1) * per] = o.reshape(t, per, d)
            continue
        for i in range(t):
            for h in range(hk):
                blocks = [m for m in ids[b][i][h if case["lists"] > 1 else 0] if m >= 0]
                at = torch.cat([torch.arange(m * page, (m + 1) * page) for m in blocks] +
                               [torch.arange(n // page * page, n + t)]).to(DEV)
                rows = s["table"][b].long()[at // page] * page + at % page
                cols, cells = slice(h * d // 2, (h + 1) * d // 2), slice(h * d // 32, (h + 1) * d // 32)
                k, v = _decoded(s["kc"][rows, cols], s["ks"][rows, cells]), _decoded(s["vc"][rows, cols], s["vs"][rows, cells])
                seen = torch.cat([torch.ones(at.numel() - t, dtype=torch.bool, device=DEV), bits[i]])
                q = s["q"][b, i, h * per:(h + 1) * per].double()
                out[b, i, h * per:(h + 1) * per] = _attend(q, k, v, seen.expand(per, -1))
    return out
