"""Measured cases of the attention path: norms and rotation of queries and keys,
attention over packed prompts, attention of drafted tokens over the paged MXFP4
cache, and the bookkeeping of that cache's pages.

Each operator has a plain form (elementary torch operations in 32 bits) and the
library's calls (own = True); `exact` is its definition in 64 bits.  The cache is
`fp4_kv_append_mx`'s: a row holds one token's kv_heads * head_dim values as E2M1
codes (two to a byte) with a UE8M0 scale per 32; row page * page_size + i is
token i of a page.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 1e6


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: 64 rows of 64 + 8 heads, where the launch counts
        {"name": "norm_rope_decode", "op": "norm_rope", "tokens": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "interleaved": False, "w_f32": False},
        # a prompt of 8192 tokens, whole heads rotated
        {"name": "norm_rope_prompt", "op": "norm_rope", "tokens": 8192, "q_heads": 64, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "interleaved": False, "w_f32": False},
        # an odd number of tokens, heads of 96 of which 64 values are rotated in neighbouring pairs, fp32 weights
        {"name": "norm_rope_odd", "op": "norm_rope", "tokens": 4097, "q_heads": 20, "kv_heads": 4, "head_dim": 96,
         "rot_dim": 64, "interleaved": True, "w_f32": True},
        # a batch of short chat turns, packed, some of a few tokens, with padding rows at the end
        {"name": "prompt_short", "op": "prompt", "seqs": 24, "low": 3, "high": 421, "pad": 13, "q_heads": 16,
         "kv_heads": 16, "head_dim": 64},
        # four documents in one prefill batch of about 8k tokens
        {"name": "prompt_packed", "op": "prompt", "seqs": 4, "low": 1100, "high": 2900, "pad": 0, "q_heads": 64,
         "kv_heads": 8, "head_dim": 128},
        # one long prompt
        {"name": "prompt_long", "op": "prompt", "seqs": 1, "low": 16384, "high": 16384, "pad": 0, "q_heads": 32,
         "kv_heads": 4, "head_dim": 128},
        # one user, one token, a short context: latency
        {"name": "tree_one_token", "op": "tree", "batch": 1, "drafts": 1, "ragged": False, "low": 1500, "high": 1500,
         "page": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128},
        # a speculative serving step: 64 sequences of all lengths, trees of up to 8 drafted tokens
        {"name": "tree_batch", "op": "tree", "batch": 64, "drafts": 8, "ragged": True, "low": 0, "high": 8191,
         "page": 64, "q_heads": 64, "kv_heads": 8, "head_dim": 128},
        # long contexts, a wide tree
        {"name": "tree_long", "op": "tree", "batch": 4, "drafts": 16, "ragged": False, "low": 90001, "high": 131072,
         "page": 128, "q_heads": 32, "kv_heads": 8, "head_dim": 128},
        # after a speculative step: give up the rejected rows, reserve, append the drafted rows, keep the accepted ones
        {"name": "pages_speculate", "op": "speculate", "batch": 64, "drafts": 8, "low": 200, "high": 4096, "page": 64,
         "d": 1024},
        # parallel sampling: the old samples end, every prompt is forked again, each sample takes its next token
        {"name": "pages_fork", "op": "fork", "parents": 16, "children": 8, "low": 500, "high": 4096, "page": 64, "d": 1024},
        # pages moved from one cache to another
        {"name": "pages_copy", "op": "copy", "pages": 8192, "page": 64, "d": 1024},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "prompt", "tree", "speculate", "fork", "copy"])
    if op == "norm_rope":
        d = rng.choice([32, 64, 96, 128, 192, 256])
        kv = rng.choice([1, 2, 4, 8])
        inter = rng.random() < 0.5
        return {"op": op, "tokens": _log(rng, 1, 8192), "q_heads": kv * rng.choice([1, 2, 4, 5, 8]), "kv_heads": kv,
                "head_dim": d, "rot_dim": 16 * rng.randint(1, d // 16), "interleaved": inter,
                "w_f32": rng.random() < 0.5}
    d = rng.choice([64, 64, 128, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 8])
    if op == "prompt":
        seqs = _log(rng, 1, 32)
        high = _log(rng, 1, 11000 // seqs)
        return {"op": op, "seqs": seqs, "low": rng.randint(0, high), "high": high, "pad": rng.choice([0, 0, 5]),
                "q_heads": kv * min(group, 4 if kv == 8 else 8), "kv_heads": kv, "head_dim": d}
    if op == "tree":
        batch = _log(rng, 1, 64)
        high = _log(rng, 1, 400000 // batch // max(1, kv * d // 512))
        return {"op": op, "batch": batch, "drafts": rng.choice([1, 1, 2, 5, 8, 17, 33, 64]) if batch <= 8
                else rng.choice([1, 1, 2, 5, 8]),
                "ragged": rng.random() < 0.5, "low": rng.randint(0, high), "high": high,
                "page": rng.choice([16, 32, 48, 64, 128]), "q_heads": kv * group, "kv_heads": kv, "head_dim": d}
    width = rng.choice([96, 256, 512, 1024])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "speculate":
        high = _log(rng, 16, 4096)
        return {"op": op, "batch": _log(rng, 1, 64), "drafts": rng.choice([1, 3, 8, 16, 64]), "low": rng.randint(1, high),
                "high": high, "page": page, "d": width}
    if op == "fork":
        high = _log(rng, 16, 4096)
        return {"op": op, "parents": _log(rng, 1, 16), "children": rng.randint(1, 8), "low": rng.randint(1, high),
                "high": high, "page": page, "d": width}
    return {"op": "copy", "pages": _log(rng, 1, 4096), "page": page, "d": width}


def _lens(case, n):
    """n lengths between the case's low and high, the same for every seed."""
    r = random.Random(f"{case['low']}-{case['high']}-{n}")
    return [r.randint(case["low"], case["high"]) for _ in range(n)]


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


def _tables(g, lens, page, columns, spare):
    """Page table, counts, lengths and references of sequences of these lengths, over
    shuffled pages, with `spare` pages left free."""
    counts = [-(-n // page) for n in lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=g, device=DEV).int()
    table = torch.full((len(lens), max(1, columns)), -1, dtype=torch.int32, device=DEV)
    held = torch.arange(table.shape[1], device=DEV) < _i32(counts)[:, None]
    table[held] = order[:sum(counts)]
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order[:sum(counts)].long()] = 1
    return table, _i32(counts), _i32(lens), refs


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
    g, op = _gen(seed), case["op"]
    if op == "norm_rope":
        n, hq, hk, d, rot = (case[k] for k in ("tokens", "q_heads", "kv_heads", "head_dim", "rot_dim"))
        qkv = (_normal(g, n, hq + 2 * hk, d) * (0.5 + 2 * torch.rand(1, hq + 2 * hk, 1, generator=g, device=DEV))).bfloat16()
        places = 131072 if n <= 256 else 2 * n
        turns = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angles = torch.arange(places, dtype=torch.float64, device=DEV)[:, None] * turns
        # a decode step's sequences stand anywhere, a prompt's tokens one after another
        positions = torch.randint(0, places, (n,), generator=g, device=DEV)
        if n > 256:
            positions = positions[:1] % n + torch.arange(n, device=DEV)
        weights = (1 + 0.2 * _normal(g, 2, d)).to(torch.float32 if case["w_f32"] else torch.bfloat16)
        return {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "q_weight": weights[0].contiguous(),
                "k_weight": weights[1].contiguous(),
                "cos_sin": torch.cat([angles.cos(), angles.sin()], 1).float(),
                "positions": positions.int(),
                "q_out": torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV),
                "k_out": torch.empty(n, hk, d, dtype=torch.bfloat16, device=DEV)}
    if op == "prompt":
        lens = _lens(case, case["seqs"])
        hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        n = sum(lens) + case["pad"]
        qkv = _normal(g, n, hq + 2 * hk, d).bfloat16()
        return {"case": case, "lens": lens, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:],
                "cu": _i32([0, *np.cumsum(lens).tolist()]),
                "out": torch.zeros(n, hq, d, dtype=torch.bfloat16, device=DEV)}
    if op == "tree":
        batch, drafts, page, d = case["batch"], case["drafts"], case["page"], case["kv_heads"] * case["head_dim"]
        lens = _lens(case, batch)
        columns = -(-(case["high"] + drafts) // page)
        table, _, _, refs = _tables(g, [n + drafts for n in lens], page, columns, 3)
        kc, ks = _cache(g, refs.numel() * page, d)
        vc, vs = _cache(g, refs.numel() * page, d)
        r = random.Random(seed + 1)
        shape = (batch, drafts, case["q_heads"], case["head_dim"])
        return {"case": case, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": table, "lens": _i32(lens),
                "q": _normal(g, *shape).bfloat16(), "masks": _tree_masks(seed, batch, drafts),
                "drafted": _i32([r.randint(1, drafts) if case["ragged"] else drafts for _ in lens]),
                "out": torch.zeros(shape, dtype=torch.bfloat16, device=DEV)}
    page, d = case["page"], case["d"]
    if op == "copy":
        n = case["pages"]
        kc, ks = _cache(g, n * page, d)
        vc, vs = _cache(g, n * page, d)
        to = torch.randperm(n + 5, generator=g, device=DEV)[:n].int()
        return {"case": case, "from": torch.randperm(n, generator=g, device=DEV).int(), "to": to,
                "source": (kc, ks, vc, vs),
                "target": tuple(torch.zeros((n + 5) * page, t.shape[1], dtype=torch.uint8, device=DEV)
                                for t in (kc, ks, vc, vs))}
    r = random.Random(seed + 1)
    if op == "speculate":
        batch, drafts = case["batch"], case["drafts"]
        lens = _lens(case, batch)
        columns = -(-(case["high"] + drafts) // page)
        table, counts, seq_lens, refs = _tables(g, lens, page, columns, batch * (1 + drafts // page) + 9)
        kept = [sorted(r.sample(range(drafts), r.randint(0, min(drafts, 6)))) for _ in lens]
        more = {"base": _i32(lens), "drafted": _i32([drafts] * batch),
                "accepted": _i32([k + [-1] * (drafts - len(k)) for k in kept]), "n_accepted": _i32([len(k) for k in kept]),
                "new_k": _normal(g, batch * drafts, d).bfloat16(), "new_v": _normal(g, batch * drafts, d).bfloat16()}
    else:
        parents, children, drafts = case["parents"], case["children"], 1
        lens = _lens(case, parents)
        batch = parents * (1 + children)
        columns = -(-(case["high"] + 1) // page)
        # the samples hold nothing before the first pass, and what it gave them from then on
        table, counts, seq_lens, refs = _tables(g, lens + [0] * (batch - parents), page, columns, 2 * batch)
        ids = list(range(parents, batch))
        more = {"samples": _i32(ids), "pairs": _i32([[(i - parents) // children, i] for i in ids]),
                "drafted": _i32([0] * parents + [1] * len(ids)),
                "new_k": _normal(g, batch, d).bfloat16(), "new_v": _normal(g, batch, d).bfloat16()}
    kc, ks = _cache(g, refs.numel() * page, d)
    vc, vs = _cache(g, refs.numel() * page, d)
    return {"case": case, "cache": (kc, ks, vc, vs), "table": table, "counts": counts, "lens": seq_lens, "refs": refs,
            "seqs": torch.arange(batch, dtype=torch.int32, device=DEV),
            "slots": torch.full((batch, drafts), -1, dtype=torch.int32, device=DEV),
            "short": torch.zeros(1, dtype=torch.int32, device=DEV), **more}


# ------------------------------------------------------------------ plain forms

def _norm_rope(x, w, cos, sin, interleaved):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    rot = 2 * cos.shape[-1]
    turned, rest = x[..., :rot], x[..., rot:]
    a, b = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :rot // 2], turned[..., rot // 2:])
    both = [a * cos - b * sin, b * cos + a * sin]
    turned = torch.stack(both, -1).flatten(-2) if interleaved else torch.cat(both, -1)
    return torch.cat([turned, rest], -1).bfloat16()


def _softmax_product(scores, hidden, v):
    """Rows of softmax(scores) v over what is not hidden; zero where all is."""
    scores = scores.masked_fill(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-3e38)
    p = torch.exp(scores - top)
    return (p @ v) / p.sum(-1, keepdim=True).clamp_min(1e-38)


def _prompt(q, k, v):
    """One sequence: q [n, q_heads, d], k and v [n, kv_heads, d]."""
    n, hq, d = q.shape
    hk = k.shape[1]
    q = q.float().reshape(n, hk, hq // hk, d).permute(1, 2, 0, 3)
    k, v = (t.float().transpose(0, 1).unsqueeze(1).contiguous() for t in (k, v))
    later = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
    out = _softmax_product(q @ k.transpose(-1, -2) * d ** -0.5, later, v)
    return out.permute(2, 0, 1, 3).reshape(n, hq, d).bfloat16()


def _values(codes, scales):
    lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    x = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1)
    x = x.reshape(*scales.shape, 32)
    return torch.ldexp(x, scales.int().unsqueeze(-1) - 127).flatten(-2)


def _tree(s):
    case = s["case"]
    page, hq, hk, d = case["page"], case["q_heads"], case["kv_heads"], case["head_dim"]
    batch, drafts = s["q"].shape[:2]
    at = torch.arange(case["high"] + drafts, device=DEV)
    rows = s["table"][:, at // page].long().clamp_min(0) * page + at % page
    k, v = (_values(c[rows], e[rows]).reshape(batch, at.numel(), hk, d).transpose(1, 2)
            for c, e in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
    q = s["q"].float().reshape(batch, drafts, hk, hq // hk, d).transpose(1, 2).reshape(batch, hk, -1, d)
    rank = at - s["lens"][:, None]                                     # of a drafted token, negative before them
    seen = (s["masks"][:, :, None] >> rank.clamp(0, 63)[:, None]) & 1 == 1
    seen = (rank[:, None] < 0) | (seen & (rank < s["drafted"][:, None])[:, None])
    hidden = ~seen[:, None, :, None].expand(batch, 1, drafts, hq // hk, at.numel()).reshape(batch, 1, -1, at.numel())
    out = _softmax_product(q @ k.transpose(-1, -2) * d ** -0.5, hidden, v)
    out = out.reshape(batch, hk, drafts, hq // hk, d).transpose(1, 2).reshape(batch, drafts, hq, d)
    used = torch.arange(drafts, device=DEV) < s["drafted"][:, None]
    return torch.where(used[:, :, None, None], out, 0.0).bfloat16()


def _free(s, seqs, keep):
    page = s["case"]["page"]
    seqs = seqs.long()
    left = torch.minimum(keep, s["lens"][seqs])
    pages = (left + page - 1) // page
    at = torch.arange(s["table"].shape[1], device=DEV)
    table = s["table"][seqs]
    gone = (at >= pages[:, None]) & (at < s["counts"][seqs][:, None])
    s["refs"].index_add_(0, table.clamp_min(0).flatten().long(), -gone.flatten().int())
    s["table"][seqs] = torch.where(gone, -1, table)
    s["counts"][seqs], s["lens"][seqs] = pages.int(), left


def _fork(s, pairs):
    page, (a, b) = s["case"]["page"], pairs.long().unbind(1)
    pages = (s["lens"][a] + page - 1) // page
    held = torch.arange(s["table"].shape[1], device=DEV) < pages[:, None]
    table = torch.where(held, s["table"][a], -1)
    s["refs"].index_add_(0, table.clamp_min(0).flatten().long(), held.flatten().int())
    s["table"][b], s["counts"][b], s["lens"][b] = table, pages, s["lens"][a]


def _reserve(s, new):
    """Pages for `new` more tokens of each sequence, lowest free ones first; a page that
    others hold too is copied before a sequence writes into it.  Gives the tokens' rows."""
    page, lens, counts, table, refs = s["case"]["page"], s["lens"], s["counts"], s["table"], s["refs"]
    n = table.shape[0]
    at = torch.arange(table.shape[1], device=DEV)
    last = (lens // page).long()
    old = table.gather(1, last.clamp_max(table.shape[1] - 1)[:, None])[:, 0].clamp_min(0).long()
    shared = (new > 0) & (lens % page > 0) & (last < counts) & (refs[old] > 1)
    need = ((lens + new + page - 1) // page - counts).clamp_min(0)
    want = need + shared.int()
    first = want.cumsum(0) - want
    free = torch.argsort((refs != 0).int(), stable=True).int()
    copied = shared[:, None] & (at == last[:, None])
    fresh = (at >= counts[:, None]) & (at < (counts + need)[:, None])
    rank = torch.where(copied, first[:, None], first[:, None] + shared[:, None] + at - counts[:, None])
    taken = copied | fresh
    picked = free[rank.clamp(0, free.numel() - 1).long()]
    s["table"].copy_(torch.where(taken, picked, table))
    refs.index_add_(0, old, -shared.int())
    refs.index_add_(0, picked.flatten().long(), taken.flatten().int())
    counts += need
    i = torch.arange(page, device=DEV)
    target = s["table"].gather(1, last.clamp_max(table.shape[1] - 1)[:, None]).long()
    row = shared[:, None] & (i < (lens % page)[:, None])
    to, source = (target * page + i)[row], (old[:, None] * page + i)[row]
    c = s["cache"]
    c[0][to], c[1][to], c[2][to], c[3][to] = c[0][source], c[1][source], c[2][source], c[3][source]
    j = torch.arange(s["slots"].shape[1], device=DEV)
    where = (lens[:, None] + j).long()
    slots = s["table"].gather(1, (where // page).clamp_max(table.shape[1] - 1)) * page + where % page
    s["slots"].copy_(torch.where(j < new[:, None], slots, -1))
    s["short"].zero_()


def _append(s):
    slots = s["slots"].flatten().long()
    used = slots >= 0
    kc, ks, vc, vs = s["cache"]
    kc[slots[used]], ks[slots[used]] = _mx_quantize(s["new_k"][used])
    vc[slots[used]], vs[slots[used]] = _mx_quantize(s["new_v"][used])


def _compact(s, accepted, n_accepted):
    page, width = s["case"]["page"], accepted.shape[1]
    j = torch.arange(width, device=DEV)
    used = j < n_accepted[:, None]
    where = torch.stack([s["lens"][:, None] + accepted.clamp_min(0), s["lens"][:, None] + j]).long()
    table = s["table"][None].expand(2, -1, -1)
    rows = table.gather(2, (where // page).clamp_max(table.shape[2] - 1)) * page + where % page
    source, to = rows[0][used].long(), rows[1][used].long()
    c = s["cache"]
    c[0][to], c[1][to], c[2][to], c[3][to] = c[0][source], c[1][source], c[2][source], c[3][source]
    s["lens"] += n_accepted


def _copy(s):
    page, (a, b) = s["case"]["page"], (s["from"].long(), s["to"].long())
    f, t = s["source"], [c.view(-1, page, c.shape[1]) for c in s["target"]]
    t[0][b], t[1][b] = f[0].view(-1, page, f[0].shape[1])[a], f[1].view(-1, page, f[1].shape[1])[a]
    t[2][b], t[3][b] = f[2].view(-1, page, f[2].shape[1])[a], f[3].view(-1, page, f[3].shape[1])[a]


def _state(s):
    return [s["table"], s["counts"], s["lens"], s["refs"], s["slots"], s["short"], *s["cache"]]


# ------------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "norm_rope":
        cos, sin = s["cos_sin"][s["positions"].long()].unsqueeze(1).chunk(2, -1)
        return [_norm_rope(s["q"], s["q_weight"], cos, sin, s["case"]["interleaved"]),
                _norm_rope(s["k"], s["k_weight"], cos, sin, s["case"]["interleaved"])]
    if op == "prompt":
        parts = [_prompt(*t) for t in zip(*(s[x][:sum(s["lens"])].split(s["lens"]) for x in "qkv")) if t[0].shape[0]]
        return torch.cat([*parts, torch.zeros_like(s["out"][sum(s["lens"]):])])
    if op == "tree":
        return _tree(s)
    if op == "copy":
        _copy(s)
        return list(s["target"])
    if op == "speculate":
        _free(s, s["seqs"], s["base"])
        _reserve(s, s["drafted"])
        _append(s)
        _compact(s, s["accepted"], s["n_accepted"])
    else:
        _free(s, s["samples"], torch.zeros_like(s["samples"]))
        _fork(s, s["pairs"])
        _reserve(s, s["drafted"])
        _append(s)
    return _state(s)


def _run_own(s):
    import block_scaled_fp4_mx_amd as F

    op = s["case"]["op"]
    if op == "norm_rope":
        F.fp4_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["cos_sin"],
                           q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=s["case"]["interleaved"])
        return [s["q_out"], s["k_out"]]
    if op == "prompt":
        F.fp4_attn_prompt(s["q"], s["k"], s["v"], s["cu"], s["out"])
        return s["out"]
    page = s["case"]["page"]
    if op == "tree":
        cache = F.KvCache(s["kc"], s["ks"], s["vc"], s["vs"], page)
        if "ws" not in s:
            s["ws"] = torch.empty(F.fp4_attn_tree_workspace_bytes(*s["q"].shape, s["case"]["kv_heads"]),
                                  dtype=torch.uint8, device=DEV)
        F.fp4_attn_tree_mx(s["q"], cache, s["table"], s["lens"], s["out"], s["ws"], draft_lens=s["drafted"],
                           tree_mask=s["masks"])
        return s["out"]
    if op == "copy":
        F.fp4_kv_copy_pages(F.KvCache(*s["source"], page), F.KvCache(*s["target"], page), s["from"], s["to"])
        return list(s["target"])
    cache = F.KvCache(*s["cache"], page)
    pages = F.KvPages(s["table"], s["counts"], s["lens"], s["refs"])
    if "ws" not in s:
        s["ws"] = torch.empty(F.fp4_kv_reserve_workspace_bytes(s["table"].shape[0], s["refs"].numel()),
                              dtype=torch.uint8, device=DEV)
    if op == "speculate":
        F.fp4_kv_free(pages, s["seqs"], page, keep_lens=s["base"])
    else:
        F.fp4_kv_free(pages, s["samples"], page)
        F.fp4_kv_fork(pages, s["pairs"], page)
    F.fp4_kv_reserve(cache, pages, s["drafted"], s["slots"], s["short"], s["ws"])
    F.fp4_kv_append_mx(s["new_k"], s["slots"].view(-1), cache.k_codes, cache.k_scales)
    F.fp4_kv_append_mx(s["new_v"], s["slots"].view(-1), cache.v_codes, cache.v_scales)
    if op == "speculate":
        F.fp4_kv_compact(cache, pages, s["accepted"], s["n_accepted"])
    return _state(s)


# ------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "norm_rope":
        heads = (case["q_heads"] + case["kv_heads"]) * case["tokens"]
        table = case["tokens"] * (4 * case["rot_dim"] + 4)
        weights = 2 * case["head_dim"] * (4 if case["w_f32"] else 2)
        return {"bytes": 4 * heads * case["head_dim"] + table + weights,
                "flops": heads * (4 * case["head_dim"] + 3 * case["rot_dim"])}
    if op == "prompt":
        lens = _lens(case, case["seqs"])
        width = 2 * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * width * sum(lens) + 4 * (len(lens) + 1), "flops": 4 * case["head_dim"] * case["q_heads"] * pairs}
    if op == "tree":
        tokens = sum(n + case["drafts"] for n in _lens(case, case["batch"]))
        row = case["kv_heads"] * case["head_dim"] * 17 // 32
        q = case["batch"] * case["drafts"] * case["q_heads"] * case["head_dim"]
        return {"bytes": 2 * row * tokens + 4 * q + 8 * case["batch"] * case["drafts"] + 4 * (tokens // case["page"]),
                "flops": 4 * case["drafts"] * case["q_heads"] * case["head_dim"] * tokens}
    row = 2 * (case["d"] * 17 // 32)                                   # a token's keys and values
    if op == "copy":
        return {"bytes": 2 * row * case["page"] * case["pages"] + 8 * case["pages"], "flops": 0}
    if op == "speculate":
        lens = _lens(case, case["batch"])
        pages = sum(-(-n // case["page"]) for n in lens)
        new = case["batch"] * case["drafts"]
        return {"bytes": new * (4 * case["d"] + row) + new * row // 2 + 4 * pages + 40 * case["batch"], "flops": 8 * new * case["d"]}
    lens = _lens(case, case["parents"])
    copied = sum(n % case["page"] for n in lens) * case["children"]
    pages = sum(-(-n // case["page"]) for n in lens)
    new = case["parents"] * case["children"]
    return {"bytes": 2 * row * copied + new * (4 * case["d"] + row) + 4 * pages * (1 + 4 * case["children"]),
            "flops": 8 * new * case["d"]}


# ------------------------------------------------------------------------ exact

def exact(case, seed):
    op = case["op"]
    if op == "norm_rope":
        s = prepare(case, seed)
        half = case["rot_dim"] // 2
        row = s["cos_sin"].double()[s["positions"].long()]
        turn = torch.complex(row[:, :half], row[:, half:])[:, None]
        outs = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            y = x.double()
            y = w.double() * y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / case["head_dim"] + EPS)
            first = slice(0, 2 * half, 2) if case["interleaved"] else slice(0, half)
            second = slice(1, 2 * half, 2) if case["interleaved"] else slice(half, 2 * half)
            z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn
            y[..., first], y[..., second] = z.real, z.imag
            outs.append(y)
        return outs
    if op == "prompt":
        s = prepare(case, seed)
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        per, start = case["q_heads"] // case["kv_heads"], 0
        for n in s["lens"]:
            at = torch.arange(n, device=DEV)
            for h in range(case["q_heads"] if n else 0):
                q, k, v = (s[x][start:start + n, i].double() for x, i in (("q", h), ("k", h // per), ("v", h // per)))
                logits = torch.mm(q, k.t().contiguous()) / math.sqrt(case["head_dim"])
                logits.masked_fill_(at[None] > at[:, None], -math.inf)
                out[start:start + n, h] = torch.softmax(logits, 1) @ v
            start += n
        return out
    if op == "tree":
        s = prepare(case, seed)
        page, per, d = case["page"], case["q_heads"] // case["kv_heads"], case["head_dim"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
        value = torch.tensor(np.concatenate([grid, -grid]), device=DEV)
        masks, drafted, lens = (s[x].cpu().tolist() for x in ("masks", "drafted", "lens"))
        for b, n in enumerate(lens):
            t = drafted[b]
            at = torch.arange(n + t, device=DEV)
            rows = s["table"][b].long()[at // page] * page + at % page
            kv = []
            for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
                two = torch.stack([value[(codes[rows] % 16).long()], value[(codes[rows] // 16).long()]], 2)
                scale = torch.pow(2.0, scales[rows].double() - 127)
                kv.append(two.reshape(n + t, -1) * scale.repeat_interleave(32, 1))
            bits = [[(masks[b][i] >> j) & 1 == 0 for j in range(t)] for i in range(t)]
            hidden = torch.zeros(t, n + t, dtype=torch.bool, device=DEV)
            hidden[:, n:] = torch.tensor(bits, device=DEV)
            for h in range(case["q_heads"]):
                cols = slice(h // per * d, (h // per + 1) * d)
                logits = torch.mm(s["q"][b, :t, h].double(), kv[0][:, cols].t().contiguous()) / math.sqrt(d)
                out[b, :t, h] = torch.softmax(logits.masked_fill(hidden, -math.inf), 1) @ kv[1][:, cols]
        return out
    return None                                                        # rows and indices, nothing computed
