"""Plain definitions of the attention path: head norms with rotation, causal
attention over packed prompts, attention of drafted tokens over a paged MXFP4
cache, all in float64, and the cache's pages as ordinary Python loops.

Cache layout and the stored values are oracle.quant's (MXFP4 rows).
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import quant as Q


# ------------------------------------------------------------- norms and rotation

def norm_rope(xbits, weight, eps, cos_sin, positions, interleaved):
    """xbits uint16 [tokens, heads, d] (bf16); weight float64 [d]; cos_sin
    [places, rot] or None.  Returns (y, size): the float64 result and, for each
    value, the sum of the magnitudes of the terms it is made of.  Rows of
    positions outside the table come back as NaN (nothing is written there)."""
    x = F.bf16_bits_to_f64(xbits)
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight
    size = np.abs(y)
    if cos_sin is None:
        return y, size
    half = cos_sin.shape[1] // 2
    out, size = y.copy(), size.copy()
    for t, pos in enumerate(positions):
        if not 0 <= pos < len(cos_sin):
            out[t] = np.nan
            continue
        for i in range(half):
            c, s = float(cos_sin[pos, i]), float(cos_sin[pos, half + i])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            size[t, :, a] = np.abs(y[t, :, a] * c) + np.abs(y[t, :, b] * s)
            size[t, :, b] = np.abs(y[t, :, b] * c) + np.abs(y[t, :, a] * s)
    return out, size


# ---------------------------------------------------------------------- attention

def attend(q, k, v, visible, scale):
    """q [m, d], k and v [n, d] float64, visible bool [m, n].  Returns (o, size):
    softmax-weighted sums and the weighted sums of |v|; rows that see nothing
    are zero."""
    s = np.where(visible, scale * (q @ k.T), -np.inf)
    with np.errstate(invalid="ignore"):
        p = np.exp(s - np.max(s, axis=1, keepdims=True, initial=-1e300))
    p = np.where(visible, p, 0.0)
    total = p.sum(axis=1, keepdims=True)
    p = p / np.where(total > 0, total, 1.0)
    v = np.where(visible.any(axis=0)[:, None], v, 0.0)
    return p @ v, p @ np.abs(v)


def attn_prompt(qbits, kbits, vbits, cu, scale):
    """Causal attention inside each sequence [cu[s], cu[s+1]); bf16 bits
    [tokens, heads, d].  Rows outside every sequence are NaN."""
    q, k, v = (F.bf16_bits_to_f64(b) for b in (qbits, kbits, vbits))
    group = q.shape[1] // k.shape[1]
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for a, b in zip(cu[:-1], cu[1:]):
        n = b - a
        for h in range(q.shape[1] if n > 0 else 0):
            out[a:b, h], size[a:b, h] = attend(q[a:b, h], k[a:b, h // group], v[a:b, h // group],
                                               np.tril(np.ones((n, n), bool)), scale)
    return out, size


def cache_rows(table_row, page_size, num_pages, n):
    """Cache rows of positions 0..n-1, -1 where the table names no page of the pool."""
    rows = np.full(n, -1, np.int64)
    for i in range(n):
        p = i // page_size
        page = table_row[p] if p < len(table_row) else -1
        if 0 <= page < num_pages:
            rows[i] = int(page) * page_size + i % page_size
    return rows


def attn_tree_mx(qbits, kc, ks, vc, vs, page_size, table, seq_lens, kv_heads, scale, draft_lens=None, tree_mask=None):
    """qbits uint16 [batch, drafts, q_heads, d].  Rows i >= draft_lens[b] are NaN."""
    q = F.bf16_bits_to_f64(qbits)
    batch, drafts, q_heads, d = q.shape
    group = q_heads // kv_heads
    out, size = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(batch):
        t = drafts if draft_lens is None else min(max(int(draft_lens[b]), 0), drafts)
        n = max(int(seq_lens[b]), 0)
        rows = cache_rows(table[b], page_size, len(kc) // page_size, n + t)
        live = rows >= 0
        k = Q.mx_dequant_f64(kc[np.maximum(rows, 0)], ks[np.maximum(rows, 0)]).reshape(-1, kv_heads, d)
        v = Q.mx_dequant_f64(vc[np.maximum(rows, 0)], vs[np.maximum(rows, 0)]).reshape(-1, kv_heads, d)
        visible = np.tile(live, (t, 1))
        for i in range(t):
            for j in range(t):
                seen = j <= i if tree_mask is None else (int(tree_mask[b, i]) >> j) & 1
                visible[i, n + j] &= bool(seen)
        for h in range(q_heads):
            out[b, :t, h], size[b, :t, h] = attend(q[b, :t, h], k[:, h // group], v[:, h // group], visible, scale)
    return out, size


# -------------------------------------------------------------------------- pages

class Pages:
    """The page state and the cache it speaks of, on the host.  arrays: the
    cache's row arrays (codes and scales of keys and values).  Page ids outside the
    pool, counts outside the table's rows and negative lengths are not followed."""

    def __init__(self, table, counts, lens, refs, page_size, arrays):
        self.table, self.counts, self.lens, self.refs = (np.array(a) for a in (table, counts, lens, refs))
        self.page_size, self.arrays = page_size, [np.array(a) for a in arrays]

    def pages_of(self, n):
        return -(-int(n) // self.page_size)

    def held(self, b):
        return min(max(int(self.counts[b]), 0), self.table.shape[1])

    def inside(self, page):
        return 0 <= page < len(self.refs)

    def row(self, b, pos):
        page = int(self.table[b, pos // self.page_size])
        return page * self.page_size + pos % self.page_size if self.inside(page) else -1

    def reserve(self, new, max_new):
        """Returns (slots, short)."""
        batch, width = self.table.shape
        slots = np.full((batch, max_new), -1, np.int32)
        jobs, short, wanted = [], 0, 0
        for b in range(batch):
            n, add = max(int(self.lens[b]), 0), max(int(new[b]), 0)
            if add == 0:
                continue
            pages = self.pages_of(n + add)
            short += max(pages - width, 0)
            last = n // self.page_size
            shared = (n % self.page_size > 0 and last < self.held(b) and self.inside(self.table[b, last]) and
                      self.refs[self.table[b, last]] > 1)
            need = max(min(pages, width) - self.held(b), 0)
            wanted += need + shared
            jobs.append((b, n, add, last, shared, need))
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        short += max(wanted - len(free), 0)
        if short:
            return slots, short
        for b, n, add, last, shared, need in jobs:
            if shared:
                old, page = int(self.table[b, last]), free.pop(0)
                for a in self.arrays:
                    for i in range(n % self.page_size):
                        a[page * self.page_size + i] = a[old * self.page_size + i]
                self.table[b, last] = page
                self.refs[old] -= 1
                self.refs[page] = 1
            self.counts[b] = self.held(b)
            for _ in range(need):
                page = free.pop(0)
                self.table[b, self.counts[b]] = page
                self.counts[b] += 1
                self.refs[page] = 1
            for j in range(min(add, max_new)):
                slots[b, j] = self.row(b, n + j)
        return slots, 0

    def fork(self, pairs):
        batch = len(self.table)
        targets = [int(t) for _, t in pairs]
        for i, (s, t) in enumerate(pairs):
            if not (0 <= s < batch and 0 <= t < batch) or t in targets[:i] or s in targets or self.counts[t]:
                continue
            n = min(self.pages_of(max(int(self.lens[s]), 0)), self.held(s))
            self.table[t, :n] = self.table[s, :n]
            for p in self.table[s, :n]:
                if self.inside(p):
                    self.refs[p] += 1
            self.counts[t], self.lens[t] = n, min(max(int(self.lens[s]), 0), n * self.page_size)

    def free(self, seqs, keep=None):
        for i, b in enumerate(seqs):
            if not 0 <= b < len(self.table) or b in list(seqs[:i]):
                continue
            n = min(max(int(self.lens[b]), 0), 0 if keep is None else max(int(keep[i]), 0))
            kept = min(self.pages_of(n), self.held(b))
            for p in range(kept, self.held(b)):
                if self.inside(self.table[b, p]):
                    self.refs[self.table[b, p]] -= 1
                self.table[b, p] = -1
            self.counts[b], self.lens[b] = kept, min(n, kept * self.page_size)

    def may_write(self, b, page, lens, commits):
        """Whether sequence b may move rows onto a page: it holds it alone, or it is the
        page of its first uncommitted row, and no other holder's tokens reach as far,
        nor does another holder commit in the same call."""
        if self.refs[page] == 1:
            return True
        last = lens[b] // self.page_size
        if lens[b] % self.page_size == 0 or self.table[b, last] != page:
            return False
        return not any(o != b and last < self.held(o) and self.table[o, last] == page and
                       (commits[o] or lens[o] > lens[b]) for o in range(len(self.table)))

    def compact(self, accepted, accepted_lens, slots=None):
        """slots: of the reservation that gave the rows; what it did not grant stays uncommitted."""
        lens = [max(int(n), 0) for n in self.lens]
        commits = [n > 0 and (slots is None or slots[o][0] >= 0) for o, n in enumerate(accepted_lens)]
        for b, n in enumerate(lens):
            room = max(self.held(b) * self.page_size - n, 0)
            m = max(int(accepted_lens[b]), 0)
            if accepted is not None:
                m = min(m, accepted.shape[1])
            m = min(m, room)
            if slots is not None:
                rows = [self.row(b, n + i) for i in range(min(room, slots.shape[1]))]
                given = [i < len(rows) and int(slots[b][i]) == rows[i] >= 0 for i in range(slots.shape[1])]
                m = min(m, (given + [False]).index(False))
            moves = []
            for i in range(m if accepted is not None else 0):
                j = int(accepted[b, i])
                if 0 <= j < room and j != i and (slots is None or (j < len(given) and given[j])):
                    source, to = self.row(b, n + j), self.row(b, n + i)
                    if source >= 0 and to >= 0 and self.may_write(b, to // self.page_size, lens, commits):
                        moves.append((source, to))
            for a in self.arrays if moves else []:
                source, to = np.array(moves).T
                a[to] = a[source]
            if m:
                self.lens[b] = n + m
