"""GPU parity of the attention of drafted tokens over the paged MXFP4 cache
(fp4_attn_tree_mx) with the float64 definition; tolerance in attn_check.py."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
import workloads as W
from attn_check import check, norm
from gpu_util import DEV
from oracle import attn as A
from oracle import quant as Q

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Step:
    """Queries, a cache of quantized normal vectors and a shuffled page table."""

    def __init__(self, seed, lens, drafts, q_heads, kv_heads, d, page_size, draft_lens=None, masks=None, spare=2, width=0):
        rng = np.random.default_rng(seed)
        self.lens, self.drafts, self.heads, self.d, self.ps = list(lens), drafts, (q_heads, kv_heads), d, page_size
        batch = len(self.lens)
        counts = [-(-(max(n, 0) + drafts) // page_size) for n in self.lens]
        pages = sum(counts) + spare
        width = max(width, max(counts))
        order = rng.permutation(pages)
        self.table, at = np.full((batch, width), -1, np.int32), 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        kv = W.bf16_bits(W.to_bf16(rng.standard_normal((2, pages * page_size, kv_heads * d)) *
                                   np.exp2(rng.integers(-2, 3, (2, pages * page_size, 1)))))
        self.kc, self.ks = Q.mx_quantize(kv[0])
        self.vc, self.vs = Q.mx_quantize(kv[1])
        self.q = W.bf16_bits(W.to_bf16(rng.standard_normal((batch, drafts, q_heads, d))))
        self.draft_lens, self.masks = draft_lens, masks

    def device(self):
        t = lambda a: torch.from_numpy(a.copy()).to(DEV)
        return dict(q=W.from_bits(self.q).to(DEV), cache=F.KvCache(t(self.kc), t(self.ks), t(self.vc), t(self.vs), self.ps),
                    page_table=t(self.table), seq_lens=_i32(self.lens),
                    out=torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device=DEV),
                    workspace=torch.full((F.fp4_attn_tree_workspace_bytes(*self.q.shape, self.heads[1]),), 0xFF,
                                         dtype=torch.uint8, device=DEV),
                    draft_lens=None if self.draft_lens is None else _i32(self.draft_lens),
                    tree_mask=None if self.masks is None else
                    torch.from_numpy(self.masks.astype(np.uint64).view(np.int64)).to(DEV))

    def check(self, out, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        ref, size = A.attn_tree_mx(self.q, self.kc, self.ks, self.vc, self.vs, self.ps, self.table, self.lens, self.heads[1],
                                   scale, self.draft_lens, self.masks)
        k = Q.mx_dequant_f64(self.kc, self.ks).reshape(-1, self.d)
        v = Q.mx_dequant_f64(self.vc, self.vs)
        check(out, ref, size, self.d, max(self.lens) + self.drafts, scale, norm(self.q), float(np.sqrt((k * k).sum(-1)).max()),
              np.abs(v).max())
        untouched = out.cpu().float().numpy()[np.isnan(ref)]
        assert (untouched == 7.0).all()

    def run(self, scale=None):
        a = self.device()
        F.fp4_attn_tree_mx(**a, scale=scale)
        self.check(a["out"], scale)
        return a


def _tree(seed, batch, drafts):
    rng = np.random.default_rng(seed)
    m = np.zeros((batch, drafts), np.uint64)
    for b in range(batch):
        for i in range(drafts):
            m[b, i] = (m[b, rng.integers(max(0, i - 4), i)] if i else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
    return m


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,drafts", [(1, 1, 1), (8, 1, 1), (4, 4, 3), (10, 2, 5), (16, 8, 1)])
def test_shapes(d, q_heads, kv_heads, drafts):
    Step(d + q_heads, [0, 1, 31, 32, 33, 200], drafts, q_heads, kv_heads, d, 16).run()


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 112, 256])
def test_pages_that_end_inside_a_step(page_size):
    Step(page_size, [page_size - 1, page_size, page_size + 1, 5 * page_size + 17], 2, 8, 2, 128, page_size).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 8, 2, 1), (128, 8, 1, 1), (128, 16, 2, 8), (256, 4, 2, 3)])
def test_long_contexts_split_over_workgroups(d, q_heads, kv_heads, drafts):
    Step(d, [9001], drafts, q_heads, kv_heads, d, 64).run()


def test_ragged_batch_split_and_whole():
    """Sequences that ranges cut, several to a range, and ranges of several sequences."""
    lens = [3000, 0, 5, 64, 2049, 1, 900, 0, 0, 40, 31, 777]
    Step(1, lens, 4, 8, 8, 64, 32, masks=_tree(1, len(lens), 4)).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 24, 12, 9), (128, 16, 8, 9), (128, 12, 6, 4), (128, 15, 5, 2),
                                                       (256, 8, 4, 4), (256, 10, 10, 3)])
def test_ragged_batches_of_other_heads(d, q_heads, kv_heads, drafts):
    lens = [1700, 0, 5, 64, 2049, 1, 300, 0, 0, 40, 31, 777]
    Step(d + drafts, lens, drafts, q_heads, kv_heads, d, 32, masks=_tree(2, len(lens), drafts)).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 8, 4, 2), (128, 8, 8, 4), (128, 32, 4, 5), (256, 8, 4, 1)])
def test_one_long_context_in_many_pieces(d, q_heads, kv_heads, drafts):
    Step(d, [17003], drafts, q_heads, kv_heads, d, 128).run()


def test_more_sequences_than_lanes():
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 130, 150).tolist()
    draft_lens = rng.integers(0, 3, 150).tolist()
    Step(2, lens, 2, 4, 2, 64, 16, draft_lens=draft_lens).run()


@pytest.mark.parametrize("d,drafts", [(64, 64), (128, 64), (128, 33), (256, 17)])
def test_trees(d, drafts):
    Step(drafts, [100, 0, 31], drafts, 16, 2, d, 48, masks=_tree(drafts, 3, drafts)).run()


def test_rows_that_see_nothing_and_bits_behind_the_last_draft():
    masks = np.array([[0, 1, 2, 0], [0, 0, 0, 0], [~np.uint64(0)] * 4], np.uint64)
    s = Step(4, [0, 0, 37], 4, 8, 2, 64, 16, draft_lens=[3, 4, 2], masks=masks)
    out = s.run()["out"]
    assert (out[0, 0] == 0).all() and (out[1] == 0).all()


def test_what_is_not_seen_may_hold_anything():
    """Scale bytes 255 and 0xFF codes behind every sequence, on free pages and in hidden drafts' place."""
    s = Step(5, [5, 70, 16], 3, 4, 2, 128, 16, draft_lens=[1, 2, 0], spare=4)
    rows = np.ones(len(s.kc), bool)
    for b, (n, t) in enumerate(zip(s.lens, s.draft_lens)):
        rows[A.cache_rows(s.table[b], 16, len(s.kc) // 16, n + t)] = False
    for c, e in ((s.kc, s.ks), (s.vc, s.vs)):
        c[rows], e[rows] = 0xFF, 0xFF
    s.run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 4, 2, 6), (128, 16, 2, 6), (128, 8, 8, 9), (256, 4, 4, 5)])
def test_drafted_values_past_the_range_reach_only_rows_that_see_them(d, q_heads, kv_heads, drafts):
    """Blocks of drafted values with the largest scales: infinite in bf16 (code 7 at
    2^126), near the end of its range (code 1) and no number (scale byte 255), in a
    sequence of one piece and in one of several; rows that do not see them, and other
    values of those that do, are as without."""
    lens = [40, 2500]
    s = Step(11, lens, drafts, q_heads, kv_heads, d, 64, masks=_tree(11, 2, drafts))
    group, odd = q_heads // kv_heads, []
    for b, n in enumerate(lens):
        for token, block, code, scale in ((1, 0, 0x77, 253), (2, 1, 0x11, 253), (drafts - 1, kv_heads * d // 32 - 1, 0x22, 255)):
            row = A.cache_rows(s.table[b], 64, len(s.kc) // 64, n + drafts)[n + token]
            s.vc[row, 16 * block:16 * block + 16], s.vs[row, block] = code, 0
            odd.append((b, token, block, row, scale))
    a = s.device()
    for *_, block, row, scale in odd:
        a["cache"].v_scales[row, block] = scale
    F.fp4_attn_tree_mx(**a)
    ref, size = A.attn_tree_mx(s.q, s.kc, s.ks, s.vc, s.vs, 64, s.table, lens, kv_heads, d ** -0.5, None, s.masks)
    got = a["out"].cpu().float().numpy()
    k_norm = float(np.sqrt((Q.mx_dequant_f64(s.kc, s.ks).reshape(-1, d) ** 2).sum(-1)).max())
    for b, token, block, row, scale in odd:
        head, at = block * 32 // d, block * 32 % d
        heads, values = slice(head * group, (head + 1) * group), slice(at, at + 32)
        sees = np.array([int(s.masks[b, i]) >> token & 1 for i in range(drafts)], bool)
        assert sees.any() and not sees.all()
        if token == 2:                                       # finite: its own reference and magnitudes
            s.vs[row, block] = scale
            r, z = A.attn_tree_mx(s.q, s.kc, s.ks, s.vc, s.vs, 64, s.table, lens, kv_heads, d ** -0.5, None, s.masks)
            s.vs[row, block] = 0
            only = np.full_like(r, np.nan)
            only[b, sees, heads, values] = r[b, sees, heads, values]
            check(a["out"], only, z, d, 2500 + drafts, d ** -0.5, norm(s.q), k_norm, 2.0 ** 125)
        else:
            x = got[b, sees, heads, values]
            assert (x == np.inf).all() if scale == 253 else not np.isfinite(x).any()
        ref[b, sees, heads, values] = np.nan
    check(a["out"], ref, size, d, 2500 + drafts, d ** -0.5, norm(s.q), k_norm, np.abs(Q.mx_dequant_f64(s.vc, s.vs)).max())


def test_cache_offsets_past_32_bits_and_the_end_of_the_workspace():
    """Pages beyond the first 4 GiB of codes, between others; bytes behind the workspace stay."""
    heads, d, ps, pages = 16, 128, 64, 1 << 16               # codes: 4 GiB each
    rng = np.random.default_rng(12)
    s = Step(12, [700, 90], 3, 32, heads, d, ps)
    small = s.device()
    used = len(s.kc) // ps
    far = np.sort(rng.choice(np.arange(pages - 64, pages), used, replace=False))[rng.permutation(used)]
    far[::3] = rng.permutation(np.arange(1, 1 + len(far[::3])))
    big = [torch.empty((pages * ps, x.shape[1]), dtype=torch.uint8, device=DEV) for x in small["cache"][:4]]
    assert pages * ps * heads * d // 2 == 1 << 32
    to, at = _i32(far), torch.arange(used, dtype=torch.int32, device=DEV)
    cache = F.KvCache(*big, ps)
    F.fp4_kv_copy_pages(small["cache"], cache, at, to)
    back = F.KvCache(*(torch.zeros_like(x) for x in small["cache"][:4]), ps)
    F.fp4_kv_copy_pages(cache, back, to, at)
    assert all(torch.equal(x, y) for x, y in zip(back[:4], small["cache"][:4]))
    table = np.where(s.table >= 0, far[np.maximum(s.table, 0)], -1).astype(np.int32)
    size = F.fp4_attn_tree_workspace_bytes(*s.q.shape, heads)
    ws = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    F.fp4_attn_tree_mx(**small | dict(cache=cache, page_table=torch.from_numpy(table).to(DEV), workspace=ws[:size]))
    s.check(small["out"])
    assert (ws[size:] == 0xA5).all()


def test_two_streams_with_a_workspace_each():
    """Calls that run at once; each is as it is alone."""
    steps = [Step(20 + i, [5000 + 700 * i, 10], 2, 8, 2, 128, 32) for i in range(2)]
    args = [s.device() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, stream in zip(args, streams):
            F.fp4_attn_tree_mx(**a, stream=stream)
    torch.cuda.synchronize()
    for s, a in zip(steps, args):
        s.check(a["out"])


def test_ids_outside_the_pool_and_short_tables_are_not_seen():
    s = Step(6, [200, 100, 90, -5], 2, 4, 2, 64, 16)
    s.table[0, 3], s.table[0, 7], s.table[1, 0] = -1, 1 << 30, -9
    s.table = s.table[:, :6].copy()                      # 96 positions; the first two sequences' drafts lie behind them
    s.run()


def test_empty_pool_empty_table_and_empty_batch():
    s = Step(7, [10, 0], 2, 4, 2, 64, 16)
    a = s.device()
    none = torch.zeros((0, 64), dtype=torch.uint8, device=DEV), torch.zeros((0, 4), dtype=torch.uint8, device=DEV)
    F.fp4_attn_tree_mx(**a | dict(cache=F.KvCache(*none, *none, 16)))
    assert (a["out"] == 0).all()
    a = s.device()
    F.fp4_attn_tree_mx(**a | dict(page_table=a["page_table"][:, :0].contiguous()))
    assert (a["out"] == 0).all()
    e = torch.empty((0, 2, 4, 64), dtype=torch.bfloat16, device=DEV)
    F.fp4_attn_tree_mx(e, a["cache"], a["page_table"][:0], a["seq_lens"][:0], e, a["workspace"][:0])


def test_scales_strides_and_large_scores():
    s = Step(8, [300, 65], 3, 8, 2, 128, 64)
    for scale in (0.0, -0.3, 2.0):                       # 2.0: a few tokens take all the weight
        s.run(scale)
    a = s.device()
    wide = torch.full((2, 3, 12, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    qw = wide.clone()
    qw[:, :, :8] = a["q"]
    F.fp4_attn_tree_mx(**a | dict(q=qw[:, :, :8], out=wide[:, :, 2:10]))
    s.check(wide[:, :, 2:10])
    assert (wide[:, :, :2] == 7).all() and (wide[:, :, 10:] == 7).all()


def test_rising_scores_move_the_reference():
    """Keys that grow along the sequence, so the running reference moves many times, and one far outlier."""
    s = Step(9, [700], 2, 4, 2, 64, 16)
    grow = np.repeat(np.linspace(110, 131, 45).astype(np.uint8), 16)
    rows = A.cache_rows(s.table[0], 16, len(s.kc) // 16, 702)
    s.ks[rows] = grow[:702, None]
    s.run(0.05)


def test_same_call_same_bits():
    s = Step(10, [5000, 300, 40], 4, 16, 4, 128, 64)
    a = s.run()
    first = a["out"].clone()
    for _ in range(3):
        a["workspace"].fill_(0xFF)
        F.fp4_attn_tree_mx(**a)
        assert torch.equal(first.view(torch.int16), a["out"].view(torch.int16))


def test_side_stream_and_replayed_graph_with_growing_lengths():
    """Captured once; the lengths, the queries and the table change between replays."""
    s = Step(11, [400, 90, 1000], 2, 8, 2, 128, 32, width=40)
    a = s.device()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        F.fp4_attn_tree_mx(**a)
    torch.cuda.current_stream().wait_stream(side)
    s.check(a["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp4_attn_tree_mx(**a)
    for k, lens in enumerate(([400, 90, 1000], [1, 2, 3], [400, 0, 17], [390, 91, 999])):
        s.lens = lens
        s.q = W.bf16_bits(W.to_bf16(np.random.default_rng(k).standard_normal(s.q.shape)))
        a["seq_lens"].copy_(_i32(lens))
        a["q"].copy_(W.from_bits(s.q))
        a["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        s.check(a["out"])
        torch.ones(1000, device=DEV).sum().item()
