"""GPU parity of the attention of sequences that share prefixes (fp4_attn_shared_mx)
with the float64 definition of the attention over each sequence's own table;
tolerance in attn_check.py (the parts that are joined are within its sums' share)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
from gpu_util import DEV
from oracle import attn as A
from test_gpu_attn_tree import Step, _i32, _tree

pytestmark = pytest.mark.gpu


class Shared(Step):
    """groups: (sequences, tokens of the prefix); lens are whole lengths.  The pages that lie
    wholly in a prefix are the group's first sequence's; the others hold the same rows."""

    def __init__(self, seed, groups, lens, drafts, q_heads, kv_heads, d, page_size, before=0, **kw):
        super().__init__(seed, lens, drafts, q_heads, kv_heads, d, page_size, **kw)
        self.bounds = np.cumsum([before] + [n for n, _ in groups]).astype(np.int32)
        self.prefix = np.array([p for _, p in groups], np.int32)
        for (n, p), first in zip(groups, self.bounds):
            rows = A.cache_rows(self.table[first], page_size, len(self.kc) // page_size, p)
            for b in range(first + 1, first + n):
                if self.lens[b] < p:
                    continue                                        # by itself
                self.table[b, :p // page_size] = self.table[first, :p // page_size]
                own = A.cache_rows(self.table[b], page_size, len(self.kc) // page_size, p)
                for x in (self.kc, self.ks, self.vc, self.vs):
                    x[own] = x[rows]

    def device(self):
        batch, drafts = self.q.shape[:2]
        need = F.fp4_attn_shared_workspace_bytes(batch, drafts, self.heads[0], self.d, self.heads[1], len(self.prefix))
        return super().device() | dict(groups=_i32(self.bounds), prefix_lens=_i32(self.prefix),
                                       workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV))

    def run(self, scale=None):
        a = self.device()
        F.fp4_attn_shared_mx(**a, scale=scale)
        self.check(a["out"], scale)
        return a


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,drafts", [(1, 1, 1), (8, 1, 1), (4, 4, 3), (10, 2, 5), (16, 8, 1), (24, 12, 2)])
def test_shapes(d, q_heads, kv_heads, drafts):
    Shared(d + q_heads, [(3, 96), (1, 32), (2, 65)], [96, 130, 97, 50, 65, 80], drafts, q_heads, kv_heads, d, 16).run()


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 112])
@pytest.mark.parametrize("prefix", [0, 1, 31, 32, 33, 63, 64, 100, 257])
def test_prefixes_that_end_anywhere(prefix, page_size):
    Shared(prefix, [(4, prefix)], [prefix, prefix + 1, prefix + 40, prefix + 129], 2, 8, 2, 128, page_size).run()


@pytest.mark.parametrize("members", [1, 2, 7, 33, 70])
@pytest.mark.parametrize("d,q_heads,kv_heads", [(64, 5, 1), (128, 8, 4), (256, 6, 2)])
def test_rows_of_many_sequences(members, d, q_heads, kv_heads):
    rng = np.random.default_rng(members)
    Shared(members, [(members, 200)], (200 + rng.integers(0, 60, members)).tolist(), 1, q_heads, kv_heads, d, 16).run()


def test_sequences_outside_groups_and_empty_groups():
    lens = [40, 300, 0, 128, 140, 200, 64, 65, 500, 20, 0]
    x = Shared(1, [(0, 50), (3, 128), (0, 7), (2, 64)], lens, 2, 4, 2, 64, 16, before=3)
    x.run()
    x.bounds[:] = 0                                         # all groups empty
    x.run()


def test_sequences_shorter_than_their_prefix():
    Shared(2, [(4, 160), (3, 96)], [200, 10, 159, 160, 95, 300, 0], 3, 8, 2, 128, 32, draft_lens=[3, 2, 3, 1, 3, 0, 3]).run()


@pytest.mark.parametrize("groups", [63, 64, 65, 130])
def test_more_groups_than_lanes(groups):
    rng = np.random.default_rng(groups)
    sizes = rng.integers(0, 3, groups)
    spec = [(int(n), int(p)) for n, p in zip(sizes, rng.integers(0, 90, groups))]
    lens = [p + int(rng.integers(0, 40)) for n, p in spec for _ in range(n)] + [5]
    Shared(groups, spec, lens, 1, 2, 1, 64, 16).run()


@pytest.mark.parametrize("groups", [64, 70, 150])
def test_many_rows_of_more_groups_than_lanes(groups):
    rng = np.random.default_rng(groups)
    sizes = rng.integers(0, 3, groups)
    sizes[62:66] = 0                                        # none where the lanes' groups end
    spec = [(int(n), int(p)) for n, p in zip(sizes, rng.integers(0, 200, groups))]
    lens = [p + int(rng.integers(0, 40)) for n, p in spec for _ in range(n)] + [5]
    Shared(groups, spec, lens, 50, 4, 2, 64, 16, masks=_tree(1, len(lens), 50)).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 8, 2, 1), (128, 16, 2, 3), (128, 8, 1, 1), (256, 4, 2, 1)])
def test_long_prefixes_split_over_workgroups(d, q_heads, kv_heads, drafts):
    Shared(d, [(5, 6000)], [6000, 6100, 6001, 7200, 6031], drafts, q_heads, kv_heads, d, 64).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,members", [(64, 6, 1, 40), (64, 4, 2, 40), (128, 4, 1, 70), (128, 4, 2, 40), (256, 3, 1, 40)])
def test_many_rows_over_long_prefixes(d, q_heads, kv_heads, members):
    """More rows than a workgroup has, and tiles and runs of pages that end anywhere."""
    rng = np.random.default_rng(d)
    x = Shared(d, [(members, 1500), (members, 97)], (1500 + rng.integers(0, 40, 2 * members)).tolist(), 1, q_heads, kv_heads, d, 48)
    x.run()
    x.table[:, 3], x.table[:, 17] = -1, 1 << 28             # not seen by any
    x.run(scale=-0.2)


def test_long_own_parts_and_whole_prefixes_in_one_range():
    """Ranges with several whole prefixes, and sequences that ranges cut."""
    lens = [64, 3000, 64, 40, 33, 2049, 70, 96, 100, 1000]
    Shared(3, [(2, 64), (3, 33), (2, 64), (2, 96)], [max(n, 96) for n in lens], 2, 8, 8, 64, 32, masks=_tree(1, len(lens), 2)).run()


@pytest.mark.parametrize("d,drafts", [(64, 64), (128, 33), (256, 17)])
def test_trees(d, drafts):
    Shared(drafts, [(3, 100)], [100, 131, 117], drafts, 4, 2, d, 48, masks=_tree(drafts, 3, drafts)).run()


def test_masks_that_leave_the_own_part_empty():
    masks = np.array([[0, 1], [0, 0], [0, 2]], np.uint64)
    x = Shared(4, [(3, 64)], [64, 64, 64], 2, 4, 2, 64, 16, masks=masks)
    x.run()
    y = Shared(5, [(3, 0)], [0, 0, 0], 2, 4, 2, 64, 16, masks=masks)
    out = y.run()["out"]
    assert (out[1] == 0).all() and (out[0, 0] == 0).all()


def test_no_groups_and_one_sequence_groups_are_the_tree_attention():
    lens = [300, 20, 0, 77]
    x = Shared(6, [], lens, 2, 8, 2, 128, 16)
    a, t = x.run(), Step.device(x)
    F.fp4_attn_tree_mx(**t)
    assert torch.equal(a["out"], t["out"])
    Shared(6, [(1, 256), (1, 20), (1, 0), (1, 33)], lens, 2, 8, 2, 128, 16).run()


def test_bounds_that_do_not_ascend_stay_in_range():
    """Not a meaningful call, but one that reads and writes nothing outside its arrays: whatever
    group a sequence finds, it is one that names it, and its first sequence's table serves."""
    x = Shared(7, [(4, 64)], [70, 90, 100, 64], 1, 4, 2, 64, 16)
    for bounds in ([0, 4, -5], [4, 0, 4], [100, 0, 2], [0, 100, 3]):
        a = x.device()
        a |= dict(groups=_i32(bounds), prefix_lens=_i32([64, 64]))
        a["workspace"] = torch.zeros(F.fp4_attn_shared_workspace_bytes(4, 1, 4, 64, 2, 2), dtype=torch.uint8, device=DEV)
        F.fp4_attn_shared_mx(**a)
        x.check(a["out"])


def test_prefixes_past_the_table_and_negative_ones():
    x = Shared(8, [(2, 60), (2, 40)], [64, 64, 50, 49], 1, 4, 2, 64, 16)
    x.prefix[:] = [-3, 2 ** 31 - 1]
    x.run()                                                 # longer than both: each by itself
    full = x.table.shape[1] * 16
    x.table[2:] = x.table[1]
    x.lens = [64, 64, 2 ** 31 - 1, 2 ** 31 - 1]
    a = x.device()
    F.fp4_attn_shared_mx(**a)
    x.lens = [64, 64, full, full]                           # the drafted tokens have no row either way
    x.check(a["out"])


def test_missing_pages_of_the_prefix_are_not_seen():
    x = Shared(10, [(3, 128)], [150, 128, 200], 1, 8, 4, 128, 16)
    x.table[:3, 2], x.table[:3, 7] = -1, len(x.kc)
    x.run()


def test_what_is_not_seen_may_hold_anything():
    x = Shared(11, [(3, 64)], [70, 64, 90], 2, 4, 2, 128, 16, draft_lens=[1, 2, 0], spare=4)
    rows = np.ones(len(x.kc), bool)
    for b, (n, t) in enumerate(zip(x.lens, x.draft_lens)):
        rows[A.cache_rows(x.table[b], 16, len(x.kc) // 16, n + t)] = False
    for c, e in ((x.kc, x.ks), (x.vc, x.vs)):
        c[rows], e[rows] = 0xFF, 0xFF
    x.run()


def test_rows_of_other_sequences_may_hold_anything():
    """Queries behind a sequence's drafts are no numbers; they stand among the prefix's rows."""
    x = Shared(12, [(4, 96)], [96, 100, 130, 97], 3, 8, 2, 64, 16, draft_lens=[1, 3, 0, 2])
    a = x.device()
    for b, t in enumerate(x.draft_lens):
        a["q"][b, t:] = float("nan")
    F.fp4_attn_shared_mx(**a)
    x.check(a["out"])


def test_negative_scale_and_strided_rows():
    x = Shared(13, [(3, 64)], [100, 65, 64], 2, 8, 2, 64, 16)
    x.run(scale=-0.3)
    a = x.device()
    wide = torch.full((3, 2, 12, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    wide_q = torch.zeros_like(wide)
    wide_q[:, :, 2:10] = a["q"]
    a["q"], a["out"] = wide_q[:, :, 2:10], wide[:, :, 4:]
    F.fp4_attn_shared_mx(**a)
    x.check(a["out"])
    assert (wide[:, :, :4] == 7.0).all()


def test_replays_and_the_end_of_the_workspace():
    x = Shared(14, [(4, 2000), (2, 64)], [2000, 2900, 2031, 2400, 64, 90], 2, 16, 4, 128, 32)
    a = x.run()
    want = a["out"].clone()
    ws = torch.full((a["workspace"].numel() + 512,), 0xEE, dtype=torch.uint8, device=DEV)
    args = a | dict(workspace=ws[:-512])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp4_attn_shared_mx(**args)
    for _ in range(3):
        a["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], want)
    assert (ws[-512:] == 0xEE).all()


@pytest.mark.parametrize("members", [3, 90])
def test_an_empty_pool_table_batch_and_no_drafts(members):
    """By the walk and with many rows."""
    x = Shared(15, [(members, 64)], [70] * members, 1, 4, 2, 64, 16)
    a = x.device()
    F.fp4_attn_shared_mx(**(a | dict(cache=F.KvCache(*(t[:0] for t in a["cache"][:4]), 16))))
    assert (a["out"] == 0).all()
    a["out"].fill_(7.0)
    F.fp4_attn_shared_mx(**(a | dict(page_table=a["page_table"][:, :0])))
    assert (a["out"] == 0).all()
    a["out"].fill_(7.0)
    F.fp4_attn_shared_mx(**(a | dict(draft_lens=_i32([0] * members))))
    assert (a["out"] == 7.0).all()
    F.fp4_attn_shared_mx(a["q"][:0], a["cache"], a["page_table"][:0], a["seq_lens"][:0], a["groups"], a["prefix_lens"], a["out"][:0],
                         a["workspace"])


@pytest.mark.parametrize("d,q_heads,kv_heads", [(64, 10, 2), (128, 8, 2), (256, 4, 1)])
def test_many_rows_replayed_and_the_end_of_the_workspace(d, q_heads, kv_heads):
    rng = np.random.default_rng(d)
    lens = (900 + rng.integers(0, 200, 45)).tolist()
    x = Shared(16, [(40, 900), (5, 333)], lens, 1, q_heads, kv_heads, d, 16, draft_lens=rng.integers(0, 2, 45).tolist())
    a = x.run()
    want = a["out"].clone()
    ws = torch.full((a["workspace"].numel() + 512,), 0xEE, dtype=torch.uint8, device=DEV)
    args = a | dict(workspace=ws[:-512])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp4_attn_shared_mx(**args)
    for _ in range(3):
        a["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], want)
    assert (ws[-512:] == 0xEE).all()
