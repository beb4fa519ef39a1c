"""GPU parity of the attention over selected cache blocks (fp4_attn_blocks_mx) with the
float64 definition; tolerance in attn_check.py."""
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
from test_gpu_attn_tree import Step, _i32, _tree

pytestmark = pytest.mark.gpu


class Blocks(Step):
    """A Step with a list of blocks for every drafted token, and every key/value head where lists > 1."""

    def __init__(self, seed, lens, drafts, q_heads, kv_heads, d, page_size, n_select, lists=1, **kw):
        super().__init__(seed, lens, drafts, q_heads, kv_heads, d, page_size, **kw)
        rng = np.random.default_rng(seed + 1)
        self.ids = np.full((len(self.lens), drafts, lists, n_select), -1, np.int32)
        for b, i, l in np.ndindex(*self.ids.shape[:3]):
            full = max(self.lens[b], 0) // page_size
            chosen = np.sort(rng.permutation(full)[:n_select])
            self.ids[b, i, l, :len(chosen)] = chosen

    def device(self):
        a = super().device()
        batch, drafts = self.q.shape[:2]
        need = F.fp4_attn_blocks_workspace_bytes(batch, drafts, self.heads[0], self.d, self.heads[1])
        return a | dict(block_ids=_i32(self.ids), workspace=torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV))

    def check(self, out, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        ref, size = A.attn_blocks_mx(self.q, self.kc, self.ks, self.vc, self.vs, self.ps, self.table, self.lens, self.heads[1],
                                     scale, self.ids, self.draft_lens, self.masks)
        k = Q.mx_dequant_f64(self.kc, self.ks).reshape(-1, self.d)
        v = Q.mx_dequant_f64(self.vc, self.vs)
        check(out, ref, size, self.d, self.ids.shape[3] * self.ps + self.ps + self.drafts, scale, norm(self.q),
              float(np.sqrt((k * k).sum(-1)).max()), np.abs(v).max())
        assert (out.cpu().float().numpy()[np.isnan(ref)] == 7.0).all()

    def run(self, scale=None):
        a = self.device()
        F.fp4_attn_blocks_mx(**a, scale=scale)
        self.check(a["out"], scale)
        return a


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,drafts,lists", [(1, 1, 1, 1), (8, 1, 1, 1), (4, 4, 3, 4), (10, 2, 5, 1), (10, 2, 2, 2),
                                                           (16, 8, 1, 8), (24, 12, 2, 1)])
def test_shapes(d, q_heads, kv_heads, drafts, lists):
    Blocks(d + q_heads, [0, 1, 15, 16, 33, 200, 500], drafts, q_heads, kv_heads, d, 16, 6, lists).run()


@pytest.mark.parametrize("page_size", [16, 32, 48, 64, 112, 256])
@pytest.mark.parametrize("lists", [1, 2])
def test_pages_that_end_inside_a_step(page_size, lists):
    Blocks(page_size, [page_size - 1, page_size, page_size + 1, 5 * page_size + 17], 2, 8, 2, 128, page_size, 3, lists).run()


@pytest.mark.parametrize("q_heads,kv_heads", [(17, 1), (40, 1), (80, 2), (64, 1)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_more_heads_than_a_row_tile(q_heads, kv_heads, d):
    Blocks(q_heads, [300, 40], 2, q_heads, kv_heads, d, 32, 4, masks=_tree(1, 2, 2)).run()


@pytest.mark.parametrize("d,q_heads,kv_heads,drafts,lists", [(64, 8, 2, 1, 1), (128, 8, 1, 1, 1), (128, 16, 2, 3, 2), (256, 4, 2, 2, 1)])
def test_many_blocks_split_over_workgroups(d, q_heads, kv_heads, drafts, lists):
    Blocks(d, [9001], drafts, q_heads, kv_heads, d, 64, 120, lists).run()


def test_ragged_batch_of_drafts_and_trees():
    lens = [3000, 0, 5, 64, 2049, 1, 900, 0, 0, 40, 31, 777]
    draft_lens = [4, 0, 1, 4, 2, 3, 4, 4, 0, 1, 2, 3]
    Blocks(1, lens, 4, 8, 8, 64, 32, 20, masks=_tree(1, len(lens), 4), draft_lens=draft_lens).run()
    Blocks(2, lens, 4, 8, 4, 128, 32, 20, 4, masks=_tree(1, len(lens), 4), draft_lens=draft_lens).run()


def test_more_sequences_than_lanes():
    rng = np.random.default_rng(2)
    Blocks(2, rng.integers(0, 130, 150).tolist(), 2, 4, 2, 64, 16, 4, draft_lens=rng.integers(0, 3, 150).tolist()).run()


def test_lists_in_any_order_with_holes_repeats_and_strangers():
    x = Blocks(3, [16 * 20 + 5, 16 * 3, 16 * 9], 2, 4, 2, 128, 16, 12, 2)
    rng = np.random.default_rng(3)
    x.ids = rng.permuted(x.ids, axis=-1)                    # -1 anywhere
    x.ids[0, 0, 0, :4] = [7, 7, 7, 3]                       # counted three times
    x.ids[0, 1, 1, :5] = [20, 1 << 30, -(1 << 31), 21, 19]  # the incomplete block and beyond: nothing
    x.run()


def test_pages_missing_from_the_pool():
    x = Blocks(4, [16 * 30 + 5, 16 * 4 + 1], 2, 4, 2, 64, 16, 8)
    x.table[0, x.ids[0, 0, 0, 0]], x.table[0, 30], x.table[1, 2] = -1, 1 << 29, len(x.kc)
    x.run()


def test_a_list_that_names_nothing_leaves_the_rest():
    x = Blocks(5, [16 * 10, 16 * 10 + 3, 5], 2, 4, 4, 64, 16, 3, masks=np.array([[0, 2], [1, 1], [1, 3]], np.uint64))
    x.ids[:] = -1
    out = x.run()["out"]
    assert (out[0, 0] == 0).all()                           # nothing behind the last block, and no drafted token seen
    x.ids = x.ids[..., :0]
    assert torch.equal(x.run()["out"], out)


def test_all_blocks_are_the_tree_attention():
    """With every block listed the rows are fp4_attn_tree_mx's tokens, in its order."""
    for lists in (1, 2):
        x = Blocks(6, [16 * 40 + 7, 16 * 3], 1, 8, 2, 128, 16, 40, lists)
        out, a = x.run()["out"], Step.device(x)
        F.fp4_attn_tree_mx(**a)
        Step.check(x, a["out"])
        if lists == 1:
            assert torch.equal(out, a["out"])


def test_what_is_not_listed_may_hold_anything():
    x = Blocks(7, [16 * 20 + 5, 70, 16], 3, 4, 2, 128, 16, 5, draft_lens=[1, 2, 0], spare=4)
    rows = np.ones(len(x.kc), bool)
    for b, n in enumerate(x.lens):
        full, at = n // 16, A.cache_rows(x.table[b], 16, len(x.kc) // 16, n + x.draft_lens[b])
        rows[at[full * 16:]] = False
        for m in np.unique(x.ids[b, :x.draft_lens[b]]):
            if m >= 0:
                rows[at[m * 16:m * 16 + 16]] = False
    for c, e in ((x.kc, x.ks), (x.vc, x.vs)):
        c[rows], e[rows] = 0xFF, 0xFF
    x.run()


@pytest.mark.parametrize("d,lists", [(64, 1), (128, 2), (256, 1)])
def test_drafted_values_past_the_range_reach_only_rows_that_see_them(d, lists):
    x = Blocks(8, [16 * 6 + 3, 40], 4, 4, 2, d, 16, 3, lists, masks=np.array([[1, 2, 5, 8], [1, 3, 4, 12]], np.uint64))
    for b, j in ((0, 1), (1, 2)):
        row = A.cache_rows(x.table[b], 16, len(x.kc) // 16, x.lens[b] + 4)[x.lens[b] + j]
        x.vs[row, 0], x.vc[row, :16] = 255, 0x77
    a = x.device()
    F.fp4_attn_blocks_mx(**a)
    out = a["out"].float().cpu().numpy()
    group = 2
    sees = [(b, i) for b in range(2) for i in range(4) if (int(x.masks[b, i]) >> (1, 2)[b]) & 1]
    for b in range(2):
        for i in range(4):
            assert np.isnan(out[b, i, :group, :32]).all() == ((b, i) in sees), (b, i)
    for row in sees:                                        # the rest as if they were not there
        a["out"][row][:group, :32] = 0.0
    x.vs[x.vs == 255] = 127
    ref = A.attn_blocks_mx(x.q, x.kc, x.ks, x.vc, x.vs, 16, x.table, x.lens, 2, d ** -0.5, x.ids, None, x.masks)
    for row in sees:
        ref[0][row][:group, :32] = 0.0
    k = Q.mx_dequant_f64(x.kc, x.ks).reshape(-1, d)
    check(a["out"], *ref, d, 80, d ** -0.5, norm(x.q), float(np.sqrt((k * k).sum(-1)).max()),
          np.abs(Q.mx_dequant_f64(x.vc, x.vs)).max())


def test_scales_of_either_sign_and_strided_rows():
    x = Blocks(9, [200, 77], 2, 8, 2, 64, 16, 5)
    x.run(scale=-0.3)
    x.run(scale=0.0)
    a = x.device()
    wide = torch.full((2, 2, 12, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    wide_q = torch.zeros_like(wide)
    wide_q[:, :, 2:10] = a["q"]
    a["q"], a["out"] = wide_q[:, :, 2:10], wide[:, :, 4:]
    F.fp4_attn_blocks_mx(**a)
    x.check(a["out"])
    assert (wide[:, :, :4] == 7.0).all()


def test_an_empty_pool_table_and_batch():
    x = Blocks(10, [40, 3], 1, 4, 2, 64, 16, 2)
    a = x.device()
    F.fp4_attn_blocks_mx(**(a | dict(cache=F.KvCache(*(t[:0] for t in a["cache"][:4]), 16))))
    assert (a["out"] == 0).all()
    a["out"].fill_(7.0)
    F.fp4_attn_blocks_mx(**(a | dict(page_table=a["page_table"][:, :0])))
    assert (a["out"] == 0).all()
    F.fp4_attn_blocks_mx(a["q"][:0], a["cache"], a["page_table"][:0], a["seq_lens"][:0], a["block_ids"][:0], a["out"][:0], a["workspace"])


def test_replays_and_the_end_of_the_workspace():
    x = Blocks(11, [4000, 900, 31], 2, 16, 4, 128, 32, 50, 4)
    a = x.run()
    want = a["out"].clone()
    ws = torch.full((a["workspace"].numel() + 512,), 0xEE, dtype=torch.uint8, device=DEV)
    args = a | dict(workspace=ws[:-512])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp4_attn_blocks_mx(**args)
    for _ in range(3):
        a["out"].fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a["out"], want)
    assert (ws[-512:] == 0xEE).all()
