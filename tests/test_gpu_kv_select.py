"""GPU parity of the selection of cache blocks (fp4_kv_select_mx): the blocks equal to
the oracle's, ties and all, and the scores to their exact values (they are sums of
fewer than 2^24 units of their smallest product in every case here, so fp32 is exact)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
import workloads as W
from gpu_util import DEV
from oracle import attn as A
from oracle import quant as Q

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Index:
    """Entries of normal vectors, shuffled pages, queries."""

    def __init__(self, seed, lens, drafts, lists, dim, page_size, width=0, spread=1):
        rng = np.random.default_rng(seed)
        self.lens, self.page_size = np.asarray(lens), page_size
        counts = [max(int(n), 0) // page_size + 1 for n in lens]
        pages = sum(counts) + 2
        order, at = rng.permutation(pages), 0
        self.table = np.full((len(lens), max(width, max(counts))), -1, np.int32)
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        e = rng.standard_normal((pages, lists, dim)) * np.exp2(rng.integers(-spread, spread + 1, (pages, lists, dim // 32)).repeat(32, -1))
        self.codes, self.scales = Q.mx_quantize(W.bf16_bits(W.to_bf16(e)).reshape(pages, -1))
        self.q = W.bf16_bits(W.to_bf16(rng.standard_normal((len(lens), drafts, lists, dim))))

    def run(self, n_select, draft_lens=None, n_first=0, n_recent=0, scores=True, workspace=None):
        t = lambda a: torch.from_numpy(a.copy()).to(DEV)
        shape = (*self.q.shape[:3], n_select)
        ids = torch.full(shape, -7, dtype=torch.int32, device=DEV)
        out = torch.full(shape, 7.0, device=DEV) if scores else None
        ws = torch.full((F.fp4_kv_select_workspace_bytes(*self.q.shape[:3], self.table.shape[1]),), 0xFF, dtype=torch.uint8,
                        device=DEV) if workspace is None else workspace
        F.fp4_kv_select_mx(W.from_bits(self.q).to(DEV), t(self.codes), t(self.scales), t(self.table), _i32(self.lens),
                           self.page_size, ids, ws, draft_lens=None if draft_lens is None else _i32(draft_lens), scores=out,
                           n_first=n_first, n_recent=n_recent)
        return ids.cpu().numpy(), None if out is None else out.cpu().numpy()

    def check(self, n_select, draft_lens=None, n_first=0, n_recent=0):
        ids, out = self.run(n_select, draft_lens, n_first, n_recent)
        alone, _ = self.run(n_select, draft_lens, n_first, n_recent, scores=False)
        assert np.array_equal(ids, alone)
        want = A.block_scores(self.q, self.codes, self.scales, self.table, self.lens, self.page_size)
        for b, i, l in np.ndindex(*ids.shape[:3]):
            if draft_lens is not None and i >= draft_lens[b]:
                assert (ids[b, i, l] == -7).all() and (out[b, i, l] == 7.0).all()
                continue
            complete = min(max(int(self.lens[b]), 0) // self.page_size, self.table.shape[1])
            chosen = A.select_blocks(want[b, i, l], complete, n_select, n_first, n_recent)
            n = len(chosen)
            assert ids[b, i, l, :n].tolist() == chosen, (b, i, l)
            assert (out[b, i, l, :n] == want[b, i, l][chosen]).all()
            assert (ids[b, i, l, n:] == -1).all() and (out[b, i, l, n:] == -np.inf).all()


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 256, 512])
@pytest.mark.parametrize("lists,drafts", [(1, 1), (3, 5), (8, 1)])
def test_shapes(dim, lists, drafts):
    Index(dim + lists, [0, 15, 16, 17, 16 * 17 + 3, 16 * 70], drafts, lists, dim, 16).check(9)


@pytest.mark.parametrize("page_size", [16, 48, 64, 112])
@pytest.mark.parametrize("n_select", [1, 2, 64, 200])
def test_pages_and_numbers(page_size, n_select):
    Index(page_size, [page_size * n + page_size // 2 for n in (1, 2, 63, 64, 65, 300)], 2, 1, 64, page_size).check(n_select)


@pytest.mark.parametrize("drafts", [16, 17, 33, 64])
def test_many_drafts(drafts):
    Index(drafts, [700, 90], drafts, 2, 128, 16).check(5, draft_lens=[drafts, drafts // 2])


@pytest.mark.parametrize("dim", [64, 160])
def test_more_queries_than_compute_units(dim):
    Index(dim, [16 * 90, 16 * 200 + 1, 30, 0, 16 * 130], 30, 2, dim, 16).check(20, draft_lens=[30, 17, 30, 1, 0])


@pytest.mark.parametrize("drafts,width", [(64, 0), (41, 0), (31, 1100)])
def test_more_queries_than_one_launch_takes(drafts, width):
    Index(drafts, [16 * 90, 16 * 200 + 1, 30, 16 * 130, 16], drafts, 3, 64, 16, width=width).check(20)


@pytest.mark.parametrize("blocks", [511, 512, 513, 1024, 1025, 2048, 2049, 4000, 8191])
def test_many_blocks_in_registers(blocks):
    Index(blocks, [16 * blocks + 5, 100], 2, 1, 64, 16).check(50)


def test_more_blocks_than_registers_hold():
    Index(3, [16 * 9001, 16 * 8192, 16 * 700], 1, 1, 32, 16).check(129)


@pytest.mark.parametrize("n_select", [1, 3, 4, 5, 40])
@pytest.mark.parametrize("n_first,n_recent", [(1, 0), (0, 3), (2, 2), (3, 100), (1000, 0)])
def test_first_and_recent_blocks(n_select, n_first, n_recent):
    Index(7, [16 * 60 + 3, 16 * 3, 16, 5], 2, 2, 32, 16).check(n_select, n_first=n_first, n_recent=n_recent)


def test_ties_go_to_the_lowest_block():
    """Equal entries all over, and a few better and worse ones between them."""
    x = Index(8, [16 * 1500, 16 * 40], 1, 1, 32, 16)
    x.codes[:], x.scales[:] = x.codes[0], x.scales[0]
    x.check(33)
    better = x.table[0, [3, 700, 1499]]
    x.scales[better] += 1                                   # twice the score, whose sign differs by query
    x.check(33)
    x.q[:] = 0
    x.check(7)
    x.q[:] = 0x8000                                         # scores of -0 and 0 are equal
    x.codes[x.table[0, ::2]] ^= 0x88
    x.check(7)


def test_many_scores_on_both_sides_of_the_threshold():
    """A few far scores, so that all others lie in one part between the least and the largest."""
    x = Index(15, [16 * 1800], 3, 1, 64, 16)
    x.scales[x.table[0, [40, 900]]] += 14
    x.scales[x.table[0, 1000:1040]] -= 14
    for n in (1, 2, 3, 60, 1000):
        x.check(n)


def test_scores_without_a_number_come_last():
    """Scale bytes of 255 (no number), and infinite sums of both signs."""
    x = Index(9, [16 * 30 + 1], 3, 1, 64, 16)
    x.scales[x.table[0, [2, 5, 9]], 0] = 255
    ids, out = x.run(30)
    assert np.array_equal(ids, np.broadcast_to(np.arange(30), ids.shape))
    assert (out[..., [2, 5, 9]] == -np.inf).all() and np.isfinite(np.delete(out, [2, 5, 9], -1)).all()
    ids, out = x.run(28)
    assert np.array_equal(ids, np.broadcast_to(np.delete(np.arange(30), [5, 9]), ids.shape))


def test_far_apart_scales_are_summed_exactly():
    """Blocks of an entry 2^7 apart: the smallest product still counts."""
    x = Index(10, [16 * 64], 4, 1, 128, 16)
    x.scales[:] = (127 + np.array([0, -7, -3, -7])).astype(np.uint8)
    x.check(20)


def test_pages_that_are_not_in_the_pool_are_no_blocks():
    x = Index(11, [16 * 50, 16 * 20, 16 * 90], 2, 1, 64, 16, width=60)
    x.table[0, [0, 7, 49]] = [-1, len(x.codes), 1 << 30]
    x.check(48)
    x.check(3, n_first=2, n_recent=2)
    x.table[1, :20] = -5
    x.check(4)


def test_a_length_past_the_table_and_a_negative_one():
    x = Index(12, [16 * 40, 16 * 40], 1, 1, 32, 16)
    x.lens = np.array([2 ** 31 - 1, -3])
    x.check(10)


def test_empty_calls():
    x = Index(13, [100], 1, 1, 32, 16)
    t = lambda a: torch.from_numpy(a.copy()).to(DEV)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    ids = torch.full((1, 1, 1, 3), -7, dtype=torch.int32, device=DEV)
    q, ws = W.from_bits(x.q).to(DEV), torch.empty(4096, dtype=torch.uint8, device=DEV)
    F.fp4_kv_select_mx(q, t(x.codes)[:0], t(x.scales)[:0], t(x.table), _i32(x.lens), 16, ids, ws)      # no pool
    assert (ids == -1).all()
    ids.fill_(-7)
    F.fp4_kv_select_mx(q, t(x.codes), t(x.scales), t(x.table)[:, :0], _i32(x.lens), 16, ids, none)     # no table
    assert (ids == -1).all()
    F.fp4_kv_select_mx(q, t(x.codes), t(x.scales), t(x.table), _i32(x.lens), 16, ids[..., :0].contiguous(), ws)
    F.fp4_kv_select_mx(q[:0], t(x.codes), t(x.scales), t(x.table)[:0], _i32([]), 16, ids[:0], ws)
    assert (ids == -1).all()


def test_strided_queries_a_guarded_workspace_and_replays():
    x = Index(14, [16 * 200 + 3, 16 * 77], 3, 2, 64, 16)
    want, _ = x.run(17)
    need = F.fp4_kv_select_workspace_bytes(*x.q.shape[:3], x.table.shape[1])
    ws = torch.full((need + 256,), 0xEE, dtype=torch.uint8, device=DEV)
    t = lambda a: torch.from_numpy(a.copy()).to(DEV)
    wide = torch.zeros((2, 3, 5, 64), dtype=torch.bfloat16, device=DEV)
    wide[:, :, 1:3] = W.from_bits(x.q).to(DEV)
    args = (wide[:, :, 1:3], t(x.codes), t(x.scales), t(x.table), _i32(x.lens), 16)
    ids = torch.zeros(want.shape, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        F.fp4_kv_select_mx(*args, ids, ws[:need])
    for _ in range(3):
        ids.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(ids.cpu().numpy(), want)
    assert (ws[need:] == 0xEE).all()
