"""GPU parity of the cache's page operations with the host's loops: tables,
counts, lengths, references, slots and every byte of the cache, exactly."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
from oracle import attn as A
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Both:
    """The same state on the host (A.Pages) and on the GPU."""

    def __init__(self, seed, batch, width, num_pages, page_size, d, values=True):
        rng = np.random.default_rng(seed)
        rows = num_pages * page_size
        arrays = [rng.integers(0, 256, (rows, w), dtype=np.uint8) for w in ((d // 2, d // 32) * (2 if values else 1))]
        self.host = A.Pages(np.full((batch, width), -1, np.int32), np.zeros(batch, np.int32), np.zeros(batch, np.int32),
                            np.zeros(num_pages, np.int32), page_size, arrays)
        h = self.host
        t = [torch.from_numpy(a.copy()).to(DEV) for a in arrays] + [None] * (0 if values else 2)
        self.cache = F.KvCache(*t, page_size)
        self.pages = F.KvPages(*(torch.from_numpy(a.copy()).to(DEV) for a in (h.table, h.counts, h.lens, h.refs)))
        # guard words behind the bytes that the query asks for
        need = F.fp4_kv_reserve_workspace_bytes(batch, num_pages)
        self.ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        self.need = need

    def reserve(self, new, max_new):
        slots = torch.full((len(new), max_new), 77, dtype=torch.int32, device=DEV)
        short = _i32([-5])
        F.fp4_kv_reserve(self.cache, self.pages, _i32(new), slots, short, self.ws[:self.need])
        want, lack = self.host.reserve(new, max_new)
        assert np.array_equal(slots.cpu().numpy(), want)
        assert short.item() == lack
        assert (self.ws[self.need:] == 0xA5).all()
        self.check()
        return slots

    def fork(self, pairs):
        F.fp4_kv_fork(self.pages, _i32(pairs).reshape(-1, 2), self.cache.page_size)
        self.host.fork(pairs)
        self.check()

    def free(self, seqs, keep=None):
        F.fp4_kv_free(self.pages, _i32(seqs), self.cache.page_size, keep_lens=None if keep is None else _i32(keep))
        self.host.free(seqs, keep)
        self.check()

    def compact(self, accepted, n):
        F.fp4_kv_compact(self.cache, self.pages, None if accepted is None else _i32(accepted), _i32(n))
        self.host.compact(None if accepted is None else np.asarray(accepted), n)
        self.check()

    def commit(self, accepted, n, slots):
        """A commit that follows the reservation's slots."""
        F.fp4_kv_compact_reserved(self.cache, self.pages, None if accepted is None else _i32(accepted), _i32(n), slots)
        self.host.compact(None if accepted is None else np.asarray(accepted), n, slots.cpu().numpy())
        self.check()

    def write(self, slots, seed):
        """Fills the reserved rows with other bytes, as an append would."""
        rng = np.random.default_rng(seed)
        rows = slots.cpu().numpy().ravel()
        rows = rows[rows >= 0]
        for h, t in zip(self.host.arrays, self.cache):
            h[rows] = rng.integers(0, 256, (len(rows), h.shape[1]), dtype=np.uint8)
            t[torch.from_numpy(rows).long().to(DEV)] = torch.from_numpy(h[rows]).to(DEV)

    whole = True            # False once a test has put something into the state that no call does

    def check(self):
        h = self.host
        for name, got, want in zip(F.KvPages._fields, self.pages, (h.table, h.counts, h.lens, h.refs)):
            assert np.array_equal(got.cpu().numpy(), want), name
        for got, want in zip(self.cache, h.arrays):
            assert np.array_equal(got.cpu().numpy(), want)
        if not self.whole:
            return
        # every reference is a table entry, and the other way round
        entries = [int(p) for row, n in zip(h.table, h.counts) for p in row[:n]]
        assert np.array_equal(np.bincount(entries, minlength=len(h.refs)), h.refs)


@pytest.mark.parametrize("page_size,d,values", [(16, 32, True), (48, 96, True), (64, 1024, True), (32, 256, False), (16, 512, True)])
def test_serving_steps(page_size, d, values):
    """Prompts, a fork of everything, drafted steps of both sides, a cut and an end."""
    s = Both(page_size + d, 8, 12, 40, page_size, d, values)
    prompts = [5 * page_size + 3, page_size, 1, 0, 0, 0, 0, 0]
    s.write(s.reserve(prompts, max(prompts)), 1)
    s.compact(None, prompts)
    s.fork([(0, 3), (1, 4), (2, 5), (0, 6), (0, 3), (6, 7), (4, 4), (9, 2), (0, -1)])
    for step in range(3):
        rng = np.random.default_rng(step)
        new = rng.integers(0, 18, 8)
        s.write(s.reserve(new, 17), 10 + step)
        acc = [rng.permutation(17).tolist() for _ in range(8)]
        s.compact(acc, [rng.integers(0, n + 1) for n in new])
    s.free([3, 0, 3, -1, 8], [page_size + 1, 2 * page_size, 0, 0, 0])
    s.write(s.reserve([1] * 8, 1), 30)                 # sequences cut inside a shared page write into copies
    s.free([0, 6])
    s.free(list(range(8)))
    assert (s.host.refs == 0).all()


def test_every_holder_of_a_page_writes_at_once():
    """Four sequences on one partly filled page: each gets a copy, the page itself becomes free."""
    s = Both(3, 4, 5, 10, 16, 64)   # 9 free pages: 4 copies and 5 new ones
    s.write(s.reserve([10, 0, 0, 0], 10), 1)
    s.compact(None, [10, 0, 0, 0])
    s.fork([(0, 1), (0, 2), (0, 3)])
    shared = int(s.host.table[0, 0])
    s.write(s.reserve([1, 7, 2, 64], 7), 2)
    assert s.host.refs[shared] == 0


def test_reserve_twice_gives_the_same_rows():
    s = Both(4, 3, 6, 12, 16, 64)
    a = s.reserve([5, 0, 20], 20)
    b = s.reserve([5, 0, 20], 20)
    assert torch.equal(a, b)


def test_what_does_not_fit_is_refused_whole():
    s = Both(5, 3, 4, 6, 16, 64)
    s.reserve([16, 33, 1], 33)                          # all 6 pages
    s.reserve([0, 0, 17], 17)                           # the pool is empty: nothing, for nobody
    s.free([0])
    s.reserve([16, 17, 1], 4)                           # one page for sequence 0, none lacks
    s.free([0, 1, 2])
    s.reserve([1, 65, 0], 2)                            # a row of 4 pages cannot hold 65 tokens
    s.reserve([-3, 0, 0], 1)                            # negative: none
    s.reserve([64, 32, 0], 0)


@pytest.mark.parametrize("num_pages,batch", [(8193, 5), (20000, 1300)])
def test_large_pools_and_batches(num_pages, batch):
    """More pages than one round of the scan and more sequences than threads."""
    s = Both(6, batch, 4, num_pages, 16, 32)
    rng = np.random.default_rng(0)
    s.reserve(rng.integers(0, 60, batch), 3)
    s.compact(None, rng.integers(0, 60, batch))
    s.free(rng.permutation(batch)[:batch // 2])
    s.reserve(rng.integers(0, 5, batch), 3)


def test_accepted_rows_may_cross():
    """A permutation of 64 rows over several pages, an index listed twice, indices that point nowhere."""
    s = Both(7, 3, 8, 24, 16, 1024)
    s.write(s.reserve([64 + 9, 30, 30], 73), 1)
    s.compact(None, [9, 3, 0])
    rng = np.random.default_rng(1)
    acc = np.stack([rng.permutation(64), np.full(64, 2), np.arange(64)[::-1]])
    acc[2, 5] = 1 << 30
    acc[2, 6] = -4
    s.compact(acc, [64, 5, 28])
    s.compact(acc, [100, 100, -1])                      # lengths never pass the pages


@pytest.mark.parametrize("committed", [10, 16, 40])
def test_a_fork_between_a_reservation_and_its_commit(committed):
    """The source still moves its accepted rows, on the page that is shared now; the
    targets keep theirs and write into copies."""
    s = Both(8, 4, 6, 24, 16, 64)
    s.write(s.reserve([committed, 3, 0, 0], committed), 1)
    s.compact(None, [committed, 3, 0, 0])
    s.write(s.reserve([20, 1, 0, 0], 20), 2)
    s.fork([(0, 2), (0, 3)])
    s.compact([[19, 0, 7, 2, 18] + [0] * 15, [0] * 20, [0] * 20, [0] * 20], [5, 1, 0, 0])
    s.write(s.reserve([2, 1, 8, 9], 9), 3)
    s.compact([[1, 0], [0, 0], [7, 1], [8, 8]], [2, 1, 2, 2])


def test_a_commit_without_a_reservation_moves_nothing_that_others_see():
    s = Both(9, 2, 4, 8, 16, 64)
    s.write(s.reserve([10, 0], 10), 1)
    s.compact(None, [10, 0])
    s.fork([(0, 1)])
    s.free([0], [5])
    before = [a.clone() for a in s.cache[:4]]
    F.fp4_kv_compact(s.cache, s.pages, _i32([[3], [0]]), _i32([1, 0]))
    assert all(torch.equal(a, b) for a, b in zip(s.cache[:4], before))
    assert s.pages.seq_lens.tolist() == [6, 10]


@pytest.mark.parametrize("forks", [2, 8, 70])
def test_sharers_that_commit_unreserved_rows_in_one_call_move_nothing(forks):
    """Each of them sees as far as the others, and all lengths grow in the call: whose
    workgroup comes first may not matter."""
    s = Both(11, forks, 4, 2 * forks, 16, 64)
    s.write(s.reserve([10] + [0] * (forks - 1), 10), 1)
    s.compact(None, [10] + [0] * (forks - 1))
    s.fork([(0, i) for i in range(1, forks)])
    before = [a.clone() for a in s.cache[:4]]
    s.compact([[1 + (b + i) % 5 for i in range(3)] for b in range(forks)], [1 + b % 3 for b in range(forks)])
    assert all(torch.equal(a, b) for a, b in zip(s.cache[:4], before))


def _same(s, before):
    return all(torch.equal(a, b) for a, b in zip((*s.cache[:4], *s.pages), before))


def _copy(s):
    return [a.clone() for a in (*s.cache[:4], *s.pages)]


@pytest.mark.parametrize("accepted", [None, [[1, 2, 0]] * 3])
def test_a_refused_reservation_commits_nothing(accepted):
    """10 of 16 rows used, the pool full: the rest of the page is no reservation, of a
    page held alone (sequence 2) or by two that commit in one call."""
    s = Both(12, 3, 4, 2, 16, 64)
    s.write(s.reserve([10, 0, 10], 10), 1)
    s.compact(None, [10, 0, 10])
    s.fork([(0, 1)])
    before = _copy(s)
    slots = s.reserve([3, 3, 30], 30)                   # two copies and two pages lack
    assert (slots == -1).all()
    s.commit(accepted, [3, 2, 3], slots)
    assert _same(s, before) and s.pages.seq_lens.tolist() == [10, 10, 10]


def test_only_what_the_reservation_granted_is_committed():
    s = Both(13, 5, 8, 30, 16, 64)
    prompts = [70, 16, 0, 5, 9]
    slots = s.reserve(prompts, 40)                      # of sequence 0's rows 40 are in slots
    s.write(slots, 1)
    s.commit(None, [70, 20, 4, 5, 8], slots)            # more than was reserved, nothing reserved, fewer
    assert s.pages.seq_lens.tolist() == [40, 16, 0, 5, 8]
    before = _copy(s)
    s.commit(None, [1, 1, 1, 1, 1], slots)              # the same slots again
    assert _same(s, before)
    slots = s.reserve([4, 20, 0, 12, 1], 20)
    s.write(slots, 2)
    acc = np.tile(np.arange(20)[::-1], (5, 1))          # 19, 18, ..: past the reserved ones in most
    s.commit(acc, [3, 20, 2, 20, 1], slots)
    assert s.pages.seq_lens.tolist() == [43, 36, 0, 17, 9]
    slots = s.reserve([4, 4, 4, 4, 4], 4)
    s.free([3], [3])                                    # its rows are let go between
    before = _copy(s)
    s.commit([[3, 1, 0, 2]] * 5, [0, 0, 0, 4, 0], slots)
    assert _same(s, before)


@pytest.mark.parametrize("committed", [10, 16, 30])
def test_a_second_reservation_starts_the_step_anew(committed):
    """Drafts reserved and appended before a fork, then reserved again: on a shared page
    the slots are a copy's, so the old ones commit nothing, and the new ones what is
    appended to them; elsewhere the slots are the same."""
    s = Both(15, 3, 6, 16, 16, 64)
    slots = s.reserve([committed, 0, 0], committed)
    s.write(slots, 1)
    s.commit(None, [committed, 0, 0], slots)
    old = s.reserve([6, 0, 0], 6)
    s.write(old, 2)
    s.fork([(0, 1)])
    new = s.reserve([6, 0, 0], 6)
    assert torch.equal(old, new) == (committed % 16 == 0)
    if committed % 16:
        before = _copy(s)
        s.commit([[5, 1, 0]] * 3, [3, 0, 0], old)
        n = int(s.pages.seq_lens[0]) - committed
        assert n == 0 and _same(s, before)
    s.write(new, 3)
    drafts = [a[new[0].long()].clone() for a in s.cache[:4]]
    s.commit([[5, 1, 0]] * 3, [3, 0, 0], new)
    for a, d in zip(s.cache, drafts):
        assert torch.equal(a[new[0, :3].long()], d[[5, 1, 0]])


def test_steps_that_outgrow_the_pool_replayed():
    """A captured step goes on being replayed when the pool is full: lengths and bytes
    stay, and it takes up again when pages are free."""
    s = Both(14, 3, 6, 9, 16, 64)
    slots = s.reserve([30, 3, 17], 30)
    s.write(slots, 1)
    s.commit(None, [30, 3, 17], slots)
    s.fork([(0, 1)])                                    # not done: sequence 1 holds pages
    new, n = _i32([9, 5, 12]), _i32([3, 5, 2])
    acc = _i32([[8, 0, 4, 1, 2], [0, 1, 2, 3, 4], [3, 7, 0, 0, 0]])
    slots, short = torch.zeros((3, 12), dtype=torch.int32, device=DEV), _i32([0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp4_kv_reserve(s.cache, s.pages, new, slots, short, s.ws)
        F.fp4_kv_compact_reserved(s.cache, s.pages, acc, n, slots)
    lacks = []
    for i in range(14):
        if i == 11:
            s.free([2])
        graph.replay()
        torch.cuda.synchronize()
        want, lack = s.host.reserve([9, 5, 12], 12)
        s.host.compact(acc.cpu().numpy(), [3, 5, 2], want)
        assert np.array_equal(slots.cpu().numpy(), want) and short.item() == lack
        s.check()
        lacks.append(lack > 0)
        torch.ones(1000, device=DEV).sum().item()
    assert lacks[10] and not lacks[0] and not lacks[11]


def test_ids_outside_are_not_followed():
    """Table entries outside the pool and counts outside the row: no access, no fault."""
    s = Both(8, 4, 4, 10, 16, 64)
    s.reserve([16, 16, 16, 0], 16)
    s.pages.page_table[0, 0] = 1 << 30
    s.pages.page_table[1, 0] = -7
    s.pages.page_counts[2] = 99
    s.pages.seq_lens[:] = _i32([9, 9, 9, 0])
    F.fp4_kv_fork(s.pages, _i32([[0, 3]]), 16)
    slots, short = torch.zeros((4, 2), dtype=torch.int32, device=DEV), _i32([0])
    F.fp4_kv_reserve(s.cache, s.pages, _i32([2, 2, 2, 2]), slots, short, s.ws)
    F.fp4_kv_compact(s.cache, s.pages, _i32([[1, 0]] * 4), _i32([2] * 4))
    F.fp4_kv_free(s.pages, _i32([0, 1, 2, 3]), 16)
    torch.cuda.synchronize()
    assert slots[0].tolist() == [-1, -1] and slots[1].tolist() == [-1, -1]
    for got, want in zip(s.cache[:1], s.host.arrays):
        assert got.shape == want.shape


ODD = [("table", (0, 0), 1 << 30), ("table", (0, 2), 40), ("table", (1, 0), -7), ("table", (2, 1), -1),
       ("table", (3, 0), -1 << 31), ("counts", 2, 99), ("counts", 2, -3), ("counts", 0, 1), ("counts", 3, 1 << 30),
       ("lens", 1, -5), ("lens", 1, 60), ("lens", 4, (1 << 31) - 1), ("lens", 2, 0)]


@pytest.mark.parametrize("field,at,value", ODD)
def test_an_odd_entry_reaches_nothing_else(field, at, value):
    """One table entry, count or length that no call leaves, then every call: all bytes of
    the cache, references, counts, lengths, tables and slots are those of the host's
    loops, which skip it; what other sequences have is untouched by it."""
    s = Both(16, 6, 5, 40, 16, 64)
    lens = [40, 9, 33, 16, 12, 0]
    slots = s.reserve(lens, 40)
    s.write(slots, 1)
    s.commit(None, lens, slots)
    getattr(s.host, field)[at] = value
    s.pages[{"table": 0, "counts": 1, "lens": 2}[field]][at] = value
    s.whole = False
    s.fork([(0, 5), (1, 5), (2, 4)])
    slots = s.reserve([3, 4, 5, 6, 7, 2], 7)
    s.write(slots, 2)
    s.commit([[2, 0, 1]] * 6, [2, 3, 1, 3, 2, 2], slots)
    s.compact([[4, 1, 0]] * 6, [1, 2, 0, 1, 0, 0])
    s.free([0, 3, 2], [17, 0, 20])
    s.free([5, 1, 0, 4])


@pytest.mark.parametrize("page_size,d,n,values", [(16, 32, 1, True), (48, 96, 7, True), (64, 1024, 33, True), (16, 512, 200, False)])
def test_copy_pages(page_size, d, n, values):
    rng = np.random.default_rng(n)
    a, b = (Both(i, 1, 1, n + 3, page_size, d, values) for i in (1, 2))
    src, dst = rng.permutation(n + 3)[:n].astype(np.int32), rng.permutation(n + 3)[:n].astype(np.int32)
    if n > 5:
        src[1], dst[2], src[4] = -1, n + 3, 1 << 30
    F.fp4_kv_copy_pages(a.cache, b.cache, _i32(src), _i32(dst))
    for s, d_, t in zip(a.host.arrays, b.host.arrays, b.cache):
        for i, j in zip(src, dst):
            if 0 <= i < n + 3 and 0 <= j < n + 3:
                d_[j * page_size:(j + 1) * page_size] = s[i * page_size:(i + 1) * page_size]
        assert np.array_equal(t.cpu().numpy(), d_)
    a.check()


def test_copy_pages_within_one_cache():
    s = Both(9, 1, 1, 12, 32, 128)
    F.fp4_kv_copy_pages(s.cache, s.cache, _i32([0, 1, 2]), _i32([9, 3, 11]))
    for h in s.host.arrays:
        for i, j in ((0, 9), (1, 3), (2, 11)):
            h[32 * j:32 * j + 32] = h[32 * i:32 * i + 32]
    s.check()


def test_replayed_graph():
    """Reserve, commit and free captured once and replayed, with eager work between the replays."""
    s = Both(10, 4, 8, 30, 16, 64)
    s.reserve([20, 3, 0, 16], 20)
    s.compact(None, [20, 3, 0, 16])
    new, n, seqs = _i32([5, 1, 9, 2]), _i32([2, 1, 3, 0]), _i32([2])
    acc = _i32([[4, 0, 1], [0, 1, 2], [8, 2, 3], [0, 0, 0]])
    slots, short = torch.zeros((4, 9), dtype=torch.int32, device=DEV), _i32([0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp4_kv_reserve(s.cache, s.pages, new, slots, short, s.ws)
        F.fp4_kv_compact(s.cache, s.pages, acc, n)
        F.fp4_kv_free(s.pages, seqs, 16)
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want, lack = s.host.reserve([5, 1, 9, 2], 9)
        s.host.compact(acc.cpu().numpy(), [2, 1, 3, 0])
        s.host.free([2])
        assert lack == 0 and np.array_equal(slots.cpu().numpy(), want)
        s.check()
        torch.ones(1000, device=DEV).sum().item()
