"""A serving loop over long contexts as it runs: reserved rows take rotated keys and values
(fp4_kv_append_rope_mx), an index entry for every complete page takes its mean, a step
selects blocks (fp4_kv_select_mx), attends over them (fp4_attn_blocks_mx), and forks attend
over their common prefix (fp4_attn_shared_mx), with the exact forms beside every step."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
import workloads as W
from attn_check import check, norm
from gpu_util import DEV
from oracle import attn as A
from oracle import formats as FM
from oracle import quant as Q
from test_gpu_attn_serving import D, HK, HQ, PAGE, POOL, ROT, Server, _chain, _i32

pytestmark = pytest.mark.gpu

SELECT, SCALE = 3, D ** -0.5


class Sparse(Server):
    def __init__(self, batch):
        super().__init__(batch)
        z = lambda w: torch.zeros((POOL, w), dtype=torch.uint8, device=DEV)
        self.index = (z(HK * D // 2), z(HK * D // 32))
        self.angles = self.table.cpu().numpy()

    def rows(self, seed, tokens, positions, slots, q_out):
        """Rotates and appends; the rotated queries equal the exact form's, and the host's copy of the rows."""
        qkv = self.projected(seed, tokens)
        F.fp4_kv_append_rope_mx(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], self.cache, slots.view(-1), q_out=q_out,
                                positions=positions, cos_sin=self.table)
        q, k, v = np.split(W.bf16_bits(qkv), [HQ, HQ + HK], axis=1)
        at = positions.cpu().numpy()
        q, k = (A.turned_bf16(x, self.angles, at, False) for x in (q, k))
        live = at >= 0
        assert np.array_equal(W.bf16_bits(q_out)[live], q[live])
        return q, k, v

    def enter(self):
        """The entry of every complete page: its keys' mean."""
        table, pages, means = self.pages.page_table.cpu().numpy(), [], []
        for b, tokens in enumerate(self.host):
            for n in range(len(tokens) // PAGE):
                k = FM.bf16_bits_to_f64(np.stack([t[0] for t in tokens[n * PAGE:(n + 1) * PAGE]]))
                pages.append(table[b, n])
                means.append(k.mean(0).reshape(-1))
        _, first = np.unique(pages, return_index=True)      # forks share pages, and with them entries
        F.fp4_kv_append_mx(W.to_bf16(np.stack(means)[first]).to(DEV), _i32(np.array(pages)[first]), *self.index)

    def prompts(self, seed, lens):
        total = sum(lens)
        slots = torch.empty((self.batch, max(lens)), dtype=torch.int32, device=DEV)
        F.fp4_kv_reserve(self.cache, self.pages, _i32(lens), slots, self.short, self.ws)
        assert self.short.item() == 0
        q_out = torch.empty((total, HQ, D), dtype=torch.bfloat16, device=DEV)
        _, k, v = self.rows(seed, total, _i32(np.concatenate([np.arange(n) for n in lens])),
                            torch.cat([slots[b, :n] for b, n in enumerate(lens)]), q_out)
        F.fp4_kv_compact_reserved(self.cache, self.pages, None, _i32(lens), slots)
        at = 0
        for b, n in enumerate(lens):
            self.host[b] += [(k[at + i], v[at + i]) for i in range(n)]
            at += n
        self.enter()

    def stored(self):
        rows = [x.cpu().numpy() for x in (self.cache.k_codes, self.cache.k_scales, self.cache.v_codes, self.cache.v_scales)]
        table, lens = self.pages.page_table.cpu().numpy(), self.pages.seq_lens.cpu().numpy()
        for b, tokens in enumerate(self.host):
            at = A.cache_rows(table[b], PAGE, POOL, len(tokens))
            for j in range(2 if tokens else 0):
                codes, scales = Q.mx_quantize(np.stack([t[j] for t in tokens]).reshape(len(tokens), -1))
                assert np.array_equal(rows[2 * j][at], codes) and np.array_equal(rows[2 * j + 1][at], scales)
        return rows, table, lens

    def step(self, seed, drafts, masks, accepted, groups, prefix):
        width, batch = max(drafts), self.batch
        slots = torch.empty((batch, width), dtype=torch.int32, device=DEV)
        F.fp4_kv_reserve(self.cache, self.pages, _i32(drafts), slots, self.short, self.ws)
        assert self.short.item() == 0
        depth = [[bin(int(m)).count("1") - 1 for m in row] for row in masks]
        pos = [len(self.host[b]) + depth[b][i] if i < drafts[b] else -1 for b in range(batch) for i in range(width)]
        q = torch.empty((batch, width, HQ, D), dtype=torch.bfloat16, device=DEV)
        qb, k, v = (x.reshape(batch, width, -1, D) for x in self.rows(seed, batch * width, _i32(pos), slots, q.flatten(0, 1)))
        qb = W.bf16_bits(q)
        byte = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)
        common = dict(draft_lens=_i32(drafts))
        tree = common | dict(tree_mask=torch.from_numpy(masks.view(np.int64)).to(DEV))
        state = (self.pages.page_table, self.pages.seq_lens)
        ids = torch.full((batch, width, HK, SELECT), -7, dtype=torch.int32, device=DEV)
        F.fp4_kv_select_mx(q[:, :, ::HQ // HK].contiguous(), *self.index, *state, PAGE, ids,
                           byte(F.fp4_kv_select_workspace_bytes(batch, width, HK, self.pages.page_table.shape[1])), n_first=1, **common)
        outs = [torch.full((batch, width, HQ, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        F.fp4_attn_blocks_mx(q, self.cache, *state, ids, outs[0], byte(F.fp4_attn_blocks_workspace_bytes(batch, width, HQ, D, HK)),
                             **tree)
        F.fp4_attn_shared_mx(q, self.cache, *state, _i32(groups), _i32(prefix), outs[1],
                             byte(F.fp4_attn_shared_workspace_bytes(batch, width, HQ, D, HK, len(prefix))), **tree)

        rows, table, lens = self.stored()
        assert lens.tolist() == [len(h) for h in self.host]
        scores = A.block_scores(qb[:, :, ::HQ // HK], *(x.cpu().numpy() for x in self.index), table, lens, PAGE)
        got = ids.cpu().numpy()
        for b, i, l in np.ndindex(*got.shape[:3]):
            chosen = A.select_blocks(scores[b, i, l], lens[b] // PAGE, SELECT, 1) if i < drafts[b] else [-7] * SELECT
            assert got[b, i, l].tolist() == chosen + [-1] * (SELECT - len(chosen))
        kd, vd = Q.mx_dequant_f64(*rows[:2]).reshape(-1, D), Q.mx_dequant_f64(*rows[2:])
        sizes = (max(lens) + width, SCALE, norm(qb[np.array(pos).reshape(batch, width) >= 0]),
                 float(np.sqrt((kd * kd).sum(-1)).max()), np.abs(vd).max())
        args = (qb, *rows, PAGE, table, lens, HK, SCALE)
        for out, (ref, size) in zip(outs, (A.attn_blocks_mx(*args, got, drafts, masks), A.attn_tree_mx(*args, drafts, masks))):
            check(out, ref, size, D, *sizes)
            assert (out.float().cpu().numpy()[np.isnan(ref)] == 7.0).all()

        most = max(1, max(len(a) for a in accepted))
        F.fp4_kv_compact_reserved(self.cache, self.pages, _i32([a + [-1] * (most - len(a)) for a in accepted]),
                                  _i32([len(a) for a in accepted]), slots)
        for b, kept in enumerate(accepted):
            self.host[b] += [(k[b, i], v[b, i]) for i in kept]
        self.enter()
        self.stored()

    def fork(self, pairs):
        F.fp4_kv_fork(self.pages, _i32(pairs), PAGE)
        for a, b in pairs:
            self.host[b] = list(self.host[a])


def test_prompts_forks_and_steps_of_drafts():
    s = Sparse(5)
    s.prompts(1, [93, 0, 0, 70, 0])
    s.fork([[0, 1], [0, 2], [3, 4]])
    groups, prefix = [0, 3, 5], [93, 70]
    tree = np.array([[1, 3, 5, 11, 21]] * 5, np.uint64)
    s.step(2, [1] * 5, _chain(5, 1), [[0]] * 5, groups, prefix)
    s.step(3, [5, 5, 2, 0, 4], tree, [[0, 2, 4], [0], [], [], [0, 1]], groups, prefix)
    F.fp4_kv_free(s.pages, _i32([1, 4]), PAGE, keep_lens=_i32([64, 0]))     # one shorter than the prefix, one ended
    s.host[1], s.host[4] = s.host[1][:64], []
    s.step(4, [3, 3, 3, 3, 3], tree[:, :3], [[0, 2], [0, 1], [0], [0, 1], [0]], groups, prefix)
    s.step(5, [1] * 5, _chain(5, 1), [[0]] * 5, [0, 3, 3, 4], [64, 10, 0])    # a shorter prefix, an empty group, one of no tokens


def _layer(seed):
    """Buffers of one layer's decode step over 24 forks of 700 tokens, and the step."""
    g = torch.Generator().manual_seed(seed)
    batch, n, pages = 24, 700, 64
    bf = lambda *shape: torch.randn(shape, generator=g).bfloat16().to(DEV)
    z = lambda rows, w: torch.zeros((rows, w), dtype=torch.uint8, device=DEV)
    w = HK * D
    cache = F.KvCache(*(z((pages + batch) * PAGE, x) for x in (w // 2, w // 32) * 2), PAGE)
    F.fp4_kv_append_mx(bf(n, w), _i32(range(n)), cache.k_codes, cache.k_scales)
    F.fp4_kv_append_mx(bf(n, w), _i32(range(n)), cache.v_codes, cache.v_scales)
    index = (z(pages + batch, w // 2), z(pages + batch, w // 32))
    F.fp4_kv_append_mx(bf(n // PAGE, w), _i32(range(n // PAGE)), *index)
    table = np.tile(np.arange(n // PAGE + 1), (batch, 1))
    table[:, n // PAGE] = pages + np.arange(batch)
    state = (_i32(table), _i32([n] * batch))
    slots, pos = _i32((pages + np.arange(batch)) * PAGE + n % PAGE), _i32([n] * batch)
    ang = torch.arange(800)[:, None] * 1e4 ** (-torch.arange(0, ROT, 2) / ROT)
    angles = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
    qkv = bf(batch, HQ + 2 * HK, D)
    q = torch.empty((batch, HQ, D), dtype=torch.bfloat16, device=DEV)
    ids = torch.empty((batch, 1, HK, SELECT), dtype=torch.int32, device=DEV)
    outs = [torch.empty((batch, 1, HQ, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    groups, prefix = _i32([0, batch]), _i32([n // PAGE * PAGE])
    byte = lambda n: torch.empty(n, dtype=torch.uint8, device=DEV)
    works = (byte(F.fp4_kv_select_workspace_bytes(batch, 1, HK, table.shape[1])),
             byte(F.fp4_attn_blocks_workspace_bytes(batch, 1, HQ, D, HK)),
             byte(F.fp4_attn_shared_workspace_bytes(batch, 1, HQ, D, HK, 1)))

    def step():
        F.fp4_kv_append_rope_mx(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], cache, slots, q_out=q, positions=pos,
                                cos_sin=angles, norm=True)
        F.fp4_kv_select_mx(q[:, None, :HK], *index, *state, PAGE, ids, works[0])
        F.fp4_attn_blocks_mx(q[:, None], cache, *state, ids, outs[0], works[1])
        F.fp4_attn_shared_mx(q[:, None], cache, *state, groups, prefix, outs[1], works[2])
    return qkv, step, (q, ids, *outs, *cache[:4])


def test_layers_on_two_streams_at_once():
    layers = [_layer(s) for s in (1, 2)]
    want = []
    for qkv, step, results in layers:
        step()
        want.append([r.clone() for r in results])
        for r in results[:4]:
            r.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for (_, step, _), stream in zip(layers, streams):
            with torch.cuda.stream(stream):
                step()
    torch.cuda.synchronize()
    for (_, _, results), w in zip(layers, want):
        assert all(torch.equal(r, x) for r, x in zip(results, w))


def test_a_captured_step_follows_its_inputs():
    qkv, step, results = _layer(3)
    inputs = [torch.randn(qkv.shape, generator=torch.Generator().manual_seed(40 + i)).bfloat16().to(DEV) for i in range(4)]
    want = []
    for x in inputs:
        qkv.copy_(x)
        step()
        want.append([r.clone() for r in results])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in (2, 0, 3, 1, 1):
        qkv.copy_(inputs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(r, x) for r, x in zip(results, want[i]))
        (inputs[i] * 2).sum().item()
