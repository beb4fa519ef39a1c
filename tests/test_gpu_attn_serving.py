"""The attention path as a serving loop runs it: two layers of a toy model take
prompts and steps of drafted tokens through norms and rotation, attention over the
prompt, the paged cache (reserve, append, commit, fork, cut) and attention over it,
with the float64 definitions beside every step."""
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

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, POOL, WIDTH = 8, 2, 64, 16, 64, 12
ROT = 64


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Server:
    def __init__(self, batch):
        self.batch = batch
        rows, d = POOL * PAGE, HK * D
        z = lambda w: torch.zeros((rows, w), dtype=torch.uint8, device=DEV)
        self.cache = F.KvCache(z(d // 2), z(d // 32), z(d // 2), z(d // 32), PAGE)
        self.pages = F.KvPages(torch.full((batch, WIDTH), -1, dtype=torch.int32, device=DEV), _i32([0] * batch),
                               _i32([0] * batch), _i32([0] * POOL))
        self.ws = torch.empty(F.fp4_kv_reserve_workspace_bytes(batch, POOL), dtype=torch.uint8, device=DEV)
        self.short = _i32([0])
        ang = np.arange(400)[:, None] * 1e4 ** (-np.arange(0, ROT, 2) / ROT)
        self.table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(DEV)
        self.qw, self.kw = (torch.linspace(0.5, 1.5, D, device=DEV).flip(i).contiguous() for i in ([], [0]))
        self.host = [[] for _ in range(batch)]                        # (k, v) bf16 bits of every committed token

    def projected(self, seed, tokens):
        x = torch.randn((tokens, HQ + 2 * HK, D), generator=torch.Generator().manual_seed(seed))
        return x.bfloat16().to(DEV)

    def rotate(self, qkv, positions):
        """Norms and rotation in place, checked."""
        before = W.bf16_bits(qkv)
        q, k = qkv[:, :HQ], qkv[:, HQ:HQ + HK]
        F.fp4_qk_norm_rope(q, k, q, k, positions, self.table, self.qw, self.kw)
        for x, b, w in ((q, before[:, :HQ], self.qw), (k, before[:, HQ:HQ + HK], self.kw)):
            ref, size = A.norm_rope(b, w.double().cpu().numpy(), 1e-6, self.table.cpu().numpy(), positions.cpu().numpy(), False)
            err = np.abs(FM.bf16_bits_to_f64(W.bf16_bits(x)) - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size).all()

    def append(self, qkv, slots):
        n = qkv.shape[0]
        F.fp4_kv_append_mx(qkv[:, HQ:HQ + HK].reshape(n, -1), slots.view(-1), self.cache.k_codes, self.cache.k_scales)
        F.fp4_kv_append_mx(qkv[:, HQ + HK:].reshape(n, -1), slots.view(-1), self.cache.v_codes, self.cache.v_scales)

    def prompts(self, seed, lens):
        """lens: tokens of each sequence, 0 for none."""
        cu = np.concatenate([[0], np.cumsum(lens)])
        qkv = self.projected(seed, int(cu[-1]))
        self.rotate(qkv, _i32(np.concatenate([np.arange(n) for n in lens])))
        out = torch.zeros((int(cu[-1]), HQ, D), dtype=torch.bfloat16, device=DEV)
        F.fp4_attn_prompt(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:], _i32(cu), out)
        bits = W.bf16_bits(qkv)
        q, k, v = np.split(bits, [HQ, HQ + HK], axis=1)
        ref, size = A.attn_prompt(q, k, v, cu, D ** -0.5)
        check(out, ref, size, D, max(lens), D ** -0.5, norm(q), norm(k), np.abs(FM.bf16_bits_to_f64(v)).max())
        slots = torch.empty((self.batch, max(lens)), dtype=torch.int32, device=DEV)
        F.fp4_kv_reserve(self.cache, self.pages, _i32(lens), slots, self.short, self.ws)
        assert self.short.item() == 0
        flat = torch.cat([slots[b, :n] for b, n in enumerate(lens)])
        self.append(qkv, flat)
        F.fp4_kv_compact(self.cache, self.pages, None, _i32(lens))
        for b, n in enumerate(lens):
            self.host[b] += [(k[cu[b] + i], v[cu[b] + i]) for i in range(n)]

    def step(self, seed, drafts, masks, accepted):
        """drafts: drafted tokens of each sequence (0: it sits out); accepted: which of them stay."""
        width = max(drafts)
        slots = torch.empty((self.batch, width), dtype=torch.int32, device=DEV)
        F.fp4_kv_reserve(self.cache, self.pages, _i32(drafts), slots, self.short, self.ws)
        assert self.short.item() == 0
        qkv = self.projected(seed, self.batch * width)
        lens = [len(h) for h in self.host]
        depth = [[bin(int(m)).count("1") - 1 for m in row] for row in masks]
        pos = [lens[b] + depth[b][i] if i < drafts[b] else -1 for b in range(self.batch) for i in range(width)]
        live = [p >= 0 for p in pos]
        before = qkv.clone()
        F.fp4_qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, :HQ], qkv[:, HQ:HQ + HK], _i32(pos), self.table, self.qw,
                           self.kw)
        dead = torch.tensor([not x for x in live], device=DEV)
        assert torch.equal(qkv[dead].view(torch.int16), before[dead].view(torch.int16))
        self.append(qkv, slots)
        q = qkv[:, :HQ].unflatten(0, (self.batch, width))
        out = torch.full((self.batch, width, HQ, D), 7.0, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(F.fp4_attn_tree_workspace_bytes(self.batch, width, HQ, D, HK), dtype=torch.uint8, device=DEV)
        F.fp4_attn_tree_mx(q, self.cache, self.pages.page_table, self.pages.seq_lens, out, ws, draft_lens=_i32(drafts),
                           tree_mask=torch.from_numpy(masks.view(np.int64)).to(DEV))
        bits = W.bf16_bits(qkv).reshape(self.batch, width, HQ + 2 * HK, D)
        for b, n in enumerate(drafts):
            if not n:
                continue
            tokens = self.host[b] + [(bits[b, i, HQ:HQ + HK], bits[b, i, HQ + HK:]) for i in range(n)]
            k, v = (np.stack([t[j] for t in tokens]).reshape(len(tokens), -1) for j in (0, 1))
            kq, vq = Q.mx_quantize(k), Q.mx_quantize(v)
            ref, size = A.attn_tree_mx(bits[b:b + 1, :n, :HQ], *(np.pad(a, ((0, -len(a) % PAGE), (0, 0))) for a in (*kq, *vq)),
                                       PAGE, np.arange(-(-len(tokens) // PAGE))[None], [lens[b]], HK, D ** -0.5, [n],
                                       masks[b:b + 1, :n])
            kd = Q.mx_dequant_f64(*kq).reshape(-1, D)
            check(out[b:b + 1, :n], ref, size, D, len(tokens), D ** -0.5, norm(bits[b, :n, :HQ]),
                  float(np.sqrt((kd * kd).sum(-1)).max()), np.abs(Q.mx_dequant_f64(*vq)).max())
        assert (out[_i32(drafts)[:, None] <= torch.arange(width, device=DEV)] == 7.0).all()
        most = max(1, max(len(a) for a in accepted))
        F.fp4_kv_compact(self.cache, self.pages, _i32([a + [-1] * (most - len(a)) for a in accepted]), _i32([len(a) for a in accepted]))
        for b, kept in enumerate(accepted):
            self.host[b] += [(bits[b, i, HQ:HQ + HK], bits[b, i, HQ + HK:]) for i in kept]
        assert self.pages.seq_lens.tolist() == [len(h) for h in self.host]


def _chain(batch, width):
    return np.array([[(1 << (i + 1)) - 1 for i in range(width)]] * batch, np.uint64)


def test_layers_each_with_their_cache_and_page_state():
    """Two layers take the same calls: each has its own rows (copies of shared pages and
    moved drafts included; every step is checked against them), and their page states
    stay equal."""
    layers = [Server(4), Server(4)]
    for i, s in enumerate(layers):
        s.prompts(10 + i, [21, 7, 0, 0])
        F.fp4_kv_fork(s.pages, _i32([[0, 2], [0, 3]]), PAGE)
        s.host[2], s.host[3] = list(s.host[0]), list(s.host[0])
    tree = np.array([[1, 3, 5, 11, 21]] * 4, np.uint64)
    for step, (drafts, kept) in enumerate([([5, 5, 5, 5], [[0, 2, 4], [0], [0, 1, 3], []]),
                                           ([5, 2, 5, 3], [[0, 1], [], [0, 2], [0, 2]]),
                                           ([1, 1, 1, 1], [[0], [0], [0], [0]])]):
        for i, s in enumerate(layers):
            s.step(20 + 2 * step + i, drafts, tree[:, :max(drafts)], kept)
        for a, b in zip(layers[0].pages, layers[1].pages):
            assert torch.equal(a, b)
    assert not torch.equal(layers[0].cache.k_codes, layers[1].cache.k_codes)


def test_prompts_steps_forks_and_cuts():
    s = Server(5)
    s.prompts(1, [37, 16, 5, 0, 0])
    s.step(2, [1, 1, 1, 0, 0], _chain(5, 1), [[0], [0], [0], [], []])
    # a tree: 0 -> 1 -> 3, 0 -> 2 -> 4; the accepted path skips rows
    tree = np.array([[1, 3, 5, 11, 21]] * 5, np.uint64)
    s.step(3, [5, 5, 3, 0, 0], tree, [[0, 2, 4], [0], [], [], []])
    F.fp4_kv_fork(s.pages, _i32([[0, 3], [1, 4]]), PAGE)
    s.host[3], s.host[4] = list(s.host[0]), list(s.host[1])
    s.step(4, [5, 1, 5, 5, 2], tree, [[0, 1, 3], [0], [0, 2], [0, 2, 4], []])
    F.fp4_kv_free(s.pages, _i32([3, 1]), PAGE, keep_lens=_i32([20, 0]))
    s.host[3], s.host[1] = s.host[3][:20], []
    s.step(5, [2, 0, 2, 2, 1], _chain(5, 2), [[0, 1], [], [0], [0, 1], [0]])
    s.prompts(6, [0, 21, 0, 0, 0])
    s.step(7, [1, 1, 1, 1, 1], _chain(5, 1), [[0]] * 5)
    F.fp4_kv_free(s.pages, _i32(range(5)), PAGE)
    assert (s.pages.page_refs == 0).all() and (s.pages.page_table == -1).all()
