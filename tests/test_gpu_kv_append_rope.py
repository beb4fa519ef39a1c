"""GPU parity of the append with the rotation on the way (fp4_kv_append_rope_mx):
every byte against the oracle without the head norms, and against fp4_qk_norm_rope
and two fp4_kv_append_mx with them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
import workloads as W
from gpu_util import DEV, describe_mismatch, host_u8
from oracle import attn as A
from oracle import quant as Q

pytestmark = pytest.mark.gpu
PLACES = 700


def _table(rot, places=PLACES):
    ang = np.arange(places)[:, None] * 1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def _i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


class Case:
    """Columns of one projection, an odd page size, shuffled slots of which some are -1 or past the cache."""

    def __init__(self, seed, tokens, hq, hk, d, rot, spread=6, page=48):
        rng = np.random.default_rng(seed)
        x = rng.standard_normal((tokens, hq + 2 * hk, d)) * np.exp2(rng.integers(-spread, spread + 1, (tokens, hq + 2 * hk, 1)))
        x[rng.random(x.shape) < 0.02] = 0.0
        self.qkv = W.to_bf16(x).to(DEV)
        self.q, self.k, self.v = self.qkv[:, :hq], self.qkv[:, hq:hq + hk], self.qkv[:, hq + hk:]
        self.pages = -(-tokens // page) + 1
        slots = rng.permutation(self.pages * page)[:tokens]
        slots[rng.random(tokens) < 0.1] = -1
        if tokens > 2:
            slots[1] = self.pages * page                          # the first row past the cache
        self.slots, self.page, self.hk, self.d = slots.astype(np.int32), page, hk, d
        self.positions = rng.integers(0, PLACES, tokens).astype(np.int32)
        self.table = _table(rot)
        self.q_out = torch.full((tokens, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)

    def cache(self, values=True):
        rows, d = self.pages * self.page, self.hk * self.d
        fill = lambda w, b: torch.full((rows, w), b, dtype=torch.uint8, device=DEV)
        return F.KvCache(fill(d // 2, 0xA5), fill(d // 32, 0x5A), fill(d // 2, 0xC3) if values else None,
                         fill(d // 32, 0x3C) if values else None, self.page)


def _same(got, want, names=("k_codes", "k_scales", "v_codes", "v_scales")):
    for n, a, b in zip(names, got, want):
        assert np.array_equal(a, b), describe_mismatch(n, a, b)


SHAPES = [(1, 1, 1, 32, 32), (3, 5, 1, 32, 16), (7, 8, 2, 64, 64), (65, 20, 4, 96, 64), (17, 64, 8, 128, 128),
          (33, 6, 3, 192, 96), (5, 16, 2, 256, 256), (9, 4, 4, 224, 160), (300, 64, 8, 128, 128), (2, 3, 1, 160, 112),
          (130, 0, 2, 128, 48)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", SHAPES)
def test_rotated_rows_and_cache_bytes(tokens, hq, hk, d, rot, interleaved):
    c = Case(tokens + d, tokens, hq, hk, d, rot)
    c.positions[tokens // 2] = -1 if interleaved else PLACES      # padding: nothing of it is written
    cache = c.cache()
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, cache, _i32(c.slots), c.q_out, _i32(c.positions), torch.from_numpy(c.table).to(DEV),
                            interleaved=interleaved)
    live = (c.positions >= 0) & (c.positions < PLACES)
    got = W.bf16_bits(c.q_out)
    want = A.turned_bf16(W.bf16_bits(c.q), c.table, c.positions, interleaved)
    assert np.array_equal(got[live], want[live]), describe_mismatch("q_out", got[live], want[live])
    assert (c.q_out.cpu().float().numpy()[~live] == 7.0).all()
    keys = A.turned_bf16(W.bf16_bits(c.k), c.table, c.positions, interleaved)
    slots = np.where(live, c.slots, -1)
    start = [host_u8(t) for t in c.cache()[:4]]
    _same([host_u8(t) for t in cache[:4]], [*Q.kv_append_mx(start[0], start[1], keys.reshape(tokens, -1), slots),
                                            *Q.kv_append_mx(start[2], start[3], W.bf16_bits(c.v).reshape(tokens, -1), slots)])


@pytest.mark.parametrize("interleaved,weight", [(False, None), (True, torch.float32), (False, torch.bfloat16)])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", SHAPES[1:-1] + [(2100, 40, 8, 128, 128)])
def test_with_norms_it_is_the_three_calls(tokens, hq, hk, d, rot, interleaved, weight):
    c = Case(7 * tokens + d, tokens, hq, hk, d, rot)
    c.positions[0] = -5
    cos_sin, positions, slots = torch.from_numpy(c.table).to(DEV), _i32(c.positions), _i32(c.slots)
    w = [None, None] if weight is None else \
        list((1 + 0.3 * torch.randn((2, d), generator=torch.Generator().manual_seed(d))).to(DEV, weight))
    one, three = c.cache(), c.cache()
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, one, slots, c.q_out, positions, cos_sin, norm=True, q_weight=w[0], k_weight=w[1],
                            eps=1e-5, interleaved=interleaved)
    qo, ko = torch.full_like(c.q_out, 7.0), torch.zeros((tokens, hk, d), dtype=torch.bfloat16, device=DEV)
    F.fp4_qk_norm_rope(c.q, c.k, qo, ko, positions, cos_sin, w[0], w[1], 1e-5, interleaved)
    kept = torch.where((positions >= 0) & (positions < PLACES), slots, -1)
    F.fp4_kv_append_mx(ko.flatten(1), kept, three.k_codes, three.k_scales)
    F.fp4_kv_append_mx(c.v.reshape(tokens, -1), kept, three.v_codes, three.v_scales)
    _same([W.bf16_bits(c.q_out)], [W.bf16_bits(qo)], ["q_out"])
    _same([host_u8(t) for t in one[:4]], [host_u8(t) for t in three[:4]])


def test_without_rotation_it_is_two_appends():
    c = Case(5, 90, 4, 3, 96, 0)
    one, two = c.cache(), c.cache()
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, one, _i32(c.slots), c.q_out)
    for x, at in ((c.k, 0), (c.v, 2)):
        F.fp4_kv_append_mx(x.flatten(1).contiguous(), _i32(c.slots), two[at], two[at + 1])
    assert torch.equal(c.q_out, c.q)
    _same([host_u8(t) for t in one[:4]], [host_u8(t) for t in two[:4]])


def test_queries_in_place_keys_only_and_no_queries():
    c = Case(6, 40, 8, 2, 64, 64)
    cos_sin, positions, slots = torch.from_numpy(c.table).to(DEV), _i32(c.positions), _i32(c.slots)
    whole, keys, bare = c.cache(), c.cache(values=False), c.cache()
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, whole, slots, c.q_out, positions, cos_sin)
    F.fp4_kv_append_rope_mx(None, c.k, c.v, bare, slots, None, positions, cos_sin)
    _same([host_u8(t) for t in bare[:4]], [host_u8(t) for t in whole[:4]])
    before = c.qkv.clone()
    F.fp4_kv_append_rope_mx(c.q, c.k, None, keys, slots, c.q, positions, cos_sin)       # q_out is q
    assert torch.equal(c.q, c.q_out) and torch.equal(c.qkv[:, 8:], before[:, 8:])
    _same([host_u8(t) for t in keys[:2]], [host_u8(t) for t in whole[:2]])


def test_far_rows_of_a_large_cache():
    """Cache rows whose codes lie more than 2^32 bytes in."""
    hk, d, page = 4, 256, 64
    pages = (1 << 32) // (page * hk * d // 2) + 3
    rows = pages * page
    empty = lambda w: torch.empty((rows, w), dtype=torch.uint8, device=DEV)
    cache = F.KvCache(empty(hk * d // 2), empty(hk * d // 32), empty(hk * d // 2), empty(hk * d // 32), page)
    slots = np.array([rows - 1, 5, rows - page, rows // 2], np.int32)
    rng = np.random.default_rng(3)
    x = W.to_bf16(rng.standard_normal((4, 2 * hk, d))).to(DEV)
    table, positions = _table(d), np.array([0, 1, 699, 350], np.int32)
    F.fp4_kv_append_rope_mx(None, x[:, :hk], x[:, hk:], cache, _i32(slots), None, _i32(positions), torch.from_numpy(table).to(DEV))
    keys = A.turned_bf16(W.bf16_bits(x[:, :hk]), table, positions, False).reshape(4, -1)
    at = torch.from_numpy(slots.astype(np.int64)).to(DEV)
    want = [*Q.mx_quantize(keys), *Q.mx_quantize(W.bf16_bits(x[:, hk:]).reshape(4, -1))]
    _same([host_u8(t[at]) for t in cache[:4]], want)


def test_captured_and_on_another_stream():
    c = Case(8, 64, 16, 4, 128, 128)
    cos_sin, positions, slots = torch.from_numpy(c.table).to(DEV), _i32(c.positions), _i32(c.slots)
    eager, caught = c.cache(), c.cache()
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, eager, slots, c.q_out, positions, cos_sin)
    out, side, graph = torch.zeros_like(c.q_out), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        F.fp4_kv_append_rope_mx(c.q, c.k, c.v, caught, slots, out, positions, cos_sin)
    for _ in range(3):
        out.zero_()
        for t in caught[:4]:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.q_out)
        used = torch.from_numpy(c.slots[(c.slots >= 0) & (c.slots < c.pages * c.page)].astype(np.int64)).to(DEV)
        for a, b in zip(caught[:4], eager[:4]):
            assert torch.equal(a[used], b[used])


def test_an_empty_call_and_an_empty_cache():
    c = Case(9, 12, 4, 2, 64, 64)
    cos_sin = torch.from_numpy(c.table).to(DEV)
    cache = c.cache()
    F.fp4_kv_append_rope_mx(c.q[:0], c.k[:0], c.v[:0], cache, _i32(c.slots[:0]), c.q_out[:0], _i32(c.positions[:0]), cos_sin)
    _same([host_u8(t) for t in cache[:4]], [host_u8(t) for t in c.cache()[:4]])
    none = F.KvCache(*(t[:0] for t in cache[:4]), c.page)
    F.fp4_kv_append_rope_mx(c.q, c.k, c.v, none, _i32(c.slots), c.q_out, _i32(c.positions), cos_sin)
    want = A.turned_bf16(W.bf16_bits(c.q), c.table, c.positions, False)
    _same([W.bf16_bits(c.q_out)], [want], ["q_out"])
