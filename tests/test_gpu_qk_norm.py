"""GPU parity of the head norms with rotation (fp4_qk_norm_rope) with the
float64 definition.

Tolerance of a value y made of terms of total magnitude S: the rounding to bf16
(half a step, 2^-8 |y|) and fp32 arithmetic before it.  There a value passes at
most 8 + 5 additions of the sum of squares (half of whose relative error reaches
the root), its scaling, the reciprocal root (2 steps), two products with the
norm and the weight, and two products and a sum of the rotation: below
32 roundings of 2^-24 relative to S, that is 2^-19 S.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
import workloads as W
from oracle import attn as A
from oracle import formats as FM
from gpu_util import DEV

pytestmark = pytest.mark.gpu


def _table(places, rot):
    turns = 1e6 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(places)[:, None] * turns
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).to(DEV)


def _inputs(seed, tokens, hq, hk, d):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((tokens, hq + 2 * hk, d)) * np.exp2(rng.integers(-6, 7, (tokens, hq + 2 * hk, 1)))
    return W.to_bf16(x).to(DEV), 1 + 0.3 * rng.standard_normal((2, d))


def _close(got, ref, size):
    got = FM.bf16_bits_to_f64(W.bf16_bits(got))
    live = ~np.isnan(ref)
    assert live.any() or ref.size == 0
    err, tol = np.abs(got - ref)[live], (2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size)[live]
    assert (err <= tol).all(), f"{(err > tol).sum()} values off, worst {np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance"


def _check(q, k, qo, ko, weights, cos_sin, positions, interleaved, eps=1e-6):
    table = None if cos_sin is None else cos_sin.cpu().numpy()
    pos = None if positions is None else positions.cpu().numpy()
    for x, o, w in ((q, qo, weights[0]), (k, ko, weights[1])):
        _close(o, *A.norm_rope(W.bf16_bits(x), w, eps, table, pos, interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rot", [(1, 1, 1, 16, 16), (3, 5, 1, 32, 16), (7, 8, 2, 64, 64), (65, 20, 4, 96, 64),
                                                (17, 64, 8, 128, 128), (33, 6, 3, 192, 96), (5, 16, 2, 256, 256),
                                                (9, 4, 4, 240, 160), (300, 64, 8, 128, 128), (2, 3, 1, 112, 112)])
def test_norm_rope_shapes(tokens, hq, hk, d, rot, interleaved):
    qkv, w = _inputs(tokens + d, tokens, hq, hk, d)
    wt = torch.from_numpy(w).to(DEV, torch.float32 if d % 64 else torch.bfloat16)
    q, k = qkv[:, :hq], qkv[:, hq:hq + hk]                       # columns of one projection
    qo = torch.full((tokens, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    ko = torch.full((tokens, hk, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    cos_sin = _table(500, rot)
    positions = torch.from_numpy(np.random.default_rng(1).integers(0, 500, tokens).astype(np.int32)).to(DEV)
    F.fp4_qk_norm_rope(q, k, qo, ko, positions, cos_sin, wt[0].contiguous(), wt[1].contiguous(), interleaved=interleaved)
    _check(q, k, qo, ko, wt.double().cpu().numpy(), cos_sin, positions, interleaved)


@pytest.mark.parametrize("hq,hk,d,rot,interleaved", [(28, 4, 128, 128, False), (40, 8, 128, 64, True), (56, 8, 128, 96, False),
                                                     (64, 8, 128, 128, True), (20, 4, 96, 64, True), (130, 7, 64, 64, False),
                                                     (30, 3, 256, 256, False), (100, 25, 32, 32, True), (260, 5, 16, 16, False)])
def test_many_tokens(hq, hk, d, rot, interleaved):
    """Enough tokens that a group of lanes takes 2 to 5 heads; some of them checked."""
    tokens = 4096 * 256 // (1 << max(1, (d // 8 - 1).bit_length())) // (hq + hk) + 3
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn((tokens, hq + hk, d), generator=g, device=DEV).bfloat16()
    wt = (1 + 0.3 * torch.randn((2, d), generator=g, device=DEV)).float()
    cos_sin = _table(300, rot)
    positions = torch.randint(0, 300, (tokens,), generator=g, device=DEV).int()
    qo = torch.full((tokens, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    ko = torch.full((tokens, hk, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    F.fp4_qk_norm_rope(x[:, :hq], x[:, hq:], qo, ko, positions, cos_sin, wt[0].contiguous(), wt[1].contiguous(),
                       interleaved=interleaved)
    some = torch.tensor([0, 1, 2, tokens // 2, tokens - 2, tokens - 1], device=DEV)
    _check(x[some, :hq], x[some, hq:], qo[some], ko[some], wt.double().cpu().numpy(), cos_sin, positions[some], interleaved)
    # every token's result depends on that token alone
    q1, k1 = torch.empty_like(qo[:50]), torch.empty_like(ko[:50])
    for t in range(0, tokens, 50):
        n = min(50, tokens - t)
        F.fp4_qk_norm_rope(x[t:t + n, :hq], x[t:t + n, hq:], q1[:n], k1[:n], positions[t:t + n], cos_sin, wt[0].contiguous(),
                           wt[1].contiguous(), interleaved=interleaved)
        assert torch.equal(q1[:n], qo[t:t + n]) and torch.equal(k1[:n], ko[t:t + n])


def test_rows_whose_offsets_pass_32_bits():
    """Tokens 2 GiB apart."""
    qkv, _ = _inputs(12, 4, 3, 1, 64)
    ld = (1 << 30) + 8
    base = torch.empty(3 * ld + 1024, dtype=torch.bfloat16, device=DEV)
    x, out = base.as_strided((4, 4, 64), (ld, 64, 1)), base.as_strided((4, 4, 64), (ld, 64, 1), 512)
    x.copy_(qkv[:, :4])
    F.fp4_qk_norm_rope(x[:, :3], x[:, 3:], out[:, :3], out[:, 3:])
    _check(qkv[:, :3], qkv[:, 3:4], out[:, :3], out[:, 3:], np.ones((2, 64)), None, None, False)


def test_norms_alone_without_weights_and_zero_rows():
    qkv, _ = _inputs(3, 11, 4, 2, 128)
    qkv[4] = 0
    q, k = qkv[:, :4], qkv[:, 4:6]
    qo, ko = torch.empty_like(q.contiguous()), torch.empty_like(k.contiguous())
    F.fp4_qk_norm_rope(q, k, qo, ko, eps=1e-5)
    _check(q, k, qo, ko, np.ones((2, 128)), None, None, False, eps=1e-5)
    assert (qo[4] == 0).all()


def test_in_place_inside_one_projection_and_padding_tokens():
    """In place: the value columns and the rows of tokens outside the table stay as they were."""
    qkv, w = _inputs(5, 37, 8, 2, 128)
    wt = torch.from_numpy(w).to(DEV, torch.float32)
    before = qkv.clone()
    cos_sin = _table(64, 128)
    pos = np.arange(37, dtype=np.int32)
    pos[[0, 9, 36]] = [-1, 64, 1 << 30]
    positions = torch.from_numpy(pos).to(DEV)
    q, k = qkv[:, :8], qkv[:, 8:10]
    F.fp4_qk_norm_rope(q, k, q, k, positions, cos_sin, wt[0].contiguous(), wt[1].contiguous())
    _check(before[:, :8], before[:, 8:10], q, k, wt.double().cpu().numpy(), cos_sin, positions, False)
    assert torch.equal(qkv[:, 10:].view(torch.int16), before[:, 10:].view(torch.int16))
    for t in (0, 9, 36):
        assert torch.equal(qkv[t].view(torch.int16), before[t].view(torch.int16))


def test_queries_alone_keys_alone_and_nothing():
    qkv, _ = _inputs(8, 6, 3, 1, 64)
    none = torch.empty((6, 0, 64), dtype=torch.bfloat16, device=DEV)
    q = qkv[:, :3]
    qo = torch.empty((6, 3, 64), dtype=torch.bfloat16, device=DEV)
    F.fp4_qk_norm_rope(q, none, qo, none)
    ko = torch.empty_like(qo)
    F.fp4_qk_norm_rope(none, q, none, ko)
    assert torch.equal(qo, ko)
    _close(qo, *A.norm_rope(W.bf16_bits(q), np.ones(64), 1e-6, None, None, False))
    empty = torch.empty((0, 3, 64), dtype=torch.bfloat16, device=DEV)
    F.fp4_qk_norm_rope(empty, empty, empty, empty)


def test_another_stream_and_a_replayed_graph():
    """The call on a side stream, and captured once and replayed on new inputs."""
    qkv, w = _inputs(9, 50, 8, 2, 128)
    wt = torch.from_numpy(w).to(DEV, torch.bfloat16)
    cos_sin, positions = _table(50, 128), torch.arange(50, dtype=torch.int32, device=DEV)
    q, k = qkv[:, :8], qkv[:, 8:10]
    outs = [torch.zeros((50, h, 128), dtype=torch.bfloat16, device=DEV) for h in (8, 2)]

    def call():
        F.fp4_qk_norm_rope(q, k, *outs, positions, cos_sin, wt[0].contiguous(), wt[1].contiguous())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    _check(q, k, *outs, wt.double().cpu().numpy(), cos_sin, positions, False)
    graph = torch.cuda.CUDAGraph()
    weights = wt[0].contiguous(), wt[1].contiguous()
    with torch.cuda.graph(graph):
        F.fp4_qk_norm_rope(q, k, *outs, positions, cos_sin, *weights)
    for seed in (1, 2, 3):
        qkv.copy_(_inputs(seed, 50, 8, 2, 128)[0])
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _check(q, k, *outs, wt.double().cpu().numpy(), cos_sin, positions, False)
