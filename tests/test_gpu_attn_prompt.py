"""GPU parity of the causal attention over packed prompts (fp4_attn_prompt) with
the float64 definition; tolerance in attn_check.py."""
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

pytestmark = pytest.mark.gpu


class Batch:
    """One projection [tokens, q_heads + 2 kv_heads, d] of packed sequences, NaN in the padding rows."""

    def __init__(self, seed, lens, q_heads, kv_heads, d, pad=0, front=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.cu = np.concatenate([[front], front + np.cumsum(lens)]).astype(np.int32)
        n = int(self.cu[-1]) + pad
        self.heads, self.d = (q_heads, kv_heads), d
        x = rng.standard_normal((n, q_heads + 2 * kv_heads, d)) * spread
        x[:front], x[self.cu[-1]:] = np.nan, np.nan
        self.bits = W.bf16_bits(W.to_bf16(x))

    def run(self, scale=None, bits=None, out=None, x=None):
        hq, hk = self.heads
        x = W.from_bits(self.bits).to(DEV) if x is None else x
        out = torch.full((x.shape[0], hq, self.d), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        F.fp4_attn_prompt(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], torch.from_numpy(self.cu).to(DEV), out, scale=scale)
        self.check(out, scale)
        return out

    def check(self, out, scale=None):
        hq, hk = self.heads
        scale = self.d ** -0.5 if scale is None else scale
        q, k, v = np.split(self.bits, [hq, hq + hk], axis=1)
        ref, size = A.attn_prompt(q, k, v, self.cu, scale)
        rows = np.zeros(len(q), bool)
        rows[self.cu[0]:self.cu[-1]] = True
        check(out, ref, size, self.d, int(np.diff(self.cu).max(initial=0)), scale, norm(q[rows]), norm(k[rows]),
              np.abs(FM.bf16_bits_to_f64(v[rows])).max(initial=0.0))
        assert (out.cpu().float().numpy()[np.isnan(ref)] == 7.0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (4, 2), (16, 2), (10, 1)])
def test_ragged_packed_sequences(d, q_heads, kv_heads):
    Batch(d + q_heads, [1, 2, 31, 0, 32, 33, 64, 65, 127, 128, 129, 0, 200], q_heads, kv_heads, d, pad=3).run()


@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (256, 1), (64, 1500), (128, 1023), (128, 1025), (256, 700)])
def test_one_sequence(d, n):
    Batch(n, [n], 8, 4, d).run()


def test_rows_outside_every_sequence_may_hold_anything():
    Batch(1, [70, 5, 130], 4, 4, 128, pad=40, front=9).run()


def test_more_sequences_than_rows_in_a_tile():
    Batch(2, np.random.default_rng(0).integers(0, 4, 400).tolist(), 2, 1, 64).run()


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(scale):
    Batch(3, [150, 67], 8, 8, 128).run(scale)


def test_rising_scores_move_the_reference():
    b = Batch(4, [600], 2, 1, 64, spread=1.0)
    k = FM.bf16_bits_to_f64(b.bits[:, 2:3]) * np.exp2(np.linspace(-3, 6, 600))[:, None, None]
    b.bits[:, 2:3] = W.bf16_bits(W.to_bf16(k))
    b.run(0.1)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_hidden_keys_and_values_that_are_no_numbers(d):
    """Only rows that see an infinite value or one that is no number have it, each in
    its own place; rows that see such a key are no numbers."""
    hq, hk, seqs = 4, 2, [(0, 330), (330, 400)]
    b = Batch(8, [330, 70], hq, hk, d)
    b.bits[[150, 290, 345, 399], hq + hk:] &= 0x807F         # tiny values where the bad ones will stand
    bad = W.from_bits(b.bits).to(DEV)
    expected = np.zeros((400, hq, d))                        # added to the result
    for token, head, first, last, value in ((150, 0, 3, 4, np.nan), (150, 1, 0, d, np.inf), (290, 0, 17, 40, -np.inf),
                                            (345, 1, 1, 2, np.nan), (399, 0, 0, d, np.nan)):
        bad[token, hq + hk + head, first:last] = value
        end = 330 if token < 330 else 400
        expected[token:end, 2 * head:2 * head + 2, first:last] += value
    for token, head in ((200, 0), (360, 1)):
        bad[token, hq + head] = np.nan
        expected[token:(330 if token < 330 else 400), 2 * head:2 * head + 2] = np.nan
    out = torch.full((400, hq, d), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp4_attn_prompt(bad[:, :hq], bad[:, hq:hq + hk], bad[:, hq + hk:], torch.from_numpy(b.cu).to(DEV), out)
    q, k, v = np.split(b.bits, [hq, hq + hk], axis=1)
    ref, size = A.attn_prompt(q, k, v, b.cu, d ** -0.5)
    got = out.cpu().float().numpy()
    odd = ~np.isfinite(expected)
    np.testing.assert_array_equal(got[odd], expected[odd])
    ref[odd] = np.nan
    check(out, ref, size, d, 330, d ** -0.5, norm(q), norm(k), np.abs(FM.bf16_bits_to_f64(v)).max())


def test_rows_whose_offsets_pass_32_bits():
    """Query, key, value and result rows 32 MB apart."""
    b = Batch(9, [3, 130, 20], 4, 2, 64)
    ld = (1 << 24) - 8
    base = torch.empty(153 * ld, dtype=torch.bfloat16, device=DEV)
    x = base.as_strided((153, 8, 64), (ld, 64, 1))
    x.copy_(W.from_bits(b.bits).to(DEV))
    out = base.as_strided((153, 4, 64), (ld, 64, 1), 1024)
    out.fill_(7.0)
    b.run(x=x, out=out)


def test_separate_tensors_wide_rows_and_no_rows():
    b = Batch(5, [90, 40], 4, 2, 64)
    x = W.from_bits(b.bits).to(DEV)
    wide = torch.full((130, 9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp4_attn_prompt(x[:, :4].contiguous(), x[:, 4:6].contiguous(), x[:, 6:], torch.from_numpy(b.cu).to(DEV), wide[:, 3:7])
    b.check(wide[:, 3:7])
    assert (wide[:, :3] == 7).all() and (wide[:, 7:] == 7).all()
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    F.fp4_attn_prompt(e, e, e, torch.zeros(3, dtype=torch.int32, device=DEV), e)
    F.fp4_attn_prompt(x[:, :4], x[:, 4:6], x[:, 6:], torch.zeros(1, dtype=torch.int32, device=DEV), wide[:, 3:7])


def test_bounds_outside_the_rows_are_cut_off():
    """cu_seqlens values outside [0, tokens] are taken as the nearest bound."""
    b = Batch(6, [60, 100], 2, 2, 64)
    b.cu = np.array([-5, 60, 160, 1 << 30, 1 << 30], np.int32)
    x = W.from_bits(b.bits).to(DEV)
    out = torch.full((160, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp4_attn_prompt(x[:, :2], x[:, 2:4], x[:, 4:], torch.from_numpy(b.cu).to(DEV), out)
    b.cu = np.array([0, 60, 160], np.int32)
    b.check(out)


def test_same_call_same_bits_side_stream_and_replayed_graph():
    b = Batch(7, [300, 17, 90], 8, 2, 128)
    x, cu = W.from_bits(b.bits).to(DEV), torch.from_numpy(b.cu).to(DEV)
    out = b.run(x=x)
    again = torch.full_like(out, 7.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        F.fp4_attn_prompt(x[:, :8], x[:, 8:10], x[:, 10:], cu, again)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp4_attn_prompt(x[:, :8], x[:, 8:10], x[:, 10:], cu, again)
    for seed, lens in ((1, [407]), (2, [1, 405, 1]), (3, [100, 100, 207])):
        new = Batch(seed, lens + [0] * (3 - len(lens)), 8, 2, 128)
        x.copy_(W.from_bits(new.bits))
        cu.copy_(torch.from_numpy(new.cu))
        again.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        new.check(again)
