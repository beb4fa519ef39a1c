"""Host-side refusals of the serving step's entry points over the paged cache (append
with rotation, shared prefixes, selected blocks), and pins of their oracle (no GPU
needed): the documented status before any HIP call, and the binding's checks."""
import struct
from fractions import Fraction

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
from oracle import attn as A
from oracle import formats as FM

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, HIPERR = 0, -1, -2, -3, -4, -5, -6
M = 1 << 20             # 16-byte aligned, never dereferenced by rejected calls


def _cache(**kw):
    v = dict(k_codes=20 * M, k_scales=21 * M, v_codes=22 * M, v_scales=23 * M, num_pages=10, d=128, page_size=16) | kw
    return struct.pack("=4Q3q", *(v[n] or 0 for n in v))


def _error():
    return F.lib.fp4_last_error().decode()


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _int(*s):
    return torch.zeros(s, dtype=torch.int32)


BAD_CACHES = [(dict(page_size=24), SHAPE), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
              (dict(k_codes=None), INVALID), (dict(k_scales=20 * M + 4), ALIGN), (dict(v_codes=None), INVALID),
              (dict(v_scales=M + 8), ALIGN), (dict(num_pages=1 << 28), SHAPE)]


# ------------------------------------------------------------- append with rotation

def _append(q=M, k=2 * M, v=3 * M, tokens=4, hq=4, hk=2, d=64, ld_q=256, ld_k=128, ld_v=128, norm=1, qw=None, kw=None, dt=0,
            eps=1e-6, table=5 * M, places=100, rot=64, pos=6 * M, qo=7 * M, ld_qo=256, cache=None, slots=8 * M):
    return F.lib.fp4_kv_append_rope_mx(q, k, v, tokens, hq, hk, d, ld_q, ld_k, ld_v, norm, qw, kw, dt, eps, table, places, rot, 0,
                                       pos, qo, ld_qo, cache or _cache(), slots, None)


def test_append_rejections():
    assert _append(tokens=-1) == INVALID and _append(hq=-1) == INVALID and _append(hk=0) == INVALID
    for d in (0, 16, 48, 288):
        assert _append(d=d) == SHAPE, d
    assert _append(rot=80) == SHAPE and _append(rot=24) == SHAPE and _append(rot=-16) == SHAPE
    assert _append(dt=2) == INVALID and _append(tokens=1 << 24) == SHAPE
    assert _append(eps=-1.0) == INVALID and _append(eps=float("nan")) == INVALID
    assert _append(norm=0, qw=M) == INVALID and _append(norm=0, kw=M) == INVALID
    assert _append(ld_q=248) == INVALID and _append(ld_q=260) == ALIGN and _append(ld_v=120) == INVALID
    for name in ("q", "k", "v", "qo", "table", "pos", "slots"):
        assert _append(**{name: None}) == INVALID, name
        assert _append(**{name: 9 * M + 2}) == ALIGN, name
    assert _append(qw=M + 8) == ALIGN and _append(kw=M + 8) == ALIGN and _append(places=-1) == INVALID
    for kw, status in BAD_CACHES:
        assert _append(cache=_cache(**kw)) == status, kw
    assert _append(cache=_cache(d=256)) == SHAPE
    assert _append(tokens=0, q=None, k=None, v=None, slots=None) == OK
    assert _append(hq=0, cache=_cache(num_pages=0), k=None, v=None, slots=None) == OK


def test_append_refuses_outputs_over_inputs_and_one_another():
    def overlap(what, **kw):
        assert _append(**kw) == INVALID and _error() == what, (kw, _error())

    # the cache: 160 rows of 64 bytes of codes and 4 of scales; q rows of 512 bytes, k and v of 256
    overlap("q_out overlaps q without being q itself", qo=M + 16)
    overlap("q_out overlaps q without being q itself", qo=M, ld_qo=264)
    overlap("q_out overlaps k", qo=2 * M)
    overlap("q_out overlaps v", qo=3 * M + 3 * 256)
    overlap("q_out overlaps q_weight", qw=7 * M + 4 * 512 - 16)
    overlap("q_out overlaps k_weight", kw=7 * M)
    overlap("q_out overlaps cos_sin", table=7 * M - 100 * 64 * 4 + 16)
    overlap("q_out overlaps positions", pos=7 * M)
    overlap("q_out overlaps slots", slots=7 * M + 16)
    overlap("q_out overlaps k_codes", qo=20 * M + 160 * 64 - 16)
    overlap("q_out overlaps v_scales", qo=23 * M)
    overlap("k_codes overlaps q", q=20 * M, qo=20 * M + 512 * 64)
    overlap("k_scales overlaps k", k=21 * M - 1008)
    overlap("v_codes overlaps v", v=22 * M)
    overlap("k_codes overlaps k_weight", kw=20 * M + 64)
    overlap("v_scales overlaps slots", slots=23 * M + 4)
    overlap("v_codes overlaps k_codes", cache=_cache(v_codes=20 * M))
    overlap("v_scales overlaps k_codes", cache=_cache(v_scales=20 * M + 160 * 64 - 16))


def test_binding_checks_the_append():
    x = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    q, k, v = x[:, :2], x[:, 2:4], x[:, 4:]
    cache = F.KvCache(_u8(160, 64), _u8(160, 4), _u8(160, 64), _u8(160, 4), 16)
    out, slots = torch.zeros((4, 2, 64), dtype=torch.bfloat16), _int(4)
    with pytest.raises(TypeError, match="bfloat16"):
        F.fp4_kv_append_rope_mx(q.float(), k, v, cache, slots, out)
    with pytest.raises(TypeError, match="v must be a torch tensor"):
        F.fp4_kv_append_rope_mx(q, k, None, cache, slots, out)
    with pytest.raises(TypeError, match="q_out"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots)
    with pytest.raises(ValueError, match="v has shape"):
        F.fp4_kv_append_rope_mx(q, k, v[:3], cache, slots, out)
    with pytest.raises(ValueError, match="q has shape"):
        F.fp4_kv_append_rope_mx(q[:3], k, v, cache, slots, out)
    with pytest.raises(ValueError, match="q_out has shape"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots, out[:, :1])
    with pytest.raises(ValueError, match="slots has shape"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, _int(5), out)
    with pytest.raises(TypeError, match="slots"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots.long(), out)
    with pytest.raises(ValueError, match="heads of k"):
        F.fp4_kv_append_rope_mx(q, x[:, ::3], v, cache, slots, out)
    with pytest.raises(TypeError, match="positions"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots, out, None, torch.zeros((8, 64)))
    with pytest.raises(ValueError, match="positions"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots, out, _int(3), torch.zeros((8, 64)))
    with pytest.raises(ValueError, match="k_weight"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots, out, norm=True, k_weight=torch.ones(32))
    with pytest.raises(ValueError, match="k_codes"):
        F.fp4_kv_append_rope_mx(q, k, v, cache._replace(page_size=48), slots, out)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_kv_append_rope_mx(q, k, v, cache, slots, out)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_turn_in_exact_arithmetic(interleaved):
    """Every turned value by fractions: two fp32 roundings, then bf16's; a quarter turn swaps the pair."""
    rng = np.random.default_rng(1)
    bits = FM.bf16_rne_of_f64(rng.standard_normal((6, 2, 64)) * np.exp2(rng.integers(-9, 9, (6, 2, 1))))
    ang = rng.standard_normal((5, 16)) * 100
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
    table[4, :16], table[4, 16:] = 0.0, 1.0
    pos = np.array([0, 1, 2, 3, 4, 9])
    got = A.turned_bf16(bits, table, pos, interleaved)
    assert np.array_equal(got[5], bits[5]) and np.array_equal(got[..., 32:], bits[..., 32:])
    value = lambda b: FM.bf16_bits_to_fraction(int(b))
    for t in range(5):
        for i in range(16):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, 16 + i)
            c, s = Fraction(float(table[t, i])), Fraction(float(table[t, 16 + i]))
            for h in range(2):
                x, y = value(bits[t, h, a]), value(bits[t, h, b])
                for at, z in ((a, x * c - FM.round_fp32(y * s)), (b, y * c + FM.round_fp32(x * s))):
                    assert FM.round_bf16(FM.round_fp32(z)) == value(got[t, h, at])
    a, b = (np.arange(0, 32, 2), np.arange(1, 32, 2)) if interleaved else (np.arange(16), np.arange(16, 32))
    assert np.array_equal(got[4][:, b], bits[4][:, a]) and np.array_equal(got[4][:, a], bits[4][:, b] ^ 0x8000)
