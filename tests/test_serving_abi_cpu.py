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


# ------------------------------------------------------- attention over the cache

def _shared(q=M, ld_q=256, cache=None, table=2 * M, max_pages=4, lens=3 * M, dlens=None, mask=None, groups=4 * M, prefix=5 * M,
            n=2, batch=3, drafts=2, hq=4, hk=2, d=64, scale=0.125, out=6 * M, ld_out=256, ws=8 * M, nbytes=None):
    nbytes = F.lib.fp4_attn_shared_workspace_bytes(3, 2, 4, 64, 2, 2) if nbytes is None else nbytes
    return F.lib.fp4_attn_shared_mx(q, ld_q, cache or _cache(), table, max_pages, lens, dlens, mask, groups, prefix, n, batch,
                                    drafts, hq, hk, d, scale, out, ld_out, ws, nbytes, None)


def _blocks(q=M, ld_q=256, cache=None, table=2 * M, max_pages=4, lens=3 * M, dlens=None, mask=None, ids=4 * M, lists=1, n=5,
            batch=3, drafts=2, hq=4, hk=2, d=64, scale=0.125, out=6 * M, ld_out=256, ws=8 * M, nbytes=None):
    nbytes = F.lib.fp4_attn_blocks_workspace_bytes(3, 2, 4, 64, 2) if nbytes is None else nbytes
    return F.lib.fp4_attn_blocks_mx(q, ld_q, cache or _cache(), table, max_pages, lens, dlens, mask, ids, lists, n, batch, drafts,
                                    hq, hk, d, scale, out, ld_out, ws, nbytes, None)


@pytest.mark.parametrize("call", [_shared, _blocks])
def test_attention_rejections_in_common(call):
    assert call(hq=0) == INVALID and call(hk=0) == INVALID and call(hq=5) == SHAPE and call(hq=8192) == SHAPE
    assert call(d=96) == SHAPE and call(d=128) == SHAPE               # no such head; not the cache's width
    for kw, status in BAD_CACHES:
        assert call(cache=_cache(**kw)) == status, kw
    assert call(cache=_cache(v_codes=None, v_scales=None)) == INVALID
    assert call(drafts=0) == INVALID and call(drafts=65) == INVALID
    assert call(batch=-1) == INVALID and call(max_pages=-1) == INVALID
    assert call(batch=65536) == SHAPE and call(max_pages=1 << 31) == SHAPE
    for scale in (float("inf"), float("nan"), 2.0 ** 127 * 1.5):
        assert call(scale=scale) == INVALID
    for name in ("q", "out"):
        assert call(**{name: None}) == INVALID and call(**{name: M + 8}) == ALIGN
    for name in ("table", "lens"):
        assert call(**{name: None}) == INVALID and call(**{name: M + 2}) == ALIGN
    assert call(dlens=M + 2) == ALIGN and call(mask=M + 4) == ALIGN
    assert call(ld_q=248) == INVALID and call(ld_out=260) == ALIGN
    assert call(out=M + 256) == INVALID and "overlaps" in _error()
    assert call(ws=None) == WORKSPACE and call(nbytes=64) == WORKSPACE and call(ws=M + 8) == ALIGN
    assert call(batch=0, q=None, out=None, table=None, lens=None, ws=None) == OK


def test_shared_prefix_rejections():
    assert _shared(n=-1) == INVALID and _shared(n=1 << 20) == SHAPE
    assert _shared(groups=None) == INVALID and _shared(prefix=None) == INVALID
    assert _shared(groups=M + 2) == ALIGN and _shared(prefix=M + 1) == ALIGN
    need = F.lib.fp4_attn_shared_workspace_bytes(3, 2, 4, 64, 2, 2)
    assert _shared(nbytes=need - 1) == WORKSPACE
    assert _shared(hq=4096, hk=1, drafts=64, batch=60000, cache=_cache(d=64)) == SHAPE     # rows past 2^31
    size = F.lib.fp4_attn_shared_workspace_bytes
    assert 0 < size(3, 2, 4, 64, 2, 0) < need < size(300, 2, 4, 64, 2, 2)
    for bad in ((0, 2, 4, 64, 2, 2), (65536, 2, 4, 64, 2, 2), (3, 65, 4, 64, 2, 2), (3, 2, 5, 64, 2, 2), (3, 2, 4, 96, 2, 2),
                (3, 2, 4, 64, 2, -1), (60000, 64, 4096, 64, 1, 1)):
        assert size(*bad) == 0, bad


def test_block_attention_rejections():
    assert _blocks(lists=3) == INVALID and _blocks(lists=0) == INVALID and _blocks(n=-1) == INVALID
    assert _blocks(n=1 << 20) == SHAPE and _blocks(ids=None) == INVALID and _blocks(ids=M + 2) == ALIGN
    assert _blocks(hq=4096, hk=4096, drafts=64, lists=4096, cache=_cache(d=4096 * 64), ld_q=4096 * 64, ld_out=4096 * 64) == SHAPE
    need = F.lib.fp4_attn_blocks_workspace_bytes(3, 2, 4, 64, 2)
    assert _blocks(nbytes=need - 1) == WORKSPACE and _blocks(nbytes=need - 1, lists=2) == WORKSPACE
    assert F.lib.fp4_attn_blocks_workspace_bytes(3, 0, 4, 64, 2) == 0 and F.lib.fp4_attn_blocks_workspace_bytes(0, 2, 4, 64, 2) == 0


def _select(q=M, ld_q=128, codes=2 * M, scales=3 * M, pages=10, lists=2, dim=64, table=4 * M, max_pages=4, lens=5 * M, dlens=None,
            page=16, batch=3, drafts=2, n=5, first=0, recent=0, ids=6 * M, out=None, ws=8 * M, nbytes=None):
    nbytes = F.lib.fp4_kv_select_workspace_bytes(3, 2, 2, 4) if nbytes is None else nbytes
    return F.lib.fp4_kv_select_mx(q, ld_q, codes, scales, pages, lists, dim, table, max_pages, lens, dlens, page, batch, drafts, n,
                                  first, recent, ids, out, ws, nbytes, None)


def test_select_rejections():
    for name in ("batch", "max_pages", "pages", "n", "first", "recent"):
        assert _select(**{name: -1}) == INVALID, name
    assert _select(drafts=0) == INVALID and _select(drafts=65) == INVALID and _select(lists=0) == INVALID
    for dim in (0, 16, 48, 544):
        assert _select(dim=dim) == SHAPE, dim
    assert _select(page=24) == SHAPE and _select(page=0) == INVALID
    assert _select(batch=65536) == SHAPE and _select(lists=4097) == SHAPE and _select(n=1 << 20) == SHAPE
    assert _select(max_pages=1 << 31) == SHAPE and _select(pages=1 << 31) == SHAPE
    assert _select(batch=60000, drafts=64, lists=4) == SHAPE
    assert _select(ld_q=120) == INVALID and _select(ld_q=132) == ALIGN
    for name in ("q", "codes", "scales", "table", "lens", "ids"):
        assert _select(**{name: None}) == INVALID, name
    assert _select(q=M + 8) == ALIGN and _select(codes=M + 8) == ALIGN
    for name in ("table", "lens", "dlens", "ids", "out"):
        assert _select(**{name: M + 2}) == ALIGN, name
    assert F.lib.fp4_kv_select_workspace_bytes(3, 2, 2, 4) == 3 * 2 * 2 * 16 * 4
    assert _select(ws=None) == WORKSPACE and _select(nbytes=767) == WORKSPACE and _select(ws=M + 8) == ALIGN
    assert _select(batch=0, q=None, ws=None) == OK and _select(n=0, q=None, ids=None, ws=None) == OK


def test_binding_checks_the_selection_and_its_attention():
    q = torch.zeros((3, 2, 2, 64), dtype=torch.bfloat16)
    codes, scales, ids, ws = _u8(10, 64), _u8(10, 4), _int(3, 2, 2, 5), _u8(1 << 16)
    args = lambda **kw: list((dict(q=q, codes=codes, scales=scales, table=_int(3, 4), lens=_int(3), page=16, ids=ids, ws=ws) | kw).values())
    with pytest.raises(TypeError, match="q must be torch.bfloat16"):
        F.fp4_kv_select_mx(*args(q=q.float()))
    for kw in (dict(codes=_u8(10, 32)), dict(scales=_u8(9, 4)), dict(q=q[:, :, :1])):
        with pytest.raises(ValueError, match="index_codes"):
            F.fp4_kv_select_mx(*args(**kw))
    for bad in (_int(3, 2, 5), _int(2, 2, 2, 5), _int(3, 2, 1, 5)):
        with pytest.raises(ValueError, match="block_ids"):
            F.fp4_kv_select_mx(*args(ids=bad))
    with pytest.raises(ValueError, match="scores has shape"):
        F.fp4_kv_select_mx(*args(), scores=torch.zeros(3, 2, 2, 4))
    with pytest.raises(ValueError, match="draft_lens"):
        F.fp4_kv_select_mx(*args(), draft_lens=_int(2))
    with pytest.raises(ValueError, match="page_table"):
        F.fp4_kv_select_mx(*args(table=_int(2, 4)))
    with pytest.raises(ValueError, match="too large"):
        F.fp4_kv_select_mx(*args(), n_first=1 << 40)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_kv_select_mx(*args())
    cache = F.KvCache(_u8(160, 64), _u8(160, 4), _u8(160, 64), _u8(160, 4), 16)
    x = torch.zeros((3, 2, 4, 64), dtype=torch.bfloat16)
    for bad in (_int(3, 2, 3, 5), _int(3, 2, 5), _int(3, 1, 1, 5)):
        with pytest.raises(ValueError, match="block_ids"):
            F.fp4_attn_blocks_mx(x, cache, _int(3, 4), _int(3), bad, x, ws)
    with pytest.raises(ValueError, match="no values"):
        F.fp4_attn_blocks_mx(x, cache._replace(v_codes=None, v_scales=None), _int(3, 4), _int(3), ids, x, ws)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_attn_blocks_mx(x, cache, _int(3, 4), _int(3), ids, x, ws)
    with pytest.raises(ValueError, match="groups has shape"):
        F.fp4_attn_shared_mx(x, cache, _int(3, 4), _int(3), _int(2), _int(2), x, ws)
    with pytest.raises(ValueError, match="prefix_lens"):
        F.fp4_attn_shared_mx(x, cache, _int(3, 4), _int(3), _int(2), _int(1, 1), x, ws)
    with pytest.raises(TypeError, match="groups"):
        F.fp4_attn_shared_mx(x, cache, _int(3, 4), _int(3), _int(2).long(), _int(1), x, ws)
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_attn_shared_mx(x, cache, _int(3, 4), _int(3), _int(2), _int(1), x, ws)


# ------------------------------------------------------------------ oracle pins

def test_oracle_selection_by_hand():
    s = np.array([1.0, 5.0, np.nan, 5.0, -2.0, 5.0, 0.0])
    pick = lambda n, first=0, recent=0, complete=7: A.select_blocks(s, complete, n, first, recent)
    assert pick(2) == [1, 3] and pick(3) == [1, 3, 5] and pick(4) == [0, 1, 3, 5] and pick(9) == [0, 1, 3, 4, 5, 6]
    assert pick(3, 1, 0) == [0, 1, 3] and pick(3, 0, 3) == [4, 5, 6] and pick(2, 1, 2) == [0, 5]
    assert pick(1, 3, 0) == [0] and pick(3, 3, 0) == [0, 1, 3] and pick(2, 0, 0, 1) == [0] and pick(2, 0, 0, 0) == []


def test_oracle_scores_by_hand():
    """One block of ones (code 2) against entries of 1 .. in two pages: 32 times the entry's value."""
    q = FM.bf16_rne_of_f64(np.full((1, 1, 1, 32), 4.0))                      # code 6 (4) at scale 1
    codes = np.full((3, 16), 0x22, np.uint8)                                 # ones
    codes[1], codes[2] = 0xAA, 0x77                                          # minus one, six
    scales = np.array([[127], [128], [126]], np.uint8)
    got = A.block_scores(q, codes, scales, np.array([[2, 0, 1, -1, 7]]), [16 * 5], 16)
    assert got[0, 0, 0, :3].tolist() == [32 * 4 * 3.0, 32 * 4.0, -32 * 8.0] and np.isnan(got[0, 0, 0, 3:]).all()
    assert np.isnan(A.block_scores(q, codes, scales, np.array([[2, 0, 1, -1, 7]]), [31], 16)[0, 0, 0, 1:]).all()


def test_oracle_listed_blocks_are_the_tree_attention_of_their_tokens():
    """All blocks listed: every token; a list of some: the tree attention over a table of them."""
    from oracle import quant as Q
    rng = np.random.default_rng(3)
    bits = lambda *s: FM.bf16_rne_of_f64(rng.standard_normal(s))
    kc, ks = Q.mx_quantize(bits(96, 64))
    vc, vs = Q.mx_quantize(bits(96, 64))
    q, table = bits(1, 2, 4, 32), np.array([[5, 2, 0, 4]])
    args = (kc, ks, vc, vs, 16)
    ids = np.broadcast_to(np.arange(3), (1, 2, 1, 3))
    want = A.attn_tree_mx(q, *args, table, [53], 2, 0.2)
    got = A.attn_blocks_mx(q, *args, table, [53], 2, 0.2, ids)
    assert np.allclose(got[0], want[0], rtol=1e-12, atol=1e-12) and np.allclose(got[1], want[1], rtol=1e-12)
    some = np.array([[[[2, -1, 0]], [[2, 9, 0]]]])
    want = A.attn_tree_mx(q, *args, np.array([[0, 5, 4]]), [37], 2, 0.2)
    got = A.attn_blocks_mx(q, *args, table, [53], 2, 0.2, some)
    assert np.allclose(got[0], want[0], rtol=1e-12, atol=1e-12)
