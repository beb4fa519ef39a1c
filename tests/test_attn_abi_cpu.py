"""Host-side refusals of the attention path's entry points: the documented
status before any HIP call, and the binding's checks (no GPU needed)."""
import struct

import pytest
import torch

import block_scaled_fp4_mx_amd as F

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, HIPERR = 0, -1, -2, -3, -4, -5, -6
FAKE = 1 << 20          # 16-byte aligned, never dereferenced by rejected calls
FAR = 1 << 40


def _norm(q=FAKE, k=2 * FAKE, tokens=4, hq=4, hk=2, d=64, ld_q=256, ld_k=128, qw=None, kw=None, dt=0, eps=1e-6, table=FAKE,
          places=100, rot=64, pos=FAKE, qo=3 * FAKE, ld_qo=256, ko=4 * FAKE, ld_ko=128):
    return F.lib.fp4_qk_norm_rope(q, k, tokens, hq, hk, d, ld_q, ld_k, qw, kw, dt, eps, table, places, rot, 0, pos, qo,
                                  ld_qo, ko, ld_ko, None)


def test_norm_rope_rejections():
    assert _norm(tokens=-1) == INVALID
    assert _norm(d=24) == SHAPE and _norm(d=272) == SHAPE and _norm(d=0) == SHAPE
    assert _norm(rot=80) == SHAPE and _norm(rot=24) == SHAPE and _norm(rot=-16) == SHAPE
    assert _norm(dt=2) == INVALID
    assert _norm(eps=-1.0) == INVALID and _norm(eps=float("nan")) == INVALID and _norm(eps=float("inf")) == INVALID
    assert _norm(ld_q=248) == INVALID and _norm(ld_q=260) == ALIGN and _norm(ld_ko=120) == INVALID
    assert _norm(q=None) == INVALID and _norm(ko=None) == INVALID and _norm(q=FAKE + 8) == ALIGN
    assert _norm(qw=FAKE + 8) == ALIGN and _norm(table=None) == INVALID and _norm(pos=None) == INVALID
    assert _norm(pos=FAKE + 2) == ALIGN and _norm(places=-1) == INVALID
    assert _norm(tokens=1 << 24) == SHAPE
    # overlaps: shifted in place, an output over the other input or output
    assert _norm(qo=FAKE + 16) == INVALID and b"overlaps" in F.lib.fp4_last_error()
    assert _norm(qo=FAKE, ld_qo=264) == INVALID
    assert _norm(qo=2 * FAKE) == INVALID and _norm(ko=FAKE) == INVALID and _norm(ko=3 * FAKE) == INVALID
    assert _norm(tokens=0, q=None, k=None, qo=None, ko=None) == OK
    assert _norm(hq=0, hk=0, q=None, k=None, qo=None, ko=None) == OK


def test_norm_rope_outputs_over_what_all_heads_read():
    """Weights, angles and positions are read by workgroups that others may be ahead of.
    The defaults: q_out 4 rows of 512 bytes at 3 MiB, k_out 4 of 256 at 4 MiB, the
    table 25600 bytes and the positions 16 at 1 MiB, the weights 128 bytes (bf16)."""
    qo, ko = 3 * FAKE, 4 * FAKE

    def overlap(what, **kw):
        assert _norm(**kw) == INVALID and F.lib.fp4_last_error().decode() == what, kw

    overlap("q_out overlaps q_weight", qw=qo)
    overlap("q_out overlaps q_weight", qw=qo + 3 * 512 + 496)
    overlap("q_out overlaps k_weight", kw=qo - 112)
    overlap("q_out overlaps k_weight", kw=qo - 240, dt=1)
    overlap("k_out overlaps k_weight", kw=ko + 16)
    overlap("q_out overlaps cos_sin", table=qo - 25600 + 16)
    overlap("k_out overlaps cos_sin", table=ko)
    overlap("q_out overlaps positions", pos=qo + 4)
    overlap("k_out overlaps positions", pos=ko - 12)
    overlap("k_out overlaps cos_sin", table=ko - 16, places=1 << 62)
    # rows of 512 bytes 1024 apart: the weights between two of them are no overlap, up to the next row they are
    overlap("q_out overlaps q_weight", qw=qo + 1024 - 112, ld_qo=512)
    # what does not overlap passes, down to the last pair of the check
    for kw in (dict(qw=qo + 512, ld_qo=512), dict(qw=qo + 2048), dict(kw=qo - 128), dict(table=qo - 25600), dict(kw=ko + 1024),
               dict(qw=qo + 3 * 1024 + 512, ld_qo=512)):
        overlap("k_out overlaps positions", pos=ko + 1020, **kw)


def _cache(**kw):
    v = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, num_pages=10, d=64, page_size=16) | kw
    return struct.pack("=4Q3q", *(v[n] or 0 for n in v))


def _pages(**kw):
    v = dict(page_table=FAKE, page_counts=FAKE, seq_lens=FAKE, page_refs=FAKE, batch=3, max_pages=4, num_pages=10) | kw
    return struct.pack("=4Q3q", *(v[n] or 0 for n in v))


BAD_CACHES = [(dict(d=48), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=0), INVALID), (dict(num_pages=-1), INVALID),
              (dict(k_codes=None), INVALID), (dict(k_scales=FAKE + 4), ALIGN), (dict(v_codes=None), INVALID),
              (dict(v_scales=FAKE + 8), ALIGN), (dict(num_pages=1 << 28, page_size=16), SHAPE)]
BAD_PAGES = [(dict(batch=-1), INVALID), (dict(page_table=None), INVALID), (dict(page_counts=FAKE + 2), ALIGN),
             (dict(seq_lens=None), INVALID), (dict(page_refs=None), INVALID), (dict(batch=1 << 20), SHAPE),
             (dict(num_pages=1 << 31), SHAPE), (dict(max_pages=-2), INVALID)]


def test_page_operations_reject_bad_states():
    lib, need = F.lib, F.lib.fp4_kv_reserve_workspace_bytes(3, 10)
    for kw, status in BAD_CACHES:
        assert lib.fp4_kv_reserve(_cache(**kw), _pages(), FAKE, FAKE, 4, FAKE, FAKE, need, None) == status, kw
        assert lib.fp4_kv_compact(_cache(**kw), _pages(), FAKE, 4, FAKE, None) == status, kw
        assert lib.fp4_kv_copy_pages(_cache(**kw), _cache(), FAKE, FAKE, 2, None) == status, kw
        assert lib.fp4_kv_copy_pages(_cache(), _cache(**kw), FAKE, FAKE, 2, None) == status, kw
    for kw, status in BAD_PAGES:
        assert lib.fp4_kv_reserve(_cache(), _pages(**kw), FAKE, FAKE, 4, FAKE, FAKE, need, None) == status, kw
        assert lib.fp4_kv_fork(_pages(**kw), FAKE, 2, 16, None) == status, kw
        assert lib.fp4_kv_free(_pages(**kw), FAKE, 2, None, 16, None) == status, kw
        assert lib.fp4_kv_compact(_cache(), _pages(**kw), FAKE, 4, FAKE, None) == status, kw


def test_page_operations_reject_bad_arguments():
    lib, need = F.lib, F.lib.fp4_kv_reserve_workspace_bytes(3, 10)
    assert need == 16 + 3 * 16 + 10 * 4 and lib.fp4_kv_reserve_workspace_bytes(0, 10) == 0

    def reserve(new=FAKE, slots=FAKE, max_new=4, short=FAKE, ws=FAKE, n=need, pages=None):
        return lib.fp4_kv_reserve(_cache(), pages or _pages(), new, slots, max_new, short, ws, n, None)

    assert reserve(new=None) == INVALID and reserve(slots=None) == INVALID and reserve(short=None) == INVALID
    assert reserve(max_new=-1) == INVALID and reserve(short=FAKE + 1) == ALIGN
    assert reserve(ws=None) == WORKSPACE and reserve(n=need - 1) == WORKSPACE and reserve(ws=FAKE + 4) == ALIGN
    assert reserve(pages=_pages(num_pages=9)) == INVALID
    assert reserve(pages=_pages(batch=0)) == OK
    assert lib.fp4_kv_fork(_pages(), None, 2, 16, None) == INVALID
    assert lib.fp4_kv_fork(_pages(), FAKE, -1, 16, None) == INVALID
    assert lib.fp4_kv_fork(_pages(), FAKE, 2, 20, None) == SHAPE
    assert lib.fp4_kv_fork(_pages(), FAKE, 1 << 20, 16, None) == SHAPE
    assert lib.fp4_kv_fork(_pages(), None, 0, 16, None) == OK
    assert lib.fp4_kv_free(_pages(), None, 2, None, 16, None) == INVALID
    assert lib.fp4_kv_free(_pages(), FAKE, 2, FAKE + 2, 16, None) == ALIGN
    assert lib.fp4_kv_free(_pages(), FAKE, 2, None, 0, None) == INVALID
    assert lib.fp4_kv_free(_pages(), FAKE, 1 << 20, None, 16, None) == SHAPE
    assert lib.fp4_kv_compact(_cache(), _pages(), FAKE, 65, FAKE, None) == INVALID
    assert lib.fp4_kv_compact(_cache(), _pages(), FAKE, 4, None, None) == INVALID
    assert lib.fp4_kv_compact(_cache(), _pages(num_pages=11), FAKE, 4, FAKE, None) == INVALID
    copy = lib.fp4_kv_copy_pages
    assert copy(_cache(), _cache(d=96), FAKE, FAKE, 2, None) == INVALID
    assert copy(_cache(), _cache(page_size=32), FAKE, FAKE, 2, None) == INVALID
    assert copy(_cache(), _cache(v_codes=None, v_scales=None), FAKE, FAKE, 2, None) == INVALID
    assert copy(_cache(), _cache(), FAKE, None, 2, None) == INVALID
    assert copy(_cache(), _cache(), FAKE, FAKE, -1, None) == INVALID
    assert copy(_cache(), _cache(), FAKE, FAKE, 1 << 24, None) == SHAPE
    assert copy(_cache(), _cache(), None, None, 0, None) == OK


def test_commit_of_a_reservation_rejects_bad_arguments():
    def commit(cache=None, pages=None, accepted=FAKE, most=4, lens=FAKE, slots=FAKE, max_new=4):
        return F.lib.fp4_kv_compact_reserved(cache or _cache(), pages or _pages(), accepted, most, lens, slots, max_new, None)

    for kw, status in BAD_CACHES:
        assert commit(cache=_cache(**kw)) == status, kw
    for kw, status in BAD_PAGES:
        assert commit(pages=_pages(**kw)) == status, kw
    assert commit(slots=None) == INVALID and commit(slots=FAKE + 2) == ALIGN and commit(max_new=-1) == INVALID
    assert commit(most=65) == INVALID and commit(lens=None) == INVALID and commit(pages=_pages(num_pages=11)) == INVALID
    assert commit(pages=_pages(batch=0)) == OK
    assert commit(pages=_pages(batch=0), slots=None, lens=None, accepted=None) == OK      # nothing is read
    assert commit(max_new=0) == OK                                                        # nothing was reserved


def test_binding_checks_the_commit_of_a_reservation():
    cache = F.KvCache(_u8(160, 32), _u8(160, 2), _u8(160, 32), _u8(160, 2), 16)
    pages = F.KvPages(_int(3, 4), _int(3), _int(3), _int(10))
    for bad in (_int(2, 4), _int(3), _int(12)):
        with pytest.raises(ValueError, match="slots has shape"):
            F.fp4_kv_compact_reserved(cache, pages, _int(3, 4), _int(3), bad)
    with pytest.raises(TypeError, match="slots"):
        F.fp4_kv_compact_reserved(cache, pages, None, _int(3), None)
    with pytest.raises(TypeError, match="slots"):
        F.fp4_kv_compact_reserved(cache, pages, None, _int(3), _int(3, 4).long())
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_kv_compact_reserved(cache, pages, None, _int(3), _int(3, 4))


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _int(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_binding_checks_the_attention_path():
    x = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="bfloat16"):
        F.fp4_qk_norm_rope(x.float(), x, x, x)
    with pytest.raises(ValueError, match="tokens, heads"):
        F.fp4_qk_norm_rope(x[0], x, x, x)
    with pytest.raises(ValueError, match="heads of q"):
        F.fp4_qk_norm_rope(x[:, ::2], x, x, x)
    with pytest.raises(ValueError, match="k has shape"):
        F.fp4_qk_norm_rope(x, x[:3], x, x[:3])
    with pytest.raises(ValueError, match="q_out and k_out"):
        F.fp4_qk_norm_rope(x, x, x[:, :2], x)
    with pytest.raises(ValueError, match="q_weight"):
        F.fp4_qk_norm_rope(x, x, x, x, q_weight=torch.ones(32))
    with pytest.raises(TypeError, match="k_weight"):
        F.fp4_qk_norm_rope(x, x, x, x, q_weight=torch.ones(64), k_weight=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="positions"):
        F.fp4_qk_norm_rope(x, x, x, x, torch.zeros(4, dtype=torch.int64), torch.zeros((8, 64)))
    with pytest.raises(TypeError, match="positions"):
        F.fp4_qk_norm_rope(x, x, x, x, None, torch.zeros((8, 64)))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_qk_norm_rope(x, x, x, x)
    cache = F.KvCache(_u8(160, 32), _u8(160, 2), _u8(160, 32), _u8(160, 2), 16)
    pages = F.KvPages(_int(3, 4), _int(3), _int(3), _int(10))
    with pytest.raises(ValueError, match="k_scales"):
        F.fp4_kv_compact(cache._replace(k_scales=_u8(160, 3)), pages, _int(3, 4), _int(3))
    with pytest.raises(ValueError, match="both"):
        F.fp4_kv_compact(cache._replace(v_codes=None), pages, _int(3, 4), _int(3))
    with pytest.raises(ValueError, match="keys"):
        F.fp4_kv_compact(cache._replace(v_codes=_u8(144, 32)), pages, _int(3, 4), _int(3))
    with pytest.raises(ValueError, match="num_pages"):
        F.fp4_kv_compact(cache._replace(page_size=48), pages, _int(3, 4), _int(3))
    with pytest.raises(ValueError, match="page_table"):
        F.fp4_kv_fork(pages._replace(page_counts=_int(2)), _int(1, 2), 16)
    with pytest.raises(ValueError, match="pairs"):
        F.fp4_kv_fork(pages, _int(2), 16)
    with pytest.raises(ValueError, match="keep_lens"):
        F.fp4_kv_free(pages, _int(3), 16, keep_lens=_int(2))
    with pytest.raises(ValueError, match="accepted"):
        F.fp4_kv_compact(cache, pages, _int(2, 4), _int(3))
    with pytest.raises(ValueError, match="slots"):
        F.fp4_kv_reserve(cache, pages, _int(3), _int(2, 4), _int(1), _u8(200))
    with pytest.raises(TypeError, match="workspace"):
        F.fp4_kv_reserve(cache, pages, _int(3), _int(3, 4), _int(1), _int(200))
    with pytest.raises(ValueError, match="dst_pages"):
        F.fp4_kv_copy_pages(cache, cache, _int(2), _int(3))
    with pytest.raises(ValueError, match="GPU"):
        F.fp4_kv_copy_pages(cache, cache, _int(2), _int(2))


def _tree(q=FAKE, ld_q=512, cache=None, table=FAKE, width=4, lens=FAKE, nd=None, mask=None, batch=2, drafts=4, hq=8, hk=1, d=64,
          scale=0.1, out=FAR, ld_out=512, ws=FAKE, n=1 << 40):
    return F.lib.fp4_attn_tree_mx(q, ld_q, cache or _cache(), table, width, lens, nd, mask, batch, drafts, hq, hk, d, scale, out,
                                  ld_out, ws, n, None)


def test_binding_survives_what_is_no_cache_no_tensor_and_no_strided_tensor():
    x = torch.zeros((4, 6, 64), dtype=torch.bfloat16)
    pages = F.KvPages(_int(3, 4), _int(3), _int(3), _int(10))
    with pytest.raises(TypeError, match="KvPages, got list"):
        F.fp4_kv_fork(list(pages), _int(1, 2), 16)
    with pytest.raises(TypeError, match="KvCache, got"):
        F.fp4_kv_compact(pages, pages, _int(3, 4), _int(3))
    with pytest.raises(TypeError, match="q must be a torch tensor, got NoneType"):
        F.fp4_attn_prompt(None, x, x, _int(2), x)
    with pytest.raises(TypeError):
        F.fp4_kv_fork(pages, _int(1, 2), "16")
    with pytest.raises(TypeError):
        F.fp4_qk_norm_rope(x, x, x, x, eps="small")
    with pytest.raises(OverflowError):
        F.fp4_kv_fork(pages, _int(1, 2), 1 << 70)
    with pytest.raises(ValueError, match="GPU, got a meta tensor"):
        F.fp4_qk_norm_rope(x.to("meta"), x, x, x)
    with pytest.raises((RuntimeError, ValueError)):
        F.fp4_kv_fork(pages._replace(page_refs=_int(10).to_sparse()), _int(1, 2), 16)
    with pytest.raises(TypeError, match="arguments"):
        F._binding.fp4_kv_fork(pages)


def test_attn_tree_rejections():
    for kw, status in BAD_CACHES:
        assert _tree(cache=_cache(**kw)) == status, kw
    assert _tree(cache=_cache(v_codes=None, v_scales=None)) == INVALID
    assert _tree(d=96) == SHAPE and _tree(d=32) == SHAPE and _tree(hq=3, hk=2) == SHAPE and _tree(hk=2) == SHAPE
    assert _tree(hq=0) == INVALID and _tree(hk=0) == INVALID and _tree(hq=8192) == SHAPE
    assert _tree(drafts=0) == INVALID and _tree(drafts=65) == INVALID and _tree(batch=-1) == INVALID
    assert _tree(batch=65536) == SHAPE and _tree(width=-1) == INVALID
    assert _tree(scale=float("nan")) == INVALID and _tree(scale=float("inf")) == INVALID
    assert _tree(q=None) == INVALID and _tree(out=None) == INVALID and _tree(table=None) == INVALID
    assert _tree(lens=None) == INVALID and _tree(q=FAKE + 8) == ALIGN and _tree(nd=FAKE + 2) == ALIGN
    assert _tree(mask=FAKE + 4) == ALIGN and _tree(ld_q=508) == INVALID and _tree(ld_out=516) == ALIGN
    assert _tree(out=FAKE) == INVALID and b"overlaps" in F.lib.fp4_last_error()
    need = F.lib.fp4_attn_tree_workspace_bytes(2, 4, 8, 64, 1)
    assert need > 0 and _tree(n=need - 1) == WORKSPACE and _tree(ws=None) == WORKSPACE and _tree(ws=FAKE + 4) == ALIGN
    assert F.lib.fp4_attn_tree_workspace_bytes(2, 4, 8, 96, 1) == 0
    assert F.lib.fp4_attn_tree_workspace_bytes(0, 4, 8, 64, 1) == 0
    assert _tree(batch=0, q=None, out=None) == OK


def test_binding_checks_the_tree_attention():
    cache = F.KvCache(_u8(160, 64), _u8(160, 4), _u8(160, 64), _u8(160, 4), 16)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    args = dict(q=q, cache=cache, page_table=_int(2, 5), seq_lens=_int(2), out=torch.zeros_like(q), workspace=_u8(16))

    def refuses(match, error=ValueError, **kw):
        with pytest.raises(error, match=match):
            F.fp4_attn_tree_mx(**args | kw)

    refuses("bfloat16", TypeError, q=q.float())
    refuses("batch, drafts", q=q[0])
    refuses("heads of q", q=q[:, :, ::2])
    refuses("one pitch", q=torch.zeros((4, 3, 4, 64), dtype=torch.bfloat16)[::2])
    refuses("out has shape", out=q[:1])
    refuses("no values", cache=cache._replace(v_codes=None, v_scales=None))
    refuses("head_dim", cache=F.KvCache(_u8(160, 48), _u8(160, 3), _u8(160, 48), _u8(160, 3), 16))
    refuses("page_table", page_table=_int(3, 5))
    refuses("page_table", TypeError, page_table=_int(2, 5).long())
    refuses("seq_lens", seq_lens=_int(3))
    refuses("draft_lens", draft_lens=_int(3))
    refuses("tree_mask", TypeError, tree_mask=_int(2, 3))
    refuses("tree_mask", tree_mask=_int(2, 4).long())
    refuses("GPU")


def _prompt(q=FAKE, k=2 * FAKE, v=3 * FAKE, cu=FAKE, seqs=2, tokens=8, hq=4, hk=2, d=64, ld_q=256, ld_k=128, ld_v=128,
            scale=0.1, out=4 * FAKE, ld_out=256):
    return F.lib.fp4_attn_prompt(q, k, v, cu, seqs, tokens, hq, hk, d, ld_q, ld_k, ld_v, scale, out, ld_out, None)


def test_attn_prompt_rejections():
    assert _prompt(d=80) == SHAPE and _prompt(hq=3) == SHAPE and _prompt(hk=0) == INVALID
    assert _prompt(tokens=-1) == INVALID and _prompt(seqs=-1) == INVALID
    assert _prompt(tokens=1 << 31) == SHAPE and _prompt(seqs=1 << 20) == SHAPE
    assert _prompt(tokens=1 << 30, hq=64, hk=2, ld_q=4096, ld_out=4096) == SHAPE
    assert _prompt(scale=float("nan")) == INVALID and _prompt(scale=float("-inf")) == INVALID
    assert _prompt(q=None) == INVALID and _prompt(k=None) == INVALID and _prompt(v=None) == INVALID
    assert _prompt(cu=None) == INVALID and _prompt(out=None) == INVALID
    assert _prompt(q=FAKE + 8) == ALIGN and _prompt(cu=FAKE + 2) == ALIGN
    assert _prompt(ld_q=248) == INVALID and _prompt(ld_k=132) == ALIGN and _prompt(ld_v=120) == INVALID
    assert _prompt(ld_out=255) == INVALID
    for kw in (dict(out=FAKE), dict(out=2 * FAKE), dict(out=3 * FAKE), dict(out=FAKE + 64)):
        assert _prompt(**kw) == INVALID and b"overlaps" in F.lib.fp4_last_error()
    # columns of one array: outputs beside the inputs in the same rows do not overlap them
    assert _prompt(tokens=0, q=None) == OK and _prompt(seqs=0, q=None) == OK


def test_attn_prompt_refuses_what_its_offsets_cannot_hold():
    """Rows of a tile are 32-bit offsets apart, and a launch has fewer than 2^32 threads."""
    assert _prompt(ld_k=1 << 24) == SHAPE and _prompt(ld_v=1 << 24) == SHAPE and b"2^24" in F.lib.fp4_last_error()
    assert _prompt(tokens=1 << 30, hq=1, hk=1) == SHAPE
    assert _prompt(tokens=1 << 29, hq=4, hk=2, d=256, ld_q=1024, ld_k=512, ld_v=512, ld_out=1024) == SHAPE
    assert b"row tiles" in F.lib.fp4_last_error()


@pytest.mark.parametrize("call,batch", [(_tree, "batch"), (_prompt, "seqs")])
def test_scales_that_fp32_cannot_hold_times_log2_e(call, batch):
    """2^128 / log2(e) is 2.36e38: the kernels' factor would be infinite, and 0 times it no number."""
    for scale in (2.5e38, -3.3e38, 1.8e38):
        assert call(scale=scale) == INVALID and b"2^127" in F.lib.fp4_last_error()
    for scale in (2.0 ** 127, -2.0 ** 127, 0.0, 1e-45):
        assert call(scale=scale, **{batch: 0}) == OK


def test_weights_of_absent_heads_are_ignored():
    """A dangling weight pointer of heads that a call has none of is no error: the
    call is refused for its own fault only (a table that is missing)."""
    assert _norm(hk=0, k=None, ko=None, kw=FAKE + 2, table=None) == INVALID
    assert _norm(hq=0, q=None, qo=None, qw=FAKE + 2, table=None) == INVALID


def test_binding_checks_the_prompt_attention():
    x = torch.zeros((8, 4, 64), dtype=torch.bfloat16)
    args = dict(q=x, k=x[:, :2], v=x[:, :2], cu_seqlens=_int(3), out=x.clone())

    def refuses(match, error=ValueError, **kw):
        with pytest.raises(error, match=match):
            F.fp4_attn_prompt(**args | kw)

    refuses("bfloat16", TypeError, v=x.half())
    refuses("heads of k", k=x[:, ::2])
    refuses("k and v", k=x[:7, :2])
    refuses("k and v", v=x[:, :1])
    refuses("out has shape", out=x[:, :2])
    refuses("cu_seqlens", TypeError, cu_seqlens=_int(3).long())
    refuses("cu_seqlens", cu_seqlens=_int(0))
    refuses("GPU")
