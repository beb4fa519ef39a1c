"""Work space sizes of the long contexts' entry points (no GPU needed)."""
import block_scaled_fp4_mx_amd as F


def test_no_selection_workspace_for_sizes_that_the_call_refuses():
    size = F.lib.fp4_kv_select_workspace_bytes
    assert size(32768, 64, 4, 4) == 0 and size(60000, 64, 4, 4) == 0        # 2^23 queries and more
    for batch, drafts, lists in ((32767, 64, 4), (65535, 64, 2), (65535, 64, 1)):
        assert batch * drafts * lists < 1 << 23
        assert size(batch, drafts, lists, 4) == batch * drafts * lists * 16 * 4


HEADS = [(64, 8, 128, 1), (32, 8, 128, 1), (20, 4, 64, 3), (4, 2, 256, 2), (8, 1, 64, 1), (96, 1, 128, 1), (5, 5, 64, 64), (24, 12, 256, 7)]


def test_a_shared_prefix_workspace_serves_smaller_steps():
    """A workspace for a batch and a number of groups serves every smaller one of either."""
    size = F.lib.fp4_attn_shared_workspace_bytes
    batches, groups = [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 33, 63, 64, 65, 128, 1000, 65535], [0, 1, 2, 3, 4, 6, 8, 15, 16, 17, 63, 64, 65, 1000]
    for q_heads, kv_heads, d, drafts in HEADS:
        at = {(b, g): size(b, drafts, q_heads, d, kv_heads, g) for b in batches for g in groups}
        assert min(at.values()) > 0
        for i, b in enumerate(batches):
            for j, g in enumerate(groups):
                assert i == 0 or at[batches[i - 1], g] <= at[b, g], (q_heads, kv_heads, d, drafts, b, g)
                assert j == 0 or at[b, groups[j - 1]] <= at[b, g], (q_heads, kv_heads, d, drafts, b, g)


def test_the_other_workspaces_serve_smaller_batches():
    for q_heads, kv_heads, d, drafts in HEADS:
        sizes = [F.lib.fp4_attn_blocks_workspace_bytes(b, drafts, q_heads, d, kv_heads) for b in (1, 2, 64, 65535)]
        assert 0 < sizes[0] and sizes == sorted(sizes)
    select = F.lib.fp4_kv_select_workspace_bytes
    for a, b in (((1, 1, 1, 5), (2, 1, 1, 5)), ((3, 2, 4, 16), (3, 2, 4, 17)), ((3, 2, 4, 16), (3, 3, 4, 16))):
        assert 0 < select(*a) < select(*b)
