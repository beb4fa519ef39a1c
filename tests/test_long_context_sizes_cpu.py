"""Work space sizes of the long contexts' entry points (no GPU needed)."""
import block_scaled_fp4_mx_amd as F


def test_no_selection_workspace_for_sizes_that_the_call_refuses():
    size = F.lib.fp4_kv_select_workspace_bytes
    assert size(32768, 64, 4, 4) == 0 and size(60000, 64, 4, 4) == 0        # 2^23 queries and more
    for batch, drafts, lists in ((32767, 64, 4), (65535, 64, 2), (65535, 64, 1)):
        assert batch * drafts * lists < 1 << 23
        assert size(batch, drafts, lists, 4) == batch * drafts * lists * 16 * 4
