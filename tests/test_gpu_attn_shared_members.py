"""Which sequences share a prefix (fp4_attn_shared_mx), where their lengths end near it;
float64 definition and tolerance as in test_gpu_attn_shared.py."""
from __future__ import annotations

import pytest

import block_scaled_fp4_mx_amd as F
from test_gpu_attn_shared import Shared

pytestmark = pytest.mark.gpu


# Averages of up to 64 rows to a group take the walk, more the workgroups for many rows.
@pytest.mark.parametrize("d,q_heads,kv_heads,drafts", [(64, 8, 2, 2), (128, 4, 2, 1), (128, 16, 1, 5), (256, 8, 2, 3)])
@pytest.mark.parametrize("prefix", [33, 100, 127])
def test_sequences_a_few_tokens_shorter_than_their_prefix(prefix, d, q_heads, kv_heads, drafts):
    """Lengths between the prefix's last whole tile and its end: such a sequence has a context
    of its own, of which the group's first one knows nothing."""
    whole = prefix // 32 * 32
    lens = [prefix + 30, whole, prefix - 1, prefix, whole - 1, prefix + 1, whole + (prefix - whole) // 2]
    x = Shared(prefix + d, [(len(lens), prefix)], lens, drafts, q_heads, kv_heads, d, 16)
    x.run()


def test_sequences_as_long_as_the_table_and_shorter_than_their_prefix():
    """The table ends before the prefix does."""
    x = Shared(1, [(3, 64)], [64, 64, 64], 1, 4, 2, 64, 16)
    x.table = x.table[:, :4].copy()
    x.table[1, 0] = x.table[1, 1]
    x.prefix[:] = 200                                       # each by itself
    x.run()
    x.lens, x.prefix[:] = [200, 200, 199], 200
    x.table[1] = x.table[0]                                 # the first two share what the table has
    a = x.device()
    F.fp4_attn_shared_mx(**a)
    x.lens = [64, 64, 64]                                   # nor do the drafted tokens have a row
    x.check(a["out"])
