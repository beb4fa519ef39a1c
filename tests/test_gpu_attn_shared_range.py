"""Drafted values past bf16's range behind a shared prefix (fp4_attn_shared_mx): they
reach only the rows that see them.  Tolerance in attn_check.py."""
from __future__ import annotations

import numpy as np
import pytest

import block_scaled_fp4_mx_amd as F
from attn_check import check, norm
from oracle import attn as A
from oracle import quant as Q
from test_gpu_attn_shared import Shared
from test_gpu_attn_tree import _tree

pytestmark = pytest.mark.gpu


# The first four by the walk (up to 64 rows to a group), the others with many rows.
@pytest.mark.parametrize("d,q_heads,kv_heads,members,drafts", [(64, 4, 2, 3, 6), (128, 8, 2, 2, 6), (128, 4, 4, 3, 9), (256, 4, 2, 3, 5),
                                                               (64, 4, 1, 8, 6), (128, 8, 2, 5, 6), (256, 4, 1, 6, 5)])
def test_drafted_values_past_the_range_reach_only_rows_that_see_them(d, q_heads, kv_heads, members, drafts):
    """As for the attention without a prefix: infinite in bf16 (code 7 at 2^126), near the end of
    its range (code 1) and no number (scale byte 255), in a sequence whose own tokens are one
    piece and in one whose own tokens are several."""
    lens = [1000 + 37 * b for b in range(members)]
    lens[-1] = 4200
    x = Shared(d + drafts, [(members, 1000)], lens, drafts, q_heads, kv_heads, d, 48, masks=_tree(11, members, drafts))
    group, odd = q_heads // kv_heads, []
    for b in (0, members - 1):
        for token, block, code, scale in ((1, 0, 0x77, 253), (2, 1, 0x11, 253), (drafts - 1, kv_heads * d // 32 - 1, 0x22, 255)):
            row = A.cache_rows(x.table[b], 48, len(x.kc) // 48, lens[b] + drafts)[lens[b] + token]
            x.vc[row, 16 * block:16 * block + 16], x.vs[row, block] = code, 0
            odd.append((b, token, block, row, scale))
    a = x.device()
    for *_, block, row, scale in odd:
        a["cache"].v_scales[row, block] = scale
    F.fp4_attn_shared_mx(**a)

    def reference():
        return A.attn_tree_mx(x.q, x.kc, x.ks, x.vc, x.vs, 48, x.table, lens, kv_heads, d ** -0.5, None, x.masks)

    ref, size = reference()
    got = a["out"].cpu().float().numpy()
    k_norm = float(np.sqrt((Q.mx_dequant_f64(x.kc, x.ks).reshape(-1, d) ** 2).sum(-1)).max())
    for b, token, block, row, scale in odd:
        head, at = block * 32 // d, block * 32 % d
        heads, values = slice(head * group, (head + 1) * group), slice(at, at + 32)
        sees = np.array([int(x.masks[b, i]) >> token & 1 for i in range(drafts)], bool)
        assert sees.any() and not sees.all()
        if token == 2:                                       # finite: its own reference and magnitudes
            # where no value of the same block is infinite or no number
            others = [t for c, t, at_block, *_ in odd if (c, at_block) == (b, block) and t != token]
            alone = sees & ~np.array([any(int(x.masks[b, i]) >> t & 1 for t in others) for i in range(drafts)])
            x.vs[row, block] = scale
            r, z = reference()
            x.vs[row, block] = 0
            only = np.full_like(r, np.nan)
            only[b, alone, heads, values] = r[b, alone, heads, values]
            check(a["out"], only, z, d, 4200 + drafts, d ** -0.5, norm(x.q), k_norm, 2.0 ** 125)
        else:
            y = got[b, sees, heads, values]
            assert (y == np.inf).all() if scale == 253 else not np.isfinite(y).any()
        ref[b, sees, heads, values] = np.nan
    check(a["out"], ref, size, d, 4200 + drafts, d ** -0.5, norm(x.q), k_norm, np.abs(Q.mx_dequant_f64(x.vc, x.vs)).max())
