"""What the rows of one wave have to do with one another in the attention over shared
prefixes (fp4_attn_shared_mx): nothing."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import block_scaled_fp4_mx_amd as F
from test_gpu_attn_shared import Shared

pytestmark = pytest.mark.gpu


def _bits(a, **kw):
    a["out"].fill_(7.0)
    F.fp4_attn_shared_mx(**(a | kw))
    return a["out"].view(torch.int16).clone()


# Few rows to a group take the walk, more than 64 the workgroups for many rows.
@pytest.mark.parametrize("d,q_heads,kv_heads,members", [(64, 4, 2, 5), (128, 4, 2, 5), (256, 4, 2, 5),
                                                        (64, 4, 2, 30), (128, 4, 2, 30), (256, 4, 2, 30)])
def test_a_sequence_has_the_same_bits_beside_any_others(d, q_heads, kv_heads, members):
    """Lengths and groups as they are, other queries beside it: the queries behind the drafts,
    which may be anything, and those of other sequences."""
    rng = np.random.default_rng(d + members)
    lens = (1100 + rng.integers(0, 60, members)).tolist()
    draft_lens = rng.integers(1, 4, members)
    x = Shared(d, [(members, 1100)], lens, 3, q_heads, kv_heads, d, 48, draft_lens=draft_lens.tolist())
    a = x.device()
    q = a["q"].clone()
    live = torch.arange(3, device=q.device) < torch.from_numpy(draft_lens).to(q.device)[:, None]
    want = _bits(a)
    x.check(a["out"])
    for other in (30 * q, -q, torch.full_like(q, float("nan")), torch.full_like(q, float("inf"))):
        a["q"] = torch.where(live[:, :, None, None], q, other)
        assert torch.equal(_bits(a), want)
    for factor in (30.0, -1.0, 0.0):
        mine = torch.from_numpy(rng.random(members) < 0.5).to(q.device)
        a["q"] = torch.where(mine[:, None, None, None], q, factor * q)
        assert torch.equal(_bits(a)[mine], want[mine])
