"""The selection of cache blocks (fp4_kv_select_mx) for as many queries as it takes, more
than one grid of workgroups has; blocks and scores equal to a plain selection in 64 bits."""
from __future__ import annotations

import pytest
import torch

import block_scaled_fp4_mx_amd as F
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,drafts,lists", [(65535, 33, 2), (65535, 64, 1)])
def test_queries_past_one_grid(batch, drafts, lists):
    """4325310 queries (2^22 and more), and 4194240; up to 4 blocks for each, the best one."""
    dim, page, columns, pages = 32, 16, 4, 7
    g = torch.Generator(device=DEV)
    g.manual_seed(batch + drafts)
    q = torch.randint(-6, 7, (batch, drafts, lists, dim), generator=g, device=DEV, dtype=torch.int8).bfloat16()
    q[..., 0] = 6.0                                         # every block's scale is 1, and 5 rounds to 4
    codes = torch.randint(0, 256, (pages, lists * dim // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (pages, lists), generator=g, device=DEV, dtype=torch.uint8)
    table = torch.randint(-1, pages, (batch, columns), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(0, page * columns + 9, (batch,), generator=g, device=DEV, dtype=torch.int32)
    ids = torch.full((batch, drafts, lists, 1), -7, dtype=torch.int32, device=DEV)
    out = torch.full(ids.shape, 7.0, device=DEV)
    ws = torch.empty(F.fp4_kv_select_workspace_bytes(batch, drafts, lists, columns), dtype=torch.uint8, device=DEV)
    F.fp4_kv_select_mx(q, codes, scales, table, lens, page, ids, ws, scores=out)

    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    value = torch.cat([value, -value])
    entries = torch.stack([value[(codes & 15).long()], value[(codes >> 4).long()]], -1).reshape(pages, lists, dim)
    entries = entries * torch.exp2(scales.double() - 127)[..., None]
    rounded = torch.where(q.abs() == 5, 4 * q.sign(), q).double()
    there = (table >= 0) & (torch.arange(columns, device=DEV) < (lens // page)[:, None])
    for l in range(lists):
        scores = (rounded[:, :, l].reshape(-1, dim) @ entries[:, l].t().contiguous()).reshape(batch, drafts, pages)
        scores = scores.gather(2, table.clamp_min(0).long()[:, None].expand(-1, drafts, -1))
        scores.masked_fill_(~there[:, None], -torch.inf)
        best = scores.amax(2, keepdim=True)
        at = torch.where(scores == best, torch.arange(columns, device=DEV), columns).amin(2)
        want = torch.where(best[..., 0] == -torch.inf, -1, at)
        assert torch.equal(ids[:, :, l, 0].long(), want)
        assert torch.equal(out[:, :, l, 0].double(), best[..., 0])
