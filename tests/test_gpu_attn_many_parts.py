"""kda_attn_paged with more parts than a grid of 2^32 threads holds."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from serve_ref import DEV

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("d,dtype,hint", [(16, BF, 1), (16, F32, 1), (64, BF, 0)])
def test_more_parts_than_a_grid_holds(d, dtype, hint):
    # 2^24 single tokens and more, of which every one sees itself alone: the result
    # is its value. Without a hint both kernels' grids are that large.
    B, H, page, pool = (1 << 19) + 3, 32, 16, 61
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((pool, H, page, d), generator=g, device=DEV).to(dtype) for _ in range(2))
    q = torch.randn((B, H, d), generator=g, device=DEV, dtype=torch.bfloat16).to(dtype)
    at = torch.arange(B, dtype=torch.int32, device=DEV)
    table = (at * 7 % pool).view(B, 1).contiguous()
    kept = torch.zeros(B, dtype=torch.int32, device=DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    o, lse = kda.kda_attn_paged(q, k, v, table, kept, cu, max_new=hint, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o, v[table[:, 0].long(), :, 0])
    # one score: d products, each cut off or rounded to fp32, and the scale
    for rows in (slice(0, 1000), slice(B - 1000, B)):
        kk = k[table[rows, 0].long(), :, 0].double()
        s = (q[rows].double() * kk).sum(-1) / d ** 0.5
        bound = (d + 4) * 2.0 ** -23 * (q[rows].double() * kk).abs().sum(-1) / d ** 0.5 + 2.0 ** -22 * s.abs()
        assert bool(((lse[rows].double() - s).abs() <= bound).all())
