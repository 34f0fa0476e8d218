"""kda_attn_paged with scores that are past fp32: they count as infinite, in every kernel."""
import pytest
import torch

import serve_ref as R
import test_gpu_attn_paged as paged

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,d", [(1, 128), (8, 64), (70, 64), (300, 128), (40, 16)])
def test_scores_past_fp32_count_as_infinite(n, d, dtype):
    # q.k is finite, its product with the scale is not. +infinity: the row is not finite;
    # -infinity: the position has no weight
    c = R.attn_case([n], [200], 4, 2, d, 16, dtype, seed=90)
    c["q"] *= 2.0 ** -9
    c["q"][:, :, 0] = 2.0 ** 60
    at = torch.arange(200 + n)
    c["kc"][c["table"][0, at // 16].long(), :, at % 16, 0] = 0.0
    row = c["kc"][c["table"][0, 0].long(), :, 5]
    row[:] = 0.0
    scale = 2.0 ** 8
    mag = R.attn(c, scale)[3]
    for x in (2.0 ** 60, -(2.0 ** 60)):
        row[:, 0] = x
        o, lse = paged.call(c, scale=scale)
        if x > 0:
            assert bool(torch.isnan(o).all()) and not bool(torch.isfinite(lse).any())
        else:
            paged.verdict(c, o, lse, (*R.attn(c, scale)[:3], mag))
