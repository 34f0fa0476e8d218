"""Latent and expanded attention of scores that are past fp32: they count as infinite."""
import pytest
import torch

import full_ref as R
import test_gpu_attn_expanded as expanded
import test_gpu_attn_latent as latent
from full_ref import BF, F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,dn", [(1, 128), (70, 64), (300, 128)])
def test_expanded_scores_past_fp32_count_as_infinite(n, dn, dtype):
    # q.k is finite, its product with the scale is not. +infinity: the row is not finite;
    # -infinity: the position has no weight
    c = R.expanded_case([n], [n + 200], 2, dn, dtype, seed=82)
    c["q"] *= 2.0 ** -9
    c["q"][:, :, dn] = 2.0 ** 60
    c["kv"][5, :, :dn] = 0.0
    c["pe_all"][5], c["pe_all"][:, 0] = 0.0, 0.0
    c["scale"] = 2.0 ** 8
    mag = R.expanded(c)[3]               # of the scores that are finite
    for x in (2.0 ** 60, -(2.0 ** 60)):
        c["pe_all"][5, 0] = x
        o, lse = expanded.call(c, scale=c["scale"])
        if x > 0:
            assert bool(torch.isnan(o).all()) and not bool(torch.isfinite(lse).any())
        else:
            ref = R.expanded(c)
            expanded.verdict(c, o, lse, (*ref[:3], mag))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,Hq", [(1, 8), (40, 8), (1, 128)])
def test_latent_scores_past_fp32_count_as_infinite(n, Hq, dtype):
    c = R.latent_case([n], [200], Hq, 128, 16, dtype, seed=83)
    c["q"] *= 2.0 ** -9
    c["q"][:, :, 130] = 2.0 ** 60
    at = torch.arange(200 + n)
    c["cache"][c["table"][0, at // 16].long(), at % 16, 130] = 0.0
    row = c["cache"][c["table"][0, 0].long(), 5]
    row[:] = 0.0
    c["scale"] = 2.0 ** 8
    mag = R.latent(c)[3]
    for x in (2.0 ** 60, -(2.0 ** 60)):
        row[130] = x
        o, lse = latent.call(c)
        if x > 0:
            assert bool(torch.isnan(o).all()) and not bool(torch.isfinite(lse).any())
        else:
            latent.verdict(c, o, lse, (*R.latent(c)[:3], mag))
