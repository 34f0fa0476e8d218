"""Latent and expanded attention of values near the end of their range: the sums over the
keys, which are not normalised, stay inside fp32 up to the limit that the header names."""
import math

import pytest
import torch

import full_ref as R
import test_gpu_attn_expanded as expanded
import test_gpu_attn_latent as latent
from full_ref import BF, F32

pytestmark = pytest.mark.gpu


def latent_scores(Hq, n, keys, dc, scores, values, dtype, seed=80):
    """Every position's score (log2 domain) is given, the same for all rows; values in [1, 2) times
    `values`, of one sign, so that nothing of a sum cancels."""
    c = R.latent_case([n], [keys - n], Hq, dc, 16, dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    c["q"][:] = 0.0
    c["q"][:, :, dc + 1] = 1.0
    at = torch.arange(keys)
    page = c["table"][0, at // 16].long()
    c["cache"][page, at % 16] = ((1.0 + torch.rand((keys, dc + 64), generator=g)) * values).to(dtype)
    c["cache"][page, at % 16, dc:] = 0.0
    c["cache"][page, at % 16, dc + 1] = (scores / (c["scale"] * math.log2(math.e))).to(dtype)
    return c


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [23.0, 15.5, 8.5])
@pytest.mark.parametrize("Hq,n,dc", [(16, 1, 512), (64, 1, 512), (20, 4, 256), (7, 1, 128)])
def test_latent_step_of_keys_far_above_the_first(Hq, n, dc, size, dtype):
    # a whole step of keys `size` above all before them, with values of 2^100: their weights
    # relative to the first step's maximum would carry the sum of 32 past fp32
    scores = torch.zeros(160)
    scores[32:64] = size
    latent.check(latent_scores(Hq, n, 160, dc, scores, 2.0 ** 100, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lag", [0.0, 3.9, 7.9])
@pytest.mark.parametrize("Hq,n,dc", [(16, 1, 512), (64, 2, 512), (7, 1, 128)])
def test_latent_values_at_their_limit(Hq, n, dc, lag, dtype):
    # values of up to 2^108 of 1024 positions, all but the first step's `lag` above it
    scores = torch.full((1024,), lag)
    scores[:32] = 0.0
    latent.check(latent_scores(Hq, n, 1024, dc, scores, 2.0 ** 107, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lag", [0.0, 7.9, 23.0])
@pytest.mark.parametrize("n,dn", [(1, 128), (300, 64), (40, 128)])
def test_expanded_values_at_their_limit(n, dn, lag, dtype):
    c = R.expanded_case([n], [1024], 2, dn, dtype, seed=81)
    g = torch.Generator().manual_seed(81)
    c["q"][:] = 0.0
    c["q"][:, :, dn + 1] = 1.0
    scores = torch.full((1024,), lag)
    scores[:64] = 0.0
    c["pe_all"][:] = 0.0
    c["pe_all"][:, -63] = (scores / (c["scale"] * math.log2(math.e))).to(dtype)
    c["kv"][..., dn:] = ((1.0 + torch.rand((1024, 2, dn), generator=g)) * 2.0 ** 107).to(dtype)
    expanded.check(c)
