"""kda_attn_paged of values near the end of their range: the sums over the positions, which
are not normalised, stay inside fp32 up to the limit that the header names."""
import math

import pytest
import torch

import serve_ref as R
import test_gpu_attn_paged as paged

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lag", [0.0, 7.9, 23.0])
@pytest.mark.parametrize("n,d", [(1, 128), (40, 64), (20, 32), (150, 128)])
def test_values_at_their_limit(n, d, lag, dtype):
    # values of up to 2^108 of 1024 positions, all but the first 128 `lag` above those (log2)
    c = R.attn_case([n], [1024 - n], 2, 1, d, 16, dtype, seed=91)
    g = torch.Generator().manual_seed(91)
    at = torch.arange(1024)
    page = c["table"][0, at // 16].long()
    c["q"][:] = 0.0
    c["q"][:, :, 1] = 1.0
    scores = torch.full((1024,), lag)
    scores[:128] = 0.0
    c["kc"][page, 0, at % 16] = 0.0
    c["kc"][page, 0, at % 16, 1] = (scores * math.sqrt(d) / math.log2(math.e)).to(dtype)
    c["vc"][page, 0, at % 16] = ((1.0 + torch.rand((1024, d), generator=g)) * 2.0 ** 107).to(dtype)
    paged.check(c)
