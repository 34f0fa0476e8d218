"""Latent attention over positions that are not finite: what their row does to the rows
that see them."""
import pytest
import torch

import full_ref as R
import test_gpu_attn_latent as latent
from full_ref import BF, F32

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n,ctx", [(2, 8, 3), (8, 20, 70), (50, 3, 40), (16, 1, 300), (16, 8, 300)])
@pytest.mark.parametrize("what", [INF, -INF])
def test_latent_row_that_sees_an_infinite_value_is_not_finite(Hq, n, ctx, what, dtype):
    c = R.latent_case([n, 2], [ctx, 20], Hq, 256, 16, dtype, seed=84)
    ref = R.latent(c)
    pos = ctx + n - 1
    c["cache"][c["table"][0, pos // 16], pos % 16, 0:256:3] = what
    o, lse = latent.call(c)
    seen = n - 1
    assert not bool(torch.isfinite(o[seen, :, 0:256:3]).any())
    o[seen], lse[seen] = ref[0][seen].to(dtype), ref[1][seen].float()
    latent.verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n,ctx", [(2, 8, 3), (8, 20, 70), (50, 3, 40), (16, 1, 300)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_latent_infinite_scores(Hq, n, ctx, sign, dtype):
    # one infinite positional channel: a score of +infinity makes a row not finite, one of
    # -infinity takes the position out of it
    c = R.latent_case([n, 2], [ctx, 20], Hq, 256, 16, dtype, seed=85)
    c["q"][:n, :, 300] = c["q"][:n, :, 300].abs() + 0.125
    pos = ctx + n - 1
    x = c["cache"][c["table"][0, pos // 16], pos % 16]
    x[300] = -1e38
    ref = R.latent(c)                    # a weight of 0 in 64 bits as well
    x[300] = sign * INF
    o, lse = latent.call(c)
    seen = n - 1
    if sign > 0:
        assert bool(torch.isnan(o[seen]).all()) and not bool(torch.isfinite(lse[seen]).any())
        o[seen], lse[seen] = ref[0][seen].to(dtype), ref[1][seen].float()
    # (the bound's share of the scores' size: that of the finite ones)
    x[300] = 0.0
    mag = R.latent(c)[3]
    latent.verdict(c, o, lse, (ref[0], ref[1], ref[2], mag))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,dc,keys,odd", [
    (16, 512, 129, range(128, 129)),                   # a last piece of one position
    (16, 256, 64 * 9, range(192, 256)),                # one of nine pieces, and ...
    (4, 128, 64 * 17 + 1, [*range(128, 192), *range(640, 704)])])   # two that the same lanes join
def test_latent_infinite_values_whose_scores_are_all_there_is(Hq, dc, keys, odd, dtype):
    # c holds -infinity where q is positive: scores of -infinity, weights of 0, and 0 times
    # the value is NaN, also where a piece of the keys has no other position
    c = R.latent_case([1], [keys - 1], Hq, dc, 64, dtype, seed=86)
    c["q"][:, :, 3] = c["q"][:, :, 3].abs() + 0.125
    at = torch.tensor(list(odd))
    c["cache"][c["table"][0, at // 64].long(), at % 64, 3] = -INF
    o, _ = latent.call(c)
    assert bool(torch.isnan(o[:, :, 3]).all())
