"""kda_latent_append of rows from the least subnormal to the largest finite numbers, under
a bound of the roundings that there are."""
import pytest
import torch

import test_gpu_latent_append as append
from full_ref import BF, F32, HALF

pytestmark = pytest.mark.gpu


def bound(y, dtype):
    # The sum of squares, its root and the quotient are fp64, fewer than 600 roundings of
    # 2^-53; the factor and its two products are rounded to fp32, and the result to bf16.
    # Below the normal numbers a rounding is half of the least one.
    half = 3 * 2.0 ** -24 * (1 + 2.0 ** -10)
    if dtype == BF:
        half = HALF[BF] * (1 + 2.0 ** -10) + half
    return half * y.abs() + (2.0 ** -134 if dtype == BF else 2.0 ** -150)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dc", [128, 512])
@pytest.mark.parametrize("w", [False, True])
def test_latents_of_all_sizes(w, dc, dtype):
    # eps 0: the normalisation knows no size. Rows from the least subnormal numbers to the
    # largest finite ones, and of ordinary size
    n = 40
    c = append.case([n], [5], dc, dtype, w=w, eps=0.0, seed=87)
    g = torch.Generator().manual_seed(88)
    x = torch.randn((n, dc), generator=g, dtype=torch.float64)
    x[:30] /= x[:30].abs().amax(1, keepdim=True)
    size = torch.tensor([1e-44, 1e-42, 1e-39, 1.1e-38, 3e-38, 1e-20, 1e20, 8e37, 1.7e38, 3.38e38],
                        dtype=torch.float64).repeat(4)
    size[30:] = torch.exp(torch.randn(10, generator=g, dtype=torch.float64))
    rows = (x * size[:, None]).float().to(dtype)
    assert bool(torch.isfinite(rows).all())
    rows[:, 0] = torch.where(rows[:, 0] == 0, torch.tensor(1e-38, dtype=dtype), rows[:, 0])
    c["kv"][:, :dc] = rows
    cache, out, _ = append.call(c)
    y = rows.double()
    y = y / torch.sqrt((y * y).mean(1, keepdim=True))
    if w:
        y = y * c["w"].double()
    got = out[:, :dc].double()
    assert bool(torch.isfinite(got).all())
    worst = ((got - y).abs() / bound(y, dtype)).amax(1)
    print(f"[latents] worst error / bound {float(worst.max()):.3f}", flush=True)
    assert float(worst.max()) <= 1.0, worst
