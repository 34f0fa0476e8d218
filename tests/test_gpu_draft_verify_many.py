"""kda_draft_verify of more requests than a grid of 2^32 threads, or its second
dimension, holds."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from serve_ref import DEV

pytestmark = pytest.mark.gpu


def test_more_requests_than_a_grid_holds():
    # rows of two tokens, quarters: all sums and products with u are exact
    B = (1 << 24) + 5
    g = torch.Generator(device=DEV).manual_seed(1)
    p0 = torch.randint(0, 5, (B,), generator=g, device=DEV) / 4
    p = torch.stack([p0, 1 - p0], 1).view(B, 1, 2)
    u = torch.randint(0, 256, (B, 1), generator=g, device=DEV) / 256
    x = torch.empty((B, 0), dtype=torch.int32, device=DEV)
    commit, tokens = kda.kda_draft_verify(p, None, x, u)
    torch.cuda.synchronize()
    assert bool((commit == 1).all())
    assert torch.equal(tokens[:, 0], (u[:, 0] >= p0).int())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_more_requests_of_several_parts_than_a_launch_takes(dtype):
    # one drafted token of 70000 requests, over 4100 tokens of which three have mass
    B, V, hot = 70000, 4100, (7, 4095, 4099)
    g = torch.Generator(device=DEV).manual_seed(2)
    p = torch.zeros((B, 2, V), dtype=dtype, device=DEV)
    for y, mass in zip(hot, (0.25, 0.5, 0.25)):
        p[:, :, y] = mass
    u = torch.randint(0, 256, (B, 2), generator=g, device=DEV) / 256
    n = torch.randint(-1, 2, (B,), generator=g, device=DEV).int()
    x = torch.full((B, 1), hot[1], dtype=torch.int32, device=DEV)
    commit, tokens = kda.kda_draft_verify(p, None, x, u, n_draft=n)
    torch.cuda.synchronize()
    # the certain draft stays for u < 0.5; without it 7 and 4099 have half each
    stays, drafted = u[:, 0] < 0.5, n == 1
    assert torch.equal(commit, torch.where(n < 0, 0, 1 + (stays & drafted).int()).int())
    v = u[:, 1]
    after = torch.where(v < 0.25, hot[0], torch.where(v < 0.75, hot[1], hot[2]))
    rest = torch.where(v < 0.5, hot[0], hot[2])
    first = torch.where(n < 0, -1, torch.where(~drafted, after, torch.where(stays, hot[1], rest)))
    second = torch.where(drafted & stays, after, -1)
    assert torch.equal(tokens, torch.stack([first, second], 1).int())
