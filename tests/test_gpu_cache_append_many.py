"""kda_cache_append of more tokens than a grid of 2^32 threads has workgroups for."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from serve_ref import DEV

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_grid_holds():
    # rows of more than 8 KB are a token a workgroup: 2^24 of them take 146 GB, which
    # keys and values share here; a few of them have a slot
    T, H, d, page, pool = (1 << 24) + 9, 17, 128, 16, 4
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < T * H * d * 4 + (4 << 30):
        pytest.skip("needs 150 GB of device memory")
    k = torch.empty((T, H, d), device=DEV)
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    at = [0, 1, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, T - 1]
    for i, t in enumerate(at):
        k[t] = torch.arange(H * d, device=DEV).view(H, d) + 10000.0 * i
        slots[t] = 7 * i + 3
    kc, vc = (torch.full((pool, H, page, d), -1.0, device=DEV) for _ in range(2))
    want = kc.clone()
    for i, t in enumerate(at):
        s = 7 * i + 3
        want[s // page, :, s % page] = k[t]
    kda.kda_cache_append(k, k, slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, want) and torch.equal(vc, want)
    del k
    torch.cuda.empty_cache()
