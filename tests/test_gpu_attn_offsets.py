"""kda_attn_paged where cu_new decreases: rows claimed once are right, and a call
whose requests claim more than its rows writes none."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints
from test_gpu_attn_paged import verdict

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def run(q, kc, vc, table, kept, cu, hint):
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    kda.kda_attn_paged(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV).contiguous(), ints(kept),
                       ints(cu), o=o, lse=lse, max_new=hint)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("empty", [1, 300])
@pytest.mark.parametrize("n,hint", [(2, 0), (2, 2), (60, 0), (60, 1)])
def test_rows_claimed_once_in_any_order(n, hint, empty, dtype):
    # the second request's rows first, then (offsets decrease) the first one's
    c = R.attn_case([n, n + 3], [900, 40], 4, 2, 64, 16, dtype, seed=80, spare_rows=2)
    ref = R.attn(c)
    kept = [c["kept"][1]] + [5] * empty + [c["kept"][0]]
    cu = [n, 2 * n + 3] + [0] * empty + [n]
    table = torch.cat([c["table"][1:], c["table"][:1].expand(empty, -1), c["table"][:1]])
    o, lse = run(c["q"], c["kc"], c["vc"], table, kept, cu, hint)
    verdict(c, o, lse, ref)


@pytest.mark.parametrize("hint", [0, 1])
def test_more_claims_than_rows_write_nothing(hint):
    # 40 requests claim the first 8192 rows, one the 40 rows behind them: more parts
    # than a call of 8232 rows has workgroups and partial results for
    c = R.attn_case([8232], [0], 1, 1, 128, 64, BF, seed=81)
    cu = [0, 8192] * 40 + [8232]
    o, lse = run(c["q"], c["kc"], c["vc"], c["table"].expand(80, -1), [0] * 80, cu, hint)
    assert bool((o == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs", [1, 100, 150])
@pytest.mark.parametrize("d", [16, 64])
def test_more_claims_of_small_calls_write_nothing(pairs, d, dtype):
    # one block of requests and two
    c = R.attn_case([40], [30], 2, 1, d, 16, dtype, seed=82)
    cu = [0, 40] * pairs + [0, 1]
    B = len(cu) - 1
    o, lse = run(c["q"], c["kc"], c["vc"], c["table"].expand(B, -1), [30] * B, cu, 0)
    assert bool((o == 7).all()) and bool((lse == 7).all())
