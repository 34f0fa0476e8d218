"""kda_attn_paged over pools of several GB, with much and with little of them in use.

Keys and values of more than the last-level cache may hold are read past it: the
work of a call decides, so both kinds run here at every width and kernel that has
them. Tables repeat pages, as requests with a shared prefix do."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints
from test_gpu_attn_paged import verdict

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
PAGE, HKV, POOL = 128, 8, 9000
DISTINCT = 4                                   # requests with pages of their own


@pytest.fixture(scope="module", params=[64, 128])
def pool(request):
    d = request.param
    # 2.4 GB (d of 64: 1.2 GB) each for K and V, NaN but for what a test puts at the end
    return [torch.full((POOL, HKV, PAGE, d), float("nan"), dtype=BF, device=DEV) for _ in range(2)]


def run(pool, n, ctx, G, copies, max_new):
    """The distinct requests, and copies of each of them: the copies' results are
    the same bits, and the first ones those of the plain form."""
    kc, vc = pool
    d = kc.shape[3]
    small = R.attn_case(n, ctx, HKV * G, HKV, d, PAGE, BF, seed=d + copies)
    used = small["kc"].shape[0]
    kc[POOL - used:], vc[POOL - used:] = small["kc"].to(DEV), small["vc"].to(DEV)
    table = torch.where((small["table"] >= 0) & (small["table"] < used),
                        small["table"] + POOL - used, small["table"]).to(DEV)
    T = small["cu"][-1]
    q = small["q"].to(DEV).repeat(copies, 1, 1)
    cu = [0]
    for x in list(n) * copies:
        cu.append(cu[-1] + x)
    o, lse = kda.kda_attn_paged(q, kc, vc, table.repeat(copies, 1), ints(list(ctx) * copies), ints(cu),
                                max_new=max_new, want_lse=True)
    torch.cuda.synchronize()
    verdict(small, o[:T].cpu(), lse[:T].cpu(), R.attn(small))
    for i in range(copies):
        assert torch.equal(o[i * T:(i + 1) * T], o[:T]), f"copy {i}"
        assert torch.equal(lse[i * T:(i + 1) * T], lse[:T]), f"copy {i}"


# rows of a request: 2 (one row group), 24 (two), and 24 beside a prompt of 80
@pytest.mark.parametrize("n,hint", [([1, 1, 1, 1], 1), ([12, 9, 12, 11], 12), ([1, 12, 40, 5], 40)])
@pytest.mark.parametrize("copies", [1, 60, 100])
def test_much_and_little_of_a_pool(pool, n, hint, copies):
    # 4 requests of 2100 positions are 34 MB at width 128 and 17 at 64; 240 of them
    # 2.1 and 1.0 GB; 400 are more than one block of requests
    ctx = [2100, 1999, 2300, 2150]
    run(pool, n, ctx, 2, copies, hint)


def test_hint_too_small(pool):
    # rows of a request in several tiles of the streams, which read its keys again
    run(pool, [70, 1, 33, 2], [2100, 1999, 2300, 2150], 2, 60, 1)


@pytest.mark.parametrize("n", [1, 12])
def test_replays_with_lengths_of_both_kinds(pool, n):
    # one captured call of more than a block of requests, replayed with lengths that
    # read little and much; each replay gives what the eager call gives
    kc, vc = pool
    d, B = kc.shape[3], 300
    small = R.attn_case([n] * 3, [2500] * 3, 2 * HKV, HKV, d, PAGE, BF, seed=5 + n)
    used = small["kc"].shape[0]
    kc[POOL - used:], vc[POOL - used:] = small["kc"].to(DEV), small["vc"].to(DEV)
    table = torch.where((small["table"] >= 0) & (small["table"] < used),
                        small["table"] + POOL - used, small["table"]).to(DEV).repeat(B // 3, 1)
    q = small["q"].to(DEV).repeat(B // 3, 1, 1)
    cu = ints([n * i for i in range(B + 1)])
    kept = ints([2500] * B)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    ws = torch.empty(kda.kda_attn_paged_workspace_size(q.shape[0], B, 2 * HKV, HKV, d, n, BF),
                     dtype=torch.uint8, device=DEV)

    def step():
        kda.kda_attn_paged(q, kc, vc, table, kept, cu, o=o, lse=lse, max_new=n, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for length in (2500, 100, 2400, 30, 2500):
        kept.fill_(length)
        o.zero_()
        step()
        torch.cuda.synchronize()
        ro, rl = o.clone(), lse.clone()
        o.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ro) and torch.equal(lse, rl), length
        c = dict(small, kept=[length] * 3)
        verdict(c, o[:3 * n].cpu(), lse[:3 * n].cpu(), R.attn(c))
