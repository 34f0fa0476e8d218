"""kda_attn_latent against the dense fp64 form.

Unused cache rows, table entries and query rows hold NaN or nonsense
(full_ref.latent_case), so every case also checks that they do not reach the result."""
import random

import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, ints

pytestmark = pytest.mark.gpu


def call(c, *, want_lse=True, sentinel=7.0, **kw):
    T, Hq, _ = c["q"].shape
    o = torch.full((T, Hq, c["dc"]), sentinel, dtype=c["q"].dtype, device=DEV)
    lse = torch.full((T, Hq), sentinel, device=DEV) if want_lse else None
    kda.kda_attn_latent(c["q"].to(DEV), c["cache"].to(DEV), c["table"].to(DEV).contiguous(),
                        ints(c["kept"]), ints(c["cu"]), dc=c["dc"], scale=c["scale"], o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    return o.cpu(), None if lse is None else lse.cpu()


def verdict(c, o, lse, ref, sentinel=7.0):
    n = [y - x for x, y in zip(c["cu"], c["cu"][1:])]
    keys = max([min(max(a, 0) + b, c["table"].shape[1] * c["page"]) for a, b in zip(c["kept"], n)] + [1])
    return R.check_attention(o, lse, ref, c["cu"][-1], c["q"].shape[2], keys, sentinel, "latent")


def check(c, **kw):
    ref = R.latent(c)
    o, lse = call(c, **kw)
    verdict(c, o, lse, ref)
    return o, lse


CASES = [
    # n, ctx, Hq, dc, page
    ([1], [0], 1, 128, 16), ([1], [1], 4, 256, 16), ([1], [15], 16, 512, 64), ([1], [16], 32, 512, 64),
    ([1], [1000], 32, 512, 64), ([1, 1, 1], [0, 63, 64], 16, 512, 64), ([1], [129], 128, 512, 64),
    ([1] * 20, list(range(0, 400, 20)), 20, 256, 32), ([8], [120], 16, 512, 64),
    ([8, 3, 5], [1, 300, 1400], 5, 512, 256), ([7, 0, 2], [9, 50, 31], 6, 128, 16),
    ([4] * 5, [33 * i for i in range(5)], 12, 512, 1024), ([17], [0], 2, 512, 16),
    ([33], [5], 4, 512, 16), ([64, 1, 0, 130], [0, 777, 20, 100], 3, 256, 32),
    ([129], [1], 2, 128, 128), ([40, 1, 1, 20], [10, 2000, 0, 555], 16, 512, 64),
    ([3], [200], 64, 512, 64), ([1, 2], [700, 64], 64, 512, 16), ([200], [0], 1, 512, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_plain(i, dtype):
    n, ctx, Hq, dc, page = CASES[i]
    c = R.latent_case(n, ctx, Hq, dc, page, dtype, seed=i, spare_rows=i % 4)
    check(c, max_new=max(n) if i % 2 else 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dc", [128, 512])
def test_hint_does_not_matter_for_the_result(dc, dtype):
    c = R.latent_case([9, 1, 30, 2], [40, 700, 64, 1000], 8, dc, 32, dtype, seed=50)
    ref = R.latent(c)
    for hint in (0, 1, 4, 8, 9, 30, 10**6):
        o, lse = call(c, max_new=hint)
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-4, 0.3, 1.0])
def test_scale_and_peaked_rows(scale, dtype):
    c = R.latent_case([6, 1], [100, 300], 8, 256, 16, dtype, seed=51)
    c["scale"] = scale
    check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n", [(4, 1), (40, 1), (100, 2)])
def test_rising_and_falling_scores(Hq, n, dtype):
    # scores that grow along the keys move the running maximum in every step; falling
    # ones leave it at the first
    for sign in (1.0, -1.0):
        c = R.latent_case([n, 1], [400, 70], Hq, 128, 16, dtype, seed=52)
        c["q"][:c["cu"][-1]] = 1.0
        for i, total in enumerate((400 + n, 71)):
            for pos in range(total):
                c["cache"][c["table"][i, pos // 16], pos % 16] = sign * 0.03125 * pos
        check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("big", [0, 90])
@pytest.mark.parametrize("Hq,n,dc", [(3, 1, 128), (16, 2, 512), (40, 1, 512), (20, 5, 256), (7, 40, 128)])
def test_maxima_that_jump(Hq, n, dc, big, dtype):
    # peaks anywhere, for all rows, for some or for none; with values of 2^90, which a
    # weight far above 1 must not carry out of fp32
    c = R.latent_case([n, n, 1], [900, 333, 2100], Hq, dc, 16, dtype, seed=70)
    T = c["cu"][-1]
    rows = torch.arange(T * Hq).view(T, Hq) % 5
    c["q"][:T, :, dc + 1] = torch.tensor([0.0, 1.0, 0.5, -1.0, 0.03125])[rows].to(dtype)
    if big:
        c["q"][:T, :, :dc] = 0.0
    for i, total in enumerate((900 + n, 333 + n, 2101)):
        x = R.jumps(total, 70 + i) / (c["scale"] * 1.4427)
        pages = c["table"][i, torch.arange(total) // 16].long()
        c["cache"][pages, torch.arange(total) % 16, dc + 1] = x.to(dtype)
        c["cache"][pages, torch.arange(total) % 16, :dc] *= 2.0 ** big
    check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n,ctx,hint", [
    (128, [1] * 6, [0, 1, 700, 63, 3000, 64], 1),          # two tiles of 64 rows, or four of 32
    (64, [4, 4, 4], [5, 2000, 90], 4),                     # four
    (64, [1, 7, 0], [900, 33, 5], 4),                      # the hint's product is T, no length is
    (96, [2, 2], [40, 1500], 2),                           # three of 64, six of 32
    (128, [1], [0], 1), (128, [1], [9], 1),                # fewer units than workgroups
    (64, [1] * 300, [(37 * i) % 150 for i in range(300)], 1)])
def test_rows_of_equal_requests_side_by_side(Hq, n, ctx, hint, dtype):
    c = R.latent_case(n, ctx, Hq, 512 if len(n) < 9 else 128, 64, dtype, seed=71)
    check(c, max_new=hint)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n", [(16, 1), (128, 1), (9, 30)])
def test_workspace_of_the_named_size(Hq, n, dtype):
    c = R.latent_case([n] * 3, [1500, 40, 7], Hq, 256, 32, dtype, seed=72)
    need = kda.kda_attn_latent_workspace_size(3 * n, 3, Hq, 256, 64, n, dtype)
    ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    check(c, max_new=n, workspace=ws)
    assert bool((ws[need:] == 0xAB).all())
    check(c, max_new=n, workspace=ws[:need - 1])          # too small: another one is used


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n,ctx", [(2, 8, 3), (8, 20, 70), (50, 3, 40), (16, 8, 300)])
@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan")])
def test_masked_positions_stay_out(Hq, n, ctx, what, dtype):
    # the last token's row is not finite: the tokens before it do not see it
    c = R.latent_case([n, 2], [ctx, 20], Hq, 256, 16, dtype, seed=53)
    ref = R.latent(c)
    pos = ctx + n - 1
    for cols in (slice(0, 256, 3), slice(256, 320, 5)):
        row = c["cache"][c["table"][0, pos // 16], pos % 16]
        keep = row.clone()
        row[cols] = what
        o, lse = call(c)
        row.copy_(keep)
        seen = c["cu"][1] - 1
        if what != what:
            assert bool(torch.isnan(o[seen]).all()) and bool(torch.isnan(lse[seen]).all())
        o[seen], lse[seen] = ref[0][seen].to(o.dtype), ref[1][seen].float()
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [(1, 500), (8, 300), (30, 90)])
def test_seen_nan_gives_nan(n, ctx, dtype):
    c = R.latent_case([n, 2], [ctx, 20], 8, 128, 16, dtype, seed=54)
    ref = R.latent(c)
    for pos in range(0, 90, 3):
        c["cache"][c["table"][0, pos // 16], pos % 16, pos % 192] = float("nan")
    o, lse = call(c)
    assert bool(torch.isnan(o[:n]).all()) and bool(torch.isnan(lse[:n]).all())
    o[:n], lse[:n] = ref[0][:n].to(o.dtype), ref[1][:n].float()
    verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_lowest_scores_and_none(dtype):
    # scores at the type's lowest values keep their order; -infinity alone gives 0
    c = R.latent_case([1, 1], [70, 70], 3, 128, 16, dtype, seed=55)
    c["q"][0] = 0
    c["q"][0, :, 191] = 1.0
    for i in range(2):
        c["cache"][c["table"][i, :5].long(), :, 191] = -1e38
    check(c)
    c["q"][0, :, 191] = float("inf")
    c["cache"][c["table"][0, :5].long(), :, 191] = -1.0
    o, lse = call(c)
    assert not o[0].any() and bool((lse[0] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n", [(4, 1), (40, 1), (5, 30)])
def test_pages_outside_the_pool_are_masked(Hq, n, dtype):
    c = R.latent_case([n, n, n], [200, 90, 0], Hq, 512, 16, dtype, seed=56)
    c["table"][0, 3] = -1
    c["table"][0, 0] = c["cache"].shape[0]
    c["table"][0, 8] = 2**31 - 1
    c["table"][2] = -2**31                      # a request without any valid page
    o, lse = check(c)
    rows = slice(c["cu"][2], c["cu"][3])
    assert not o[rows].any() and bool((lse[rows] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 12])
def test_positions_past_the_table_are_masked(n, dtype):
    c = R.latent_case([n, n], [500, 100], 6, 256, 16, dtype, seed=57, width=40)
    c["table"] = c["table"][:, :20].contiguous()          # 320 positions
    c["kept"][1] = -5                                     # counts as 0
    check(c)
    c["kept"][0] = 2**31 - 1
    check(c)
    c["table"] = c["table"][:, :0].contiguous()
    o, _ = check(c)
    assert not o.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pool", [0, 1])
def test_no_pool(pool, dtype):
    c = R.latent_case([2, 1], [3, 0], 4, 128, 16, dtype, seed=58)
    c["cache"] = c["cache"][:pool].contiguous()
    c["table"][:] = pool
    o, lse = check(c)
    assert not o[:3].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("empty", [1, 300])
@pytest.mark.parametrize("n,hint", [(2, 0), (2, 2), (20, 1)])
def test_offsets_in_any_order(n, hint, empty, dtype):
    # the second request's rows first, then (offsets decrease) the first one's
    c = R.latent_case([n, n + 3], [900, 40], 4, 128, 16, dtype, seed=59, spare_rows=2)
    ref = R.latent(c)
    d = dict(c, kept=[c["kept"][1]] + [5] * empty + [c["kept"][0]],
             cu=[n, 2 * n + 3] + [0] * empty + [n],
             table=torch.cat([c["table"][1:], c["table"][:1].expand(empty, -1), c["table"][:1]]))
    o, lse = call(d, max_new=hint)
    verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs", [1, 100, 150])
def test_more_claims_than_rows_write_nothing(pairs, dtype):
    c = R.latent_case([40], [30], 2, 128, 16, dtype, seed=60)
    cu = [0, 40] * pairs + [0, 1]
    B = len(cu) - 1
    o, lse = call(dict(c, cu=cu, kept=[30] * B, table=c["table"].expand(B, -1)))
    assert bool((o == 7).all()) and bool((lse == 7).all())


def test_cache_past_32_bit_offsets():
    pool, page, W = 60000, 128, 576
    assert pool * page * W > 1 << 32
    cache = torch.empty((pool, page, W), dtype=BF, device=DEV)
    for n, Hq in ((1, 16), (3, 50)):
        c = R.latent_case([n, n], [700, 300], Hq, 512, page, BF, seed=61)
        used = c["cache"].shape[0]
        cache[pool - used:] = c["cache"].to(DEV)
        table = torch.where((c["table"] >= 0) & (c["table"] < used), c["table"] + pool - used,
                            c["table"]).contiguous()
        o, lse = kda.kda_attn_latent(c["q"].to(DEV), cache, table.to(DEV), ints(c["kept"]),
                                     ints(c["cu"]), dc=512, scale=c["scale"], want_lse=True)
        verdict(c, o.cpu(), lse.cpu(), R.latent(c))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [256, 257, 1100, 17000])
def test_many_requests(B, dtype):
    n = [(i * 7) % 4 for i in range(B)]
    ctx = [(i * 131) % 90 for i in range(B)]
    if B > 5000:
        n = [x if i % 32 == 0 else 0 for i, x in enumerate(n)]
        ctx = [x if i % 32 == 0 else 0 for i, x in enumerate(ctx)]
    n[B // 2], ctx[3], n[3], n[B - 1], ctx[B - 1] = 30, 3000, 1, 2, 700
    check(R.latent_case(n, ctx, 2, 128, 16, dtype, seed=62), max_new=0 if B % 2 else 30)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,n,ctx", [(16, [1, 1], [9000, 20]), (8, [8], [20000]),
                                      (128, [1, 2], [5000, 100]), (64, [1], [3000])])
def test_long_contexts_in_parts(Hq, n, ctx, dtype):
    rel = None
    c = R.latent_case(n, ctx, Hq, 512, 64, dtype, seed=63)
    ref = R.latent(c)
    o, lse = call(c)
    verdict(c, o, lse, ref)
    # Over a whole case the roundings average out: before its rounding a result has a
    # relative error in norm of a score's 576 steps, independent, 2^-24 sqrt(576 / 3) of
    # a magnitude of 30 (below 2^-15 with the exponential's), and of the weights' two
    # terms, 2^-15. An error of size x moves a rounded bf16 value by a unit u with
    # probability x / u: sqrt(2^-7 2^-14) < 2^-10. fp32: 2^-15.
    rounded = ref[0].to(dtype).double() if dtype == BF else ref[0]
    rel = float((o.double() - rounded).norm() / ref[0].norm())
    assert rel <= (2.0 ** -10 if dtype == BF else 2.0 ** -15), rel


@pytest.mark.parametrize("Hq,n", [(16, 1), (128, 1), (8, 40)])
def test_identical_calls_and_graph_replays(Hq, n):
    c = R.latent_case([n, 1], [2000, 400], Hq, 512, 64, BF, seed=64)
    q, cache, table = (c[k].to(DEV) for k in ("q", "cache", "table"))
    kept, cu = ints(c["kept"]), ints(c["cu"])
    ws = torch.empty(max(1, kda.kda_attn_latent_workspace_size(n + 1, 2, Hq, 512, 64, n, BF)),
                     dtype=torch.uint8, device=DEV)
    o = torch.zeros((n + 1, Hq, 512), dtype=BF, device=DEV)
    lse = torch.zeros((n + 1, Hq), device=DEV)

    def step():
        kda.kda_attn_latent(q, cache, table, kept, cu, dc=512, scale=c["scale"], o=o, lse=lse, max_new=n,
                            workspace=ws)
    step()
    ro, rl = o.clone(), lse.clone()
    verdict(c, ro.cpu(), rl.cpu(), R.latent(c))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        o.zero_()
        lse.zero_()
        ws.fill_(0xFF)                       # the workspace carries nothing between calls
        if i == 2:
            step()                           # the program's own eager call between replays
            torch.cuda.synchronize()
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ro) and torch.equal(lse, rl), f"replay {i}"
    kept.copy_(ints([700, 17]))              # other lengths in the same captured call
    g.replay()
    torch.cuda.synchronize()
    c["kept"] = [700, 17]
    verdict(c, o.cpu(), lse.cpu(), R.latent(c))


def test_two_graphs_with_their_own_workspaces():
    cases = [R.latent_case([1, 1], ctx, 16, 256, 16, BF, seed=65 + i)
             for i, ctx in enumerate([[2500, 40], [300, 4000]])]
    refs, graphs, outs, keep = [], [], [], []
    for c in cases:
        dev = [c[k].to(DEV) for k in ("q", "cache", "table")] + [ints(c["kept"]), ints(c["cu"])]
        keep.append(dev)
        refs.append(R.latent(c))
        kda.kda_attn_latent(*dev, dc=256, scale=c["scale"], max_new=1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.kda_attn_latent(*dev, dc=256, scale=c["scale"], max_new=1, want_lse=True))
        graphs.append(g)
    for i in (0, 1, 1, 0):
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        for c, ref, (o, lse) in zip(cases, refs, outs):
            verdict(c, o.cpu(), lse.cpu(), ref)
        kda.kda_attn_latent(*keep[i], dc=256, scale=cases[i]["scale"])


def test_two_streams_at_once():
    cases = [R.latent_case([1] * 5, [700 * i + 10 * k for i in range(5)], 16, 512, 64, BF, seed=67 + k)
             for k in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [[c[k].to(DEV) for k in ("q", "cache", "table")] + [ints(c["kept"]), ints(c["cu"])] for c in cases]
    torch.cuda.synchronize()
    outs = [kda.kda_attn_latent(*d, dc=512, scale=c["scale"], want_lse=True, stream=s)
            for c, d, s in zip(cases, dev, streams)]
    torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cases, outs):
        verdict(c, o.cpu(), lse.cpu(), R.latent(c))


def test_refusals():
    c = R.latent_case([2, 3], [5, 6], 4, 128, 16, BF, seed=69)
    q, cache, tab = (c[k].to(DEV) for k in ("q", "cache", "table"))
    kept, cu = ints(c["kept"]), ints(c["cu"])
    good, kw = (q, cache, tab, kept, cu), dict(dc=128, scale=0.1)
    kda.kda_attn_latent(*good, **kw)
    for i, bad in ((0, q.float()), (0, q.half()), (0, q.transpose(0, 1)), (0, q[..., :128]), (1, cache.float()),
                   (1, cache.cpu()), (2, tab.long()), (2, tab[:, ::2]), (3, kept[:1]), (4, cu[:2])):
        with pytest.raises(ValueError):
            kda.kda_attn_latent(*good[:i], bad, *good[i + 1:], **kw)
    with pytest.raises(ValueError):
        kda.kda_attn_latent(*good, **kw, o=torch.empty_like(q))
    for bad in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(dc=64), dict(dc=96), dict(dc=192)):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_latent(*good, **{**kw, **bad})
    with pytest.raises(kda.KDAError):
        kda.kda_attn_latent(*good, **kw, o=q.view(-1)[:5 * 4 * 128].view(5, 4, 128))
    with pytest.raises(kda.KDAError):
        kda.kda_attn_latent(*good, **kw, max_new=-1)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = random.Random(seed)
    B = rng.choice([1, 2, 3, 7, 15])
    n = [rng.choice([0, 1, 1, 2, 8, rng.randint(1, 40)]) for _ in range(B)]
    ctx = [int(2 ** rng.uniform(0, 11.5)) for _ in range(B)]
    c = R.latent_case(n, ctx, rng.choice([1, 3, 16, 20, 64]), rng.choice([128, 256, 512]),
                      rng.choice([16, 64, 256]), rng.choice([BF, F32]), seed=seed, spare_rows=2)
    check(c, max_new=rng.choice([0, 0, max(n)]))
