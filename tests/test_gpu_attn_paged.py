"""kda_attn_paged against the dense fp64 form.

Unused cache rows, table entries and query rows hold NaN or nonsense
(serve_ref.attn_case), so every case also checks that they do not reach the
result. Bounds: serve_ref.attn_bound, element by element."""
import random

import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def call(c, *, want_lse=True, sentinel=7.0, **kw):
    o = torch.full(c["q"].shape, sentinel, dtype=c["q"].dtype, device=DEV)
    lse = torch.full(c["q"].shape[:2], sentinel, device=DEV) if want_lse else None
    dev = {k: c[k].to(DEV) for k in ("q", "kc", "vc", "table")}
    kda.kda_attn_paged(dev["q"], dev["kc"], dev["vc"], dev["table"], ints(c["kept"]),
                       ints(c["cu"]), o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    return o.cpu(), None if lse is None else lse.cpu()


def verdict(c, o, lse, ref, sentinel=7.0):
    ro, rl, spread, mag = ref
    T = c["cu"][-1]
    d, dtype = c["q"].shape[2], c["q"].dtype
    keys = max([a + b for a, b in zip(c["kept"], [y - x for x, y in zip(c["cu"], c["cu"][1:])])] + [1])
    assert bool((o[T:] == sentinel).all()), "rows behind the last request were written"
    got = o[:T].double()
    bound = R.attn_bound(ro[:T], spread[:T], mag[:T], d, keys, dtype) + 1e-30
    err = (got - ro[:T]).abs()
    assert not torch.isnan(got).any()
    worst = float((err / bound).max()) if T else 0.0
    print(f"[attn] worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0
    if lse is not None:
        assert bool((lse[T:] == sentinel).all())
        empty = torch.isinf(rl[:T])
        assert torch.equal(torch.isinf(lse[:T]), empty) and bool((lse[:T][empty] < 0).all())
        # a score's error, the sum's, and the logarithm's rounding
        lb = (d + 4) * 2.0 ** -24 * mag[:T] + (keys / 32 + 72) * 2.0 ** -24 + 2.0 ** -21 \
            + 2.0 ** -23 * rl[:T].abs()
        assert bool(((lse[:T].double() - rl[:T]).abs() <= lb)[~empty].all())


def check(c, scale=0.0, **kw):
    ref = R.attn(c, scale)
    o, lse = call(c, scale=scale, **kw)
    verdict(c, o, lse, ref)
    return o, lse


CASES = [
    # n, ctx, Hq, Hkv, d, page
    ([1], [0], 1, 1, 16, 16), ([1], [1], 4, 4, 32, 16), ([1], [15], 8, 2, 64, 16),
    ([1], [16], 8, 2, 128, 16), ([1], [1000], 32, 8, 128, 64), ([1, 1, 1], [0, 63, 64], 16, 2, 64, 64),
    ([1] * 40, list(range(0, 800, 20)), 8, 1, 128, 32),
    ([8], [120], 32, 8, 128, 64), ([8, 3, 5], [1, 300, 4000], 16, 4, 64, 256),
    ([7, 0, 2], [9, 50, 31], 6, 2, 32, 16), ([4] * 9, [33 * i for i in range(9)], 5, 1, 128, 1024),
    ([17], [0], 1, 1, 128, 16), ([33], [5], 4, 1, 64, 16), ([64, 1, 0, 130], [0, 777, 20, 100], 8, 8, 64, 32),
    ([129], [1], 12, 4, 128, 128), ([300, 1, 1, 40], [10, 3000, 0, 555], 16, 4, 128, 64),
    ([511], [1025], 2, 1, 16, 16), ([200, 2], [64, 64], 40, 1, 64, 64), ([257], [0], 3, 3, 128, 64),
    ([1, 90], [5000, 0], 48, 16, 32, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_plain(i, dtype):
    n, ctx, Hq, Hkv, d, page = CASES[i]
    c = R.attn_case(n, ctx, Hq, Hkv, d, page, dtype, seed=i, spare_rows=i % 4)
    check(c, max_new=max(n) if i % 2 else 0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_hint_does_not_matter_for_the_result(dtype):
    c = R.attn_case([90, 1, 9, 33, 2], [40, 700, 64, 0, 2000], 8, 2, 64, 32, dtype, seed=50)
    ref = R.attn(c)
    for hint in (0, 1, 4, 9, 16, 33, 90, 10**6):
        o, lse = call(c, max_new=hint)
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-4, 0.5, 3.0])
def test_scale_and_peaked_rows(dtype, scale):
    c = R.attn_case([40, 1], [100, 300], 8, 4, 64, 16, dtype, seed=51)
    check(c, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [([1, 1], [40, 3]), ([8, 5], [40, 0]), ([100, 30], [40, 0])])
def test_rising_and_falling_scores(n, ctx, dtype):
    # scores that grow along the keys move the running maximum in every tile;
    # falling ones leave it at the first
    for sign in (1.0, -1.0):
        c = R.attn_case(n, ctx, 4, 2, 64, 16, dtype, seed=52)
        c["q"][:c["cu"][-1]] = 1.0
        page = c["page"]
        for i in range(len(n)):
            total = ctx[i] + n[i]
            for pos in range(total):
                c["kc"][c["table"][i, pos // page], :, pos % page] = sign * 0.03125 * pos
        check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [(8, 3), (40, 70), (150, 0)])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_masked_values_stay_out(n, ctx, what, dtype):
    # the last token's key and value are not finite: the rows before it do not see them
    c = R.attn_case([n, 2], [ctx, 20], 8, 2, 64, 16, dtype, seed=53)
    ref = R.attn(c)
    pos = ctx + n - 1
    page = c["table"][0, pos // 16]
    c["vc"][page, :, pos % 16, ::3] = what
    for keys_too in (False, True):
        if keys_too:
            c["kc"][page, :, pos % 16, 1::2] = what
        o, lse = call(c)
        seen = c["cu"][1] - 1
        if not keys_too:
            hit = o[seen].double()
            assert not torch.isfinite(hit[:, ::3]).any()
            assert torch.isfinite(hit[:, 1::3]).all()
        o[seen], lse[seen] = ref[0][seen].to(o.dtype), ref[1][seen].float()
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [(1, 500), (8, 300), (70, 90)])
def test_seen_nan_keys_give_nan(n, ctx, dtype):
    # keys that every row sees: the rows of their heads are NaN, others are not
    c = R.attn_case([n, 2], [ctx, 20], 8, 2, 64, 16, dtype, seed=63)
    ref = R.attn(c)
    for pos in range(0, 90, 3):                     # all of some waves' keys, too
        c["kc"][c["table"][0, pos // 16], 0, pos % 16] = float("nan")
    o, lse = call(c)
    assert torch.isnan(o[:n, :4]).all() and torch.isnan(lse[:n, :4]).all()
    o[:n, :4], lse[:n, :4] = ref[0][:n, :4].to(o.dtype), ref[1][:n, :4].float()
    verdict(c, o, lse, ref)
    c["kc"][c["table"][0, :6].long()] = float("nan")
    o, lse = call(c)
    assert torch.isnan(o[:n]).all() and torch.isnan(lse[:n]).all()


@pytest.mark.parametrize("n", [1, 70])
def test_two_graphs_with_their_own_workspaces(n):
    # captured on two lengths, replayed in turn, each with the tensors it made
    cases = [R.attn_case([n, 1], ctx, 8, 2, 64, 16, BF, seed=64 + i)
             for i, ctx in enumerate([[2500, 40], [300, 4000]])]
    refs, graphs, outs, keep = [], [], [], []
    for c in cases:
        dev = [c[k].to(DEV) for k in ("q", "kc", "vc", "table")] + [ints(c["kept"]), ints(c["cu"])]
        keep.append(dev)
        refs.append(R.attn(c))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            kda.kda_attn_paged(*dev, max_new=n)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kda.kda_attn_paged(*dev, max_new=n, want_lse=True))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        graphs[i].replay()
        graphs[1 - i].replay()
        torch.cuda.synchronize()
        for c, ref, (o, lse) in zip(cases, refs, outs):
            verdict(c, o.cpu(), lse.cpu(), ref)
        kda.kda_attn_paged(*keep[i], max_new=n)     # eager calls in between


def test_overlapping_offsets_end():
    # every request claims all rows: values are unspecified, the call ends and
    # writes nothing behind its rows
    B, T = 64, 300
    c = R.attn_case([T], [700], 8, 2, 64, 16, BF, seed=66, spare_rows=3)
    dev = {k: c[k].to(DEV) for k in ("q", "kc", "vc")}
    table = c["table"].to(DEV).expand(B, -1).contiguous()
    cu = ints([0, T] * (B // 2) + [0])
    for hint in (0, 1):
        o = torch.full(c["q"].shape, 7.0, dtype=BF, device=DEV)
        kda.kda_attn_paged(dev["q"], dev["kc"], dev["vc"], table, ints([700] * B), cu, o=o,
                           max_new=hint)
        torch.cuda.synchronize()
        assert bool((o[T:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 8, 70])
def test_pages_outside_the_pool_are_masked(n, dtype):
    c = R.attn_case([n, n, n], [200, 90, 0], 8, 2, 64, 16, dtype, seed=54)
    c["table"][0, 3] = -1
    c["table"][0, 0] = c["kc"].shape[0]
    c["table"][0, 8] = 2**31 - 1
    c["table"][2] = -2**31                      # a request without any valid page
    o, lse = check(c)
    rows = slice(c["cu"][2], c["cu"][3])
    assert not o[rows].any() and bool((lse[rows] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 60])
def test_positions_past_the_table_are_masked(n, dtype):
    c = R.attn_case([n, n], [500, 100], 4, 4, 64, 16, dtype, seed=55, width=40)
    c["table"] = c["table"][:, :20].contiguous()          # 320 positions
    c["kept"][1] = -5                                     # counts as 0
    check(c)
    c["kept"][0] = 2**31 - 1
    check(c)
    c["table"] = c["table"][:, :0].contiguous()
    o, lse = check(c)
    assert not o.any()


def test_offsets_outside_are_clamped():
    # only where the result is defined: offsets inside [0, T] once clamped
    c = R.attn_case([3, 40, 2], [10, 20, 30], 4, 2, 64, 16, BF, seed=56)
    ref = R.attn(c)
    T = c["cu"][-1]
    cu = c["cu"]
    c["cu"] = [-9, cu[1], cu[2], T + 1000]
    o, lse = call(c)
    c["cu"] = cu
    verdict(c, o, lse, ref)
    # decreasing offsets: that request is empty, the call ends, the others are right
    c["cu"] = [0, 3, 0, 3]
    call(c)


def test_cache_past_32_bit_offsets():
    pool, Hkv, page, d = 40000, 8, 128, 128
    assert pool * Hkv * page * d > 1 << 32
    kc = torch.empty((pool, Hkv, page, d), dtype=BF, device=DEV)
    vc = torch.empty_like(kc)
    for n, dtype in ((1, BF), (40, BF)):
        small = R.attn_case([n, n], [700, 300], 16, Hkv, d, page, dtype, seed=57)
        used = small["kc"].shape[0]
        kc[pool - used:] = small["kc"].to(DEV)
        vc[pool - used:] = small["vc"].to(DEV)
        table = torch.where((small["table"] >= 0) & (small["table"] < used),
                            small["table"] + pool - used, small["table"]).contiguous()
        o = torch.empty_like(small["q"], device=DEV)
        _, lse = kda.kda_attn_paged(small["q"].to(DEV), kc, vc, table.to(DEV), ints(small["kept"]),
                                    ints(small["cu"]), o=o, want_lse=True)
        verdict(small, o.cpu(), lse.cpu(), R.attn(small))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [256, 257, 300, 1100, 17000])
def test_many_requests(B, dtype):
    n = [(i * 7) % 4 for i in range(B)]
    ctx = [(i * 131) % 90 for i in range(B)]
    if B > 5000:                                     # more than 64 blocks of requests
        n = [x if i % 16 == 0 else 0 for i, x in enumerate(n)]
        ctx = [x if i % 16 == 0 else 0 for i, x in enumerate(ctx)]
    n[B // 2], ctx[3], n[3], n[B - 1], ctx[B - 1] = 70, 3000, 1, 2, 700
    for hint in (0, 2):
        check(R.attn_case(n, ctx, 2, 1, 64, 16, dtype, seed=58), max_new=hint)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [([1, 1], [9000, 20]), ([8], [20000]), ([100, 1], [5000, 100])])
def test_long_contexts_in_parts(n, ctx, dtype):
    check(R.attn_case(n, ctx, 8, 2, 128, 64, dtype, seed=59))


@pytest.mark.parametrize("n", [1, 8, 200])
def test_identical_calls_and_graph_replays(n):
    c = R.attn_case([n, 1], [3000, 400], 16, 4, 128, 64, BF, seed=60)
    dev = {k: c[k].to(DEV) for k in ("q", "kc", "vc", "table")}
    kept, cu = ints(c["kept"]), ints(c["cu"])
    ws = torch.empty(max(1, kda.kda_attn_paged_workspace_size(c["q"].shape[0], 2, 16, 4, 128, n, BF)),
                     dtype=torch.uint8, device=DEV)
    o = torch.zeros_like(dev["q"])
    lse = torch.zeros(c["q"].shape[:2], device=DEV)

    def step():
        kda.kda_attn_paged(dev["q"], dev["kc"], dev["vc"], dev["table"], kept, cu, o=o, lse=lse,
                           max_new=n, workspace=ws)
    step()
    ro, rl = o.clone(), lse.clone()
    verdict(c, ro.cpu(), rl.cpu(), R.attn(c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
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
    # another length in the same captured call
    kept.copy_(ints([1200, 17]))
    g.replay()
    torch.cuda.synchronize()
    c["kept"] = [1200, 17]
    verdict(c, o.cpu(), lse.cpu(), R.attn(c))


def test_other_stream():
    c = R.attn_case([1] * 6, [800 * i for i in range(6)], 16, 2, 128, 64, BF, seed=61)
    ref = R.attn(c)
    dev = {k: c[k].to(DEV) for k in ("q", "kc", "vc", "table")}
    kept, cu = ints(c["kept"]), ints(c["cu"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = kda.kda_attn_paged(dev["q"], dev["kc"], dev["vc"], dev["table"], kept, cu,
                                want_lse=True, stream=side)
    junk = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    junk.fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    verdict(c, o.cpu(), lse.cpu(), ref)


def test_refusals():
    c = R.attn_case([2, 3], [5, 6], 4, 2, 64, 16, BF, seed=62)
    q, kc, vc, tab = (c[k].to(DEV) for k in ("q", "kc", "vc", "table"))
    kept, cu = ints(c["kept"]), ints(c["cu"])
    for bad in ((q.float(), kc, vc, tab, kept, cu), (q, kc, vc.float(), tab, kept, cu),
                (q, kc, vc[:, :1], tab, kept, cu), (q[..., :32], kc, vc, tab, kept, cu),
                (q, kc, vc, tab.long(), kept, cu), (q, kc, vc, tab, kept[:1], cu),
                (q, kc, vc, tab, kept, cu[:2]), (q.transpose(0, 1), kc, vc, tab, kept, cu),
                (q.half(), kc.half(), vc.half(), tab, kept, cu), (q, kc.cpu(), vc, tab, kept, cu),
                (q, kc, vc, tab[:, ::2], kept, cu)):
        with pytest.raises(ValueError):
            kda.kda_attn_paged(*bad)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_paged(q[:, :3].contiguous(), kc, vc, tab, kept, cu)     # 3 heads over 2
    with pytest.raises(kda.KDAError):
        kda.kda_attn_paged(q, kc, vc, tab, kept, cu, o=q)
    for s in (-1.0, float("nan")):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_paged(q, kc, vc, tab, kept, cu, scale=s)


@pytest.mark.parametrize("seed", range(10))
def test_random_batches(seed):
    # lengths from nothing to thousands of keys, cut into parts of any length
    rng = random.Random(seed)
    B = rng.choice([1, 2, 3, 7, 20])
    n = [rng.choice([0, 1, 1, 2, 8, 31, rng.randint(1, 150)]) for _ in range(B)]
    ctx = [int(2 ** rng.uniform(0, 12.5)) for _ in range(B)]
    Hkv = rng.choice([1, 2, 3])
    c = R.attn_case(n, ctx, Hkv * rng.choice([1, 3, 4]), Hkv, rng.choice([16, 32, 64, 128]),
                    rng.choice([16, 64, 256]), rng.choice([BF, F32]), seed=seed, spare_rows=2)
    check(c, max_new=rng.choice([0, 0, max(n)]))
