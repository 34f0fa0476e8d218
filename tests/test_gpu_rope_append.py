"""kda_rope_append against the 64-bit rotation and a copy of rows."""
import random

import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, ints

pytestmark = pytest.mark.gpu


def case(n, ctx, Hq, Hkv, d, rot, page, dtype, *, interleaved=False, factor=1.0, seed=0, spare=0,
         base=10000.0):
    g = torch.Generator().manual_seed(seed)
    cu = R.offsets(n)
    T = cu[-1] + spare
    pool = -(-T // page) + 2
    q, k, v = (torch.randn((T, h, d), generator=g).to(dtype) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(pool * page, generator=g)[:T].to(torch.int32)
    f, _ = kda.kda_rope_freqs(rot, base=base)
    return dict(q=q, k=k, v=v, slots=slots, kept=list(ctx), cu=cu, f=f, interleaved=interleaved,
                factor=factor, pool=pool, page=page)


def call(c, q_out=None, in_place=False, sentinel=7.0, **kw):
    T, Hkv, d = c["k"].shape
    dt = c["k"].dtype
    rope = kda.KDARope(c["f"].to(DEV), interleaved=c["interleaved"], factor=c["factor"])
    kc, vc = (torch.full((c["pool"], Hkv, c["page"], d), sentinel, dtype=dt, device=DEV)
              for _ in range(2))
    q = c["q"].to(DEV)
    out = q if in_place else torch.full(c["q"].shape, sentinel, dtype=dt, device=DEV)
    got = kda.kda_rope_append(q, c["k"].to(DEV), c["v"].to(DEV), c["slots"].to(DEV), ints(c["kept"]),
                              ints(c["cu"]), kc, vc, rope, q_out=out, **kw)
    torch.cuda.synchronize()
    assert got is out
    if not in_place:
        assert torch.equal(q.cpu().view(torch.uint8), c["q"].view(torch.uint8))
    return out.cpu(), kc.cpu(), vc.cpu()


def verdict(c, out, kc, vc, in_place=False, sentinel=7.0, pos=None):
    T, Hkv, d = c["k"].shape
    dt, rot, page = c["k"].dtype, 2 * len(c["f"]), c["page"]
    pos = R.positions(c["cu"], c["kept"], T) if pos is None else pos
    rows_k, rows_v = (x.transpose(1, 2).reshape(x.shape[0] * page, Hkv, d) for x in (kc, vc))
    for name, src in (("q", c["q"]), ("k", c["k"])):
        y, mag = R.rotate(src[..., :rot], pos, c["f"], c["interleaved"], c["factor"])
        bound = R.rotation_bound(y, mag, dt)
        written = torch.zeros(rows_k.shape[0], dtype=torch.bool)
        for t in range(T):
            slot = int(c["slots"][t])
            if name == "q":
                if pos[t] is None:
                    assert torch.equal(out[t], c["q"][t] if in_place else torch.full_like(out[t], sentinel))
                    continue
                got = out[t]
            else:
                if pos[t] is None or not 0 <= slot < rows_k.shape[0]:
                    continue
                got = rows_k[slot]
                written[slot] = True
                assert torch.equal(rows_v[slot], c["v"][t])
            assert torch.equal(got[:, rot:], src[t, :, rot:])
            assert bool(((got[:, :rot].double() - y[t]).abs() <= bound[t]).all()), (name, t)
        if name == "k":
            assert bool((rows_k[~written] == sentinel).all() and (rows_v[~written] == sentinel).all())


CASES = [
    # n, ctx, Hq, Hkv, d, rot, page
    ([1], [0], 1, 1, 16, 16, 16), ([1], [5], 4, 2, 32, 16, 16), ([3, 0, 1], [0, 9, 100], 8, 2, 64, 64, 64),
    ([1] * 9, list(range(9)), 32, 8, 128, 128, 64), ([5, 70, 2], [4000, 0, 131071], 6, 3, 128, 64, 32),
    ([33], [1000000], 5, 1, 128, 48, 256), ([1, 1], [2**31 - 2, 2**30], 3, 1, 64, 32, 16),
    ([700, 1, 400], [0, 17, 12345], 2, 1, 64, 48, 1024), ([0, 0, 4], [1, 2, 3], 40, 40, 32, 32, 128),
    ([2], [1], 0, 2, 64, 64, 16), ([2], [1], 3, 0, 64, 64, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_plain(i, interleaved, dtype):
    n, ctx, Hq, Hkv, d, rot, page = CASES[i]
    c = case(n, ctx, Hq, Hkv, d, rot, page, dtype, interleaved=interleaved,
             factor=1.0 if i % 2 else 1.4852, seed=i, spare=i % 3)
    for in_place in (False, True):
        verdict(c, *call(c, in_place=in_place), in_place=in_place)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tokens_take_the_other_split(dtype):
    # more than 4096 tokens: a wave a token instead of four
    n = [4000, 1, 0, 180]
    c = case(n, [7, 90000, 3, 0], 4, 2, 64, 32, 64, dtype, seed=50, spare=5)
    verdict(c, *call(c))


@pytest.mark.parametrize("B", [63, 64, 65, 4096, 4200, 270000])
def test_many_requests(B):
    # the search over the offsets in one, two and three steps
    rng = random.Random(B)
    n = [0] * B
    for i in [0, B - 1, B // 2, 62 % B, 63 % B, 64 % B] + [rng.randrange(B) for _ in range(30)]:
        n[i] = rng.randint(1, 3)
    ctx = [rng.randint(0, 10**6) if x else 5 for x in n]
    c = case(n, ctx, 2, 1, 16, 16, 16, F32, seed=51, spare=2)
    verdict(c, *call(c))


def test_slots_outside_are_skipped():
    c = case([40], [3], 2, 2, 32, 32, 16, BF, seed=52)
    for t, s in ((3, -1), (7, c["pool"] * 16), (9, 2**31 - 1), (20, -2**31)):
        c["slots"][t] = s
    verdict(c, *call(c))


def test_offsets_and_lengths_outside():
    # kept below 0 counts as 0; offsets are clamped to [0, T]
    c = case([3, 9, 4], [-7, 20, 30], 2, 1, 32, 32, 16, F32, seed=53, spare=2)
    verdict(c, *call(c))
    T = c["k"].shape[0]
    c["cu"] = [-5, 3, 12, T + 100]
    verdict(c, *call(c))
    # decreasing offsets: rows that one request alone claims, behind all the disorder,
    # are not demanded; the call ends and writes no slot that it was not given
    c["cu"] = [9, 3, 0, 12]
    out, kc, vc = call(c)
    rows = kc.transpose(1, 2).reshape(-1, 1, 32)
    given = torch.zeros(rows.shape[0], dtype=torch.bool)
    given[c["slots"].long()] = True
    assert bool((rows[~given] == 7).all())


def test_rotation_keeps_lengths_and_differences():
    # properties of the rotation itself: lengths stay, and q.k depends on the distance
    d, g = 64, torch.Generator().manual_seed(3)
    x = torch.randn((2, 1, d), generator=g)
    f, _ = kda.kda_rope_freqs(d)
    dots = []
    for at in (0, 1000):
        c = dict(q=x, k=x.clone(), v=x.clone(), slots=torch.tensor([0, 1], dtype=torch.int32),
                 kept=[at], cu=[0, 2], f=f, interleaved=False, factor=1.0, pool=1, page=16)
        out, kc, _ = call(c)
        assert torch.allclose(out.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
        dots.append(float(out[1, 0].double() @ kc[0, 0, 0].double()))
    assert abs(dots[0] - dots[1]) <= 64 * 4 * 2.0 ** -24 * float(x.abs().max()) ** 2 * 2


def test_values_that_are_not_finite_stay_in_their_pairs():
    c = case([4], [11], 2, 1, 64, 32, 16, F32, seed=54)
    c["q"][1, 0, 5] = float("nan")
    c["k"][2, 0, 40] = float("inf")              # not rotated: copied
    out, kc, vc = call(c)
    bad = torch.isnan(out)
    assert bad[1, 0, 5] and bad[1, 0, 21] and int(bad.sum()) == 2
    slot = int(c["slots"][2])
    row = kc.transpose(1, 2).reshape(-1, 64)[slot]
    assert torch.isinf(row[40]) and int((~torch.isfinite(row)).sum()) == 1


@pytest.mark.parametrize("tokens", [1, 300, 5000])
def test_other_stream_and_graph(tokens):
    c = case([tokens, 1], [50, 2000], 8, 2, 64, 64, 64, BF, seed=55)
    ref = call(c)
    verdict(c, *ref)
    rope = kda.KDARope(c["f"].to(DEV))
    dev = [c[k].to(DEV) for k in ("q", "k", "v", "slots")]
    kept, cu = ints(c["kept"]), ints(c["cu"])
    kc, vc = (torch.full(ref[1].shape, 7.0, dtype=BF, device=DEV) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = kda.kda_rope_append(*dev, kept, cu, kc, vc, rope, stream=side)
    torch.empty(8 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref[0]) and torch.equal(kc.cpu(), ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_rope_append(*dev, kept, cu, kc, vc, rope, q_out=out)
    for i in range(3):
        out.zero_()
        kc.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), ref[0]) and torch.equal(kc.cpu(), ref[1])
        assert torch.equal(vc.cpu(), ref[2])


def test_refusals():
    c = case([2, 3], [5, 6], 4, 2, 64, 32, 16, BF, seed=56)
    rope = kda.KDARope(c["f"].to(DEV))
    q, k, v, slots = (c[x].to(DEV) for x in ("q", "k", "v", "slots"))
    kept, cu = ints(c["kept"]), ints(c["cu"])
    kc, vc = (torch.zeros((c["pool"], 2, 16, 64), dtype=BF, device=DEV) for _ in range(2))
    good = (q, k, v, slots, kept, cu, kc, vc, rope)
    kda.kda_rope_append(*good)
    for i, bad in ((0, q.float()), (0, q.half()), (1, k[:, :1]), (1, k.float()), (2, v[:4]),
                   (3, slots.long()), (4, kept[:1]), (5, cu[:2]), (6, kc.float()), (7, vc[:1]),
                   (0, q.cpu()), (0, q.transpose(0, 1)), (3, slots.cpu())):
        with pytest.raises(ValueError):
            kda.kda_rope_append(*good[:i], bad, *good[i + 1:])
    with pytest.raises(ValueError):
        kda.kda_rope_append(*good, q_out=torch.zeros((4, 4, 64), dtype=BF, device=DEV))
    with pytest.raises(kda.KDAError):
        kda.kda_rope_append(*good, q_out=kc.view(-1)[:5 * 4 * 64].view(5, 4, 64))
    for f, kw in ((torch.ones(36, dtype=torch.float64), {}), (torch.ones(12, dtype=torch.float64), {}),
                  (torch.ones(16, dtype=torch.float64), dict(factor=float("nan"))),
                  (torch.ones(16, dtype=torch.float64), dict(factor=float("inf")))):
        with pytest.raises(kda.KDAError):
            kda.kda_rope_append(*good[:-1], kda.KDARope(f.to(DEV), **kw))
    with pytest.raises(ValueError):
        kda.KDARope(torch.ones(16, device=DEV))
    with pytest.raises(ValueError):
        kda.KDARope(torch.ones(16, dtype=torch.float64))
