"""kda_latent_append against the 64-bit normalisation and rotation."""
import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, HALF, ints

pytestmark = pytest.mark.gpu
DR = 64


def case(n, ctx, dc, dtype, *, Hq=4, dq=192, dq_out=None, page=16, interleaved=False, factor=1.0,
         w=True, normalise=True, rope=True, kv_out=True, seed=0, spare=0, eps=1e-6):
    g = torch.Generator().manual_seed(seed)
    cu = R.offsets(n)
    T = cu[-1] + spare
    pool = -(-T // page) + 2
    kv = torch.randn((T, dc + DR), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    q = torch.randn((T, Hq, dq), generator=g)
    f, _ = kda.kda_rope_freqs(DR)
    return dict(kv=kv.to(dtype), q=q.to(dtype), dq_out=dq if dq_out is None else dq_out,
                w=1 + 0.3 * torch.randn(dc, generator=g) if w and normalise else None,
                slots=torch.randperm(pool * page, generator=g)[:T].to(torch.int32), kept=list(ctx),
                cu=cu, f=f if rope else None, interleaved=interleaved, factor=factor, pool=pool,
                page=page, normalise=normalise, eps=eps, dc=dc, kv_out=kv_out)


def call(c, in_place=False, sentinel=7.0, **kw):
    T, W = c["kv"].shape
    dt = c["kv"].dtype
    rope = None if c["f"] is None else kda.KDARope(c["f"].to(DEV), interleaved=c["interleaved"],
                                                   factor=c["factor"])
    cache = torch.full((c["pool"], c["page"], W), sentinel, dtype=dt, device=DEV)
    kv, q = c["kv"].to(DEV), c["q"].to(DEV)
    out = kv if in_place else torch.full(c["kv"].shape, sentinel, dtype=dt, device=DEV)
    qo = q if in_place else torch.full((T, q.shape[1], c["dq_out"]), sentinel, dtype=dt, device=DEV)
    has_q = q.shape[1] > 0
    kda.kda_latent_append(kv, c["slots"].to(DEV), ints(c["kept"]), ints(c["cu"]), cache, rope=rope,
                          w=None if c["w"] is None else c["w"].to(DEV), normalise=c["normalise"],
                          eps=c["eps"], q=q if has_q else None, q_out=qo if has_q else None,
                          kv_out=out if c["kv_out"] else None, **kw)
    torch.cuda.synchronize()
    return cache.cpu(), out.cpu(), qo.cpu()


def verdict(c, cache, out, qo, in_place=False, sentinel=7.0):
    T, W = c["kv"].shape
    dt, dc = c["kv"].dtype, c["dc"]
    pos = R.positions(c["cu"], c["kept"], T)
    x = c["kv"][:, :dc].double()
    if c["normalise"]:
        inv = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + c["eps"])
        y = x * inv * (1 if c["w"] is None else c["w"].double())
        # the sum of squares: 8 or fewer in a lane one after the other, 2 vectors, six
        # steps over the lanes, one rounding of each square: 18 * 2^-24; half of that
        # through the root, whose own rounding, the division's, the mean's and eps's
        # and the two products': 7 more
        yb = 16 * 2.0 ** -24 * y.abs() + HALF[dt] * (1 + 2.0 ** -18) * y.abs() + 2.0 ** -140
    else:
        y, yb = x, torch.zeros_like(x)
    pe, qpe = c["kv"][:, None, dc:], c["q"][..., -DR:]
    if c["f"] is not None:
        pe, pmag = R.rotate(pe, pos, c["f"], c["interleaved"], c["factor"])
        qpe, qmag = R.rotate(qpe, pos, c["f"], c["interleaved"], c["factor"])
        pb, qb = R.rotation_bound(pe, pmag, dt), R.rotation_bound(qpe, qmag, dt)
    else:
        pe, qpe = pe.double(), qpe.double()
        pb, qb = torch.zeros_like(pe), torch.zeros_like(qpe)
    row, rb = torch.cat([y, pe[:, 0]], 1), torch.cat([yb, pb[:, 0]], 1)
    flat = cache.view(-1, W)
    written = torch.zeros(flat.shape[0], dtype=torch.bool)
    untouched = c["kv"] if in_place else torch.full_like(c["kv"], sentinel)
    base_q = c["q"] if in_place else torch.full_like(qo, sentinel)
    for t in range(T):
        slot = int(c["slots"][t])
        if pos[t] is None:
            assert torch.equal(out[t], untouched[t]) and torch.equal(qo[t], base_q[t])
            continue
        if 0 <= slot < flat.shape[0]:
            written[slot] = True
            assert bool(((flat[slot].double() - row[t]).abs() <= rb[t]).all()), t
            if c["kv_out"]:
                assert torch.equal(flat[slot], out[t])
        if c["kv_out"]:
            assert bool(((out[t].double() - row[t]).abs() <= rb[t]).all()), t
        else:
            assert torch.equal(out[t], untouched[t])
        if c["q"].shape[1]:
            assert torch.equal(qo[t, :, :-DR], base_q[t, :, :-DR])
            assert bool(((qo[t, :, -DR:].double() - qpe[t]).abs() <= qb[t]).all()), t
    assert bool((flat[~written] == sentinel).all())


CASES = [
    dict(n=[1], ctx=[0], dc=128), dict(n=[1] * 9, ctx=list(range(9)), dc=512, Hq=16, dq_out=576),
    dict(n=[3, 0, 70], ctx=[100000, 2, 9], dc=256, Hq=5, dq=64, dq_out=320, spare=3),
    dict(n=[5], ctx=[1], dc=512, Hq=0), dict(n=[2, 2], ctx=[7, 8], dc=128, w=False, kv_out=False),
    dict(n=[9], ctx=[2**31 - 20], dc=512, normalise=False, Hq=33, dq=128, page=256),
    dict(n=[4], ctx=[5], dc=256, rope=False, dq_out=72), dict(n=[4], ctx=[5], dc=512, eps=0.0, Hq=1),
    dict(n=[1000, 2], ctx=[0, 50], dc=128, Hq=2, page=64), dict(n=[1], ctx=[3], dc=512, Hq=128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_plain(i, interleaved, dtype):
    kw = dict(CASES[i])
    c = case(kw.pop("n"), kw.pop("ctx"), kw.pop("dc"), dtype, interleaved=interleaved,
             factor=1.0 if i % 2 else 1.2079, seed=i, **kw)
    verdict(c, *call(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(dtype):
    c = case([6, 40], [900, 0], 512, dtype, Hq=3, seed=30, spare=2)
    verdict(c, *call(c, in_place=True), in_place=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tokens_take_the_other_split(dtype):
    c = case([4100, 0, 30], [7, 1, 70000], 128, dtype, Hq=2, page=64, seed=31, spare=3)
    verdict(c, *call(c))


def test_rows_of_zeros_and_extremes():
    # zeros stay zeros (eps > 0) and are NaN without eps; large rows overflow nothing
    # that fits: a sum of squares up to 512 * 1e36
    c = case([3], [5], 512, F32, w=False, seed=32)
    c["kv"][0, :512] = 0
    c["kv"][1, :512] = 1e18
    cache, out, _ = call(c)
    assert not out[0, :512].any()
    assert torch.allclose(out[1, :512], torch.ones(512), rtol=1e-6)
    verdict(c, cache, out, _)
    c["eps"] = 0.0
    _, out, _ = call(c)
    assert bool(torch.isnan(out[0, :512]).all()) and bool(torch.isfinite(out[1:]).all())
    assert bool(torch.isfinite(out[0, 512:]).all())


def test_slots_outside_are_skipped():
    c = case([40], [3], 128, BF, seed=33)
    for t, s in ((3, -1), (7, c["pool"] * 16), (9, 2**31 - 1), (20, -2**31)):
        c["slots"][t] = s
    verdict(c, *call(c))


def test_identical_calls_streams_and_graphs():
    for tokens in (3, 5000):
        c = case([tokens, 1], [50, 2000], 512, BF, Hq=8, dq_out=576, seed=34)
        ref = call(c)
        rope = kda.KDARope(c["f"].to(DEV))
        kv, slots, q, w = (c[k].to(DEV) for k in ("kv", "slots", "q", "w"))
        kept, cu = ints(c["kept"]), ints(c["cu"])
        cache, out, qo = (torch.full(x.shape, 7.0, dtype=BF, device=DEV) for x in ref)

        def step(stream=None):
            kda.kda_latent_append(kv, slots, kept, cu, cache, rope=rope, w=w, q=q, q_out=qo, kv_out=out,
                                  stream=stream)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for x, y in zip((cache, out, qo), ref):
            assert torch.equal(x.cpu(), y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for i in range(3):
            for x in (cache, out, qo):
                x.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip((cache, out, qo), ref):
                assert torch.equal(x.cpu(), y)


def test_refusals():
    c = case([2, 3], [5, 6], 512, BF, seed=35)
    rope = kda.KDARope(c["f"].to(DEV))
    kv, slots, q, w = (c[k].to(DEV) for k in ("kv", "slots", "q", "w"))
    kept, cu = ints(c["kept"]), ints(c["cu"])
    cache = torch.zeros((c["pool"], 16, 576), dtype=BF, device=DEV)
    good = (kv, slots, kept, cu, cache)
    kda.kda_latent_append(*good, rope=rope, w=w, q=q, q_out=q)
    for i, bad in ((0, kv.float()), (0, kv.half()), (0, kv[:, :500]), (1, slots.long()), (1, slots[:3]),
                   (2, kept[:1]), (3, cu[:2]), (4, cache.float()), (4, cache[..., :512].contiguous()),
                   (0, kv.cpu())):
        with pytest.raises(ValueError):
            kda.kda_latent_append(*good[:i], bad, *good[i + 1:], rope=rope, w=w)
    for kw in (dict(q=q), dict(q_out=q), dict(w=w[:100]), dict(w=w.bfloat16()), dict(kv_out=kv[:2]),
               dict(q=q[:3], q_out=q[:3]), dict(q=q, q_out=q[:, :2].contiguous())):
        with pytest.raises(ValueError):
            kda.kda_latent_append(*good, rope=rope, **kw)
    small = kda.KDARope(torch.ones(16, dtype=torch.float64, device=DEV))
    for kw in (dict(rope=small), dict(eps=-1.0), dict(eps=float("nan")), dict(normalise=False, w=w),
               dict(q=q[..., :60].contiguous(), q_out=q), dict(q=q[..., :68].contiguous(), q_out=q),
               dict(dr=128), dict(kv_out=cache.view(-1)[:5 * 576].view(5, 576))):
        with pytest.raises(kda.KDAError):
            kda.kda_latent_append(*good, **kw)
