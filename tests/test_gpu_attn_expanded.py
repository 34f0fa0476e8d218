"""kda_attn_expanded against the dense fp64 form. Rows and keys outside all
requests, and what lies beside the shared part of the keys, hold NaN."""
import random

import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, ints

pytestmark = pytest.mark.gpu


def tensors(c):
    pe = c["pe_all"].to(DEV)
    return [c["q"].to(DEV), c["kv"].to(DEV), pe[:, -c["dr"]:], ints(c["cu"]), ints(c["ck"])]


def call(c, *, want_lse=True, sentinel=7.0, **kw):
    T, H, _ = c["q"].shape
    o = torch.full((T, H, c["dn"]), sentinel, dtype=c["q"].dtype, device=DEV)
    lse = torch.full((T, H), sentinel, device=DEV) if want_lse else None
    kda.kda_attn_expanded(*tensors(c), dv=c["dn"], o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    return o.cpu(), None if lse is None else lse.cpu()


def verdict(c, o, lse, ref, sentinel=7.0):
    keys = max([b - a for a, b in zip(c["ck"], c["ck"][1:])] + [1])
    return R.check_attention(o, lse, ref, c["cu"][-1], c["q"].shape[2], keys, sentinel, "expanded")


def check(c, **kw):
    ref = R.expanded(c)
    o, lse = call(c, **kw)
    verdict(c, o, lse, ref)
    return o, lse


CASES = [
    # queries, keys, heads, dn
    ([1], [1], 1, 128), ([1], [40], 3, 64), ([7], [7], 2, 128), ([64], [64], 2, 64), ([65], [65], 1, 128),
    ([31, 32, 33], [31, 40, 33], 2, 128), ([255], [255], 2, 128), ([257], [300], 1, 64),
    ([300, 1, 0, 40], [300, 900, 5, 41], 3, 128), ([1] * 30, list(range(1, 31)), 4, 64),
    ([5, 9], [3, 9], 2, 128), ([20, 3], [0, 3], 2, 64), ([600], [600], 2, 128), ([100, 513], [1200, 700], 1, 128),
    ([0, 0], [4, 0], 2, 64), ([129, 5], [2000, 5], 2, 64), ([300], [100], 1, 128)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_plain(i, dtype):
    n, keys, H, dn = CASES[i]
    c = R.expanded_case(n, keys, H, dn, dtype, seed=i, spare_rows=i % 4, spare_keys=i % 3,
                        pe_stride=[None, 576, 72][i % 3])
    check(c, max_q=max(n) if i % 2 else 0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_hint_does_not_matter_for_the_result(dtype):
    c = R.expanded_case([90, 1, 9, 300], [90, 700, 64, 500], 2, 64, dtype, seed=40)
    ref = R.expanded(c)
    for hint in (0, 1, 9, 90, 300, 10**6):
        o, lse = call(c, max_q=hint)
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-4, 0.5, 2.0])
def test_scale(scale, dtype):
    c = R.expanded_case([40, 1], [140, 300], 2, 128, dtype, seed=41)
    c["scale"] = scale
    check(c, scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rising_and_falling_scores(dtype):
    for sign in (1.0, -1.0):
        c = R.expanded_case([100, 5], [400, 70], 2, 64, dtype, seed=42)
        c["q"][:105] = 1.0
        for k0, k1 in ((0, 400), (400, 470)):
            ramp = sign * 0.03125 * torch.arange(k1 - k0, dtype=torch.float32)
            c["kv"][k0:k1, :, :64] = ramp[:, None, None].to(dtype)
            c["pe_all"][k0:k1] = ramp[:, None].to(dtype)
        check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,keys", [(8, 11), (40, 110), (300, 300), (130, 500)])
@pytest.mark.parametrize("what", [float("inf"), float("nan")])
def test_masked_values_stay_out(n, keys, what, dtype):
    # the last key and value are not finite: the queries before the last do not see them
    c = R.expanded_case([n, 2], [keys, 22], 2, 128, dtype, seed=43)
    ref = R.expanded(c)
    c["kv"][keys - 1, :, 128::3] = what
    for keys_too in (False, True):
        if keys_too:
            c["kv"][keys - 1, :, 1:128:2] = what
            c["pe_all"][keys - 1, ::2] = what
        o, lse = call(c)
        seen = n - 1
        if not keys_too:
            hit = o[seen].double()
            assert not torch.isfinite(hit[:, ::3]).any()
            assert torch.isfinite(hit[:, 1::3]).all()
        o[seen], lse[seen] = ref[0][seen].to(o.dtype), ref[1][seen].float()
        verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_values_that_are_seen(dtype):
    c = R.expanded_case([70], [300], 2, 64, dtype, seed=44)
    want, _ = call(c)
    inf = float("inf")
    for pos in (3, 64, 200):
        v = c["kv"][pos, :, 64:]
        v[:, 0], v[:, 9] = inf, -inf
        v[:, 33] = inf if pos == 3 else -inf
    o, _ = call(c)
    assert bool((o[..., 0] == inf).all()) and bool((o[..., 9] == -inf).all())
    assert bool(torch.isnan(o[..., 33]).all())
    o[..., [0, 9, 33]] = want[..., [0, 9, 33]]
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_seen_nan_keys_give_nan(dtype):
    c = R.expanded_case([70, 2], [160, 22], 2, 128, dtype, seed=45)
    ref = R.expanded(c)
    c["kv"][0:90:3, 0, 5] = float("nan")
    o, lse = call(c)
    assert bool(torch.isnan(o[:70, 0]).all()) and bool(torch.isnan(lse[:70, 0]).all())
    o[:70, 0], lse[:70, 0] = ref[0][:70, 0].to(o.dtype), ref[1][:70, 0].float()
    verdict(c, o, lse, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_outside_and_in_any_order(dtype):
    c = R.expanded_case([3, 40, 2], [13, 60, 30], 2, 64, dtype, seed=46)
    ref = R.expanded(c)
    cu, ck = c["cu"], c["ck"]
    d = dict(c, cu=[-9, cu[1], cu[2], cu[3] + 1000], ck=[-3, ck[1], ck[2], ck[3] + 50])
    o, lse = call(d)
    verdict(c, o, lse, ref)
    # the second request's rows and keys first, then (offsets decrease) the first one's
    d = dict(c, cu=[3, 43, 0, 3], ck=[13, 73, 0, 13])
    o, lse = call(d)
    assert bool((o[43:] == 7).all())
    o[43:], lse[43:] = ref[0][43:].to(dtype), ref[1][43:].float()
    verdict(c, o, lse, ref)
    # keys that decrease alone: a request without keys
    o, lse = call(dict(c, ck=[13, 0, 60, 90]))
    assert not o[:3].any() and bool((lse[:3] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pairs", [1, 150])
def test_more_claims_than_rows_write_nothing(pairs, dtype):
    c = R.expanded_case([40], [70], 1, 64, dtype, seed=47)
    cu = [0, 40] * pairs + [0, 1]
    o, lse = call(dict(c, cu=cu, ck=[0, 70] * pairs + [0, 1]))
    assert bool((o == 7).all()) and bool((lse == 7).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B", [256, 257, 1100])
def test_many_requests(B, dtype):
    n = [(i * 7) % 5 for i in range(B)]
    keys = [a + (i * 31) % 40 for i, a in enumerate(n)]
    n[B // 2], keys[B // 2], keys[3], n[B - 1], keys[B - 1] = 70, 90, 3000, 2, 700
    check(R.expanded_case(n, keys, 2, 64, dtype, seed=48), max_q=0 if B % 2 else 70)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,keys,H,dn", [([1], [9000], 2, 128), ([40], [12000], 1, 128), ([300, 7], [5000, 60], 2, 64)])
def test_long_contexts_in_parts(n, keys, H, dn, dtype):
    c = R.expanded_case(n, keys, H, dn, dtype, seed=49)
    ref = R.expanded(c)
    o, lse = call(c)
    verdict(c, o, lse, ref)
    # as in test_gpu_attn_latent.py: 2^-10 (bf16, after rounding), 2^-15 (fp32)
    rounded = ref[0].to(dtype).double() if dtype == BF else ref[0]
    rel = float((o.double() - rounded).norm() / ref[0].norm())
    assert rel <= (2.0 ** -10 if dtype == BF else 2.0 ** -15), rel


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,keys,H,dn", [([1, 40], [900, 300], 5, 64), ([300, 7], [700, 2000], 3, 128)])
def test_maxima_that_jump(n, keys, H, dn, dtype):
    c = R.expanded_case(n, keys, H, dn, dtype, seed=70)
    T = c["cu"][-1]
    rows = torch.arange(T * H).view(T, H) % 5
    c["q"][:T, :, dn + 1] = torch.tensor([0.0, 1.0, 0.5, -1.0, 0.03125])[rows].to(dtype)
    for i, total in enumerate(keys):
        c["pe_all"][c["ck"][i]:c["ck"][i + 1], -63] = (R.jumps(total, 70 + i) / (c["scale"] * 1.4427)).to(dtype)
    check(c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dn", [64, 128])
def test_workspace_of_the_named_size(dn, dtype):
    c = R.expanded_case([300, 1, 40], [1300, 700, 40], 5, dn, dtype, seed=72)
    need = kda.kda_attn_expanded_workspace_size(341, 3, 5, dn, 64, dn, 300, dtype)
    ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
    check(c, max_q=300, workspace=ws)
    assert bool((ws[need:] == 0xAB).all())
    check(c, max_q=300, workspace=ws[:need - 1])          # too small: another one is used


def test_widest_keys():
    # rows of keys and the shared part's stride have a limit
    c = R.expanded_case([2], [3], 1, 64, BF, seed=73)
    q, kv, pe, cu, ck = tensors(c)
    wide = torch.zeros(2 * (1 << 26) + 64 + 128, dtype=BF, device=DEV)
    at = wide.as_strided((3, 64), (1 << 26, 1))
    at.copy_(pe)
    o = kda.kda_attn_expanded(q, kv, at, cu, ck, dv=64, want_lse=True)
    verdict(c, o[0].cpu(), o[1].cpu(), R.expanded(c))
    wide = torch.empty((1 << 33) + 192, dtype=BF, device=DEV)    # 32 bits would cut strides to 0 and 64
    for stride in ((1 << 26) + 8, 1 << 32, (1 << 32) + 64):
        with pytest.raises(ValueError):
            kda.kda_attn_expanded(q, kv, wide.as_strided((3, 64), (stride, 1)), cu, ck, dv=64)


@pytest.mark.parametrize("n", [1, 400])
def test_identical_calls_streams_and_graphs(n):
    c = R.expanded_case([n, 30], [3000, 400], 4, 128, BF, seed=50)
    dev = tensors(c)
    ws = torch.empty(max(1, kda.kda_attn_expanded_workspace_size(n + 30, 2, 4, 128, 64, 128, 0, BF)),
                     dtype=torch.uint8, device=DEV)
    o = torch.zeros((n + 30, 4, 128), dtype=BF, device=DEV)
    lse = torch.zeros((n + 30, 4), device=DEV)

    def step(**kw):
        kda.kda_attn_expanded(*dev, dv=128, o=o, lse=lse, **kw)
    step()
    ro, rl = o.clone(), lse.clone()
    ref = R.expanded(c)
    verdict(c, ro.cpu(), rl.cpu(), ref)
    o.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    torch.empty(64 << 20, dtype=torch.uint8, device=DEV).fill_(0xFF)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(o, ro) and torch.equal(lse, rl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(workspace=ws)
    for i in range(4):
        o.zero_()
        ws.fill_(0xFF)
        if i == 2:
            step(workspace=ws)
            torch.cuda.synchronize()
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ro) and torch.equal(lse, rl), f"replay {i}"


def test_keys_past_32_bit_offsets():
    N, H, dn = 530000, 32, 128
    assert N * H * 2 * dn > 1 << 32
    c = R.expanded_case([70, 3], [400, 90], H, dn, BF, seed=51, pe_stride=576)
    kv = torch.empty((N, H, 2 * dn), dtype=BF, device=DEV)
    pe = torch.empty((N, 576), dtype=BF, device=DEV)
    kv[N - 490:] = c["kv"].to(DEV)
    pe[N - 490:] = c["pe_all"].to(DEV)
    o, lse = kda.kda_attn_expanded(c["q"].to(DEV), kv, pe[:, 512:], ints(c["cu"]),
                                   ints([N - 490, N - 90, N]), dv=dn, want_lse=True)
    verdict(c, o.cpu(), lse.cpu(), R.expanded(c))


def test_refusals():
    c = R.expanded_case([2, 3], [5, 6], 4, 64, BF, seed=52)
    q, kv, pe, cu, ck = good = tensors(c)
    kda.kda_attn_expanded(*good, dv=64)
    for i, bad in ((0, q.float()), (0, q.half()), (0, q.transpose(0, 1)), (0, q[..., :100]), (1, kv.float()),
                   (1, kv[:, :2]), (1, kv.cpu()), (2, pe[:3]), (2, pe.float()), (2, pe[:, ::2]),
                   (3, cu.long()), (3, cu[:2]), (4, ck[:2])):
        with pytest.raises(ValueError):
            kda.kda_attn_expanded(*good[:i], bad, *good[i + 1:], dv=64)
    wide = torch.zeros((11, 68), dtype=BF, device=DEV)       # rows 136 bytes apart
    with pytest.raises(ValueError):
        kda.kda_attn_expanded(q, kv, wide[:, :64], cu, ck, dv=64)
    with pytest.raises(ValueError):
        kda.kda_attn_expanded(q, kv, wide[:1, :64].expand(11, 64), cu, ck, dv=64)
    with pytest.raises(kda.KDAError):                        # 2 bytes off
        kda.kda_attn_expanded(q, kv, torch.zeros((11, 72), dtype=BF, device=DEV)[:, 1:65], cu, ck, dv=64)
    for bad in (dict(scale=-1.0), dict(scale=float("nan")), dict(max_q=-1)):
        with pytest.raises(kda.KDAError):
            kda.kda_attn_expanded(*good, dv=64, **bad)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_expanded(q[..., :96].contiguous(), kv[..., :64].contiguous(), pe, cu, ck, dv=32)
    with pytest.raises(kda.KDAError):
        kda.kda_attn_expanded(*good, dv=64, o=q.view(-1)[:5 * 4 * 64].view(5, 4, 64))


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = random.Random(seed)
    B = rng.choice([1, 2, 3, 7, 20])
    n = [rng.choice([0, 1, 2, 31, rng.randint(1, 400)]) for _ in range(B)]
    keys = [max(0, a + rng.choice([0, 0, -3, rng.randint(0, 900)])) for a in n]
    c = R.expanded_case(n, keys, rng.choice([1, 2, 5]), rng.choice([64, 128]), rng.choice([BF, F32]),
                        seed=seed, spare_rows=2, spare_keys=3, pe_stride=rng.choice([None, 128, 576]))
    check(c, max_q=rng.choice([0, 0, max(n)]))
