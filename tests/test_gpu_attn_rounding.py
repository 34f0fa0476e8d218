"""kda_attn_paged in bf16: the result is rounded, the weights on the way to it are not.

The bounds of test_gpu_attn_paged.py leave room for softmax weights of eight bits; these do not."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def call(c, **kw):
    dev = {k: c[k].to(DEV) for k in ("q", "kc", "vc", "table")}
    o, _ = kda.kda_attn_paged(dev["q"], dev["kc"], dev["vc"], dev["table"], ints(c["kept"]),
                              ints(c["cu"]), **kw)
    torch.cuda.synchronize()
    return o.cpu()


@pytest.mark.parametrize("n,ctx,Hq,Hkv,d", [
    ([1], [40], 8, 8, 128), ([1] * 7, [20, 31, 60, 64, 90, 120, 7], 16, 2, 64), ([8], [50], 16, 4, 128),
    ([6, 3], [70, 9], 5, 1, 32), ([17], [30], 4, 4, 16), ([130], [0], 4, 2, 64), ([90], [40], 4, 1, 128),
    ([60, 1, 8], [9, 100, 33], 8, 2, 128), ([70, 1], [50, 110], 8, 4, 64)])
def test_result_is_the_rounded_one(n, ctx, Hq, Hkv, d):
    # Before its rounding a result is off by at most E: the scores' part as in
    # serve_ref.attn_bound; a weight in two bf16 terms lacks 2^-15 of itself (the
    # first leaves less than 2^-7, of which the second's rounding loses 2^-8) and
    # has 2^-20 too much; two products a key in the values' sum and one in the
    # weights', each of which may lose 2^-23 where a product is cut off instead of
    # rounded. Rounding is monotone: the result lies between those of ref -+ E.
    c = R.attn_case(n, ctx, Hq, Hkv, d, 16, BF, seed=d + len(n), qscale=0.25)
    ref, _, spread, mag = R.attn(c)
    keys = max(a + b for a, b in zip(n, ctx))
    w = 2 * ((d + 2) * 2.0 ** -24 + 2.0 ** -22) * mag[..., None] + 2.0 ** -21 \
        + 2.0 ** -15 + 2.0 ** -20 + (3 * keys + 128) * 2.0 ** -23
    o = call(c).double()
    lo, hi = (ref - w * spread).to(BF).double(), (ref + w * spread).to(BF).double()
    out = (o < lo) | (o > hi)
    print(f"[attn] bf16 results outside: {int(out.sum())} of {out.numel()}, "
          f"other than the rounded reference: {int((o != ref.to(BF).double()).sum())}", flush=True)
    assert not out.any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx,Hq,Hkv,d", [
    ([1], [1000], 32, 8, 128), ([1, 1], [9000, 20], 8, 2, 64), ([8], [20000], 8, 2, 128),
    ([8, 5], [3000, 700], 8, 2, 64), ([1], [5000], 4, 2, 16), ([9], [2500], 6, 3, 32),
    ([100, 1], [5000, 100], 8, 2, 128), ([100, 1, 4], [2000, 6000, 40], 4, 4, 64),
    ([300], [900], 4, 1, 128), ([130], [4000], 4, 1, 64)])
def test_relative_error(n, ctx, Hq, Hkv, d, dtype):
    # Over a whole case the roundings average out. Let e be the result's relative
    # error in norm before its rounding: of a score's d steps, independent, 2^-24
    # sqrt(d / 3) of a magnitude of 16, below 2^-17; of a bf16 weight's two
    # terms below 2^-15. fp32: 2^-17. bf16: an error of size x moves the rounded
    # value by a unit u with probability x / u, so the norm of what moved is
    # sqrt(2^-7 e) <= 2^-10 for e up to 2^-13. (A weight of eight bits has e of
    # 2^-9.3 and moves the result by 2^-9.3; one missing value in 20000 by 2^-6.8.)
    c = R.attn_case(n, ctx, Hq, Hkv, d, 64, dtype, seed=d + len(n))
    ref, _, _, mag = R.attn(c)
    assert float(mag.max()) < 40 and float(mag.mean()) < 16
    rounded = ref.to(dtype).double() if dtype == BF else ref
    e = float((call(c).double() - rounded).norm() / ref.norm())
    print(f"[attn] relative to the rounded reference: {e:.2e}", flush=True)
    assert e <= (2.0 ** -10 if dtype == BF else 2.0 ** -17)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,ctx", [(1, 600), (8, 300), (70, 200)])
def test_infinite_values_that_are_seen(n, ctx, dtype):
    # every row sees them: their columns are infinite with their sign, NaN where
    # both signs meet; all others are as without
    c = R.attn_case([n, 1], [ctx, 30], 8, 2, 64, 16, dtype, seed=71)
    want = call(c)
    inf = float("inf")
    for pos in (3, 64, 97):
        v = c["vc"][c["table"][0, pos // 16], :, pos % 16]
        v[:, 0], v[:, 9] = inf, -inf
        v[:, 33] = inf if pos == 3 else -inf
    o = call(c)
    assert bool((o[:n, :, 0] == inf).all()) and bool((o[:n, :, 9] == -inf).all())
    assert bool(torch.isnan(o[:n, :, 33]).all())
    o[:n, :, [0, 9, 33]] = want[:n, :, [0, 9, 33]]
    assert torch.equal(o, want)
