"""Attention over so many positions that their number and its share of a part are not exact
in fp32: every position belongs to a part. The last one decides the result."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, ints

pytestmark = pytest.mark.gpu
PAGE = 1024
SCALE, KEY = 0.5, 96.0                    # the last position's score is 48, all others' 0


def pages(keys):
    """All positions in page 0, the last page's in page 1; the last position's row of it."""
    n = -(-keys // PAGE)
    table = torch.zeros((1, n), dtype=torch.int32, device=DEV)
    table[0, -1] = 1
    return table, (keys - 1) % PAGE


def check(o, lse, value):
    # the last position's weight is 1 - 2^-40 or more: its value, a few roundings of fp32 off
    o = o.double().reshape(-1, value.numel())
    assert bool(((o - value.double()).abs() <= 2.0 ** -21 * value.double().abs()).all())
    assert bool(((lse.double() - SCALE * KEY).abs() <= 2.0 ** -15).all())


def values(n, dtype):
    return (1.0 + torch.rand(n, generator=torch.Generator().manual_seed(1))).to(dtype).to(DEV)


@pytest.mark.parametrize("keys,n,d,dtype", [
    (18354817, 1, 16, BF), (21369857, 1, 128, BF), (25303809, 1, 64, F32), (18445057, 33, 64, BF),
    (20995969, 40, 128, BF), (25378305, 300, 64, BF), (1 << 24, 1, 64, BF), (100000007, 1, 64, BF)])
def test_paged(keys, n, d, dtype):
    table, row = pages(keys)
    q = torch.zeros((n, 1, d), dtype=dtype, device=DEV)
    q[-1, :, 1] = 1.0
    kc, vc = (torch.zeros((2, 1, PAGE, d), dtype=dtype, device=DEV) for _ in range(2))
    kc[1, 0, row, 1] = KEY
    v = values(d, dtype)
    vc[1, 0, row] = v
    o, lse = kda.kda_attn_paged(q, kc, vc, table, ints([keys - n]), ints([0, n]), scale=SCALE, want_lse=True)
    torch.cuda.synchronize()
    check(o[-1], lse[-1], v)


@pytest.mark.parametrize("keys,Hq,dc,dtype", [
    (21104833, 512, 128, BF), (21104833, 256, 128, F32), (167773320, 16, 128, BF), (1 << 24, 16, 512, BF),
    (100000007, 1, 256, BF)])
def test_latent(keys, Hq, dc, dtype):
    table, row = pages(keys)
    q = torch.zeros((1, Hq, dc + 64), dtype=dtype, device=DEV)
    q[..., dc + 1] = 1.0
    cache = torch.zeros((2, PAGE, dc + 64), dtype=dtype, device=DEV)
    cache[1, row, dc + 1] = KEY
    v = values(dc, dtype)
    cache[1, row, :dc] = v
    o, lse = kda.kda_attn_latent(q, cache, table, ints([keys - 1]), ints([0, 1]), dc=dc, scale=SCALE,
                                 want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, v)


@pytest.mark.parametrize("keys", [21243905, 25167233])
def test_expanded(keys):
    q = torch.zeros((1, 1, 128), dtype=BF, device=DEV)
    q[..., 65] = 1.0
    kv = torch.zeros((keys, 1, 128), dtype=BF, device=DEV)
    pe = torch.zeros((keys, 64), dtype=BF, device=DEV)
    pe[-1, 1] = KEY
    v = values(64, BF)
    kv[-1, 0, 64:] = v
    o, lse = kda.kda_attn_expanded(q, kv, pe, ints([0, 1]), ints([0, keys]), dv=64, scale=SCALE, want_lse=True)
    torch.cuda.synchronize()
    check(o, lse, v)
