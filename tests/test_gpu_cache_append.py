"""kda_cache_append: exact copies into the slots, everything else untouched."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from serve_ref import DEV, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,d,page,dtype", [
    (1, 1, 16, 16, torch.bfloat16), (1, 8, 128, 64, torch.bfloat16), (7, 3, 32, 16, torch.float32),
    (256, 8, 128, 64, torch.bfloat16), (333, 5, 64, 128, torch.float32),
    (1000, 2, 16, 1024, torch.bfloat16), (513, 40, 128, 16, torch.float32),
    (5, 300, 128, 32, torch.bfloat16)])
def test_copies_rows(T, H, d, page, dtype):
    g = torch.Generator().manual_seed(T)
    pool = -(-T // page) + 4
    slot = torch.randperm(pool * page, generator=g)[:T].to(torch.int32)
    for i, bad in zip(range(2, T, 5), [-1, pool * page, 2**31 - 1, -2**31, -page] * T):
        slot[i] = bad                                   # skipped
    k, v = (torch.randn((T, H, d), generator=g).to(dtype) for _ in range(2))
    want = [torch.full((pool, H, page, d), -2.0, dtype=dtype) for _ in range(2)]
    for t in range(T):
        s = int(slot[t])
        if 0 <= s < pool * page:
            want[0][s // page, :, s % page] = k[t]
            want[1][s // page, :, s % page] = v[t]
    kc, vc = (torch.full((pool, H, page, d), -2.0, dtype=dtype, device=DEV) for _ in range(2))
    kda.kda_cache_append(k.to(DEV), v.to(DEV), slot.to(DEV), kc, vc)
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_bit_patterns_survive():
    # NaN payloads and signed zeros are copied as they are
    bits = torch.tensor([0x7fc1, 0x8000, 0xff81, 0x0001] * 4, dtype=torch.int32).to(torch.int16)
    k = bits.view(torch.bfloat16).view(1, 1, 16).to(DEV)
    kc = torch.zeros((1, 1, 16, 16), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    kda.kda_cache_append(k, k.clone(), ints([5]), kc, vc)
    assert torch.equal(kc[0, 0, 5].cpu().view(torch.int16), bits)
    assert torch.equal(vc[0, 0, 5].cpu().view(torch.int16), bits)


def test_cache_past_32_bit_offsets():
    # element offsets beyond 2^32 in a cache that is otherwise left alone
    pool, H, page, d = 40000, 8, 128, 128
    assert pool * H * page * d > 1 << 32
    kc = torch.empty((pool, H, page, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    slots = [pool * page - 1, 0, (pool - 1) * page, pool // 2 * page + 3]
    kc[pool - 1, :, 1:page - 1] = 4.0
    k = torch.randn((4, H, d), device=DEV).to(torch.bfloat16)
    kda.kda_cache_append(k, -k, ints(slots), kc, vc)
    for t, s in enumerate(slots):
        assert torch.equal(kc[s // page, :, s % page], k[t])
        assert torch.equal(vc[s // page, :, s % page], -k[t])
    assert bool((kc[pool - 1, :, 1:page - 1] == 4.0).all())


@pytest.mark.parametrize("dtype,H", [(torch.float32, 5), (torch.bfloat16, 9)])
def test_large_calls(dtype, H):
    # more than the last-level cache holds: other loads and stores
    T, d, page = 70001, 128, 32
    pool = -(-T // page) + 1
    g = torch.Generator(device=DEV).manual_seed(3)
    k, v = (torch.randn((T, H, d), generator=g, device=DEV).to(dtype) for _ in range(2))
    slot = torch.randperm(pool * page, generator=g, device=DEV)[:T].to(torch.int32)
    slot[::1000] = -1
    kc, vc = (torch.full((pool, H, page, d), -2.0, dtype=dtype, device=DEV) for _ in range(2))
    kda.kda_cache_append(k, v, slot, kc, vc)
    keep = slot >= 0
    s = slot[keep].long()
    for cache, rows in ((kc, k), (vc, v)):
        assert torch.equal(cache[s // page, :, s % page], rows[keep])
        assert int((cache == -2.0).all(-1).sum()) >= (pool * page - int(keep.sum())) * H


def test_empty_and_refusals():
    kc = torch.zeros((2, 2, 16, 64), device=DEV)
    vc = torch.zeros_like(kc)
    k = torch.randn((3, 2, 64), device=DEV)
    s = ints([0, 1, 2])
    kda.kda_cache_append(k[:0], k[:0], s[:0], kc, vc)
    assert not kc.any()
    for bad in ((k.bfloat16(), k, s, kc, vc), (k, k[:2], s, kc, vc), (k, k, s[:2], kc, vc),
                (k, k, s.long(), kc, vc), (k, k, s, kc[:, :1], vc), (k, k, s, kc, vc[:1]),
                (k.half(), k.half(), s, kc.half(), vc.half()),
                (k.transpose(0, 1), k, s, kc, vc), (k, k, s, kc.cpu(), vc)):
        with pytest.raises(ValueError):
            kda.kda_cache_append(*bad)
    with pytest.raises(kda.KDAError):
        kda.kda_cache_append(k, k.clone(), s, kc, kc)
    flat = torch.zeros(3 * 2 * 64 + 1, device=DEV)[1:].view(3, 2, 64)      # 4-byte aligned only
    with pytest.raises(kda.KDAError):
        kda.kda_cache_append(flat, k, s, kc, vc)
