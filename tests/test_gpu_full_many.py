"""The full-attention layers' operators with more workgroups than a grid of 2^32 threads
has, and keys as far apart as they may be."""
import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, F32, ints

pytestmark = pytest.mark.gpu
GRID = 1 << 23                # workgroups of a launch, of 256 threads


def room(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"needs {gigabytes} GB of device memory")


def two_requests(T, cut):
    """The first `cut` rows from position 7 on, the others from position 1000."""
    def position(t):
        return 7 + t if t < cut else 1000 + t - cut
    return ints([7, 1000]), ints([0, cut, T]), position


def test_rope_append():
    # a token a workgroup: rows on both sides of a launch's end are checked, all others by
    # their norm, and rows of a request that begins in the second launch
    T, d, page, pool = GRID + 1000, 16, 16, 4
    room(8)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((T, 1, d), generator=g, device=DEV, dtype=BF)
    k, v = (torch.randn((T, 1, d), generator=g, device=DEV, dtype=BF) for _ in range(2))
    kept, cu, position = two_requests(T, GRID + 300)
    at = [0, 1, GRID - 2, GRID - 1, GRID, GRID + 1, GRID + 299, GRID + 300, T - 1]
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    for i, t in enumerate(at):
        slots[t] = 5 * i + 2
    kc, vc = (torch.full((pool, 1, page, d), 7.0, dtype=BF, device=DEV) for _ in range(2))
    f, _ = kda.kda_rope_freqs(d)
    out = kda.kda_rope_append(q, k, v, slots, kept, cu, kc, vc, kda.KDARope(f.to(DEV)))
    torch.cuda.synchronize()
    pos = [position(t) for t in at]
    for src, got in ((q, out[at, 0].cpu()), (k, kc.view(-1, d)[[5 * i + 2 for i in range(len(at))]].cpu())):
        y, mag = R.rotate(src[at].cpu(), pos, f, False, 1.0)
        assert bool(((got.double() - y[:, 0]).abs() <= R.rotation_bound(y, mag, BF)[:, 0]).all())
    assert torch.equal(vc.view(-1, d)[[5 * i + 2 for i in range(len(at))]], v[at, 0])
    assert int((vc.view(-1, d) != 7.0).any(1).sum()) == len(at)
    # a rotation keeps lengths: every component is off by at most 2^-8 of the pair's length
    a, b = out.float().norm(dim=-1), q.float().norm(dim=-1)
    assert bool(((a - b).abs() <= 2.0 ** -7 * b).all())


@pytest.mark.parametrize("dtype", [BF])
def test_latent_append(dtype):
    # four tokens a workgroup
    T, dc, page, pool = 4 * GRID + 1000, 128, 16, 4
    room(32)
    kv = torch.empty((T, dc + 64), dtype=dtype, device=DEV)
    kv.view(torch.int16).random_(0x3f00, 0x4000)          # 0.5 to 2
    kept, cu, position = two_requests(T, 4 * GRID + 300)
    at = [0, 3, 4 * GRID - 1, 4 * GRID, 4 * GRID + 1, 4 * GRID + 299, 4 * GRID + 300, T - 1]
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    for i, t in enumerate(at):
        slots[t] = 7 * i + 1
    cache = torch.full((pool, page, dc + 64), 7.0, dtype=dtype, device=DEV)
    f, _ = kda.kda_rope_freqs(64)
    rows = kv[at].cpu()
    kda.kda_latent_append(kv, slots, kept, cu, cache, rope=kda.KDARope(f.to(DEV)), kv_out=kv)
    torch.cuda.synchronize()
    got = kv[at].cpu()
    assert torch.equal(got, cache.view(-1, dc + 64)[[7 * i + 1 for i in range(len(at))]].cpu())
    assert int((cache.view(-1, dc + 64) != 7.0).any(1).sum()) == len(at)
    x = rows[:, :dc].double()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-6)
    # the factor and its product in fp32, the result in bf16
    assert bool(((got[:, :dc].double() - y).abs() <= (R.HALF[dtype] + 2.0 ** -22) * y.abs()).all())
    y, mag = R.rotate(rows[:, None, dc:], [position(t) for t in at], f, False, 1.0)
    assert bool(((got[:, None, dc:].double() - y).abs() <= R.rotation_bound(y, mag, dtype)).all())
    # every row was normalised
    for i in range(0, T, 1 << 22):
        norm = kv[i:i + (1 << 22), :dc].float().square().mean(1)
        assert bool(((norm - 1).abs() <= 2.0 ** -6).all())


@pytest.mark.parametrize("dtype,dn", [(BF, 64), (BF, 128), (F32, 64)])
def test_expanded(dtype, dn):
    # single tokens that see themselves alone: the result is their value
    B, H = (1 << 18) + 3, 33
    assert B * H > GRID
    room(16)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn((B, H, dn + 64), generator=g, device=DEV, dtype=BF).to(dtype)
    kv = torch.randn((B, H, 2 * dn), generator=g, device=DEV, dtype=BF).to(dtype)
    pe = torch.randn((B, 64), generator=g, device=DEV, dtype=BF).to(dtype)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    o, lse = kda.kda_attn_expanded(q, kv, pe, cu, cu, dv=dn, max_q=1, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o, kv[..., dn:])
    for rows in (slice(0, 500), slice(B - 500, B)):
        k = torch.cat([kv[rows, :, :dn], pe[rows, None].expand(-1, H, -1)], 2).double()
        s, size = ((x * y).sum(-1) / (dn + 64) ** 0.5 for x, y in
                   ((q[rows].double(), k), (q[rows].double().abs(), k.abs())))
        # a sum of products cut off or rounded to fp32, the scale, the factor log2 e and back
        assert bool(((lse[rows].double() - s).abs() <= (dn + 70) * 2.0 ** -23 * size + 2.0 ** -22).all())


@pytest.mark.parametrize("dtype,dn,n", [(BF, 64, 3), (BF, 128, 40), (F32, 64, 3)])
def test_widest_keys_of_a_whole_step(dtype, dn, n):
    # the largest stride, with as many keys as a wave fetches at once and more: every offset
    # over them, up to 15 * 2^27 bytes, is used
    keys = 20
    stride = 1 << 26
    room(12 if dtype == BF else 22)
    c = R.expanded_case([n], [max(keys, n)], 1, dn, dtype, seed=74)
    keys = max(keys, n)
    wide = torch.empty((keys - 1) * stride + 64, dtype=dtype, device=DEV)
    at = wide.as_strided((keys, 64), (stride, 1))
    at.copy_(c["pe_all"].to(DEV))
    o, lse = kda.kda_attn_expanded(c["q"].to(DEV), c["kv"].to(DEV), at, ints(c["cu"]), ints(c["ck"]), dv=dn,
                                   want_lse=True)
    torch.cuda.synchronize()
    R.check_attention(o.cpu(), lse.cpu(), R.expanded(c), n, dn + 64, keys, what="widest")
