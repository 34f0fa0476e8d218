"""Plain 64-bit forms of the full-attention layers' operators, on the host, and
their inputs (no test cases here)."""
import math

import numpy as np
import torch

DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")
# half a step of a type, relative to the value
HALF = {BF: torch.finfo(BF).eps / 2, F32: torch.finfo(F32).eps / 2}


def ints(x, dev=DEV):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(int).tolist()


# ------------------------------------------------------------------ rotation

def positions(cu, kept, T):
    """Position of each of T rows, None outside all requests (offsets in order)."""
    p = [None] * T
    for i in range(len(kept)):
        for t in range(max(cu[i], 0), min(cu[i + 1], T)):
            p[t] = max(kept[i], 0) + t - max(cu[i], 0)
    return p


def rotate(x, pos, freqs, interleaved, factor):
    """x [T, H, rot] -> (rotated, magnitude |x cos| + |x' sin|), fp64."""
    half = x.shape[-1] // 2
    x = x.double()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    angle = torch.tensor([float(p or 0) for p in pos], dtype=torch.float64)[:, None] * freqs
    c, s = factor * torch.cos(angle)[:, None], factor * torch.sin(angle)[:, None]
    pairs = [a * c - b * s, b * c + a * s]
    mags = [(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()]
    if interleaved:
        return tuple(torch.stack(v, -1).flatten(-2) for v in (pairs, mags))
    return tuple(torch.cat(v, -1) for v in (pairs, mags))


def rotation_bound(y, mag, dtype):
    # cos and sin are rounded to fp32 once (from fp64), each product once, their sum
    # once: 3 * 2^-24 of the magnitudes; then the result's own rounding
    return 3.01 * 2.0 ** -24 * mag + HALF[dtype] * (1 + 2.0 ** -20) * y.abs() + 2.0 ** -140


# ------------------------------------------------------------------ attention over latents

def latent_case(n, ctx, Hq, dc, page, dtype, *, dr=64, seed=0, spare_rows=0, qscale=1.0, width=None):
    """Random requests in scattered pages. What no position of a request uses (cache
    rows, table entries, query rows behind the last request) holds NaN or nonsense."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B, W = len(n), dc + dr
    have = [(a + b + page - 1) // page for a, b in zip(n, ctx)]
    pool = sum(have) + 3
    perm = torch.randperm(pool, generator=g).tolist()
    width = max(have + [1]) + 2 if width is None else width
    table = rng.choice([-1, pool, 2**31 - 1, -2**31], size=(B, width)).astype(np.int64)
    cache = torch.full((pool, page, W), NAN)
    at = 0
    for i in range(B):
        for j in range(have[i]):
            p = perm[at]
            at += 1
            table[i, j] = p
            rows = min(page, n[i] + ctx[i] - j * page)
            cache[p, :rows] = torch.randn((rows, W), generator=g)
    cu = offsets(n)
    q = torch.full((cu[-1] + spare_rows, Hq, W), NAN)
    q[:cu[-1]] = qscale * torch.randn((cu[-1], Hq, W), generator=g)
    return dict(q=q.to(dtype), cache=cache.to(dtype),
                table=torch.tensor(table, dtype=torch.int64).to(torch.int32), kept=list(ctx), cu=cu,
                page=page, dc=dc, scale=1 / math.sqrt(128 + dr))


def _attend(q, k, v, visible, scale):
    """q [n,H,W], k [m,H|1,W], v [m,H|1,D], visible [n,m] -> o, lse, spread, mag."""
    n, H, W = q.shape
    m = k.shape[0]
    k, v = k.expand(m, H, W).permute(1, 2, 0), v.expand(m, H, v.shape[2]).permute(1, 0, 2)
    q = q.permute(1, 0, 2)
    s = (q @ k) * scale
    s.masked_fill_(~visible[None], -math.inf)
    none = ~visible.any(1)
    top = s.amax(2, keepdim=True) if m else s.new_full((H, n, 1), -math.inf)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(2, keepdim=True)
    lse = (top + total.log())[..., 0]
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    mag = (q.abs() @ k.abs()) * scale
    mag = mag.masked_fill(~visible[None], 0.0)
    mag = mag.amax(2) if m else s.new_zeros((H, n))
    o, spread = p @ v, p @ v.abs()
    o[:, none] = 0.0
    return [x.transpose(0, 1) for x in (o, lse, spread, mag)]


def latent(c):
    """(o, lse, spread, mag) in fp64; spread = sum_j p_j |c_j|, mag the largest
    scale * sum |q||x| of a row's scores."""
    q, cache, dc, page = c["q"].double(), c["cache"].double(), c["dc"], c["page"]
    T, Hq, W = q.shape
    pool = cache.shape[0]
    o = torch.full((T, Hq, dc), NAN, dtype=torch.float64)
    lse, mag = (torch.full((T, Hq), NAN, dtype=torch.float64) for _ in range(2))
    spread = torch.zeros_like(o)
    table = c["table"].long()
    cap = table.shape[1] * page
    for i in range(len(c["kept"])):
        r0, r1 = c["cu"][i], c["cu"][i + 1]
        kept = max(c["kept"][i], 0)
        pos = torch.arange(min(kept + r1 - r0, cap))
        pg = table[i][pos // page] if len(pos) else pos
        ok = (pg >= 0) & (pg < pool)
        pos, pg = pos[ok], pg[ok]
        x = cache[pg, pos % page][:, None]
        seen = pos[None] <= kept + torch.arange(r1 - r0)[:, None]
        o[r0:r1], lse[r0:r1], spread[r0:r1], mag[r0:r1] = _attend(q[r0:r1], x, x[..., :dc], seen,
                                                                  c["scale"])
    return o, lse, spread, mag


def expanded_case(n, keys, H, dn, dtype, *, dr=64, seed=0, spare_rows=0, spare_keys=0, pe_stride=None):
    g = torch.Generator().manual_seed(seed)
    cu, ck = offsets(n), offsets(keys)
    q = torch.full((cu[-1] + spare_rows, H, dn + dr), NAN)
    q[:cu[-1]] = 1.5 * torch.randn((cu[-1], H, dn + dr), generator=g)
    kv = torch.full((ck[-1] + spare_keys, H, 2 * dn), NAN)
    kv[:ck[-1]] = torch.randn((ck[-1], H, 2 * dn), generator=g)
    pe = torch.full((ck[-1] + spare_keys, pe_stride or dr), NAN)
    pe[:ck[-1], -dr:] = torch.randn((ck[-1], dr), generator=g)
    return dict(q=q.to(dtype), kv=kv.to(dtype), pe_all=pe.to(dtype), dr=dr, cu=cu, ck=ck, dn=dn,
                scale=1 / math.sqrt(dn + dr))


def expanded(c):
    q, kv, pe, dn = c["q"].double(), c["kv"].double(), c["pe_all"].double()[:, -c["dr"]:], c["dn"]
    T, H, _ = q.shape
    o = torch.full((T, H, dn), NAN, dtype=torch.float64)
    lse, mag = (torch.full((T, H), NAN, dtype=torch.float64) for _ in range(2))
    spread = torch.zeros_like(o)
    for i in range(len(c["cu"]) - 1):
        r0, r1, k0, k1 = c["cu"][i], c["cu"][i + 1], c["ck"][i], c["ck"][i + 1]
        k = torch.cat([kv[k0:k1, :, :dn], pe[k0:k1, None].expand(k1 - k0, H, c["dr"])], 2)
        seen = torch.arange(k1 - k0)[None] <= k1 - k0 - (r1 - r0) + torch.arange(r1 - r0)[:, None]
        o[r0:r1], lse[r0:r1], spread[r0:r1], mag[r0:r1] = _attend(q[r0:r1], k, kv[k0:k1, :, dn:],
                                                                  seen, c["scale"])
    return o, lse, spread, mag


def jumps(total, seed):
    """What a position adds to its scores, in the log2 domain: nothing at most of them,
    and peaks of all sizes at some, so that a running maximum jumps by little and much."""
    g = torch.Generator().manual_seed(seed)
    kind = torch.randint(0, 40, (total,), generator=g)
    size = torch.tensor([5.0, 9.0, 20.0, 23.0, 26.0, 40.0, 70.0, 130.0, -30.0, -200.0])
    x = torch.where(kind < 10, size[kind.clamp(max=9)], torch.zeros(total))
    return x * torch.linspace(0.1, 1.0, total)


def before_rounding(spread, mag, width, keys, dtype):
    """Largest error of a result before it is rounded to its type.

    A score is a sum of `width` products in fp32: off by at most (width + 2) 2^-24
    mag; it enters the weights through exp (v_exp_f32: 2^-22 relative, and the
    rounding of its argument, of size at most 2 mag log2 e: 2^-23 mag), which moves
    numerator and denominator: factor 2. A row's weights are relative to a reference
    that may be off its maximum by 2^24, which costs nothing in fp32. Sums over the
    keys: one step a key in the weights' sum and one (bf16: two) in the values', each
    of which may lose 2^-23 where a product is cut off instead of rounded; the joins
    add fewer than 128. bf16: a weight in two bf16 terms lacks 2^-15 of itself (the
    first leaves less than 2^-7, of which the second's rounding loses 2^-8) and has
    2^-20 too much."""
    w = 2 * ((width + 2) * 2.0 ** -24 + 2.0 ** -22) * mag[..., None] + 2.0 ** -21 \
        + (3 * keys + 128) * 2.0 ** -23
    if dtype == BF:
        w = w + 2.0 ** -15 + 2.0 ** -20
    return w * spread


def check_attention(o, lse, ref, T, width, keys, sentinel=7.0, what="attn"):
    """o, lse of a call against (o, lse, spread, mag) over the first T rows; rows
    behind them keep the sentinel. The result lies between the roundings of ref -+ E
    (rounding is monotone)."""
    ro, rl, spread, mag = (x[:T] for x in ref)
    dtype = o.dtype
    assert bool((o[T:] == sentinel).all()), "rows behind the last request were written"
    got = o[:T].double()
    assert not torch.isnan(got).any()
    E = before_rounding(spread, mag, width, keys, dtype) + 1e-30
    lo, hi = (ro - E).to(dtype).double(), (ro + E).to(dtype).double()
    out = (got < lo) | (got > hi)
    rel = float((got - ro).norm() / ro.norm()) if T and float(ro.norm()) else 0.0
    print(f"[{what}] outside: {int(out.sum())} of {out.numel()}, relative error {rel:.2e}", flush=True)
    assert not out.any()
    if lse is not None:
        assert bool((lse[T:] == sentinel).all())
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse[:T]), empty) and bool((lse[:T][empty] < 0).all())
        lb = (width + 4) * 2.0 ** -24 * mag + (3 * keys + 136) * 2.0 ** -23 + 2.0 ** -21 \
            + 2.0 ** -23 * rl.abs()
        assert bool(((lse[:T].double() - rl).abs() <= lb)[~empty].all())
    return rel
