"""Plain 64-bit forms of the serving operators, on the host, and their inputs
(no test cases here). They share nothing with the GPU path: Python loops over
requests, dense gathers, fp64."""
import math

import numpy as np
import torch

DEV = torch.device("cuda:0")


def ints(x, dev=DEV):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ page plan

def plan(kept, new, pages, table, ring, ring_state, page, slots):
    """Sequential form. Returns a dict of lists; table and ring are copies."""
    B, width = len(kept), (len(table[0]) if table else 0)
    table, ring = [list(r) for r in table], list(ring)
    pool, (head, count) = len(ring), ring_state
    need = [(a + b + page - 1) // page for a, b in zip(kept, new)]
    take = [max(0, n - h) for n, h in zip(need, pages)]
    give = [max(0, h - n) for n, h in zip(need, pages)]
    status = 0
    if (any(a < 0 or b < 0 for a, b in zip(kept, new)) or any(h < 0 or h > width for h in pages)
            or any(n > width for n in need) or not 0 <= head < max(pool, 1)
            or not 0 <= count <= pool or count + sum(give) > pool):
        status = -1
    elif sum(new) > slots:
        status = -2
    elif sum(take) > count:
        status = sum(take) - count
    if status:
        return dict(table=table, ring=ring, pages=list(pages), ring_state=[head, count],
                    cu=[0] * (B + 1), slot=[-1] * slots, status=status)
    free = [ring[(head + j) % pool] for j in range(sum(take))]
    back = []
    for i in range(B):
        for j in range(take[i]):
            table[i][pages[i] + j] = free.pop(0)
        back += table[i][need[i]:pages[i]] if give[i] else []
    for j, p in enumerate(back):
        ring[(head + count + j) % pool] = p
    cu, slot = [0], []
    for i in range(B):
        for t in range(new[i]):
            pos = kept[i] + t
            slot.append(table[i][pos // page] * page + pos % page)
        cu.append(cu[-1] + new[i])
    slot += [-1] * (slots - len(slot))
    head = (head + sum(take)) % pool if sum(take) else head
    return dict(table=table, ring=ring, pages=need,
                ring_state=[head, count - sum(take) + sum(give)], cu=cu, slot=slot, status=0)


# ------------------------------------------------------------------ attention

def attn_case(n, ctx, Hq, Hkv, d, page, dtype, *, seed=0, spare_rows=0, qscale=1.5, dev=DEV,
              width=None):
    """Random requests in scattered pages. Everything that no position of a
    request uses (cache rows, table entries, query rows behind the last
    request) holds NaN or nonsense."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    B = len(n)
    have = [(a + b + page - 1) // page for a, b in zip(n, ctx)]
    pool = sum(have) + 3
    perm = torch.randperm(pool, generator=g).tolist()
    width = max(have + [1]) + 2 if width is None else width
    table = rng.choice([-1, pool, 2**31 - 1, -2**31], size=(B, width)).astype(np.int64)
    kc, vc = (torch.full((pool, Hkv, page, d), float("nan")) for _ in range(2))
    at = 0
    for i in range(B):
        for j in range(have[i]):
            p = perm[at]
            at += 1
            table[i, j] = p
            rows = min(page, n[i] + ctx[i] - j * page)
            kc[p, :, :rows] = torch.randn((Hkv, rows, d), generator=g)
            vc[p, :, :rows] = torch.randn((Hkv, rows, d), generator=g)
    cu = np.concatenate([[0], np.cumsum(n)]).astype(int).tolist()
    T = cu[-1] + spare_rows
    q = torch.full((T, Hq, d), float("nan"))
    q[:cu[-1]] = qscale * torch.randn((cu[-1], Hq, d), generator=g)
    return dict(q=q.to(dtype), kc=kc.to(dtype), vc=vc.to(dtype),
                table=torch.tensor(table, dtype=torch.int64).to(torch.int32), kept=list(ctx),
                cu=cu, page=page)


def attn(c, scale=None):
    """(o, lse, spread) in fp64: spread = sum_j p_j |v_j|, what the rounding of
    the weights p_j scales with, and the largest |q||k| sum of a row's scores."""
    q, kc, vc = c["q"].double(), c["kc"].double(), c["vc"].double()
    T, Hq, d = q.shape
    pool, Hkv, page, _ = kc.shape
    scale = 1 / math.sqrt(d) if not scale else scale
    o = torch.full((T, Hq, d), float("nan"), dtype=torch.float64)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64)
    spread = torch.zeros_like(o)
    mag = torch.zeros_like(lse)
    table = c["table"].long()
    cap = table.shape[1] * page
    for i in range(len(c["kept"])):
        n = c["cu"][i + 1] - c["cu"][i]
        total = min(max(c["kept"][i], 0) + n, cap)
        pos = torch.arange(total)
        pg = table[i][pos // page] if total else pos
        ok = (pg >= 0) & (pg < pool)
        pos, pg = pos[ok], pg[ok]
        k, v = kc[pg, :, pos % page], vc[pg, :, pos % page]       # [keys, Hkv, d]
        for t in range(n):
            r = c["cu"][i] + t
            vis = int((pos <= max(c["kept"][i], 0) + t).sum())
            if vis == 0:
                o[r], lse[r] = 0, -math.inf
                continue
            kk = k[:vis].repeat_interleave(Hq // Hkv, 1)
            vv = v[:vis].repeat_interleave(Hq // Hkv, 1)
            s = torch.einsum("hd,khd->hk", q[r], kk) * scale
            lse[r] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            o[r] = torch.einsum("hk,khd->hd", p, vv)
            spread[r] = torch.einsum("hk,khd->hd", p, vv.abs())
            mag[r] = (torch.einsum("hd,khd->hk", q[r].abs(), kk.abs()) * scale).amax(1)
    return o, lse, spread, mag


def attn_bound(ref, spread, mag, d, keys, dtype):
    """Largest |o - ref| by the roundings that the operator makes.

    A score is a sum of d products in fp32: off by at most (d + 2) 2^-24 mag;
    it enters the weights through exp (v_exp_f32: 2^-22 relative, and the
    rounding of its argument, of size at most 2 mag log2 e: 2^-23 mag), which
    moves numerator and denominator: factor 2. Sums over the keys run in fp32
    in at most keys / 32 + 64 sequential steps each of 2^-24, twice. bf16:
    each weight is rounded to bf16 (2^-8) before it multiplies the values, and
    so is the result."""
    w = 2 * ((d + 2) * 2.0 ** -24 + 2.0 ** -22) * mag[..., None] + 2.0 ** -21 \
        + 2 * (keys / 32 + 64) * 2.0 ** -24
    if dtype == torch.bfloat16:
        return (w + 2.0 ** -8) * (1 + 2.0 ** -8) * spread + 2.0 ** -8 * ref.abs()
    return w * spread + 2.0 ** -24 * ref.abs()


# ------------------------------------------------------------------ verification

def verify(p, q, x, u, n_draft=None):
    """p [B,T+1,V], q [B,T,V] or None (torch, any dtype), x [B,T], u [B,T+1]."""
    B, T1, V = p.shape
    T = T1 - 1
    p = p.double().numpy()
    q = None if q is None else q.double().numpy()
    x, u = x.numpy(), u.double().numpy()
    commit, tokens = [], []
    for b in range(B):
        n = T if n_draft is None else min(int(n_draft[b]), T)
        if n < 0:
            commit.append(0)
            tokens.append([-1] * (T + 1))
            continue
        a = 0
        while a < n:
            y = int(x[b, a])
            if not 0 <= y < V:
                break
            qt = 1.0 if q is None else q[b, a, y]
            if not u[b, a] * qt < p[b, a, y]:
                break
            a += 1
        r = p[b, a].copy()
        with np.errstate(invalid="ignore"):
            if a < n:
                if q is not None:
                    r = r - q[b, a]
                elif 0 <= int(x[b, a]) < V:
                    r[int(x[b, a])] = 0
                if not (r > 0).any():
                    r = p[b, a].copy()
            r = np.where(r > 0, r, 0.0)
            cdf = np.cumsum(r)
            above = np.nonzero(cdf > u[b, T] * cdf[-1])[0]
        if len(above):
            y = int(above[0])
        else:
            y = int(np.nonzero(r > 0)[0][-1]) if (r > 0).any() else 0
        commit.append(a + 1)
        tokens.append([int(t) for t in x[b, :a]] + [y] + [-1] * (T - a))
    return commit, tokens
