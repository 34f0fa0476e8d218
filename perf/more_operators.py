"""The full-attention layers' operators around the recurrent layer: cases, inputs, plain forms and
64-bit values.

A stack that mixes recurrent with full-attention layers has layers of grouped heads, whose queries and
keys are rotated by their positions (``rope``: rotation, and the keys and values into their cache
pages), and layers whose keys and values are one shared latent vector a token: its normalisation and
rotation on the way into the cache (``latent``), attention over that cache with the up-projections
absorbed into queries and outputs (``absorbed``), and attention of prompts over the keys and values
that were expanded from the latents (``expanded``).

With ``own`` false, ``run`` computes them from elementary torch operations; with ``own`` true it
makes the calls of this package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
GOLDEN = 0.6180339887498949
EPS = 1e-6
SCORE_BYTES = 4 << 30         # the plain attention's scores at one time


# ---------------------------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one token of every request of a decode batch: rotation of whole heads, into the pages
        dict(name="rope_step_t256", op="rope", B=256, n_lo=1, n_hi=1, ctx_lo=1, ctx_hi=16384, Hq=32,
             Hkv=8, d=128, rot=128, pairs="half", scaling="none", page=64, dtype="bf16"),
        # prompts packed into one call, resumed far into a context of 1M positions with scaled
        # frequencies; half of each head is rotated
        dict(name="rope_prompts_far", op="rope", B=24, n_lo=64, n_hi=8191, ctx_lo=4096,
             ctx_hi=1040384, Hq=32, Hkv=8, d=128, rot=64, pairs="interleaved", scaling="parts",
             page=64, dtype="bf16"),
        # one token of every request: latents normalised and rotated into the pages, with the
        # rotated part of the queries
        dict(name="latent_step_t128", op="latent", B=128, n_lo=1, n_hi=1, ctx_lo=1, ctx_hi=32768,
             Hq=32, dq=192, dq_out=576, dc=512, dr=64, norm=True, pairs="interleaved",
             scaling="none", page=64, dtype="bf16"),
        # packed prompts, fp32
        dict(name="latent_prompts_fp32", op="latent", B=9, n_lo=500, n_hi=8191, ctx_lo=1,
             ctx_hi=65536, Hq=32, dq=192, dq_out=192, dc=512, dr=64, norm=True, pairs="half",
             scaling="linear", page=64, dtype="fp32"),
        # one request, one token, a short context: latency
        dict(name="absorbed_decode_b1", op="absorbed", B=1, n_lo=1, n_hi=1, ctx_lo=1000, ctx_hi=1000,
             Hq=32, dc=512, dr=64, page=64, dtype="bf16"),
        # a full decode batch where a GPU holds 16 heads: reading the cache
        dict(name="absorbed_decode_h16", op="absorbed", B=256, n_lo=1, n_hi=1, ctx_lo=1024,
             ctx_hi=32768, Hq=16, dc=512, dr=64, page=64, dtype="bf16"),
        # a decode batch with 128 heads on one GPU: as much arithmetic as reading
        dict(name="absorbed_decode_h128", op="absorbed", B=128, n_lo=1, n_hi=1, ctx_lo=1024,
             ctx_hi=16384, Hq=128, dc=512, dr=64, page=64, dtype="bf16"),
        # 8-token drafts checked over very long contexts
        dict(name="absorbed_draft_long", op="absorbed", B=4, n_lo=8, n_hi=8, ctx_lo=65536,
             ctx_hi=262144, Hq=32, dc=512, dr=64, page=256, dtype="bf16"),
        # single tokens and chunks of prompts together, small pages, a narrower latent
        dict(name="absorbed_mixed", op="absorbed", B=16, n_lo=1, n_hi=255, ctx_lo=1, ctx_hi=8191,
             Hq=20, dc=256, dr=64, page=16, dtype="bf16"),
        # fp32, ragged
        dict(name="absorbed_fp32", op="absorbed", B=6, n_lo=1, n_hi=33, ctx_lo=1, ctx_hi=2001, Hq=16,
             dc=512, dr=64, page=32, dtype="fp32"),
        # a chunk of a long prompt over its own keys and those before it
        dict(name="expanded_chunk_t8192", op="expanded", B=1, n_lo=8192, n_hi=8192, ctx_lo=16384,
             ctx_hi=16384, H=32, dn=128, dr=64, dv=128, dtype="bf16"),
        # packed prompts of very different lengths, some over a context, narrower heads
        dict(name="expanded_ragged", op="expanded", B=21, n_lo=1, n_hi=2047, ctx_lo=1, ctx_hi=999,
             H=12, dn=64, dr=64, dv=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _fit(case, most_bytes, most_flops, keys):
    """Halves the sizes named in keys, in turn, until the case costs no more than that."""
    j = 0
    while work(case)["bytes"] > most_bytes or work(case)["flops"] > most_flops:
        key = keys[j % len(keys)]
        case[key] = max(1, case[key] // 2)
        for lo, hi in (("n_lo", "n_hi"), ("ctx_lo", "ctx_hi")):
            case[lo] = min(case[lo], case[hi])
        j += 1
    return case


def _draw_append(rng, op):
    ctx = _log_int(rng, 1, 1040384)
    n_hi = rng.choice([1, rng.randint(2, 8), _log_int(rng, 9, 8191)])
    c = dict(op=op, B=_log_int(rng, 1, 256), n_lo=1 if n_hi > 8 else n_hi, n_hi=n_hi,
             ctx_lo=max(1, ctx // rng.randint(1, 50)), ctx_hi=ctx,
             pairs=rng.choice(["half", "interleaved"]),
             scaling=rng.choice(["none", "linear", "parts"]),
             page=rng.choice([16, 32, 64, 128, 256]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "rope":
        c["Hkv"] = rng.choice([1, 2, 3, 4, 8])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
        c["d"] = rng.choice([64, 128])
        c["rot"] = rng.choice([16, 32, 48, 64, c["d"]])
    else:
        c["Hq"] = rng.choice([5, 16, 20, 32, 64, 128])
        c["dc"], c["dr"] = rng.choice([128, 256, 512]), 64
        c["dq"], c["dq_out"] = rng.choice([(192, c["dc"] + 64), (192, 192), (128, 128)])
        c["norm"] = rng.choice([True, True, False])
    return _fit(c, 2e9, math.inf, ["B", "n_hi"])


def _draw_absorbed(rng):
    kind = rng.choice(["decode", "decode", "draft", "mixed"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if kind == "decode":
        B, n_lo, n_hi, ctx = _log_int(rng, 1, 256), 1, 1, _log_int(rng, 1, 65536)
    elif kind == "draft":
        n_hi = rng.randint(2, 8)
        B, n_lo, ctx = _log_int(rng, 1, 64), n_hi, _log_int(rng, 8, 131072)
    else:
        B, n_lo, n_hi, ctx = rng.randint(2, 24), 1, _log_int(rng, 9, 511), _log_int(rng, 1, 8191)
    c = dict(op="absorbed", B=B, n_lo=n_lo, n_hi=n_hi, ctx_lo=max(1, ctx // rng.randint(1, 20)),
             ctx_hi=ctx, Hq=rng.choice([1, 5, 8, 16, 20, 32, 64, 128]),
             dc=rng.choice([128, 256, 512, 512]), dr=64, page=rng.choice([16, 32, 64, 128, 256]),
             dtype=dtype)
    return _fit(c, 2e9, 1.5e12 if dtype == "bf16" else 1.5e11, ["B", "ctx_hi", "n_hi"])


def _draw_expanded(rng):
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    n_hi, ctx = _log_int(rng, 1, 8192), _log_int(rng, 1, 16384)
    w = rng.choice([64, 128])
    c = dict(op="expanded", B=_log_int(rng, 1, 32), n_lo=max(1, n_hi // rng.choice([1, 4, 50])),
             n_hi=n_hi, ctx_lo=max(1, ctx // rng.choice([1, 4, 50])), ctx_hi=ctx,
             H=rng.choice([1, 5, 12, 16, 32]), dn=w, dr=64, dv=w, dtype=dtype)
    return _fit(c, 2e9, 2.5e12 if dtype == "bf16" else 2.5e11, ["B", "ctx_hi", "n_hi"])


def draw(rng):
    op = rng.choice(["rope", "latent", "absorbed", "absorbed", "expanded"])
    if op in ("rope", "latent"):
        return _draw_append(rng, op)
    return _draw_absorbed(rng) if op == "absorbed" else _draw_expanded(rng)


# ---------------------------------------------------------------------------------------------
# Lengths: a fixed spread over the case's range (over the logarithm), the same multiset for every
# seed, so that the work of a case does not depend on the seed; the seed permutes the requests.

def _spread(lo, hi, n, step, shift):
    return [min(hi, max(lo, int(round(math.exp(
        math.log(lo) + ((i + shift) * step % 1.0) * (math.log(hi) - math.log(lo)))))))
        for i in range(n)]


def _lengths(case):
    """(new tokens, tokens before them) of the requests."""
    return (_spread(case["n_lo"], case["n_hi"], case["B"], GOLDEN, 0.5),
            _spread(case["ctx_lo"], case["ctx_hi"], case["B"], math.sqrt(2), 0.5))


def _pages(n, page):
    return -(-n // page)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n, ctx = _lengths(case)
    T, kv = sum(n), sum(n) + sum(ctx)
    if case["op"] == "rope":
        rows = case["Hq"] + case["Hkv"]
        return {"bytes": 2 * T * (rows + case["Hkv"]) * case["d"] * e + 4 * T,
                "flops": 3 * T * rows * case["rot"]}
    if case["op"] == "latent":
        dc, dr = case["dc"], case["dr"]
        return {"bytes": e * T * (3 * (dc + dr) + 2 * case["Hq"] * dr) + 4 * T,
                "flops": T * (4 * dc * case["norm"] + 3 * (case["Hq"] + 1) * dr)}
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, ctx))
    if case["op"] == "absorbed":
        dk, dv, H = case["dc"] + case["dr"], case["dc"], case["Hq"]
        return {"bytes": e * (kv * dk + T * H * (dk + dv)), "flops": 2 * H * (dk + dv) * pairs}
    H, dk, dv = case["H"], case["dn"] + case["dr"], case["dv"]
    return {"bytes": e * (T * H * (dk + dv) + kv * (H * (case["dn"] + dv) + case["dr"])) + 4 * T * H,
            "flops": 2 * H * (dk + dv) * pairs}


# ---------------------------------------------------------------------------------------------
# Inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _requests(case, seed):
    rng = random.Random(seed)
    rows = list(zip(*_lengths(case)))
    rng.shuffle(rows)
    n, ctx = (list(c) for c in zip(*rows))
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    return n, ctx, cu


def _freqs(rot, scaling):
    """Radians a position of each pair, in 64 bits, and the factor on what is rotated."""
    base = 10000.0 if scaling == "none" else 500000.0
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if scaling == "linear":
        return f / 8.0, 1.0
    if scaling == "none":
        return f, 1.0
    # by parts: slow pairs are slowed by the factor, fast ones stay, a ramp between; 8192 positions
    # before, 128 times as many after
    factor, turns = 128.0, 8192.0 * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor), 0.1 * math.log(factor) + 1.0


def _slots(T, page, g):
    """Slots of T tokens: runs of consecutive ones in scattered pages, as prompts have them."""
    pool = _pages(T, page) + 3
    pages = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    at = torch.arange(T, device=DEV)
    return (pages[at // page].long() * page + at % page).to(torch.int32), pool


def _prepare_rope(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n, ctx, cu = _requests(case, seed)
    T, d, page = cu[-1], case["d"], case["page"]
    slot, pool = _slots(T, page, g)
    q = torch.randn((T, case["Hq"], d), generator=g, device=DEV).to(dt)
    k, v = (torch.randn((T, case["Hkv"], d), generator=g, device=DEV).to(dt) for _ in range(2))
    kc, vc = (torch.zeros((pool, case["Hkv"], page, d), dtype=dt, device=DEV) for _ in range(2))
    f, factor = _freqs(case["rot"], case["scaling"])
    return dict(case=case, q=q, k=k, v=v, slot=slot, kept=_ints(ctx), cu=_ints(cu), k_cache=kc,
                v_cache=vc, q_out=torch.empty_like(q), freqs=f.to(DEV), factor=factor)


def _prepare_latent(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n, ctx, cu = _requests(case, seed)
    T, page, width = cu[-1], case["page"], case["dc"] + case["dr"]
    slot, pool = _slots(T, page, g)
    q = torch.randn((T, case["Hq"], case["dq"]), generator=g, device=DEV).to(dt)
    # latents of very different lengths, as a projection gives them
    kv = torch.randn((T, width), generator=g, device=DEV)
    kv[:, :case["dc"]] *= torch.exp(torch.randn((T, 1), generator=g, device=DEV) - 1.0)
    w = 1.0 + 0.2 * torch.randn(case["dc"], generator=g, device=DEV)
    f, factor = _freqs(case["dr"], case["scaling"])
    return dict(case=case, q=q, kv=kv.to(dt), w=w if case["norm"] else None, slot=slot,
                kept=_ints(ctx), cu=_ints(cu), freqs=f.to(DEV), factor=factor,
                q_out=torch.zeros((T, case["Hq"], case["dq_out"]), dtype=dt, device=DEV),
                kv_out=torch.zeros((T, width), dtype=dt, device=DEV),
                cache=torch.zeros((pool, page, width), dtype=dt, device=DEV))


def _prepare_absorbed(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n, ctx, cu = _requests(case, seed)
    page, width = case["page"], case["dc"] + case["dr"]
    have = [_pages(a + b, page) for a, b in zip(n, ctx)]
    cols, pool = max(have) + 1, sum(have) + 5
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    counts = _ints(have).long()
    first = counts.cumsum(0) - counts
    col = torch.arange(cols, device=DEV)
    table = torch.where(col < counts[:, None],
                        perm[(first[:, None] + col).clamp_max(pool - 1)], -1).to(torch.int32)
    q = torch.randn((cu[-1], case["Hq"], width), generator=g, device=DEV).to(dt)
    cache = torch.randn((pool, page, width), generator=g, device=DEV, dtype=dt)
    return dict(case=case, q=q, cache=cache, table=table.contiguous(), kept=_ints(ctx), cu=_ints(cu),
                n=n, ctx=ctx, cu_host=cu, max_new=max(n), scale=1.0 / math.sqrt(192.0))


def _prepare_expanded(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    n, ctx, cu = _requests(case, seed)
    cu_k = [0]
    for a, b in zip(n, ctx):
        cu_k.append(cu_k[-1] + a + b)
    H, N = case["H"], cu_k[-1]
    q = (1.5 * torch.randn((cu[-1], H, case["dn"] + case["dr"]), generator=g, device=DEV)).to(dt)
    # keys and values as one up-projection writes them, the shared part behind the latents
    kv = torch.randn((N, H, case["dn"] + case["dv"]), generator=g, device=DEV).to(dt)
    latent = torch.randn((N, 512 + case["dr"]), generator=g, device=DEV).to(dt)
    return dict(case=case, q=q, kv=kv, pe=latent[:, 512:], cu_q=_ints(cu), cu_k=_ints(cu_k),
                max_q=max(n), cu_q_host=cu, cu_k_host=cu_k)


def prepare(case, seed):
    s = {"rope": _prepare_rope, "latent": _prepare_latent, "absorbed": _prepare_absorbed,
         "expanded": _prepare_expanded}[case["op"]](case, seed)
    if own and "freqs" in s:
        import gated_delta_rule_22_amd as kda
        s["rope"] = kda.KDARope(s["freqs"], interleaved=case["pairs"] == "interleaved",
                                factor=s["factor"])
    return s


# ---------------------------------------------------------------------------------------------
# Plain forms

def _angles(s, T):
    """cos and sin [T, pairs] of the tokens' positions: angles in 64 bits, values in 32."""
    cu, kept = s["cu"].long(), s["kept"].long()
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(cu[1:], t, right=True)
    x = (kept[r] + t - cu[r]).double()[:, None] * s["freqs"]
    return (torch.cos(x) * s["factor"]).float(), (torch.sin(x) * s["factor"]).float()


def _rotate(x, cos, sin, pairs):
    """x [T, H, rot] in 32 bits."""
    cos, sin = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_rope(s):
    c, rot, page = s["case"], s["case"]["rot"], s["case"]["page"]
    cos, sin = _angles(s, s["q"].shape[0])

    def turn(x):
        y = _rotate(x[..., :rot].float(), cos, sin, c["pairs"]).to(x.dtype)
        return torch.cat([y, x[..., rot:]], -1)

    slot = s["slot"].long()
    at, off = slot // page, slot % page
    s["k_cache"][at, :, off] = turn(s["k"])
    s["v_cache"][at, :, off] = s["v"]
    return dict(q=turn(s["q"]), k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_latent(s):
    c, page = s["case"], s["case"]["page"]
    dc, dr, dt = c["dc"], c["dr"], s["kv"].dtype
    cos, sin = _angles(s, s["kv"].shape[0])
    x = s["kv"][:, :dc].float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w"]
    pe = _rotate(s["kv"][:, None, dc:].float(), cos, sin, c["pairs"])[:, 0]
    row = torch.cat([x, pe], -1).to(dt)
    s["kv_out"].copy_(row)
    slot = s["slot"].long()
    s["cache"][slot // page, slot % page] = row
    s["q_out"][..., -dr:] = _rotate(s["q"][..., -dr:].float(), cos, sin, c["pairs"]).to(dt)
    return dict(q=s["q_out"], kv=s["kv_out"], cache=s["cache"])


def _plain_absorbed(s):
    c, page = s["case"], s["case"]["page"]
    Hq, dc = c["Hq"], c["dc"]
    out = torch.empty((s["q"].shape[0], Hq, dc), dtype=s["q"].dtype, device=DEV)
    for i, (n, ctx) in enumerate(zip(s["n"], s["ctx"])):
        m, r0 = n + ctx, s["cu_host"][i]
        kv = s["cache"][s["table"][i, :_pages(m, page)].long()].flatten(0, 1)[:m].float()
        step = max(1, SCORE_BYTES // (4 * Hq * m))
        for a in range(0, n, step):                     # blocks of rows: the scores fit the memory
            b = min(n, a + step)
            x = torch.matmul(s["q"][r0 + a:r0 + b].float().flatten(0, 1), kv.t()).mul_(s["scale"])
            if n > 1:
                limit = ctx + torch.arange(a, b, device=DEV).repeat_interleave(Hq)
                x.masked_fill_(torch.arange(m, device=DEV) > limit[:, None], -math.inf)
            x = x.sub_(x.amax(-1, keepdim=True)).exp_()
            x = x.div_(x.sum(-1, keepdim=True))
            out[r0 + a:r0 + b] = torch.matmul(x, kv[:, :dc]).view(b - a, Hq, dc)
    return dict(o=out)


def _plain_expanded(s):
    c = s["case"]
    H, dn, dv, T = c["H"], c["dn"], c["dv"], s["q"].shape[0]
    out = torch.empty((T, H, dv), dtype=s["q"].dtype, device=DEV)
    lse = torch.empty((T, H), dtype=torch.float32, device=DEV)
    scale = 1.0 / math.sqrt(dn + c["dr"])
    for i in range(c["B"]):
        q0, q1, k0, k1 = (s[x][i + j] for x in ("cu_q_host", "cu_k_host") for j in (0, 1))
        n, m = q1 - q0, k1 - k0
        kv = s["kv"][k0:k1].float()
        k = torch.cat([kv[..., :dn], s["pe"][k0:k1, None].float().expand(m, H, c["dr"])], -1)
        k, v = k.permute(1, 2, 0).contiguous(), kv[..., dn:].transpose(0, 1).contiguous()
        step = max(1, SCORE_BYTES // (4 * H * m))
        for a in range(0, n, step):
            b = min(n, a + step)
            x = torch.matmul(s["q"][q0 + a:q0 + b].float().transpose(0, 1), k).mul_(scale)
            limit = m - n + torch.arange(a, b, device=DEV)
            x.masked_fill_(torch.arange(m, device=DEV) > limit[:, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            x = x.div_(total)
            out[q0 + a:q0 + b] = torch.matmul(x, v).transpose(0, 1)
            lse[q0 + a:q0 + b] = (top + total.log())[..., 0].t()
    return dict(o=out, lse=lse)


# ---------------------------------------------------------------------------------------------
# The package's calls

def _own(s):
    import gated_delta_rule_22_amd as kda
    c = s["case"]
    if c["op"] == "rope":
        kda.kda_rope_append(s["q"], s["k"], s["v"], s["slot"], s["kept"], s["cu"], s["k_cache"],
                            s["v_cache"], s["rope"], q_out=s["q_out"])
        return dict(q=s["q_out"], k_cache=s["k_cache"], v_cache=s["v_cache"])
    if c["op"] == "latent":
        kda.kda_latent_append(s["kv"], s["slot"], s["kept"], s["cu"], s["cache"], rope=s["rope"], w=s["w"],
                              normalise=c["norm"], eps=EPS, q=s["q"], q_out=s["q_out"],
                              kv_out=s["kv_out"])
        return dict(q=s["q_out"], kv=s["kv_out"], cache=s["cache"])
    if c["op"] == "absorbed":
        o, _ = kda.kda_attn_latent(s["q"], s["cache"], s["table"], s["kept"], s["cu"], dc=c["dc"],
                                   scale=s["scale"], max_new=s["max_new"])
        return dict(o=o)
    o, lse = kda.kda_attn_expanded(s["q"], s["kv"], s["pe"], s["cu_q"], s["cu_k"], dv=c["dv"],
                                   max_q=s["max_q"], want_lse=True)
    return dict(o=o, lse=lse)


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "latent": _plain_latent, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# 64-bit values: one request (and head) at a time, from the definition

def _turned(x, position, s):
    """x [tokens, heads, rot] at the positions, as complex numbers times exp(i angle)."""
    half = x.shape[-1] // 2
    if s["case"]["pairs"] == "half":
        z = torch.complex(x[..., :half].double(), x[..., half:].double())
    else:
        z = torch.view_as_complex(x.double().unflatten(-1, (half, 2)).contiguous())
    angle = position.double()[:, None] * s["freqs"]
    z = z * torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    parts = torch.view_as_real(z)
    return torch.cat([parts[..., 0], parts[..., 1]], -1) if s["case"]["pairs"] == "half" \
        else parts.flatten(-2)


def _exact_append(case, s):
    cu, kept = s["cu"].tolist(), s["kept"].tolist()
    position = torch.cat([torch.arange(k, k + b - a, device=DEV)
                          for k, a, b in zip(kept, cu, cu[1:])])
    slot = s["slot"].long()
    if case["op"] == "rope":
        rot = case["rot"]
        q, k = (torch.cat([_turned(s[x][..., :rot], position, s), s[x][..., rot:].double()], -1)
                for x in "qk")
        out = dict(q=q)
        for name, rows in (("k_cache", k), ("v_cache", s["v"].double())):
            pool, H, page, d = s[name].shape
            x = torch.zeros((pool * page, H, d), dtype=torch.float64, device=DEV)
            x.index_copy_(0, slot, rows)
            out[name] = x.view(pool, page, H, d).transpose(1, 2).contiguous()
        return out
    dc, dr = case["dc"], case["dr"]
    c = s["kv"][:, :dc].double()
    if case["norm"]:
        c = c / torch.sqrt(c.square().sum(1, keepdim=True) / dc + EPS) * s["w"].double()
    row = torch.cat([c, _turned(s["kv"][:, None, dc:], position, s)[:, 0]], 1)
    cache = torch.zeros(s["cache"].shape, dtype=torch.float64, device=DEV)
    cache.view(-1, dc + dr).index_copy_(0, slot, row)
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    q[..., -dr:] = _turned(s["q"][..., -dr:], position, s)
    return dict(q=q, kv=row, cache=cache)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] in ("rope", "latent"):
        return _exact_append(case, s)
    if case["op"] == "absorbed":
        out = torch.zeros(s["q"].shape[:2] + (case["dc"],), dtype=torch.float64, device=DEV)
        flat, page = s["cache"].flatten(0, 1), case["page"]
        for i, (r0, r1) in enumerate(zip(s["cu_host"], s["cu_host"][1:])):
            at = torch.arange(s["ctx"][i] + r1 - r0, device=DEV)
            x = flat[s["table"][i, at // page].long() * page + at % page].double()
            for a in range(r0, r1, 32):                 # a few tokens of all heads at a time
                b = min(r1, a + 32)
                z = (s["q"][a:b].double().reshape(-1, x.shape[1]) @ x.t().contiguous()) * s["scale"]
                last = s["ctx"][i] + torch.arange(a - r0, b - r0, device=DEV)
                z = z.view(b - a, -1, at.numel())
                z[(at > last[:, None])[:, None].expand_as(z)] = -math.inf
                out[a:b] = (torch.softmax(z, -1).view(-1, at.numel()) @ x[:, :case["dc"]]).view(
                    b - a, -1, case["dc"])
        return dict(o=out)
    H, dn = case["H"], case["dn"]
    out = torch.zeros((s["q"].shape[0], H, case["dv"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["q"].shape[0], H), dtype=torch.float64, device=DEV)
    for i in range(case["B"]):
        q0, q1 = s["cu_q_host"][i:i + 2]
        k0, k1 = s["cu_k_host"][i:i + 2]
        at = torch.arange(k1 - k0, device=DEV)
        pe = s["pe"][k0:k1].double().t().contiguous()
        for h in range(H):
            k = s["kv"][k0:k1, h, :dn].double().t().contiguous()
            v = s["kv"][k0:k1, h, dn:].double().contiguous()
            for a in range(q0, q1, 4096):
                b = min(q1, a + 4096)
                q = s["q"][a:b, h].double()
                z = (q[:, :dn].contiguous() @ k + q[:, dn:].contiguous() @ pe) \
                    / math.sqrt(dn + case["dr"])
                last = k1 - k0 - (q1 - torch.arange(a, b, device=DEV))
                z[at > last[:, None]] = -math.inf
                lse[a:b, h] = torch.logsumexp(z, 1)
                out[a:b, h] = torch.softmax(z, 1) @ v
    return dict(o=out, lse=lse)
