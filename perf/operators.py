"""The serving operators around the recurrent layer: cases, inputs, plain forms and 64-bit values.

One serving step of a stack that mixes recurrent and full-attention layers gives the new tokens of
every request their cache pages (``plan``), writes their keys and values there (``append``), attends
from them over each request's pages (``attn``), and decides which drafted tokens stay (``verify``).

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
ROW_BLOCK_BYTES = 8 << 30     # the plain attention's scores at one time


# ---------------------------------------------------------------------------------------------
# Cases

def listed():
    return [
        # one decode step of a full batch: every request adds up to 8 tokens (a verified draft)
        dict(name="plan_step_b256", op="plan", B=256, new_lo=1, new_hi=8, kept_lo=1, kept_hi=16384,
             page=64, gone=0.05),
        # prompts packed into one call, many requests, small pages: hundreds of thousands of slots
        dict(name="plan_prompts_b1024", op="plan", B=1024, new_lo=1, new_hi=2048, kept_lo=1,
             kept_hi=32768, page=16, gone=0.1),
        # one token of every request into its page
        dict(name="append_step_t256", op="append", T=256, Hkv=8, d=128, page=64, dtype="bf16"),
        # 65,536 packed prompt tokens, fp32
        dict(name="append_prompts_t65536", op="append", T=65536, Hkv=8, d=128, page=64, dtype="fp32"),
        # one request, one token, a short context: latency
        dict(name="attn_decode_b1", op="attn", B=1, n_lo=1, n_hi=1, ctx_lo=1000, ctx_hi=1000, Hq=32,
             Hkv=8, d=128, page=64, dtype="bf16"),
        # a full decode batch over ragged contexts
        dict(name="attn_decode_b256", op="attn", B=256, n_lo=1, n_hi=1, ctx_lo=1024, ctx_hi=16384,
             Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # 8-token drafts checked over very long contexts
        dict(name="attn_draft_b4_long", op="attn", B=4, n_lo=8, n_hi=8, ctx_lo=65536, ctx_hi=262144,
             Hq=32, Hkv=8, d=128, page=256, dtype="bf16"),
        # a chunk of a long prompt over what is cached of it
        dict(name="attn_chunk_t8192", op="attn", B=1, n_lo=8192, n_hi=8192, ctx_lo=24576,
             ctx_hi=24576, Hq=32, Hkv=8, d=128, page=64, dtype="bf16"),
        # prompts and single tokens together, one KV head per query head, 64 wide, small pages
        dict(name="attn_mixed_d64", op="attn", B=16, n_lo=1, n_hi=1023, ctx_lo=1, ctx_hi=8191, Hq=16,
             Hkv=16, d=64, page=16, dtype="bf16"),
        # fp32, ragged
        dict(name="attn_fp32", op="attn", B=8, n_lo=5, n_hi=301, ctx_lo=1, ctx_hi=2001, Hq=16, Hkv=4,
             d=128, page=32, dtype="fp32"),
        # one request, a certain draft (no draft probabilities), an odd vocabulary, bf16
        dict(name="verify_b1_bf16", op="verify", B=1, T=3, V=32003, dtype="bf16", with_q=False),
        # a full batch of 7-token drafts over a large vocabulary
        dict(name="verify_b256", op="verify", B=256, T=7, V=131072, dtype="fp32", with_q=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_attn(rng):
    kind = rng.choice(["decode", "draft", "chunk", "mixed"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    Hq = Hkv * rng.choice([g for g in (1, 2, 3, 4, 5, 8, 16) if Hkv * g <= 40])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    if kind == "decode":
        B, n_lo, n_hi, ctx = _log_int(rng, 1, 256), 1, 1, _log_int(rng, 1, 65536)
    elif kind == "draft":
        n_hi = rng.randint(2, 8)
        B, n_lo, ctx = _log_int(rng, 1, 128), n_hi, _log_int(rng, 8, 131072)
    elif kind == "chunk":
        n_hi = _log_int(rng, 33, 8192)
        B, n_lo, ctx = rng.randint(1, 3), n_hi, _log_int(rng, 1, 24576)
    else:
        B, n_lo, n_hi, ctx = rng.randint(2, 24), 1, _log_int(rng, 9, 1023), _log_int(rng, 1, 8191)
    c = dict(op="attn", B=B, n_lo=n_lo, n_hi=n_hi, ctx_lo=max(1, ctx // rng.randint(1, 6)), ctx_hi=ctx,
             Hq=Hq, Hkv=Hkv, d=d, page=page, dtype=dtype)
    most = work(dict(op="attn", B=1, n_lo=8192, n_hi=8192, ctx_lo=24576, ctx_hi=24576, Hq=32, Hkv=8,
                     d=128, page=64, dtype="bf16"))["flops"]
    while work(c)["bytes"] > 2e9 or work(c)["flops"] > (0.5 if dtype == "bf16" else 0.05) * most:
        if c["B"] > 1:
            c["B"] = max(1, c["B"] // 2)
        else:
            c["ctx_hi"] = max(1, c["ctx_hi"] // 2)
            c["ctx_lo"] = min(c["ctx_lo"], c["ctx_hi"])
            c["n_hi"] = max(1, c["n_hi"] // 2)
            c["n_lo"] = min(c["n_lo"], c["n_hi"])
    return c


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn", "attn", "verify"])
    if op == "plan":
        kept = _log_int(rng, 8, 32768)
        return dict(op="plan", B=_log_int(rng, 1, 1024), new_lo=1, new_hi=_log_int(rng, 1, 2048),
                    kept_lo=1, kept_hi=kept, page=rng.choice([16, 32, 64, 128, 256]),
                    gone=rng.choice([0.0, 0.05, 0.3]))
    if op == "append":
        return dict(op="append", T=_log_int(rng, 1, 65536), Hkv=rng.choice([1, 2, 3, 4, 8, 16]),
                    d=rng.choice([16, 32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "fp32"]))
    if op == "verify":
        return dict(op="verify", B=_log_int(rng, 1, 256), T=rng.randint(1, 7),
                    V=_log_int(rng, 257, 131072), dtype=rng.choice(["bf16", "fp32"]),
                    with_q=rng.choice([True, True, False]))
    return _draw_attn(rng)


# ---------------------------------------------------------------------------------------------
# Lengths: a fixed spread over the case's range (over the logarithm), the same multiset for every
# seed, so that the work of a case does not depend on the seed; the seed permutes the requests.

def _spread(lo, hi, n, shift):
    return [min(hi, max(lo, int(round(math.exp(
        math.log(lo) + ((i + shift) * GOLDEN % 1.0) * (math.log(hi) - math.log(lo)))))))
        for i in range(n)]


def _attn_lengths(case):
    n = _spread(case["n_lo"], case["n_hi"], case["B"], 0.5)
    # a second sequence independent of the first: half steps of sqrt(2)
    ctx = [min(case["ctx_hi"], max(case["ctx_lo"], int(round(math.exp(
        math.log(case["ctx_lo"]) + ((i + 0.5) * math.sqrt(2) % 1.0)
        * (math.log(case["ctx_hi"]) - math.log(case["ctx_lo"]))))))) for i in range(case["B"])]
    return n, ctx


def _plan_lengths(case):
    B = case["B"]
    new = _spread(case["new_lo"], case["new_hi"], B, 0.5)
    kept = _spread(case["kept_lo"], case["kept_hi"], B, 0.25)
    ahead = [(i * 7919) % 9 for i in range(B)]          # tokens of the last step that fell away
    gone = [((i + 0.5) * math.sqrt(2) % 1.0) < case["gone"] for i in range(B)]
    had = [k + a for k, a in zip(kept, ahead)]
    new = [0 if g else n for n, g in zip(new, gone)]
    kept = [0 if g else k for k, g in zip(kept, gone)]
    return had, kept, new


def _pages(n, page):
    return -(-n // page)


def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] == "plan":
        had, kept, new = _plan_lengths(case)
        moved = sum(abs(_pages(k + n, case["page"]) - _pages(h, case["page"]))
                    for h, k, n in zip(had, kept, new))
        # three lengths in, two counts out, a slot per token, each moved page read and written
        return {"bytes": 4 * (5 * case["B"] + sum(new) + 2 * moved), "flops": 0}
    if case["op"] == "append":
        return {"bytes": 4 * case["T"] * case["Hkv"] * case["d"] * e + 4 * case["T"], "flops": 0}
    if case["op"] == "attn":
        n, ctx = _attn_lengths(case)
        kv = sum(a + b for a, b in zip(n, ctx))
        pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, ctx))
        return {"bytes": 2 * e * case["d"] * (kv * case["Hkv"] + sum(n) * case["Hq"]),
                "flops": 4 * case["d"] * case["Hq"] * pairs}
    # one row of the target for every request; the draft's row only where a token is rejected
    # (about half of the requests), and two values for each drafted token
    rows = case["B"] * (1.5 if case["with_q"] else 1.0)
    return {"bytes": int(rows * case["V"] * e) + 12 * case["B"] * case["T"],
            "flops": int(3 * rows * case["V"])}


# ---------------------------------------------------------------------------------------------
# Inputs

def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _prepare_plan(case, seed):
    rng = random.Random(seed)
    g, B, page = _gen(seed), case["B"], case["page"]
    rows = list(zip(*_plan_lengths(case)))
    rng.shuffle(rows)
    had, kept, new = (list(c) for c in zip(*rows))
    have = [_pages(h, page) for h in had]
    need = [_pages(k + n, page) for k, n in zip(kept, new)]
    width = max(have + need) + 2
    pops = sum(max(0, b - a) for a, b in zip(have, need))
    pool = sum(have) + pops + 37
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    counts = _ints(have).long()
    first = counts.cumsum(0) - counts
    col = torch.arange(width, device=DEV)
    table = torch.where(col < counts[:, None],
                        perm[(first[:, None] + col).clamp_max(pool - 1)], -1).to(torch.int32)
    free = perm[sum(have):]
    head = rng.randrange(pool)
    ring = torch.full((pool,), -1, dtype=torch.int32, device=DEV)
    ring[(head + torch.arange(free.numel(), device=DEV)) % pool] = free
    slots = sum(new) + 5                                # padded, as a captured step's is
    return dict(case=case, kept=_ints(kept), new=_ints(new), pages=_ints(have), table=table,
                ring=ring, ring_state=_ints([head, free.numel()]), slots=slots,
                out=dict(n_pages_out=torch.empty_like(_ints(have)),
                         ring_out=_ints([0, 0]), cu_new=_ints([0] * (B + 1)),
                         slot_map=torch.empty(slots, dtype=torch.int32, device=DEV),
                         status=_ints([0])))


def _prepare_append(case, seed):
    g, T, H, d, page = _gen(seed), case["T"], case["Hkv"], case["d"], case["page"]
    dt = DTYPES[case["dtype"]]
    pool = _pages(T, page) + 3
    # runs of consecutive slots in scattered pages, as prompts have them
    pages = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    at = torch.arange(T, device=DEV)
    slot = (pages[at // page].long() * page + at % page).to(torch.int32)
    k, v = (torch.randn((T, H, d), generator=g, device=DEV).to(dt) for _ in range(2))
    kc, vc = (torch.zeros((pool, H, page, d), dtype=dt, device=DEV) for _ in range(2))
    return dict(case=case, k=k, v=v, slot=slot, k_cache=kc, v_cache=vc)


def _prepare_attn(case, seed):
    rng = random.Random(seed)
    g, B, page, d = _gen(seed), case["B"], case["page"], case["d"]
    dt = DTYPES[case["dtype"]]
    rows = list(zip(*_attn_lengths(case)))
    rng.shuffle(rows)
    n, ctx = (list(c) for c in zip(*rows))
    have = [_pages(a + b, page) for a, b in zip(n, ctx)]
    width, pool = max(have) + 1, sum(have) + 5
    perm = torch.randperm(pool, generator=g, device=DEV, dtype=torch.int32)
    counts = _ints(have).long()
    first = counts.cumsum(0) - counts
    col = torch.arange(width, device=DEV)
    table = torch.where(col < counts[:, None],
                        perm[(first[:, None] + col).clamp_max(pool - 1)], -1).to(torch.int32)
    cu = [0]
    for a in n:
        cu.append(cu[-1] + a)
    q = (1.5 * torch.randn((cu[-1], case["Hq"], d), generator=g, device=DEV)).to(dt)
    kc, vc = (torch.randn((pool, case["Hkv"], page, d), generator=g, device=DEV, dtype=dt)
              for _ in range(2))
    return dict(case=case, q=q, k_cache=kc, v_cache=vc, table=table.contiguous(), kept=_ints(ctx),
                cu=_ints(cu), max_new=max(n), max_kv=max(a + b for a, b in zip(n, ctx)))


def _prepare_verify(case, seed):
    g, B, T, V = _gen(seed), case["B"], case["T"], case["V"]
    dt = DTYPES[case["dtype"]]
    z = 2.0 * torch.randn((B, T + 1, V), generator=g, device=DEV)
    p = torch.softmax(z, -1)
    z = z[:, :T].add_(torch.randn((B, T, V), generator=g, device=DEV), alpha=0.35)
    q = torch.softmax(z, -1)
    # a certain draft is the likelier to stay the likelier its token: drawn from the target's
    x = torch.multinomial((q if case["with_q"] else p[:, :T]).reshape(B * T, V), 1, generator=g)
    u = torch.rand((B, T + 1), generator=g, device=DEV)
    return dict(case=case, p=p.to(dt).contiguous(), q=q.to(dt).contiguous() if case["with_q"] else None,
                x=x.view(B, T).to(torch.int32), u=u)


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn,
            "verify": _prepare_verify}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------
# Plain forms

def _plain_plan(s):
    page, (B, width), pool = s["case"]["page"], s["table"].shape, s["ring"].numel()
    kept, new, have = s["kept"].long(), s["new"].long(), s["pages"].long()
    head, count = s["ring_state"].long().unbind()
    need = (kept + new + page - 1) // page
    pop, push = (need - have).clamp_min(0), (have - need).clamp_min(0)
    pop_end, push_end, cu_end = pop.cumsum(0), push.cumsum(0), new.cumsum(0)
    missing = (pop_end[-1] - count).clamp_min(0)
    bad = (need > width).any() | (kept < 0).any() | (new < 0).any() | (count + push_end[-1] > pool)
    status = torch.where(bad, -1, torch.where(cu_end[-1] > s["slots"], -2, missing))
    good = status == 0
    col = torch.arange(width, device=DEV)
    taken = s["ring"][(head + (pop_end - pop)[:, None] + col - have[:, None]) % pool]
    fresh = (col >= have[:, None]) & (col < need[:, None]) & good
    table = torch.where(fresh, taken, s["table"])
    back = (col >= need[:, None]) & (col < have[:, None]) & good
    to = torch.where(back, (head + count + (push_end - push)[:, None] + col - need[:, None]) % pool,
                     pool)
    ring = torch.cat([s["ring"], s["ring"][:1]])
    ring[to] = torch.where(back, s["table"], s["ring"][0])
    t = torch.arange(s["slots"], device=DEV)
    r = torch.searchsorted(cu_end, t, right=True).clamp_max(B - 1)
    pos = kept[r] + t - (cu_end - new)[r]
    slot = table[r, (pos // page).clamp(0, width - 1)] * page + pos % page
    slot = torch.where((t < cu_end[-1]) & good, slot, -1)
    cu = torch.cat([cu_end.new_zeros(1), cu_end]) * good
    state = torch.stack([(head + pop_end[-1] * good) % pool,
                         count + (push_end[-1] - pop_end[-1]) * good])
    return dict(table=table, pages=torch.where(good, need, have).to(torch.int32),
                ring=ring[:pool], ring_state=state.to(torch.int32), cu=cu.to(torch.int32),
                slot=slot.to(torch.int32), status=status.view(1).to(torch.int32))


def _plain_append(s):
    page, slot = s["case"]["page"], s["slot"].long()
    at, off = slot // page, slot % page
    s["k_cache"][at, :, off] = s["k"]
    s["v_cache"][at, :, off] = s["v"]
    return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])


def _plain_attn(s):
    c, T = s["case"], s["q"].shape[0]
    B, Hkv, d, page = c["B"], c["Hkv"], c["d"], c["page"]
    G, n_max, kv_max = c["Hq"] // Hkv, s["max_new"], s["max_kv"]
    cols = _pages(kv_max, page)
    pages = s["table"][:, :cols].clamp_min(0).long()
    kept, cu = s["kept"].long(), s["cu"].long()
    # every request padded to the longest: [B, Hkv, keys, d] and [B, Hkv, new * G, d]
    k, v = (x[pages].transpose(1, 2).reshape(B, Hkv, cols * page, d).float()
            for x in (s["k_cache"], s["v_cache"]))
    t = torch.arange(n_max, device=DEV)
    row = (cu[:-1, None] + t).clamp_max(T - 1)
    q = s["q"][row].float().view(B, n_max, Hkv, G, d).permute(0, 2, 1, 3, 4)
    key = torch.arange(cols * page, device=DEV)
    out = torch.empty((B, n_max, Hkv, G, d), device=DEV)
    step = max(1, ROW_BLOCK_BYTES // (4 * B * Hkv * G * cols * page))
    for a in range(0, n_max, step):                     # blocks of rows: the scores fit the memory
        b = min(n_max, a + step)
        x = torch.matmul(q[:, :, a:b].reshape(B, Hkv, (b - a) * G, d), k.transpose(2, 3))
        x = x.mul_(1.0 / math.sqrt(d)).view(B, Hkv, b - a, G, cols * page)
        seen = key <= (kept[:, None] + t[a:b])[..., None]            # [B, rows, keys]
        x = x.masked_fill_(~seen[:, None, :, None], -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        x = x.div_(x.sum(-1, keepdim=True)).view(B, Hkv, (b - a) * G, cols * page)
        out[:, a:b] = torch.matmul(x, v).view(B, Hkv, b - a, G, d).permute(0, 2, 1, 3, 4)
        del x, seen
    r = torch.searchsorted(cu[1:], torch.arange(T, device=DEV), right=True)
    return dict(o=out.view(B, n_max, c["Hq"], d)[r, torch.arange(T, device=DEV) - cu[r]]
                .to(s["q"].dtype))


def _plain_verify(s):
    p, q, x = s["p"], s["q"], s["x"].long()
    (B, T), V = x.shape, p.shape[-1]
    u = s["u"].double()
    pt = p[:, :T].gather(2, x[..., None])[..., 0].double()
    qt = q.gather(2, x[..., None])[..., 0].double() if q is not None else torch.ones_like(pt)
    stay = (u[:, :T] * qt < pt).long().cumprod(1)
    a = stay.sum(1)
    b = torch.arange(B, device=DEV)
    row = p[b, a].double()
    last = a.clamp_max(T - 1)
    if q is not None:
        rest = (row - q[b, last].double()).clamp_min_(0)
    else:
        rest = row.scatter(1, x[b, last][:, None], 0.0)
    use = (a < T) & (rest.sum(1) > 0)
    cdf = torch.where(use[:, None], rest, row).cumsum(1)
    y = (cdf <= (u[:, T] * cdf[:, -1])[:, None]).sum(1).clamp_max(V - 1)
    t = torch.arange(T + 1, device=DEV)
    tokens = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(t < a[:, None], tokens, torch.where(t == a[:, None], y[:, None], -1))
    return dict(n_commit=(a + 1).to(torch.int32), tokens=tokens.to(torch.int32))


# ---------------------------------------------------------------------------------------------
# The package's calls

def _own(s):
    import gated_delta_rule_22_amd as kda
    c = s["case"]
    if c["op"] == "plan":
        kda.kda_page_plan(s["kept"], s["new"], s["pages"], s["table"], s["ring"], s["ring_state"],
                          page_size=c["page"], **s["out"])
        o = s["out"]
        return dict(table=s["table"], pages=o["n_pages_out"], ring=s["ring"],
                    ring_state=o["ring_out"], cu=o["cu_new"], slot=o["slot_map"],
                    status=o["status"])
    if c["op"] == "append":
        kda.kda_cache_append(s["k"], s["v"], s["slot"], s["k_cache"], s["v_cache"])
        return dict(k_cache=s["k_cache"], v_cache=s["v_cache"])
    if c["op"] == "attn":
        o, _ = kda.kda_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kept"],
                                  s["cu"], max_new=s["max_new"])
        return dict(o=o)
    n_commit, tokens = kda.kda_draft_verify(s["p"], s["q"], s["x"], s["u"])
    return dict(n_commit=n_commit, tokens=tokens)


def run(state):
    if own:
        return _own(state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn,
            "verify": _plain_verify}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------
# 64-bit values: one request and one KV head at a time, from the definition

def exact(case, seed):
    if case["op"] in ("plan", "verify"):
        return None                                      # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        slots = s["slot"].long()
        flat = {}
        for name, rows in (("k_cache", s["k"]), ("v_cache", s["v"])):
            pool, H, page, d = s[name].shape
            x = torch.zeros((pool * page, H, d), dtype=torch.float64, device=DEV)
            x.index_copy_(0, slots, rows.double())
            flat[name] = x.view(pool, page, H, d).transpose(1, 2).contiguous()
        return flat
    if work(case)["flops"] > 8e12:
        return None
    page, G = case["page"], case["Hq"] // case["Hkv"]
    cu, kept = s["cu"].tolist(), s["kept"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for i in range(case["B"]):
        n, m = cu[i + 1] - cu[i], kept[i] + cu[i + 1] - cu[i]
        at = torch.arange(m, device=DEV)
        pg, off = s["table"][i, at // page].long(), at % page
        limit = kept[i] + torch.arange(n, device=DEV)
        for h in range(case["Hkv"]):
            kt = s["k_cache"][pg, h, off].double().t().contiguous()
            v = s["v_cache"][pg, h, off].double()
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                for hq in range(h * G, (h + 1) * G):
                    z = s["q"][cu[i] + a:cu[i] + b, hq].double() @ kt / math.sqrt(case["d"])
                    z[at[None, :] > limit[a:b, None]] = -math.inf
                    out[cu[i] + a:cu[i] + b, hq] = torch.softmax(z, 1) @ v
    return dict(o=out)
