"""The full-attention layers' calls as a stack uses them, several steps in a row.

A latent layer: page plan, latent append, then attention of the prompts over expanded
keys and values and, of the same prompts and of the steps after them, over the latent
cache with the up-projections absorbed. Both are compared with the layer written down
in fp64 from its inputs (normalisation, rotation, up-projections, softmax over the
request's whole history). A grouped layer: page plan, rotated append, kda_attn_paged.
All in fp32, so that no rounding of intermediates to eight bits hides anything; steps
also run captured in one graph."""
import math

import pytest
import torch

import full_ref as R
import gated_delta_rule_22_amd as kda
from full_ref import DEV, F32, ints

pytestmark = pytest.mark.gpu

B, H, DN, DR, DC, PAGE = 4, 4, 64, 64, 128, 16
POOL, WIDTH, N = 64, 10, 3
SCALE = 1 / math.sqrt(DN + DR)
# Everything is fp32 with sums of at most 600 terms, relative to vectors whose parts are
# of the same size: 2^-24 * 600 for a score of magnitude up to 2^3 and twice through
# the softmax, the projections' 128 terms beside it, below 2^-10; measured against the
# norm of a row, errors average to far less than 2^-14.
TOL = 2.0 ** -14


class Requests:
    """The plan's state, and its buffers."""

    def __init__(self, rows):
        self.kept, self.new = ints([0] * B), ints([0] * B)
        self.pages, self.ring = ints([0] * B), ints([0, POOL])
        self.table, self.free = ints([[-1] * WIDTH] * B), ints(list(range(POOL)))
        self.cu, self.slots, self.status = ints([0] * (B + 1)), ints([0] * rows), ints([0])
        self.ws = torch.empty(max(16, kda.kda_page_plan_workspace_size(B)), dtype=torch.uint8, device=DEV)

    def plan(self):
        kda.kda_page_plan(self.kept, self.new, self.pages, self.table, self.free, self.ring, page_size=PAGE,
                          n_pages_out=self.pages, ring_out=self.ring, cu_new=self.cu, slot_map=self.slots,
                          status=self.status, workspace=self.ws)

    def state(self):
        return [self.kept, self.pages, self.ring, self.table, self.free]


def rel(x, ref):
    return float((x.double().cpu() - ref).norm() / ref.norm())


def turn(x, pos, f):
    return R.rotate(x, pos, f, False, 1.0)[0]


def history_attention(q, k, v, kept, scale):
    """One request: q [n,H,dk], k [m,H,dk], v [m,H,dv] with m = kept + n."""
    n, m = q.shape[0], k.shape[0]
    s = torch.einsum("nhd,mhd->hnm", q, k) * scale
    s.masked_fill_(torch.arange(m)[None, None] > kept + torch.arange(n)[None, :, None], -math.inf)
    return torch.einsum("hnm,mhd->nhd", torch.softmax(s, 2), v)


@pytest.mark.parametrize("captured", [False, True])
def test_latent_layer(captured):
    g = torch.Generator().manual_seed(1)
    uk = (torch.randn((H, DN, DC), generator=g) / math.sqrt(DC)).to(DEV)
    uv = (torch.randn((H, DN, DC), generator=g) / math.sqrt(DC)).to(DEV)
    w = (1 + 0.2 * torch.randn(DC, generator=g)).to(DEV)
    f, _ = kda.kda_rope_freqs(DR)
    rope = kda.KDARope(f.to(DEV))
    prompt = [40, 1, 0, 65]
    rows = max(sum(prompt), B * N)
    r = Requests(rows)
    cache = torch.full((POOL, PAGE, DC + DR), float("nan"), device=DEV)
    q, kv = torch.zeros((rows, H, DN + DR), device=DEV), torch.zeros((rows, DC + DR), device=DEV)
    q_lat, kv_out = torch.zeros((rows, H, DC + DR), device=DEV), torch.zeros_like(kv)
    o_lat = torch.zeros((rows, H, DC), device=DEV)
    ws = torch.empty(kda.kda_attn_latent_workspace_size(rows, B, H, DC, DR, 0, F32), dtype=torch.uint8, device=DEV)
    past = [torch.zeros((0, DC + DR), dtype=torch.float64) for _ in range(B)]

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        q.copy_(torch.randn(q.shape, generator=g))
        kv.copy_(torch.randn(kv.shape, generator=g) * torch.exp(torch.randn((rows, 1), generator=g)))

    def step():
        r.plan()
        q_lat[..., :DC].copy_(torch.matmul(q[..., :DN].transpose(0, 1), uk).transpose(0, 1))
        kda.kda_latent_append(kv, r.slots, r.kept, r.cu, cache, rope=rope, w=w, q=q, q_out=q_lat, kv_out=kv_out)
        kda.kda_attn_latent(q_lat, cache, r.table, r.kept, r.cu, dc=DC, scale=SCALE, o=o_lat, workspace=ws)

    def reference(n, kept):
        """[rows, H, DN]: the layer's heads before the output projection."""
        cu, out = R.offsets(n), []
        x = kv.double().cpu()
        c = x[:, :DC] / torch.sqrt((x[:, :DC] ** 2).mean(1, keepdim=True) + 1e-6) * w.double().cpu()
        for i in range(B):
            at = slice(cu[i], cu[i + 1])
            pos = list(range(kept[i], kept[i] + n[i]))
            pe = turn(x[at, None, DC:], pos, f)[:, 0]
            past[i] = torch.cat([past[i][:kept[i]], torch.cat([c[at], pe], 1)])
            if n[i] == 0:
                continue
            qd = q[at].double().cpu()
            qd = torch.cat([qd[..., :DN], turn(qd[..., DN:], pos, f)], 2)
            k = torch.einsum("mc,hdc->mhd", past[i][:, :DC], uk.double().cpu())
            k = torch.cat([k, past[i][:, None, DC:].expand(-1, H, -1)], 2)
            v = torch.einsum("mc,hdc->mhd", past[i][:, :DC], uv.double().cpu())
            out.append(history_attention(qd, k, v, kept[i], SCALE))
        return torch.cat(out)

    def heads(T):
        return torch.matmul(o_lat[:T].transpose(0, 1), uv.transpose(1, 2).contiguous()).transpose(0, 1)

    fill(100)
    r.new.copy_(ints(prompt))
    step()
    torch.cuda.synchronize()
    T = sum(prompt)
    ref = reference(prompt, [0] * B)
    e = rel(heads(T), ref)
    print(f"[full] prompts, absorbed: {e:.2e}", flush=True)
    assert int(r.status) == 0 and e <= TOL
    # the same prompts, expanded
    up = torch.cat([uk, uv], 1)                                     # [H, DN + DN, DC]
    kv_up = torch.einsum("mc,hdc->mhd", kv_out[:T, :DC], up).contiguous()
    qr = q[:T].clone()
    qr[..., DN:] = q_lat[:T, :, DC:]
    o, _ = kda.kda_attn_expanded(qr, kv_up, kv_out[:T, DC:], r.cu, r.cu, dv=DN, max_q=max(prompt))
    e = rel(o, ref)
    print(f"[full] prompts, expanded: {e:.2e}", flush=True)
    assert e <= TOL

    r.kept.copy_(r.new)
    r.new.fill_(N)
    graph = None
    if captured:
        saved = [t.clone() for t in r.state() + [cache]]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, x in zip(r.state() + [cache], saved):
            t.copy_(x)
    for i in range(5):
        fill(200 + i)
        kept = r.kept.tolist()
        if graph is None:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert int(r.status) == 0
        e = rel(heads(B * N), reference([N] * B, kept))
        print(f"[full] step {i}: {e:.2e}", flush=True)
        assert e <= TOL
        r.kept.add_(ints([1, 3, 2, 1]))              # some of the new tokens stay


@pytest.mark.parametrize("captured", [False, True])
def test_grouped_layer(captured):
    HQ, HKV, D, ROT = 8, 2, 64, 32
    f, factor = kda.kda_rope_freqs(ROT, scaling="parts", scale=8.0, original_len=32)
    rope = kda.KDARope(f.to(DEV), interleaved=True, factor=factor)
    prompt = [33, 0, 5, 70]
    rows = max(sum(prompt), B * N)
    r = Requests(rows)
    kc, vc = (torch.full((POOL, HKV, PAGE, D), float("nan"), device=DEV) for _ in range(2))
    q = torch.zeros((rows, HQ, D), device=DEV)
    k, v = (torch.zeros((rows, HKV, D), device=DEV) for _ in range(2))
    qr, o = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.empty(max(16, kda.kda_attn_paged_workspace_size(rows, B, HQ, HKV, D, 0, F32)), dtype=torch.uint8,
                     device=DEV)
    past = [(torch.zeros((0, HKV, D), dtype=torch.float64),) * 2 for _ in range(B)]

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))

    def step():
        r.plan()
        kda.kda_rope_append(q, k, v, r.slots, r.kept, r.cu, kc, vc, rope, q_out=qr)
        kda.kda_attn_paged(qr, kc, vc, r.table, r.kept, r.cu, o=o, workspace=ws)

    def turned(x, pos):
        return torch.cat([R.rotate(x[..., :ROT], pos, f, True, factor)[0], x[..., ROT:]], 2)

    def reference(n, kept):
        cu, out = R.offsets(n), []
        for i in range(B):
            at, pos = slice(cu[i], cu[i + 1]), list(range(kept[i], kept[i] + n[i]))
            ks, vs = past[i]
            past[i] = (torch.cat([ks[:kept[i]], turned(k[at].double().cpu(), pos)]),
                       torch.cat([vs[:kept[i]], v[at].double().cpu()]))
            if n[i]:
                kk, vv = (x.repeat_interleave(HQ // HKV, 1) for x in past[i])
                out.append(history_attention(turned(q[at].double().cpu(), pos), kk, vv, kept[i],
                                             1 / math.sqrt(D)))
        return torch.cat(out)

    def compare(n, kept, what):
        torch.cuda.synchronize()
        assert int(r.status) == 0
        e = rel(o[:sum(n)], reference(n, kept))
        print(f"[full] grouped, {what}: {e:.2e}", flush=True)
        assert e <= TOL

    fill(300)
    r.new.copy_(ints(prompt))
    step()
    compare(prompt, [0] * B, "prompts")
    r.kept.copy_(r.new)
    r.new.fill_(N)
    graph = None
    if captured:
        saved = [t.clone() for t in r.state() + [kc, vc]]
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, x in zip(r.state() + [kc, vc], saved):
            t.copy_(x)
    for i in range(5):
        fill(400 + i)
        kept = r.kept.tolist()
        if graph is None:
            step()
        else:
            graph.replay()
        compare([N] * B, kept, f"step {i}")
        r.kept.add_(ints([3, 1, 1, 2]))


def test_empty_step_after_a_shortage():
    # a plan that cannot be met leaves offsets of 0 and slots of -1: the calls behind it
    # write nothing
    r = Requests(50)
    r.new.copy_(ints([40, 1, 0, 9]))
    r.ring.copy_(ints([0, 2]))
    r.plan()
    rope = kda.KDARope(kda.kda_rope_freqs(DR)[0].to(DEV))
    cache = torch.full((POOL, PAGE, DC + DR), 7.0, device=DEV)
    kv, q = torch.ones((50, DC + DR), device=DEV), torch.ones((50, H, DC + DR), device=DEV)
    q_out, kv_out, o = torch.full_like(q, 5.0), torch.full_like(kv, 5.0), torch.full((50, H, DC), 5.0, device=DEV)
    kda.kda_latent_append(kv, r.slots, r.kept, r.cu, cache, rope=rope, q=q, q_out=q_out, kv_out=kv_out)
    kda.kda_attn_latent(q, cache, r.table, r.kept, r.cu, dc=DC, scale=SCALE, o=o)
    assert int(r.status) > 0
    for x, want in ((cache, 7.0), (q_out, 5.0), (kv_out, 5.0), (o, 5.0)):
        assert bool((x == want).all())


def test_context_and_chunk_join_by_their_sums():
    # a chunk's attention over what is cached (absorbed) and over itself (expanded) join
    # to its attention over both: o = sum_i exp(lse_i - lse) o_i
    g = torch.Generator().manual_seed(9)
    ctx, n = 50, 20
    uk, uv = (torch.randn((H, DN, DC), generator=g, dtype=torch.float64) / math.sqrt(DC) for _ in range(2))
    rows = torch.randn((ctx + n, DC + DR), generator=g, dtype=torch.float64)
    q = torch.randn((n, H, DN + DR), generator=g, dtype=torch.float64)
    k = torch.cat([torch.einsum("mc,hdc->mhd", rows[:, :DC], uk), rows[:, None, DC:].expand(-1, H, -1)], 2)
    v = torch.einsum("mc,hdc->mhd", rows[:, :DC], uv)
    ref = history_attention(q, k, v, ctx, SCALE)
    kv_up = torch.cat([k[ctx:, :, :DN], v[ctx:]], 2).float().contiguous().to(DEV)
    o1, l1 = kda.kda_attn_expanded(q.float().to(DEV), kv_up, rows[ctx:, DC:].float().contiguous().to(DEV),
                                   ints([0, n]), ints([0, n]), dv=DN, want_lse=True)
    # every token alone sees the whole context and nothing else: a request of one row
    # over ctx - 1 tokens before it
    cache = torch.zeros((4, PAGE, DC + DR), device=DEV)
    cache.view(-1, DC + DR)[:ctx] = rows[:ctx].float().to(DEV)
    q_lat = torch.cat([torch.einsum("nhd,hdc->nhc", q[..., :DN], uk), q[..., DN:]], 2).float().contiguous()
    o2, l2 = kda.kda_attn_latent(q_lat.to(DEV), cache, ints([[0, 1, 2, 3]] * n), ints([ctx - 1] * n),
                                 ints(list(range(n + 1))), dc=DC, scale=SCALE, max_new=1, want_lse=True)
    o2 = torch.einsum("nhc,hdc->nhd", o2.double().cpu(), uv)
    l1, l2 = l1.double().cpu()[..., None], l2.double().cpu()[..., None]
    both = torch.logaddexp(l1, l2)
    o = torch.exp(l1 - both) * o1.double().cpu() + torch.exp(l2 - both) * o2
    assert rel(o, ref) <= TOL
