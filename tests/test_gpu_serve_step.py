"""The serving calls as a step uses them, several steps in a row.

Each step drafts tokens for every request: page plan, cache append, paged
attention, draft verification, and the recurrent layer's state advanced by
the verification's n_commit (kda_decode_multi). Requests keep what stays;
rejected tokens' pages go back. A dense copy of every request's keys and
values, kept on the host, says what the attention has to see."""
import numpy as np
import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints

pytestmark = pytest.mark.gpu

B, T, HQ, HKV, D, PAGE, V = 5, 4, 8, 2, 64, 16, 97
N = T + 1                                     # the last token and the drafts
POOL, WIDTH = 64, 12
DK = 64                                       # the recurrent layer's head


class Step:
    def __init__(self, dtype, prompt):
        self.dtype = dtype
        g = torch.Generator().manual_seed(4)
        self.kept, self.new = ints([0] * B), ints(prompt)
        self.pages, self.ring = ints([0] * B), ints([0, POOL])
        self.table, self.free = ints([[-1] * WIDTH] * B), ints(list(range(POOL)))
        self.kc, self.vc = (torch.full((POOL, HKV, PAGE, D), float("nan"), dtype=dtype, device=DEV)
                            for _ in range(2))
        self.S = 0.1 * torch.randn((B, 2, DK, DK), generator=g).to(DEV)
        self.dense = [([], []) for _ in range(B)]
        rows = max(sum(prompt), B * N)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.cu, self.slots = torch.zeros(B + 1, **i32), torch.zeros(rows, **i32)
        self.status = torch.zeros(1, **i32)
        self.q = torch.zeros((rows, HQ, D), dtype=dtype, device=DEV)
        self.k, self.v = (torch.zeros((rows, HKV, D), dtype=dtype, device=DEV) for _ in range(2))
        self.o = torch.zeros_like(self.q)
        self.p, self.x = torch.zeros((B, N, V), device=DEV), torch.zeros((B, T), **i32)
        self.qd, self.u = torch.zeros((B, T, V), device=DEV), torch.zeros((B, N), device=DEV)
        self.lin = {n: torch.zeros((B, N, 2, DK), device=DEV) for n in ("q", "k", "v", "log_alpha")}
        self.beta = torch.zeros((B, N, 2), device=DEV)
        self.n_commit = torch.zeros(B, **i32)
        self.tokens = torch.zeros((B, N), **i32)
        self.ol = torch.zeros((B, N, 2, DK), device=DEV)
        self.ws = [torch.empty(max(16, n), dtype=torch.uint8, device=DEV) for n in (
            kda.kda_page_plan_workspace_size(B),
            kda.kda_attn_paged_workspace_size(rows, B, HQ, HKV, D, N, dtype),
            kda.kda_draft_verify_workspace_size(B, T, V))]

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g).to(self.dtype))
        z = 2 * torch.randn((B, N, V), generator=g)
        self.p.copy_(torch.softmax(z, -1))
        q = torch.softmax(z[:, :T] + 0.5 * torch.randn((B, T, V), generator=g), -1)
        self.qd.copy_(q)
        self.x.copy_(torch.multinomial(q.view(-1, V), 1, generator=g).view(B, T).int())
        self.u.copy_(torch.rand((B, N), generator=g))
        for n, t in self.lin.items():
            x = torch.randn(t.shape, generator=g)
            t.copy_(-0.1 * x.abs() if n == "log_alpha" else torch.nn.functional.normalize(x, dim=-1))
        self.beta.copy_(torch.rand(self.beta.shape, generator=g))

    def attend(self):
        kda.kda_page_plan(self.kept, self.new, self.pages, self.table, self.free, self.ring,
                          page_size=PAGE, n_pages_out=self.pages, ring_out=self.ring,
                          cu_new=self.cu, slot_map=self.slots, status=self.status,
                          workspace=self.ws[0])
        kda.kda_cache_append(self.k, self.v, self.slots, self.kc, self.vc)
        kda.kda_attn_paged(self.q, self.kc, self.vc, self.table, self.kept, self.cu, max_new=N,
                           o=self.o, workspace=self.ws[1])

    def decide(self):
        kda.kda_draft_verify(self.p, self.qd, self.x, self.u, n_commit=self.n_commit,
                             tokens=self.tokens, workspace=self.ws[2])
        kda.kda_decode_multi(self.lin["q"], self.lin["k"], self.lin["v"], self.lin["log_alpha"],
                             self.beta, self.S, n_commit=self.n_commit, o=self.ol)
        self.kept.add_(self.n_commit)

    def reference(self, new, kept):
        """o of the new tokens from the dense copies (which are extended)."""
        kc, vc = self.k.cpu(), self.v.cpu()
        at, n = 0, list(new)
        tot = [a + b for a, b in zip(kept, n)]
        have = [-(-t // PAGE) for t in tot]
        c = dict(q=self.q.cpu(), kept=kept, page=PAGE,
                 cu=np.concatenate([[0], np.cumsum(n)]).astype(int).tolist())
        c["kc"] = torch.zeros((sum(have) + 1, HKV, PAGE, D), dtype=self.dtype)
        c["vc"] = torch.zeros_like(c["kc"])
        c["table"] = torch.full((B, max(have) + 1), -1, dtype=torch.int32)
        first = 0
        for i in range(B):
            ks, vs = self.dense[i]
            del ks[kept[i]:], vs[kept[i]:]
            for t in range(n[i]):
                ks.append(kc[at])
                vs.append(vc[at])
                at += 1
            for pos in range(tot[i]):
                c["kc"][first + pos // PAGE, :, pos % PAGE] = ks[pos]
                c["vc"][first + pos // PAGE, :, pos % PAGE] = vs[pos]
            c["table"][i, :have[i]] = torch.arange(first, first + have[i])
            first += have[i]
        return c, R.attn(c)


def _compare(s, c, ref, what):
    T0 = c["cu"][-1]
    ro, _, spread, mag = ref
    keys = max(a + b for a, b in zip(c["kept"], np.diff(c["cu"]).tolist()))
    bound = R.attn_bound(ro[:T0], spread[:T0], mag[:T0], D, keys, s.dtype) + 1e-30
    worst = float(((s.o[:T0].cpu().double() - ro[:T0]).abs() / bound).max())
    print(f"[serve] {what}: worst error / bound {worst:.3f}", flush=True)
    assert worst <= 1.0


def _recurrent(s, S0, commits):
    """fp64 recurrence of the committed tokens."""
    S = S0.double().cpu()
    L = {n: t.double().cpu() for n, t in s.lin.items()}
    beta = s.beta.double().cpu()
    for b, n in enumerate(commits):
        for t in range(n):
            for h in range(2):
                M = S[b, h] * L["log_alpha"][b, t, h].exp()[:, None]
                k = L["k"][b, t, h]
                S[b, h] = M + beta[b, t, h] * torch.outer(k, L["v"][b, t, h] - M.t() @ k)
    return S


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("captured", [False, True])
def test_steps(dtype, captured):
    prompt = [40, 1, 16, 0, 77]
    s = Step(dtype, prompt)
    s.fill(100)
    s.attend()                                       # the prompts
    c, ref = s.reference(prompt, [0] * B)
    _compare(s, c, ref, "prompts")
    s.kept.copy_(s.new)
    s.new.fill_(N)
    whole = None
    if captured:
        # warm up on copies of nothing: two eager calls into the same buffers
        # would advance the state, so the state is put back afterwards
        saved = [t.clone() for t in (s.kept, s.pages, s.ring, s.table, s.free, s.S, s.kc, s.vc)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s.attend()
            s.decide()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        whole = torch.cuda.CUDAGraph()
        with torch.cuda.graph(whole):
            s.attend()
            s.decide()
        for t, x in zip((s.kept, s.pages, s.ring, s.table, s.free, s.S, s.kc, s.vc), saved):
            t.copy_(x)
    for step in range(6):
        s.fill(200 + step)
        kept, S0 = s.kept.tolist(), s.S.clone()
        if captured:
            whole.replay()
            torch.cuda.synchronize()
        else:
            s.attend()
            s.decide()
        assert int(s.status) == 0
        c, ref = s.reference([N] * B, kept)
        _compare(s, c, ref, f"step {step}")
        commits, tokens = R.verify(s.p.cpu(), s.qd.cpu(), s.x.cpu(), s.u.cpu())
        assert s.n_commit.tolist() == commits and s.tokens.tolist() == tokens
        assert s.kept.tolist() == [a + b for a, b in zip(kept, commits)]
        S = _recurrent(s, S0, commits)
        e = float((s.S.double().cpu() - S).norm() / S.norm())
        assert e <= 1e-5, e
        held = [p for r, n in zip(s.table.tolist(), s.pages.tolist()) for p in r[:n]]
        head, count = s.ring.tolist()
        free = [s.free.tolist()[(head + j) % POOL] for j in range(count)]
        assert sorted(held + free) == list(range(POOL))


def test_empty_step_after_a_shortage():
    # a plan that cannot be met leaves offsets of 0 and slots of -1: the calls
    # behind it do nothing
    s = Step(torch.bfloat16, [40, 1, 16, 0, 77])
    s.fill(1)
    s.ring.copy_(ints([0, 3]))
    s.o.fill_(5.0)
    s.attend()
    assert int(s.status) > 0
    assert bool((s.o == 5.0).all()) and bool(torch.isnan(s.kc.float()).all())
    assert s.ring.tolist() == [0, 3] and s.pages.tolist() == [0] * B


def test_prefill_takes_the_plans_offsets():
    # cu_new is kda_prefill_varlen's cu_seqlens
    import oracle
    import workloads as W
    n = [70, 0, 3, 130]
    x = W.varlen_inputs(W.PREFILL_CONFIGS["batched"], n, H=2, seed=5)
    cu, *_ = kda.kda_page_plan(ints([0] * 4), ints(n), ints([0] * 4), ints([[-1] * 9] * 4),
                               ints(list(range(40))), ints([0, 40]), page_size=16, n_slots=sum(n))
    xd = {k: (t.to(DEV) if t is not None else None) for k, t in x.items()}
    assert torch.equal(cu.cpu(), x["cu_seqlens"].cpu().int())
    o, S, _ = kda.kda_prefill_varlen(xd["q"], xd["k"], xd["v"], xd["log_alpha"], xd["beta"], cu,
                                     xd["S0"])
    ro, rS, _ = oracle.prefill_varlen_f64(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"],
                                          x["cu_seqlens"], x["S0"])
    assert oracle.rel_l2(o.cpu(), ro) <= 2e-2 and oracle.rel_l2(S.cpu(), rS) <= 2e-2
