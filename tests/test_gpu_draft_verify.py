"""kda_draft_verify against the plain 64-bit form: exact integers."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV

pytestmark = pytest.mark.gpu


def make(B, T, V, dtype, with_q, seed, noise=0.4, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    z = sharp * torch.randn((B, T + 1, V), generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z[:, :T] + noise * torch.randn((B, T, V), generator=g), -1)
    src = (q if with_q else p[:, :T]).reshape(B * T, V)
    x = torch.multinomial(src, 1, generator=g).view(B, T).to(torch.int32) if T else \
        torch.zeros((B, 0), dtype=torch.int32)
    u = torch.rand((B, T + 1), generator=g)
    return p.to(dtype), (q.to(dtype) if with_q else None), x, u


def call(p, q, x, u, n_draft=None, **kw):
    c, t = kda.kda_draft_verify(p.to(DEV), None if q is None else q.to(DEV), x.to(DEV), u.to(DEV),
                                n_draft=None if n_draft is None else R.ints(n_draft), **kw)
    torch.cuda.synchronize()
    return c.tolist(), t.tolist()


def check(p, q, x, u, n_draft=None):
    want, got = R.verify(p, q, x, u, n_draft), call(p, q, x, u, n_draft)
    assert got[0] == want[0]
    assert got[1] == want[1]
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("B,T,V", [
    (1, 1, 1), (1, 3, 2), (5, 7, 17), (3, 7, 255), (16, 4, 257), (2, 7, 4095), (2, 3, 4097),
    (64, 7, 1000), (1, 5, 32003), (3, 2, 131072), (300, 1, 63), (1, 7, 262147)])
def test_matches_plain(B, T, V, with_q, dtype):
    check(*make(B, T, V, dtype, with_q, B + T + V))


def test_every_position_is_reached():
    p, q, x, u = make(400, 7, 50, torch.float32, True, 5, noise=0.7)
    want, _ = check(p, q, x, u)
    assert set(want) == set(range(1, 9))


@pytest.mark.parametrize("V", [64, 1000, 5000])
def test_ragged_drafts_and_unused_rows(V):
    p, q, x, u = make(12, 5, V, torch.float32, True, 6)
    n = [5, 0, -1, 3, 9, 1, 2, -2**31, 4, 5, 0, 2**31 - 1]
    check(p, q, x, u, n)
    check(p, None, x, u, n)


@pytest.mark.parametrize("V", [9, 4100, 20000])
def test_no_draft_samples_the_target(V):
    p, _, x, u = make(6, 0, V, torch.float32, False, 7)
    want, tok = check(p, None, x, u)
    assert want == [1] * 6
    check(p, torch.empty((6, 0, V)), x, u)


@pytest.mark.parametrize("V", [8, 64, 4096, 16384])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_borders_of_equal_steps(V, dtype):
    # p = 1 / V: every partial sum and u V are exact, and u on a border
    # belongs to the next token
    ks = [0, 1, V // 2 - 1, V // 2, V - 1]
    p = torch.full((len(ks), 1, V), 1.0 / V).to(dtype)
    u = torch.tensor([[k / V] for k in ks])
    x = torch.zeros((len(ks), 0), dtype=torch.int32)
    _, tok = check(p, None, x, u)
    assert [t[0] for t in tok] == ks


def test_acceptance_border_is_strict():
    # u q < p exactly: u q = p rejects; q = 0 keeps any token the target gives
    V = 8
    p = torch.zeros((4, 2, V))
    q = torch.zeros((4, 1, V))
    p[:, :, 5] = 0.5
    p[:, 0, 3] = torch.tensor([0.25, 0.25, 0.0, 0.25])
    q[:, 0, 3] = torch.tensor([0.5, 0.5, 0.0, 0.0])
    x = torch.full((4, 1), 3, dtype=torch.int32)
    u = torch.tensor([[0.5, 0.1], [0.4999, 0.1], [0.0, 0.1], [0.9999, 0.1]])
    want, tok = check(p, q, x, u)
    assert want == [1, 2, 1, 2]
    assert tok[0] == [5, -1]            # r = max(p - q, 0) has 5 alone


@pytest.mark.parametrize("V", [33, 9000])
def test_equal_distributions_and_empty_rest(V):
    # p = q: nothing is left of max(p - q, 0), so the target itself is drawn from
    p, _, x, u = make(20, 2, V, torch.float32, True, 8)
    q = p[:, :2].clone()
    x[:10] = -1                         # outside the vocabulary: rejected
    x[10:15, 0] = V
    u[15:] = 0.999999
    check(p, q, x, u)


@pytest.mark.parametrize("V", [70, 8200])
def test_extremes(V):
    p, q, x, u = make(9, 3, V, torch.float32, True, 9)
    p[0] = 0                            # no mass at all
    p[1, :, 3:] = 0                     # most of a row empty
    p[2, :, ::2] = float("nan")
    p[3, :, V // 2] = float("inf")
    p[4] = -p[4]
    u[5, 3] = 1.0                       # past the last border
    u[6, 3] = 0.0
    q[7] = 1e-38
    p[8] *= 1e-30
    for n in (None, [0] * 9):
        check(p, q, x, u, n)
        check(p, None, x, u, n)


def test_repeats_streams_and_workspace():
    p, q, x, u = make(40, 7, 30011, torch.float32, True, 10)
    want = check(p, q, x, u)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert call(p, q, x, u, stream=side) == want
    small = torch.empty(3, dtype=torch.uint8, device=DEV)
    assert call(p, q, x, u, workspace=small) == want      # too small: a larger one is made
    with pytest.raises(ValueError):
        call(p, q, x, u, workspace=small.cpu())


def test_rows_past_32_bit_offsets():
    # 2^32 elements of probabilities; only the rows that decide are filled
    B, T, V = 2, 7, (1 << 28) + 5
    p = torch.empty((B, T + 1, V), dtype=torch.bfloat16, device=DEV)
    x = torch.full((B, T), V - 2, dtype=torch.int32)
    for t in range(T + 1):
        p[:, t, V - 2] = 0.75
    p[:, T] = 0
    p[:, T, V - 3] = 0.25
    p[:, T, V - 2] = 0.75
    u = torch.full((B, T + 1), 0.5)
    u[1, T] = 0.125
    c, tok = kda.kda_draft_verify(p, None, x.to(DEV), u.to(DEV))
    assert c.tolist() == [8, 8]
    assert tok[:, T].tolist() == [V - 2, V - 3]


def test_refusals():
    p, q, x, u = (t.to(DEV) for t in make(3, 2, 40, torch.float32, True, 11))
    for bad in ((p, q.bfloat16(), x, u), (p[:, :2], q, x, u), (p, q[..., :39], x, u),
                (p, q, x.long(), u), (p, q, x[:2], u), (p, q, x, u[:, :2]), (p, q, x, u.double()),
                (p.half(), None, x, u), (p[..., :20], None, x, u), (p, q, x.cpu(), u)):
        with pytest.raises(ValueError):
            kda.kda_draft_verify(*bad)
    with pytest.raises(ValueError):
        kda.kda_draft_verify(p, q, x, u, n_draft=R.ints([1, 2]))
    with pytest.raises(kda.KDAError):
        kda.kda_draft_verify(p, q, x, u, n_commit=x.view(-1)[:3])
