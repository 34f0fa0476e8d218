"""Sizes that a 32-bit argument would cut are refused, not cut."""
import pytest
import torch

import gated_delta_rule_22_amd as kda
from full_ref import BF, DEV, ints

pytestmark = pytest.mark.gpu
MANY = (1 << 32) + 1          # one, in 32 bits


@pytest.fixture(scope="module")
def many():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    x = torch.zeros(2 * (MANY + 1), dtype=torch.int32, device=DEV)
    yield x
    del x
    torch.cuda.empty_cache()


def test_requests_and_positions(many):
    kept, cu, table = many[:MANY], many[MANY:2 * MANY + 1], many[:MANY].view(MANY, 1)
    wide = many[:MANY].view(1, MANY)
    q = torch.zeros((4, 2, 64), dtype=BF, device=DEV)
    k = torch.zeros((4, 1, 64), dtype=BF, device=DEV)
    kc, vc = (torch.zeros((2, 1, 16, 64), dtype=BF, device=DEV) for _ in range(2))
    slots, one, two = ints([0, 1, 2, 3]), ints([0]), ints([0, 4])
    rope = kda.KDARope(torch.ones(32, dtype=torch.float64, device=DEV))
    with pytest.raises(ValueError):
        kda.kda_rope_append(q, k, k.clone(), slots, kept, cu, kc, vc, rope)
    kv, cache = torch.zeros((4, 192), dtype=BF, device=DEV), torch.zeros((2, 16, 192), dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        kda.kda_latent_append(kv, slots, kept, cu, cache)
    ql = torch.zeros((4, 2, 192), dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        kda.kda_attn_latent(ql, cache, table, kept, cu, dc=128, scale=0.1)
    with pytest.raises(ValueError):
        kda.kda_attn_latent(ql, cache, wide, one, two, dc=128, scale=0.1)
    qe, kve = torch.zeros((4, 2, 128), dtype=BF, device=DEV), torch.zeros((4, 2, 128), dtype=BF, device=DEV)
    pe = torch.zeros((4, 64), dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        kda.kda_attn_expanded(qe, kve, pe, cu, cu, dv=64)
    for t in (kc, vc, cache):
        assert not t.any()
    with pytest.raises(ValueError):
        kda.kda_attn_paged(q, kc, vc, table, kept, cu)
    with pytest.raises(ValueError):
        kda.kda_attn_paged(q, kc, vc, wide, one, two)


def test_plan_and_vocabulary(many):
    kept, wide = many[:MANY], many[:MANY].view(1, MANY)
    table, ring, state, one = ints([[0, 1]]), ints([0, 1]), ints([0, 2]), ints([0])
    for bad in (dict(n=kept, table=many[:MANY].view(MANY, 1)), dict(table=wide), dict(ring=kept),
                dict(n_slots=MANY)):
        n = bad.get("n", one)
        with pytest.raises(ValueError):
            kda.kda_page_plan(n, n, n, bad.get("table", table), bad.get("ring", ring), state, page_size=16,
                              n_slots=bad.get("n_slots", 4))
    p = many.view(BF)[:MANY].view(1, 1, MANY)
    with pytest.raises(ValueError):
        kda.kda_draft_verify(p, None, torch.zeros((1, 0), dtype=torch.int32, device=DEV),
                             torch.zeros((1, 1), device=DEV))


def test_sequences(many):
    q, k, v = (torch.zeros((64, 1, 16), dtype=BF, device=DEV) for _ in range(3))
    gate, beta = torch.zeros((64, 1, 16), device=DEV), torch.zeros((64, 1), device=DEV)
    with pytest.raises(ValueError):
        kda.kda_prefill_varlen(q, k, v, gate, beta, many[:MANY + 1], want_state=False)


def test_tokens(many):
    # rows of no heads take no memory, and a slot each
    slots = many[:MANY]
    none = torch.zeros((MANY, 0, 64), dtype=BF, device=DEV)
    pool = torch.zeros((2, 0, 16, 64), dtype=BF, device=DEV)
    rope = kda.KDARope(torch.ones(32, dtype=torch.float64, device=DEV))
    with pytest.raises(ValueError):
        kda.kda_rope_append(none, none, none, slots, ints([0]), ints([0, 1]), pool, pool, rope)
    with pytest.raises(ValueError):
        kda.kda_cache_append(none, none, slots, pool, pool)
