"""kda_page_plan against the sequential form: exact integers."""
import random

import pytest
import torch

import gated_delta_rule_22_amd as kda
import serve_ref as R
from serve_ref import DEV, ints

pytestmark = pytest.mark.gpu


def make(seed, B, page, new_hi, kept_hi, *, gone=0.1, width_extra=2, spare=7):
    """Requests that hold the pages of an earlier length; some shrink, some end."""
    rng = random.Random(seed)
    had = [rng.randint(0, kept_hi) for _ in range(B)]
    kept = [0 if rng.random() < gone else max(0, h - rng.randint(0, 2 * page)) for h in had]
    new = [0 if rng.random() < 0.2 else rng.randint(0, new_hi) for _ in range(B)]
    pages = [-(-h // page) for h in had]
    need = [-(-(a + b) // page) for a, b in zip(kept, new)]
    width = max(pages + need + [0]) + width_extra
    take = sum(max(0, n - p) for n, p in zip(need, pages))
    pool = sum(pages) + take + spare
    ids = list(range(pool))
    rng.shuffle(ids)
    table, at = [], 0
    for p in pages:
        table.append(ids[at:at + p] + [-7] * (width - p))
        at += p
    head = rng.randrange(pool) if pool else 0
    ring = [-9] * pool
    for j, f in enumerate(ids[at:]):
        ring[(head + j) % pool] = f
    return dict(kept=kept, new=new, pages=pages, table=table, ring=ring,
                ring_state=[head, pool - at], page=page, slots=sum(new) + rng.randint(0, 5))


def call(c, *, in_place=False, **kw):
    B = len(c["kept"])
    table = ints(c["table"]).view(B, len(c["table"][0]) if B else 0)
    ring, pages, state = ints(c["ring"]), ints(c["pages"]), ints(c["ring_state"])
    if in_place:
        kw.update(n_pages_out=pages, ring_out=state)
    cu, slot, pages_out, state_out, status = kda.kda_page_plan(
        ints(c["kept"]), ints(c["new"]), pages, table, ring, state, page_size=c["page"],
        n_slots=c["slots"], **kw)
    torch.cuda.synchronize()
    return dict(table=table.tolist(), ring=ring.tolist(), pages=pages_out.tolist(),
                ring_state=state_out.tolist(), cu=cu.tolist(), slot=slot.tolist(),
                status=int(status))


def check(c, **kw):
    want = R.plan(c["kept"], c["new"], c["pages"], c["table"], c["ring"], c["ring_state"],
                  c["page"], c["slots"])
    got = call(c, **kw)
    for k in want:
        assert got[k] == want[k], k
    return want


@pytest.mark.parametrize("B,page,new_hi,kept_hi", [
    (1, 16, 1, 40), (1, 64, 5000, 0), (3, 16, 33, 100), (17, 1024, 2500, 5000), (64, 64, 8, 3000),
    (256, 64, 8, 2000), (257, 32, 100, 500), (1023, 16, 3, 200), (1024, 16, 40, 64),
    (1025, 128, 9, 300), (2500, 16, 5, 90)])
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_sequential(B, page, new_hi, kept_hi, in_place):
    c = make(B + page, B, page, new_hi, kept_hi)
    assert check(c, in_place=in_place)["status"] == 0


@pytest.mark.parametrize("slots", [4095, 4096, 4097, 70000])
def test_slot_counts_around_the_launch_shapes(slots):
    c = make(slots, 40, 16, 100, 600)
    c["slots"] = slots
    assert check(c)["status"] == 0


def test_no_requests_and_no_tokens():
    c = dict(kept=[], new=[], pages=[], table=[], ring=[3, 1], ring_state=[1, 1], page=16, slots=4)
    assert check(c)["slot"] == [-1] * 4
    c = dict(kept=[0, 0], new=[0, 0], pages=[0, 0], table=[[], []], ring=[], ring_state=[0, 0],
             page=16, slots=0)
    assert check(c)["status"] == 0
    c = make(5, 9, 16, 0, 100)          # releases only
    assert check(c)["cu"] == [0] * 10


def test_ring_wraps_and_fills():
    # the whole pool is given back, then taken again, across the ring's end
    c = dict(kept=[0, 0], new=[0, 0], pages=[3, 2], table=[[4, 2, 0], [1, 3, -1]], ring=[-1] * 5,
             ring_state=[3, 0], page=16, slots=0)
    w = check(c)
    assert w["ring"] == [0, 1, 3, 4, 2] and w["ring_state"] == [3, 5]
    c = dict(kept=[0, 0], new=[33, 17], pages=[0, 0], table=[[-1] * 3, [-1] * 3], ring=w["ring"],
             ring_state=w["ring_state"], page=16, slots=60)
    assert check(c)["ring_state"] == [3, 0]


@pytest.mark.parametrize("change,status", [
    (dict(kept=(0, -1)), -1), (dict(new=(3, -5)), -1), (dict(pages=(1, -1)), -1),
    (dict(pages=(1, 10**6)), -1), (dict(kept=(2, 10**9)), -1), (dict(new=(0, 2**31 - 1)), -1),
    (dict(ring_state=(0, -1)), -1), (dict(ring_state=(1, 10**9)), -1),
    (dict(ring_state=(0, -2**31)), -1)])
def test_bad_values_leave_an_empty_step(change, status):
    c = make(11, 20, 16, 30, 200)
    for k, (i, v) in change.items():
        c[k] = list(c[k])
        c[k][i] = v
    for in_place in (False, True):
        assert check(c, in_place=in_place)["status"] == status


def test_shortage_and_too_few_slots():
    c = make(12, 20, 16, 300, 200, gone=0.0, spare=0)
    taken = c["ring_state"][1]
    c["ring_state"] = [c["ring_state"][0], taken - 4]
    assert check(c)["status"] > 0
    c = make(13, 20, 16, 30, 200)
    c["slots"] = sum(c["new"]) - 1
    assert check(c)["status"] == -2


def test_other_stream_and_repeat():
    c = make(14, 100, 16, 200, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check(c, stream=side)
    check(c, stream=side)
    # the same inputs again, on the arrays the first call wrote to: the same outputs
    table, ring = ints(c["table"]), ints(c["ring"])
    args = (ints(c["kept"]), ints(c["new"]), ints(c["pages"]), table, ring, ints(c["ring_state"]))
    first = [t.clone() for t in kda.kda_page_plan(*args, page_size=16, n_slots=c["slots"])]
    t1, r1 = table.clone(), ring.clone()
    again = kda.kda_page_plan(*args, page_size=16, n_slots=c["slots"])
    assert all(torch.equal(x, y) for x, y in zip(first, again))
    assert torch.equal(t1, table) and torch.equal(r1, ring)


def test_random_steps_never_share_a_page():
    rng = random.Random(3)
    B, page, pool, width = 12, 16, 200, 30
    ring, state = ints(list(range(pool))), ints([0, pool])
    table, pages = ints([[-1] * width] * B), ints([0] * B)
    kept = [0] * B
    for _ in range(40):
        new = [rng.randint(0, 40) if k < 300 else 0 for k in kept]
        kept = [0 if rng.random() < 0.05 else k for k in kept]
        cu, slot, _, _, status = kda.kda_page_plan(
            ints(kept), ints(new), pages, table, ring, state, page_size=page, n_slots=600,
            n_pages_out=pages, ring_out=state)
        held = [p for r, n in zip(table.tolist(), pages.tolist()) for p in r[:n]]
        head, count = state.tolist()
        free = [ring.tolist()[(head + j) % pool] for j in range(count)]
        assert int(status) == 0
        assert sorted(held + free) == list(range(pool))
        s = slot.tolist()
        assert len(set(s[:sum(new)])) == sum(new) and set(s[sum(new):]) <= {-1}
        kept = [max(0, k + n - rng.randint(0, 9)) for k, n in zip(kept, new)]


def test_refuses_wrong_arguments():
    c = make(15, 4, 16, 30, 90)
    a = [ints(c[k]) for k in ("kept", "new", "pages", "table", "ring", "ring_state")]
    with pytest.raises(ValueError, match="n_slots"):
        kda.kda_page_plan(*a, page_size=16)
    with pytest.raises(kda.KDAError):
        kda.kda_page_plan(*a, page_size=24, n_slots=4)
    for i in range(6):
        b = list(a)
        b[i] = b[i].long()
        with pytest.raises(ValueError):
            kda.kda_page_plan(*b, page_size=16, n_slots=4)
        b[i] = a[i][..., ::2]
        with pytest.raises(ValueError):
            kda.kda_page_plan(*b, page_size=16, n_slots=4)
    with pytest.raises(kda.KDAError):       # an output over an input
        kda.kda_page_plan(*a, page_size=16, slot_map=a[1])


def test_page_ids_outside_the_pool_give_no_slot():
    c = dict(kept=[60, 0], new=[10, 3], pages=[2, 0], table=[[0, 2**26, 0], [0, 0, 0]],
             ring=[5, -3, 2**31 - 1, 1, 0, 2], ring_state=[0, 3], page=64, slots=25)
    got = call(c)
    assert got["status"] == 0
    # page 0 of request 0 is valid, its second is no page; request 1 takes page 5
    assert got["slot"][:4] == [60, 61, 62, 63] and set(got["slot"][4:10]) == {-1}
    assert got["slot"][10:13] == [320, 321, 322]


def test_many_pages_move_in_a_small_step():
    # few slots, thousands of pages given back and taken
    c = make(31, 300, 16, 2, 6000, gone=0.5)
    c["slots"] = max(c["slots"], sum(c["new"]))
    assert check(c, in_place=True)["status"] == 0


@pytest.mark.parametrize("gone", [0.0, 0.6])
def test_many_pages_over_wide_tables(gone):
    # more table entries than one workgroup takes, whatever the slots
    c = make(33, 700, 16, 3, 4000, gone=gone, spare=400)
    assert 700 * len(c["table"][0]) > 1 << 17 and sum(c["new"]) < 4096
    assert check(c, in_place=True)["status"] == 0
    assert check(c)["status"] == 0
