"""Serving C ABI without a GPU: declared symbols are exported, and every bad
argument is rejected on the host before any launch."""
import ctypes
import os
import re

import pytest
import torch

import gated_delta_rule_22_amd as kda

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
I31 = 2**31 - 1


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(kda.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return kda.load_library()


# made-up, well spaced device addresses: only where no GPU is visible, so that
# a call that wrongly passes the checks fails to launch instead of touching them
BASE = 1 << 40
no_gpu = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                            reason="fake device addresses: run only where no GPU is visible")


def P(i, off=0):
    return ctypes.c_void_p(BASE + (i << 36) + off)


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "kda_serve.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    syms = set(re.findall(r"\b(kda_[a-z0-9_]+)\s*\(", text))
    assert syms == {"kda_page_plan_workspace_size", "kda_page_plan", "kda_cache_append",
                    "kda_attn_paged_workspace_size", "kda_attn_paged",
                    "kda_draft_verify_workspace_size", "kda_draft_verify"}
    for s in syms:
        assert hasattr(lib, s) and s in kda.__all__, s


def plan(lib, **kw):
    a = dict(kept=P(0), new=P(1), pin=P(2), pout=P(3), table=P(4), ring=P(5), rin=P(6), rout=P(7),
             cu=P(8), slot=P(9), status=P(10), B=8, width=16, page=64, pool=100, slots=50,
             ws=P(11), wsz=1 << 20)
    a.update(kw)
    return lib.kda_page_plan(*[a[k] for k in ("kept", "new", "pin", "pout", "table", "ring", "rin",
                                              "rout", "cu", "slot", "status", "B", "width", "page",
                                              "pool", "slots", "ws", "wsz")], None)


@no_gpu
def test_plan_rejects(lib):
    for name in ("B", "width", "pool", "slots"):
        assert plan(lib, **{name: -1}) == INVALID, name
    for page in (0, 8, 48, 2048, -64):
        assert plan(lib, page=page) == UNSUPPORTED, page
    assert plan(lib, pool=1 << 25, page=64) == INVALID          # slots past int32
    for name in ("kept", "new", "pin", "pout", "table", "ring", "rin", "rout", "cu", "slot",
                 "status"):
        assert plan(lib, **{name: None}) == INVALID, name
        assert plan(lib, **{name: P(12, 2)}) == INVALID, name   # misaligned
    assert plan(lib, ws=None) == WORKSPACE
    assert plan(lib, wsz=kda.kda_page_plan_workspace_size(8) - 1) == WORKSPACE
    assert plan(lib, pout=P(2, 4)) == INVALID                   # partly over n_pages_in
    assert plan(lib, rout=P(6, 4)) == INVALID
    assert plan(lib, slot=P(0, 4)) == INVALID
    assert plan(lib, cu=P(9)) == INVALID                        # two outputs
    assert plan(lib, table=P(5, 8)) == INVALID
    assert plan(lib, ws=P(4, 16)) == INVALID
    assert plan(lib, B=I31, width=I31) != OK


def append(lib, **kw):
    a = dict(k=P(0), v=P(1), slot=P(2), kc=P(3), vc=P(4), T=8, H=2, d=64, page=64, pool=10, dt=1)
    a.update(kw)
    return lib.kda_cache_append(*[a[k] for k in ("k", "v", "slot", "kc", "vc", "T", "H", "d",
                                                 "page", "pool", "dt")], None)


@no_gpu
def test_append_rejects(lib):
    for name in ("T", "H", "pool"):
        assert append(lib, **{name: -1}) == INVALID, name
        assert append(lib, **{name: 0}) == OK, name             # nothing to do
    for kw in (dict(d=48), dict(d=256), dict(page=24), dict(dt=5)):
        assert append(lib, **kw) == UNSUPPORTED, kw
    for name in ("k", "v", "kc", "vc"):
        assert append(lib, **{name: None}) == INVALID, name
        assert append(lib, **{name: P(7, 8)}) == INVALID, name
    assert append(lib, slot=None) == INVALID
    assert append(lib, slot=P(7, 2)) == INVALID
    assert append(lib, kc=P(0, 256)) == INVALID
    assert append(lib, vc=P(3, 1024)) == INVALID
    assert append(lib, kc=P(2)) == INVALID
    assert append(lib, T=I31, H=I31) == INVALID


def attn(lib, **kw):
    a = dict(q=P(0), kc=P(1), vc=P(2), table=P(3), kept=P(4), cu=P(5), o=P(6), lse=P(7), T=40, B=4,
             Hq=8, Hkv=2, d=64, page=64, pool=100, width=16, max_new=0, scale=0.0, dt=1, ws=P(8),
             wsz=1 << 34)
    a.update(kw)
    return lib.kda_attn_paged(*[a[k] for k in ("q", "kc", "vc", "table", "kept", "cu", "o", "lse",
                                               "T", "B", "Hq", "Hkv", "d", "page", "pool", "width",
                                               "max_new", "scale", "dt", "ws", "wsz")], None)


@no_gpu
def test_attn_rejects(lib):
    for name in ("T", "B", "Hq", "Hkv", "pool", "width", "max_new"):
        assert attn(lib, **{name: -1}) == INVALID, name
    for name in ("T", "B", "Hq"):
        assert attn(lib, **{name: 0}) == OK, name
    assert attn(lib, Hkv=0) == INVALID
    assert attn(lib, Hkv=3) == INVALID                          # Hq not a multiple
    for kw in (dict(d=96), dict(page=8), dict(dt=2)):
        assert attn(lib, **kw) == UNSUPPORTED, kw
    for s in (-1.0, float("nan"), float("inf")):
        assert attn(lib, scale=s) == INVALID, s
    for name in ("q", "kc", "vc", "table", "kept", "cu", "o"):
        assert attn(lib, **{name: None}) == INVALID, name
    for name in ("q", "kc", "vc", "o"):
        assert attn(lib, **{name: P(9, 8)}) == INVALID, name
    for name in ("table", "kept", "cu", "lse"):
        assert attn(lib, **{name: P(9, 2)}) == INVALID, name
    need = kda.kda_attn_paged_workspace_size(40, 4, 8, 2, 64, 0, torch.bfloat16)
    if need:
        assert attn(lib, ws=None) == WORKSPACE
        assert attn(lib, wsz=need - 1) == WORKSPACE
        assert attn(lib, ws=P(8, 8)) == INVALID
        assert attn(lib, ws=P(1, 256)) == INVALID
    assert attn(lib, o=P(0)) == INVALID                         # in place
    assert attn(lib, o=P(1, 4096)) == INVALID
    assert attn(lib, lse=P(6, 16)) == INVALID
    assert attn(lib, T=I31) == INVALID                          # query rows past 32 bits
    assert attn(lib, width=1 << 26) == INVALID                  # positions past 32 bits


def verify(lib, **kw):
    a = dict(p=P(0), q=P(1), x=P(2), u=P(3), n=P(4), c=P(5), tok=P(6), B=4, T=7, V=1001, dt=0,
             ws=P(7), wsz=1 << 34)
    a.update(kw)
    return lib.kda_draft_verify(*[a[k] for k in ("p", "q", "x", "u", "n", "c", "tok", "B", "T",
                                                 "V", "dt", "ws", "wsz")], None)


@no_gpu
def test_verify_rejects(lib):
    for name in ("B", "T", "V"):
        assert verify(lib, **{name: -1}) == INVALID, name
    assert verify(lib, B=0) == OK
    assert verify(lib, V=0) == INVALID
    assert verify(lib, dt=4) == UNSUPPORTED
    for name in ("p", "x", "u", "c", "tok"):
        assert verify(lib, **{name: None}) == INVALID, name
    for name in ("p", "q"):
        assert verify(lib, **{name: P(9, 4)}) == INVALID, name
    for name in ("x", "u", "n", "c", "tok"):
        assert verify(lib, **{name: P(9, 2)}) == INVALID, name
    need = kda.kda_draft_verify_workspace_size(4, 7, 1001)
    if need:
        assert verify(lib, ws=None) == WORKSPACE
        assert verify(lib, wsz=need - 1) == WORKSPACE
        assert verify(lib, ws=P(7, 8)) == INVALID
        assert verify(lib, ws=P(1, 256)) == INVALID
    assert verify(lib, tok=P(2)) == INVALID
    assert verify(lib, c=P(6, 8)) == INVALID
    assert verify(lib, B=I31, T=I31, V=I31) == INVALID
    assert verify(lib, T=I31) == INVALID


def test_workspace_queries_refuse(lib):
    bf = torch.bfloat16
    for args in ((0, 1, 8, 2, 64, 0), (8, 0, 8, 2, 64, 0), (8, 1, 8, 3, 64, 0), (8, 1, 8, 0, 64, 0),
                 (8, 1, 8, 2, 48, 0), (8, 1, 8, 2, 64, -1), (-4, 1, 8, 2, 64, 0),
                 (I31, I31, I31, 1, 128, 0)):
        assert kda.kda_attn_paged_workspace_size(*args, bf) == 0, args
    assert kda.kda_draft_verify_workspace_size(-1, 7, 100) == 0
    assert kda.kda_draft_verify_workspace_size(4, -1, 100) == 0
    assert kda.kda_draft_verify_workspace_size(4, 7, 0) == 0
    assert kda.kda_page_plan_workspace_size(-1) == 0


def test_binding_refuses_host_tensors():
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 2, 64))
    c = torch.zeros((3, 2, 16, 64))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_page_plan(i, i, i, i.view(1, 4), i, i[:2], page_size=16, n_slots=3)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_cache_append(x, x, i, c, c)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_attn_paged(x, c, c, i.view(4, 1), i, i)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_draft_verify(x, x, i.view(4, 1), x[..., 0])
