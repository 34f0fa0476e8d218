"""Binding of the serving step's calls (``include/kda_serve.h``).

Like the rest of the package this only marshals arguments: devices, dtypes,
shapes and contiguity are checked, outputs and workspaces the caller leaves
out are allocated with torch, and the HIP kernels behind the library do the
work. Page plan, cache append, paged attention and draft verification run in
this order in a step; the verification's ``n_commit`` is the one that
``kda_decode_multi`` takes.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

import gated_delta_rule_22_amd as _kda

KDA_PLAN_OK, KDA_PLAN_INVALID, KDA_PLAN_NO_SLOTS = 0, -1, -2


def declare(lib) -> None:
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.kda_page_plan_workspace_size.argtypes = [i]
    lib.kda_page_plan_workspace_size.restype = sz
    lib.kda_page_plan.argtypes = [vp] * 11 + [i] * 5 + [vp, sz, vp]
    lib.kda_page_plan.restype = i
    lib.kda_cache_append.argtypes = [vp] * 5 + [i] * 6 + [vp]
    lib.kda_cache_append.restype = i
    lib.kda_attn_paged_workspace_size.argtypes = [i] * 7
    lib.kda_attn_paged_workspace_size.restype = sz
    lib.kda_attn_paged.argtypes = [vp] * 8 + [i] * 9 + [f, i, vp, sz, vp]
    lib.kda_attn_paged.restype = i
    lib.kda_draft_verify_workspace_size.argtypes = [i] * 3
    lib.kda_draft_verify_workspace_size.restype = sz
    lib.kda_draft_verify.argtypes = [vp] * 7 + [i] * 4 + [vp, sz, vp]
    lib.kda_draft_verify.restype = i


# A serving step makes these calls once per layer: the checks below cost about
# 0.3 us a tensor where the package's general one (which words the refusal)
# takes 1 us, and a call on the current device needs no device switch.

def _device(t: torch.Tensor, what: str) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{what} needs GPU tensors")
    return dev


def _dtype(t: torch.Tensor) -> torch.dtype:
    if t.dtype not in _kda._DTYPES:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return t.dtype


def _dims(t: torch.Tensor, name: str, n: int):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {n} dimensions")
    return shape


def _ptr(t: torch.Tensor, name: str, shape, dtype, dev) -> int:
    """The address of a tensor that is as it has to be."""
    if t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        _kda._check(t, name, shape, dtype, dev)
    return t.data_ptr()


def _out(t: Optional[torch.Tensor], shape, dtype, dev, stream) -> torch.Tensor:
    """The caller's output, or a new one."""
    return _kda._empty(shape, dtype, dev, stream) if t is None else t


def _workspace(ws: Optional[torch.Tensor], need: int, dev, stream):
    """(workspace or None, its address, its bytes): the caller's if it is large enough."""
    if ws is not None:
        if ws.device != dev:
            raise ValueError(f"workspace is on {ws.device}, expected {dev}")
        if not ws.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if ws.nbytes >= need:
            return ws, ws.data_ptr(), ws.nbytes
    if not need:
        return None, None, 0
    ws = _kda._empty((need,), torch.uint8, dev, stream)
    return ws, ws.data_ptr(), need


def _call(name: str, dev, stream, *args) -> None:
    fn = getattr(_kda.load_library(), name)
    raw = torch._C._cuda_getCurrentRawStream(dev.index) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != 0:
        raise _kda.KDAError(st, name)


@functools.lru_cache(maxsize=256)
def kda_page_plan_workspace_size(B: int) -> int:
    return int(_kda.load_library().kda_page_plan_workspace_size(B))


def kda_page_plan(kept_len: torch.Tensor, n_new: torch.Tensor, n_pages: torch.Tensor,
                  block_table: torch.Tensor, free_ring: torch.Tensor, ring: torch.Tensor, *,
                  page_size: int, n_slots: Optional[int] = None,
                  n_pages_out: Optional[torch.Tensor] = None,
                  ring_out: Optional[torch.Tensor] = None,
                  cu_new: Optional[torch.Tensor] = None,
                  slot_map: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Pages and slots of a step's new tokens. kept_len, n_new, n_pages [B];
    block_table [B,max_pages] and free_ring [n_pool], both updated in place;
    ring [2] = (head, count); all int32 on the device. The slot map has
    n_slots rows (at least the new tokens; or pass slot_map). n_pages_out and
    ring_out may be n_pages and ring themselves. Returns (cu_new [B+1],
    slot_map, n_pages_out, ring_out, status [1]); a status other than
    KDA_PLAN_OK stays on the device, and makes the step an empty one."""
    dev = _device(kept_len, "kda_page_plan")
    i32 = torch.int32
    B, = _dims(kept_len, "kept_len", 1)
    _, width = _dims(block_table, "block_table", 2)
    pool, = _dims(free_ring, "free_ring", 1)
    if slot_map is None and n_slots is None:
        raise ValueError("kda_page_plan needs n_slots or slot_map")
    if n_slots is None:
        n_slots, = _dims(slot_map, "slot_map", 1)
    n_pages_out = _out(n_pages_out, (B,), i32, dev, stream)
    ring_out = _out(ring_out, (2,), i32, dev, stream)
    cu_new = _out(cu_new, (B + 1,), i32, dev, stream)
    slot_map = _out(slot_map, (n_slots,), i32, dev, stream)
    status = _out(status, (1,), i32, dev, stream)
    ws, wsp, wsz = _workspace(workspace, kda_page_plan_workspace_size(B), dev, stream)
    _call("kda_page_plan", dev, stream, _ptr(kept_len, "kept_len", (B,), i32, dev),
          _ptr(n_new, "n_new", (B,), i32, dev), _ptr(n_pages, "n_pages", (B,), i32, dev),
          _ptr(n_pages_out, "n_pages_out", (B,), i32, dev),
          _ptr(block_table, "block_table", (B, width), i32, dev),
          _ptr(free_ring, "free_ring", (pool,), i32, dev), _ptr(ring, "ring", (2,), i32, dev),
          _ptr(ring_out, "ring_out", (2,), i32, dev), _ptr(cu_new, "cu_new", (B + 1,), i32, dev),
          _ptr(slot_map, "slot_map", (n_slots,), i32, dev),
          _ptr(status, "status", (1,), i32, dev),
          B, width, int(page_size), pool, int(n_slots), wsp, wsz)
    return cu_new, slot_map, n_pages_out, ring_out, status


def kda_cache_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                     k_cache: torch.Tensor, v_cache: torch.Tensor, *, stream=None) -> None:
    """New tokens' k, v [T,Hkv,d] into the slots slot_map [T] (int32; those
    outside the cache are skipped) of k_cache, v_cache [n_pool,Hkv,page_size,d]."""
    dev, dt = _device(k, "kda_cache_append"), _dtype(k)
    T, H, d = _dims(k, "k", 3)
    pool, _, page, _ = _dims(k_cache, "k_cache", 4)
    rows, cache = (T, H, d), (pool, H, page, d)
    _call("kda_cache_append", dev, stream, _ptr(k, "k", rows, dt, dev), _ptr(v, "v", rows, dt, dev),
          _ptr(slot_map, "slot_map", (T,), torch.int32, dev),
          _ptr(k_cache, "k_cache", cache, dt, dev), _ptr(v_cache, "v_cache", cache, dt, dev),
          T, H, d, page, pool, _kda._DTYPES[dt])


@functools.lru_cache(maxsize=256)
def kda_attn_paged_workspace_size(T: int, B: int, Hq: int, Hkv: int, d: int, max_new: int,
                                  dtype: torch.dtype) -> int:
    return int(_kda.load_library().kda_attn_paged_workspace_size(T, B, Hq, Hkv, d, max_new,
                                                                 _kda._DTYPES[dtype]))


def kda_attn_paged(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, kept_len: torch.Tensor, cu_new: torch.Tensor, *,
                   scale: float = 0.0, max_new: int = 0, o: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, want_lse: bool = False,
                   workspace: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal attention of new tokens q [T,Hq,d] (request i: rows cu_new[i] ..
    cu_new[i+1), from position kept_len[i]) over the pages block_table
    [B,max_pages] of k_cache, v_cache [n_pool,Hkv,page_size,d], which hold the
    new tokens already. scale 0 = 1/sqrt(d); max_new: the most new tokens of a
    request if known (chooses kernels only). Returns (o [T,Hq,d], lse [T,Hq]
    fp32 or None); rows outside all requests keep what they held."""
    dev, dt = _device(q, "kda_attn_paged"), _dtype(q)
    T, Hq, d = _dims(q, "q", 3)
    pool, Hkv, page, _ = _dims(k_cache, "k_cache", 4)
    B, width = _dims(block_table, "block_table", 2)
    i32, cache = torch.int32, (pool, Hkv, page, d)
    if o is None:
        o = torch.empty_like(q) if stream is None else _kda._empty(q.shape, dt, dev, stream)
    if lse is None and want_lse:
        lse = _kda._empty((T, Hq), torch.float32, dev, stream)
    need = kda_attn_paged_workspace_size(T, B, Hq, Hkv, d, max_new, dt)
    ws, wsp, wsz = _workspace(workspace, need, dev, stream)
    _call("kda_attn_paged", dev, stream, _ptr(q, "q", (T, Hq, d), dt, dev),
          _ptr(k_cache, "k_cache", cache, dt, dev), _ptr(v_cache, "v_cache", cache, dt, dev),
          _ptr(block_table, "block_table", (B, width), i32, dev),
          _ptr(kept_len, "kept_len", (B,), i32, dev), _ptr(cu_new, "cu_new", (B + 1,), i32, dev),
          _ptr(o, "o", (T, Hq, d), dt, dev),
          None if lse is None else _ptr(lse, "lse", (T, Hq), torch.float32, dev),
          T, B, Hq, Hkv, d, page, pool, width, int(max_new), float(scale), _kda._DTYPES[dt],
          wsp, wsz)
    return o, lse


@functools.lru_cache(maxsize=256)
def kda_draft_verify_workspace_size(B: int, T: int, V: int) -> int:
    return int(_kda.load_library().kda_draft_verify_workspace_size(B, T, V))


def kda_draft_verify(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor],
                     draft_tokens: torch.Tensor, u: torch.Tensor, *,
                     n_draft: Optional[torch.Tensor] = None,
                     n_commit: Optional[torch.Tensor] = None,
                     tokens: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None
                     ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Which of T drafted tokens stay, and the next one. target_probs
    [B,T+1,V], draft_probs [B,T,V] in the same dtype or None (a certain
    draft), draft_tokens int32 [B,T], u fp32 [B,T+1] in [0,1), n_draft int32
    [B] or None (T each; below 0: an unused row). Returns (n_commit int32 [B]:
    tokens that stay + 1, 0 for an unused row; tokens int32 [B,T+1]: those that
    stay, the next one, -1)."""
    dev, dt = _device(target_probs, "kda_draft_verify"), _dtype(target_probs)
    B, T1, V = _dims(target_probs, "target_probs", 3)
    T = T1 - 1
    if T < 0:
        raise ValueError("target_probs needs T + 1 >= 1 rows per request")
    i32 = torch.int32
    n_commit = _out(n_commit, (B,), i32, dev, stream)
    tokens = _out(tokens, (B, T1), i32, dev, stream)
    ws, wsp, wsz = _workspace(workspace, kda_draft_verify_workspace_size(B, T, V), dev, stream)
    _call("kda_draft_verify", dev, stream,
          _ptr(target_probs, "target_probs", (B, T1, V), dt, dev),
          None if draft_probs is None else _ptr(draft_probs, "draft_probs", (B, T, V), dt, dev),
          _ptr(draft_tokens, "draft_tokens", (B, T), i32, dev),
          _ptr(u, "u", (B, T1), torch.float32, dev),
          None if n_draft is None else _ptr(n_draft, "n_draft", (B,), i32, dev),
          _ptr(n_commit, "n_commit", (B,), i32, dev), _ptr(tokens, "tokens", (B, T1), i32, dev),
          B, T, V, _kda._DTYPES[dt], wsp, wsz)
    return n_commit, tokens
