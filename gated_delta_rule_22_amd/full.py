"""Binding of the full-attention layers' calls (``include/kda_full.h``).

In the manner of :mod:`gated_delta_rule_22_amd.serve`: checks of arguments,
outputs and workspaces the caller leaves out, and the HIP kernels behind the
library. ``kda_rope_append`` goes between ``kda_page_plan`` and
``kda_attn_paged`` in layers of grouped heads; ``kda_latent_append`` and then
``kda_attn_latent`` or, for prompts, ``kda_attn_expanded`` are the layers whose
keys and values are one latent vector a token.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

import gated_delta_rule_22_amd as _kda
from .serve import _call, _device, _dims, _dtype, _out, _ptr, _too_large, _workspace


class _RopeStruct(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("rot", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("factor", ctypes.c_float)]


def declare(lib) -> None:
    vp, i, sz, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    lib.kda_rope_append.argtypes = [vp] * 9 + [i] * 7 + [vp, i, vp]
    lib.kda_rope_append.restype = i
    lib.kda_latent_append.argtypes = [vp] * 9 + [i] * 10 + [f, vp, i, vp]
    lib.kda_latent_append.restype = i
    lib.kda_attn_latent_workspace_size.argtypes = [i] * 7
    lib.kda_attn_latent_workspace_size.restype = sz
    lib.kda_attn_latent.argtypes = [vp] * 7 + [i] * 9 + [f, i, vp, sz, vp]
    lib.kda_attn_latent.restype = i
    lib.kda_attn_expanded_workspace_size.argtypes = [i] * 8
    lib.kda_attn_expanded_workspace_size.restype = sz
    lib.kda_attn_expanded.argtypes = [vp] * 7 + [i] * 9 + [f, i, vp, sz, vp]
    lib.kda_attn_expanded.restype = i


class KDARope:
    """A rotation by positions: ``freqs`` fp64 [rot/2] on the device (radians a
    position of each pair, see :func:`kda_rope_freqs`), pairs of neighbouring
    channels (``interleaved``) or of the two halves, and a ``factor`` on what is
    rotated. Made once and kept."""

    def __init__(self, freqs: torch.Tensor, *, interleaved: bool = False, factor: float = 1.0):
        n, = _dims(freqs, "freqs", 1)
        self.freqs, self.rot = freqs, 2 * n
        self.interleaved, self.factor = bool(interleaved), float(factor)
        dev = _device(freqs, "KDARope")
        self.struct = _RopeStruct(_ptr(freqs, "freqs", (n,), torch.float64, dev), self.rot,
                                  int(self.interleaved), self.factor)
        self.ref = ctypes.addressof(self.struct)


def _rope_ref(rope: Optional[KDARope], dev) -> Optional[int]:
    if rope is None:
        return None
    if rope.freqs.device != dev:
        raise ValueError(f"rope.freqs is on {rope.freqs.device}, expected {dev}")
    return rope.ref


def kda_rope_freqs(rot: int, *, base: float = 10000.0, scaling: str = "none", scale: float = 1.0,
                   original_len: int = 0, fast: float = 32.0, slow: float = 1.0,
                   device=None) -> Tuple[torch.Tensor, float]:
    """(freqs, factor) for :class:`KDARope`: ``freqs[j] = base ** (-2 j / rot)`` in
    fp64, for contexts ``scale`` times as long as the model's own:

    - ``"none"``: as they are;
    - ``"linear"``: positions divided by ``scale``;
    - ``"base"``: a larger base, ``base * scale ** (rot / (rot - 2))``, which divides
      the slowest pair by ``scale`` and leaves the fastest;
    - ``"parts"``: pairs that turn less than ``slow`` times over ``original_len``
      positions are divided by ``scale``, those that turn more than ``fast`` times
      stay, the others in between (linearly in their turns); factor
      ``0.1 ln(scale) + 1`` for ``scale`` above 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot {rot} is not a positive even number")
    if not (base > 0 and scale > 0):
        raise ValueError("base and scale must be positive")
    exponent = -torch.arange(0, rot, 2, dtype=torch.float64) / rot
    factor = 1.0
    if scaling == "none":
        f = base ** exponent
    elif scaling == "linear":
        f = base ** exponent / scale
    elif scaling == "base":
        if rot < 4:
            raise ValueError("scaling 'base' needs rot >= 4")
        f = (base * scale ** (rot / (rot - 2))) ** exponent
    elif scaling == "parts":
        if original_len <= 0 or not fast > slow:
            raise ValueError("scaling 'parts' needs original_len > 0 and fast > slow")
        f = base ** exponent
        turns = original_len * f / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / scale)
        factor = 0.1 * math.log(scale) + 1.0 if scale > 1 else 1.0
    else:
        raise ValueError(f"unknown scaling {scaling!r}")
    return f.to(device), factor


def kda_rope_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor,
                    kept_len: torch.Tensor, cu_new: torch.Tensor, k_cache: torch.Tensor,
                    v_cache: torch.Tensor, rope: KDARope, *, q_out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """New tokens' queries q [T,Hq,d] and keys k [T,Hkv,d] rotated (the first
    rope.rot channels) by their positions (request i: rows cu_new[i] ..
    cu_new[i+1), from position kept_len[i]), keys and values v into the slots
    slot_map [T] of k_cache, v_cache [n_pool,Hkv,page_size,d]. Returns the rotated
    queries (q_out, which may be q itself); rows outside all requests are not
    written and not appended."""
    dev, dt = _device(q, "kda_rope_append"), _dtype(q)
    T, Hq, d = _dims(q, "q", 3)
    pool, Hkv, page, _ = _dims(k_cache, "k_cache", 4)
    B, = _dims(kept_len, "kept_len", 1)
    if (T | B | pool) >> 31:
        _too_large("kda_rope_append")
    i32, rows, cache = torch.int32, (T, Hkv, d), (pool, Hkv, page, d)
    if q_out is None:
        q_out = torch.empty_like(q) if stream is None else _kda._empty(q.shape, dt, dev, stream)
    _call("kda_rope_append", dev, stream, _ptr(q, "q", (T, Hq, d), dt, dev),
          _ptr(k, "k", rows, dt, dev), _ptr(v, "v", rows, dt, dev),
          _ptr(slot_map, "slot_map", (T,), i32, dev), _ptr(kept_len, "kept_len", (B,), i32, dev),
          _ptr(cu_new, "cu_new", (B + 1,), i32, dev), _ptr(q_out, "q_out", (T, Hq, d), dt, dev),
          _ptr(k_cache, "k_cache", cache, dt, dev), _ptr(v_cache, "v_cache", cache, dt, dev),
          T, B, Hq, Hkv, d, page, pool, _rope_ref(rope, dev), _kda._DTYPES[dt])
    return q_out


def kda_latent_append(kv: torch.Tensor, slot_map: torch.Tensor, kept_len: torch.Tensor,
                      cu_new: torch.Tensor, cache: torch.Tensor, *,
                      rope: Optional[KDARope] = None, w: Optional[torch.Tensor] = None,
                      normalise: bool = True, eps: float = 1e-6, dr: int = 64,
                      q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                      kv_out: Optional[torch.Tensor] = None, stream=None) -> None:
    """New tokens' latent rows kv [T,dc+dr] into the slots slot_map [T] of cache
    [n_pool,page_size,dc+dr]: the first dc channels RMS-normalised (normalise, with
    weights w fp32 [dc] or ones), the last dr rotated by the token's position (rope;
    None: as they are). kv_out [T,dc+dr] receives the same rows (it may be kv). With
    q [T,Hq,dq], the last dr channels of q_out [T,Hq,dq_out] become the last dr of q,
    rotated (q_out may be q). Requests as in kda_rope_append."""
    dev, dt = _device(kv, "kda_latent_append"), _dtype(kv)
    T, width = _dims(kv, "kv", 2)
    pool, page, _ = _dims(cache, "cache", 3)
    B, = _dims(kept_len, "kept_len", 1)
    if (T | B) >> 31:
        _too_large("kda_latent_append")
    i32 = torch.int32
    if (q is None) != (q_out is None):
        raise ValueError("kda_latent_append takes q and q_out together")
    Hq = dq = dq_out = 0
    if q is not None:
        _, Hq, dq = _dims(q, "q", 3)
        _, _, dq_out = _dims(q_out, "q_out", 3)
    _call("kda_latent_append", dev, stream, _ptr(kv, "kv", (T, width), dt, dev),
          None if w is None else _ptr(w, "w", (width - dr,), torch.float32, dev),
          _ptr(slot_map, "slot_map", (T,), i32, dev), _ptr(kept_len, "kept_len", (B,), i32, dev),
          _ptr(cu_new, "cu_new", (B + 1,), i32, dev),
          _ptr(cache, "cache", (pool, page, width), dt, dev),
          None if kv_out is None else _ptr(kv_out, "kv_out", (T, width), dt, dev),
          None if q is None else _ptr(q, "q", (T, Hq, dq), dt, dev),
          None if q is None else _ptr(q_out, "q_out", (T, Hq, dq_out), dt, dev),
          T, B, Hq, dq, dq_out, width - dr, dr, page, pool, int(normalise), float(eps),
          _rope_ref(rope, dev), _kda._DTYPES[dt])


@functools.lru_cache(maxsize=256)
def kda_attn_latent_workspace_size(T: int, B: int, Hq: int, dc: int, dr: int, max_new: int,
                                   dtype: torch.dtype) -> int:
    return int(_kda.load_library().kda_attn_latent_workspace_size(T, B, Hq, dc, dr, max_new,
                                                                  _kda._DTYPES[dtype]))


def kda_attn_latent(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                    kept_len: torch.Tensor, cu_new: torch.Tensor, *, dc: int, scale: float,
                    max_new: int = 0, o: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, want_lse: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal attention of new tokens q [T,Hq,dc+dr] (request i: rows cu_new[i] ..
    cu_new[i+1), from position kept_len[i]) over the pages block_table [B,max_pages]
    of the latent cache [n_pool,page_size,dc+dr], whose rows are the keys of all heads
    and in their first dc channels the values; it holds the new tokens already.
    max_new: the most new tokens of a request if known (chooses kernels only).
    Returns (o [T,Hq,dc], lse [T,Hq] fp32 or None); rows outside all requests keep
    what they held."""
    dev, dt = _device(q, "kda_attn_latent"), _dtype(q)
    T, Hq, dk = _dims(q, "q", 3)
    pool, page, _ = _dims(cache, "cache", 3)
    B, width = _dims(block_table, "block_table", 2)
    if (T | B | width) >> 31:
        _too_large("kda_attn_latent")
    i32, dr = torch.int32, dk - dc
    o = _out(o, (T, Hq, dc), dt, dev, stream)
    if lse is None and want_lse:
        lse = _kda._empty((T, Hq), torch.float32, dev, stream)
    need = kda_attn_latent_workspace_size(T, B, Hq, dc, dr, max_new, dt)
    ws, wsp, wsz = _workspace(workspace, need, dev, stream)
    _call("kda_attn_latent", dev, stream, _ptr(q, "q", (T, Hq, dk), dt, dev),
          _ptr(cache, "cache", (pool, page, dk), dt, dev),
          _ptr(block_table, "block_table", (B, width), i32, dev),
          _ptr(kept_len, "kept_len", (B,), i32, dev), _ptr(cu_new, "cu_new", (B + 1,), i32, dev),
          _ptr(o, "o", (T, Hq, dc), dt, dev),
          None if lse is None else _ptr(lse, "lse", (T, Hq), torch.float32, dev),
          T, B, Hq, dc, dr, page, pool, width, int(max_new), float(scale), _kda._DTYPES[dt], wsp, wsz)
    return o, lse


@functools.lru_cache(maxsize=256)
def kda_attn_expanded_workspace_size(T: int, B: int, H: int, dn: int, dr: int, dv: int, max_q: int,
                                     dtype: torch.dtype) -> int:
    return int(_kda.load_library().kda_attn_expanded_workspace_size(T, B, H, dn, dr, dv, max_q,
                                                                    _kda._DTYPES[dtype]))


def kda_attn_expanded(q: torch.Tensor, kv: torch.Tensor, k_pe: torch.Tensor, cu_q: torch.Tensor,
                      cu_k: torch.Tensor, *, dv: int, scale: float = 0.0, max_q: int = 0,
                      o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      want_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None
                      ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal attention of packed prompts q [T,H,dn+dr] over expanded keys and values
    kv [N,H,dn+dv] and the keys' shared part k_pe [N,dr], whose rows may lie apart
    (the last columns of a wider tensor). Request i has query rows cu_q[i] ..
    cu_q[i+1) and key rows cu_k[i] .. cu_k[i+1); its last query is at its last key.
    scale 0 = 1/sqrt(dn+dr); max_q: the most queries of a request if known (chooses
    kernels only). Returns (o [T,H,dv], lse [T,H] fp32 or None); rows outside all
    requests keep what they held."""
    dev, dt = _device(q, "kda_attn_expanded"), _dtype(q)
    T, H, dk = _dims(q, "q", 3)
    N, _, w = _dims(kv, "kv", 3)
    _, dr = _dims(k_pe, "k_pe", 2)
    dn = w - dv
    if dn + dr != dk:
        raise ValueError(f"q is {dk} wide, kv and k_pe make keys of {dn} + {dr}")
    B = _dims(cu_q, "cu_q", 1)[0] - 1
    if B < 0:
        raise ValueError("cu_q needs B + 1 entries")
    if (T | N | B) >> 31:
        _too_large("kda_attn_expanded")
    if k_pe.shape[0] != N or k_pe.dtype is not dt or k_pe.device != dev:
        _kda._check(k_pe, "k_pe", (N, dr), dt, dev)
    # (of a single row, or of none, the stride means nothing)
    stride_pe, column = k_pe.stride() if N > 1 else (dr, k_pe.stride(1))
    if column != 1 or stride_pe < dr or stride_pe % 8 or stride_pe > 1 << 26:
        raise ValueError("k_pe's rows must be contiguous, a multiple of 8 and at most 2^26 elements apart")
    i32 = torch.int32
    o = _out(o, (T, H, dv), dt, dev, stream)
    if lse is None and want_lse:
        lse = _kda._empty((T, H), torch.float32, dev, stream)
    need = kda_attn_expanded_workspace_size(T, B, H, dn, dr, dv, max_q, dt)
    ws, wsp, wsz = _workspace(workspace, need, dev, stream)
    _call("kda_attn_expanded", dev, stream, _ptr(q, "q", (T, H, dk), dt, dev),
          _ptr(kv, "kv", (N, H, w), dt, dev), k_pe.data_ptr(),
          _ptr(cu_q, "cu_q", (B + 1,), i32, dev), _ptr(cu_k, "cu_k", (B + 1,), i32, dev),
          _ptr(o, "o", (T, H, dv), dt, dev),
          None if lse is None else _ptr(lse, "lse", (T, H), torch.float32, dev),
          T, N, B, H, dn, dr, dv, stride_pe, int(max_q), float(scale), _kda._DTYPES[dt], wsp, wsz)
    return o, lse
