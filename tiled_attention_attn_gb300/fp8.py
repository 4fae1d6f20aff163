"""Paged key/value caches of 8-bit floating point (include/attn.h,
attn_paged_kv8): the append of new tokens, reading back, and attention of single
tokens and of trees of drafted tokens.

Like the rest of the binding this marshals arguments only.  Every operator takes
``stream`` by name (default: the current stream of its tensors' device).

Caches: ``k_pages`` and ``v_pages`` are float8_e4m3fn (num_pages, page_size, Hkv, d),
``k_scales`` and ``v_scales`` float32 (num_pages, page_size, Hkv), each pair strided
alike and as the caller likes (features contiguous, the other strides of the pages
multiples of 16): the row of a token and head is its e4m3 values times its scale.
``page_table`` is int32 (B, max_pages), ``seqlens_k`` int32 (B): key j of sequence b
is token j % page_size of page page_table[b, j // page_size].
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import Optional, Tuple

import torch

from . import attn as _attn
from .paged import _HALF, _check_int, _check_rc, _freqs, _outputs, _placed, _scratch, _stream


class _PagedKV8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("seqlens_k", ctypes.c_void_p),
                ("stride_page", ctypes.c_longlong), ("stride_token", ctypes.c_longlong),
                ("stride_head", ctypes.c_longlong), ("scale_stride_page", ctypes.c_longlong),
                ("scale_stride_token", ctypes.c_longlong), ("scale_stride_head", ctypes.c_longlong),
                ("table_stride", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


def declare(L) -> None:
    """Argument types of the entry points."""
    vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
    kv = vp   # (a _PagedKV8 by reference, or its bytes)
    L.attn_cache_append_fp8.argtypes = [vp, vp, vp, vp, ll, ll, ll, i, i, i, kv, vp, i, vp, f, i, vp, i, vp]
    L.attn_cache_read_fp8.argtypes = [vp, vp, i, i, kv, vp, vp, i, vp]
    L.attn_tree_fp8.argtypes = [vp, vp, vp, i, i, i, i, kv, vp, vp, f, i, vp, ll, vp]
    L.attn_fp8_workspace_bytes.argtypes = [i]
    L.attn_fp8_workspace_bytes.restype = ll
    for n in ("attn_cache_append_fp8", "attn_cache_read_fp8", "attn_tree_fp8"):
        getattr(L, n).restype = i


# The structure's bytes (quicker than its constructor: the small calls are the host's).
_pack = struct.Struct("6P6q6i").pack


def _cache(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
           page_table: torch.Tensor, seqlens_k: torch.Tensor) -> bytes:
    dev, shape, strides = k_pages.device, k_pages.shape, k_pages.stride()
    if k_pages.dtype != torch.float8_e4m3fn or v_pages.dtype != torch.float8_e4m3fn:
        raise TypeError("k_pages and v_pages must be float8_e4m3fn")
    if dev.type != "cuda" or len(shape) != 4 or strides[3] != 1:
        raise ValueError("k_pages is a CUDA tensor (num_pages, page_size, Hkv, d) with contiguous features")
    if v_pages.device != dev or v_pages.shape != shape or v_pages.stride() != strides:
        raise ValueError("v_pages must be laid out like k_pages")
    scale_strides = k_scales.stride()
    for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
        if s.dtype != torch.float32:
            raise TypeError(f"{name} must be float32")
        if s.device != dev or s.shape != shape[:3] or s.stride() != scale_strides:
            raise ValueError(f"{name} must be a CUDA tensor {tuple(shape[:3])}, both scales laid out alike")
    if page_table.dtype != torch.int32 or page_table.device != dev or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be an int32 CUDA tensor (B, max_pages) with contiguous rows")
    B, max_pages = page_table.shape
    _check_int(seqlens_k, "seqlens_k", dev, (B,))
    n, P, hkv, d = shape
    sp, st, sh, _ = strides
    cp, ct, ch = scale_strides
    # strides of an axis of one entry address nothing: any valid value serves
    sp, sh = sp if n > 1 else max(16, d), sh if hkv > 1 else max(16, d)
    cp, ch = cp if n > 1 else 1, ch if hkv > 1 else 1
    return _pack(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                 page_table.data_ptr(), seqlens_k.data_ptr(), sp, st, sh, cp, ct, ch,
                 page_table.stride(0) if B > 1 else max_pages, max_pages, n, P, hkv, d)


@_placed
def cache_append_fp8(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                     k_scales: torch.Tensor, v_scales: torch.Tensor, page_table: torch.Tensor, seqlens_k: torch.Tensor,
                     cu_seqlens: torch.Tensor, q: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None,
                     amplitude: float = 1.0, interleaved: bool = False, positions: Optional[torch.Tensor] = None,
                     q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """``cache_append`` into a cache of 8-bit floating point: the new tokens' k and v
    (bfloat16 or float16, (total, Hkv, d) with offsets ``cu_seqlens``) are quantised
    as they are written, each row of a token and head with the scale max |x| / 448;
    with ``freqs`` the keys are rotated before that, in float32, and the queries q
    (total, Hq, d) too, which are returned (in ``q_out`` if given) in their own
    type.  ``seqlens_k`` counts the new tokens already; ``positions`` (int32 (total))
    replaces the key index as the rotary position.  rot_dim a multiple of 16."""
    c = _cache(k_pages, v_pages, k_scales, v_scales, page_table, seqlens_k)
    dev, B = k_pages.device, page_table.shape[0]
    _check_int(cu_seqlens, "cu_seqlens", dev, (B + 1,))
    hkv, d = k_pages.shape[2:]
    if k.dtype not in _HALF:
        raise TypeError("k and v must be bfloat16 or float16")
    total = k.shape[0] if k.dim() == 3 else -1
    strides = []
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            strides.append(0)
            continue
        if t.dtype != k.dtype:
            raise TypeError("q, k and v must share one 16-bit dtype")
        H = t.shape[1] if name == "q" and t.dim() == 3 else hkv
        if t.device != dev or tuple(t.shape) != (total, H, d) or t.stride(2) != 1 or (H > 1 and t.stride(1) != d):
            raise ValueError(f"{name} is (total, H, d) on the cache's device with contiguous heads")
        strides.append(t.stride(0) if total > 1 else H * d)
    if q is not None and freqs is None:
        raise ValueError("q is only taken to be rotated: freqs are missing")
    if positions is not None:
        _check_int(positions, "positions", dev, (total,))
    f, rot = (None, 0) if freqs is None else _freqs(freqs, d)
    s = _stream(dev)
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    elif q is None and q_out is not None:
        raise ValueError("q_out without q")
    elif q is not None and (q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != dev
                            or not q_out.is_contiguous()):
        raise ValueError("q_out must be a contiguous tensor shaped like q")
    rc = _attn.lib().attn_cache_append_fp8(
        q.data_ptr() if q is not None else None, k.data_ptr() or None, v.data_ptr() or None,
        q_out.data_ptr() if q is not None else None, *strides, B, q.shape[1] if q is not None else 0, total,
        c, cu_seqlens.data_ptr(), rot, f.data_ptr() if f is not None else None, float(amplitude),
        int(bool(interleaved)), positions.data_ptr() if positions is not None else None, int(k.dtype == torch.float16),
        s) if total else 0
    _check_rc(rc, "attn_cache_append_fp8")
    return q_out


@_placed
def cache_read_fp8(k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor, v_scales: torch.Tensor,
                   page_table: torch.Tensor, seqlens_k: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
                   dtype: torch.dtype = torch.bfloat16, starts: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None,
                   v_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keys and values read back, packed as ``attn_fwd`` takes them with
    ``cu_seqlens_k``: rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of the returned
    (total, Hkv, d) tensors are the keys from starts[b] on (int32 (B), default 0) of
    sequence b, in ``dtype`` (bfloat16 or float16), rounded once.  Rows outside
    every sequence are left as they are in ``k_out`` and ``v_out``."""
    c = _cache(k_pages, v_pages, k_scales, v_scales, page_table, seqlens_k)
    dev, B = k_pages.device, page_table.shape[0]
    _check_int(cu_seqlens, "cu_seqlens", dev, (B + 1,))
    if starts is not None:
        _check_int(starts, "starts", dev, (B,))
    if dtype not in _HALF:
        raise TypeError("dtype must be bfloat16 or float16")
    if total < 0:
        raise ValueError("total must not be negative")
    s = _stream(dev)
    shape = (int(total), *k_pages.shape[2:])
    outs = []
    for name, t in (("k_out", k_out), ("v_out", v_out)):
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        elif t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
        outs.append(t)
    rc = _attn.lib().attn_cache_read_fp8(outs[0].data_ptr(), outs[1].data_ptr(), B, int(total), c,
                                         cu_seqlens.data_ptr(), starts.data_ptr() if starts is not None else None,
                                         int(dtype == torch.float16), s) if total else 0
    _check_rc(rc, "attn_cache_read_fp8")
    return outs[0], outs[1]


_ws_bytes: dict = {}


def _attend(q, cache, cu_seqlens, tree_mask, max_tokens, scale, out, lse):
    c = _cache(*cache)
    dev, B, d = cache[0].device, cache[4].shape[0], cache[0].shape[3]
    if q.dtype not in _HALF:
        raise TypeError("q must be bfloat16 or float16")
    if q.device != dev or not q.is_contiguous() or q.dim() != 3 or q.shape[2] != d:
        raise ValueError("q is a contiguous CUDA tensor (tokens, Hq, d) on the cache's device")
    T = q.shape[0]
    if cu_seqlens is not None:
        _check_int(cu_seqlens, "cu_seqlens", dev, (B + 1,))
    elif T != B:
        raise ValueError("q holds one row per sequence of page_table")
    if tree_mask is not None and (tree_mask.dtype != torch.int64 or tree_mask.device != dev or tree_mask.shape != (T,)
                                  or not tree_mask.is_contiguous()):
        raise ValueError(f"tree_mask must be a contiguous int64 tensor of shape {(T,)} on {dev}")
    if not 1 <= max_tokens <= 64:
        raise ValueError("max_tokens is between 1 and 64")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    s = _stream(dev)
    out, lse = _outputs(q, out, lse)
    if T == 0:
        return out, lse
    n = _ws_bytes.get((dev.index, d))
    if n is None:
        n = _attn.lib().attn_fp8_workspace_bytes(d)
        if n < 0:
            raise _attn.AttnError(int(n), "attn_fp8_workspace_bytes")
        _ws_bytes[(dev.index, d)] = n
    ws = _scratch(dev, s, n)
    rc = _attn.lib().attn_tree_fp8(q.data_ptr(), out.data_ptr(), lse.data_ptr(), B, q.shape[1], T, int(max_tokens),
                                   c, cu_seqlens.data_ptr() if cu_seqlens is not None else None,
                                   tree_mask.data_ptr() if tree_mask is not None else None, float(scale),
                                   int(q.dtype == torch.float16), ws.data_ptr(), ws.numel(), s)
    _check_rc(rc, "attn_tree_fp8")
    return out, lse


@_placed
def attn_tree_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                  v_scales: torch.Tensor, page_table: torch.Tensor, seqlens_k: torch.Tensor, cu_seqlens: torch.Tensor,
                  tree_mask: Optional[torch.Tensor] = None, max_tokens: Optional[int] = None,
                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                  lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of trees of drafted tokens over a cache of 8-bit floating point: q
    (total, Hq, d) with offsets ``cu_seqlens`` (int32, B + 1), the T tokens of a
    sequence being its last T keys.  Each token sees all keys before them, and of
    the T keys those t whose bit t is set in its ``tree_mask`` (int64 (total): its
    ancestors and itself); without ``tree_mask`` the tokens are a chain.
    ``max_tokens``: at least every T, at most 64 (default: 64, or total if less);
    smaller is faster.  Returns O like q and lse (Hq, total) float32; a token
    that sees no key gives 0 and -inf, rows outside every sequence are left as they
    are."""
    if max_tokens is None:
        max_tokens = max(1, min(64, q.shape[0]))
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is missing")
    return _attend(q, (k_pages, v_pages, k_scales, v_scales, page_table, seqlens_k), cu_seqlens, tree_mask, max_tokens,
                   scale, out, lse)


@_placed
def attn_decode_fp8(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, k_scales: torch.Tensor,
                    v_scales: torch.Tensor, page_table: torch.Tensor, seqlens_k: torch.Tensor,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One decoding step over a cache of 8-bit floating point: q (B, Hq, d) holds one
    query per sequence, which sees all of its seqlens_k[b] keys.  Returns O (B, Hq,
    d) and lse (Hq, B) float32."""
    return _attend(q, (k_pages, v_pages, k_scales, v_scales, page_table, seqlens_k), None, None, 1, scale, out, lse)
