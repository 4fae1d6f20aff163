"""Paged key/value caches (include/attn.h): rotary embedding with scaled
frequencies, the append of new tokens to the pages, attention of a chunk or of
single tokens over the pages, accumulated attention weights, and eviction.

Like the rest of the binding this marshals arguments only; every step runs in
the library's kernels.  Outputs and scratch memory are allocated by torch on
the call's stream; calls on several streams, from several threads, or captured
in several graphs share nothing.  Every operator takes ``stream`` by name
(default: the current stream of its tensors' device); the one with a gradient
runs on the current stream.

Caches: ``k_pages`` and ``v_pages`` are (num_pages, page_size, Hkv, d) views,
strided as the caller likes as long as the features are contiguous (slices of
one buffer, or permuted (num_pages, Hkv, page_size, d) storage); ``page_table``
is int32 (B, max_pages), ``seqlens_k`` int32 (B): key j of sequence b is token
j % page_size of page page_table[b, j // page_size].
"""

from __future__ import annotations

import ctypes
import functools
import math
import threading
from typing import Optional, Tuple

import torch

from . import attn as _attn

ATTN_DEVERR_BAD_PAGE = 0x300


class _PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("seqlens_k", ctypes.c_void_p), ("stride_page", ctypes.c_longlong),
                ("stride_token", ctypes.c_longlong), ("stride_head", ctypes.c_longlong),
                ("table_stride", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("page_size", ctypes.c_int), ("num_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("fp16", ctypes.c_int)]


def declare(L) -> None:
    """Argument types of the paged entry points."""
    vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
    kv = ctypes.POINTER(_PagedKV)
    L.attn_rotary_scaled.argtypes = [vp, vp, i, i, i, i, i, vp, f, i, i, ll, ll, vp, i, vp, vp, i, vp]
    L.attn_cache_append.argtypes = [vp, vp, vp, vp, ll, ll, ll, i, i, i, kv, vp, i, vp, f, i, vp, vp]
    L.attn_fwd_paged.argtypes = [vp, vp, vp, i, i, i, kv, vp, i, f, vp, ll, vp]
    L.attn_decode_paged.argtypes = [vp, vp, vp, i, i, kv, f, vp, ll, vp]
    L.attn_key_weights.argtypes = [vp, vp, vp, i, i, i, i, kv, vp, i, f, f, vp, ll, vp]
    L.attn_cache_evict.argtypes = [vp, i, vp, vp, vp, i, i, kv, vp, i, i, i, i, vp]
    L.attn_paged_workspace_bytes.argtypes = [i, i]
    L.attn_paged_workspace_bytes.restype = ll
    for n in ("attn_rotary_scaled", "attn_cache_append", "attn_fwd_paged", "attn_decode_paged", "attn_key_weights",
              "attn_cache_evict"):
        getattr(L, n).restype = i


_HALF = (torch.bfloat16, torch.float16)


def _placed(fn):
    """Runs fn with the device of its first tensor current and, given ``stream``
    (by name), on that stream, so that outputs and scratch memory are allocated
    there too.  The usual call, on the current device and stream, enters no
    context."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def call(*args, stream: Optional[torch.cuda.Stream] = None, **kw):
        dev = (args[0] if args else kw[name]).device
        if dev.type != "cuda" or (stream is None and dev.index == torch.cuda.current_device()):
            return fn(*args, **kw)
        with torch.cuda.device(dev):
            if stream is None:
                return fn(*args, **kw)
            if stream.device != dev:
                raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
            with torch.cuda.stream(stream):
                return fn(*args, **kw)

    return call


def _stream(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check_int(t: torch.Tensor, name: str, device, shape) -> None:
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous() or t.shape != shape:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {tuple(shape)} on {device}")


def _check_rc(rc: int, what: str) -> None:
    if rc != _attn.ATTN_OK:
        raise _attn.AttnError(rc, what)


def _cache(k_pages: torch.Tensor, v_pages: Optional[torch.Tensor], page_table: torch.Tensor,
           seqlens_k: torch.Tensor) -> _PagedKV:
    dev, dtype, shape, strides = k_pages.device, k_pages.dtype, k_pages.shape, k_pages.stride()
    if dtype not in _HALF:
        raise TypeError("k_pages and v_pages must be bfloat16 or float16")
    if dev.type != "cuda" or len(shape) != 4 or strides[3] != 1:
        raise ValueError("k_pages is a CUDA tensor (num_pages, page_size, Hkv, d) with contiguous features")
    v = None
    if v_pages is not None:
        if v_pages.dtype != dtype:
            raise TypeError("k_pages and v_pages must share one dtype")
        if v_pages.device != dev or v_pages.shape != shape or v_pages.stride() != strides:
            raise ValueError("v_pages must be laid out like k_pages")
        v = v_pages.data_ptr()
    if page_table.dtype != torch.int32 or page_table.device != dev or page_table.dim() != 2 or page_table.stride(1) != 1:
        raise ValueError("page_table must be an int32 CUDA tensor (B, max_pages) with contiguous rows")
    B, max_pages = page_table.shape
    _check_int(seqlens_k, "seqlens_k", dev, (B,))
    n, P, hkv, d = shape
    sp, st, sh, _ = strides
    # strides of an axis of one entry address nothing: any valid value serves
    sp, sh = sp if n > 1 else max(8, d), sh if hkv > 1 else max(8, d)
    return _PagedKV(k_pages.data_ptr(), v, page_table.data_ptr(), seqlens_k.data_ptr(), sp, st, sh,
                    page_table.stride(0) if B > 1 else max_pages, max_pages, n, P, hkv, d, int(dtype == torch.float16))


def _check_q(q: torch.Tensor, c: _PagedKV, k_pages: torch.Tensor) -> None:
    if q.dtype != k_pages.dtype:
        raise TypeError("q and the cache must share one 16-bit dtype")
    if q.device != k_pages.device or not q.is_contiguous() or q.dim() != 3 or q.shape[2] != c.head_dim:
        raise ValueError("q is a contiguous CUDA tensor (tokens, Hq, d) on the cache's device")


def _freqs(freqs: torch.Tensor, d: int) -> Tuple[torch.Tensor, int]:
    f = freqs if isinstance(freqs, torch.Tensor) else torch.tensor(freqs, dtype=torch.float64)
    if f.is_cuda or f.dtype != torch.float64 or f.dim() != 1 or not f.is_contiguous() or not 0 < 2 * f.numel() <= d:
        raise ValueError("freqs must be a contiguous float64 host tensor of at most d / 2 entries")
    return f, 2 * f.numel()


def rotary_freqs(rot_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                 original_len: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0) -> Tuple[torch.Tensor, float]:
    """(freqs, amplitude) for ``rotary_scaled``: the spectrum f_i = base^(-2i / rot_dim)
    (float64, radians per position), scaled for contexts ``factor`` times the
    trained length ``original_len``:

    * ``None``: as it is;
    * ``"linear"``: f / factor (position interpolation);
    * ``"ntk"``: the base times factor^(rot_dim / (rot_dim - 2)), which leaves the
      highest frequency alone and divides the lowest by factor;
    * ``"yarn"``: pairs that turn more than ``beta_fast`` times within
      original_len keep f, those below ``beta_slow`` turns take f / factor, linear in
      the pair index between; amplitude 0.1 ln(factor) + 1.
    """
    if rot_dim <= 0 or rot_dim % 2 or not base > 1.0 or not factor >= 1.0 or original_len <= 0:
        raise ValueError("rot_dim even and positive, base > 1, factor >= 1, original_len positive")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot_dim)
    if scaling is None:
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        if rot_dim == 2:
            return f, 1.0
        return (base * factor ** (rot_dim / (rot_dim - 2.0))) ** (-2.0 * i / rot_dim), 1.0
    if scaling == "yarn":
        def pair_of(turns):   # the pair that turns so often within original_len
            return rot_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
        lo = max(math.floor(pair_of(beta_fast)), 0)
        hi = min(math.ceil(pair_of(beta_slow)), rot_dim // 2 - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        ramp[f * original_len < 2.0 * math.pi * beta_slow] = 1.0   # (also where a short context leaves lo = hi)
        return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"unknown scaling {scaling!r}")


@_placed
def rotary_scaled(x: torch.Tensor, freqs: torch.Tensor, amplitude: float = 1.0, interleaved: bool = False,
                  cu_seqlens: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                  positions: Optional[torch.Tensor] = None, inverse: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotary embedding of x with the given frequencies (``rotary_freqs``; a
    float64 host tensor of rot_dim / 2 radians per position) times ``amplitude``;
    ``inverse`` turns the other way, which is its gradient.

    x is (B, L, H, d), or packed (total, H, d) with ``cu_seqlens`` or
    ``positions``; its features are contiguous, tokens and heads may be strided
    (a slice of a fused projection).  Positions are i + offsets[b] (``offsets``
    int32 (B)), or ``positions``, int32 of x's leading shape.  ``out`` may be x
    itself when x is contiguous; default a new contiguous tensor.  With
    ``cu_seqlens``, rows outside every sequence are left as they are in out.
    """
    if x.dtype not in _HALF:
        raise TypeError("x must be bfloat16 or float16")
    if not x.is_cuda or x.dim() not in (3, 4) or x.stride(-1) != 1 and x.shape[-1] > 1:
        raise ValueError("x is a CUDA tensor (B, L, H, d) or (total, H, d) with contiguous features")
    dev, H, d = x.device, x.shape[-2], x.shape[-1]
    f, rot = _freqs(freqs, d)
    total = 0
    if x.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("packed x is (total, H, d)")
        B, L = x.shape[:2]
        if B > 1 and L > 1 and x.stride(0) != L * x.stride(1):
            raise ValueError("the tokens of x must be evenly strided over batch and length")
        st = x.stride(1) if L > 1 else x.stride(0)
    else:
        if cu_seqlens is None and positions is None:
            raise ValueError("packed x needs cu_seqlens or positions")
        if cu_seqlens is not None:
            if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
                raise ValueError("cu_seqlens has B + 1 entries")
            _check_int(cu_seqlens, "cu_seqlens", dev, cu_seqlens.shape)
            B, L, total = cu_seqlens.numel() - 1, 0, x.shape[0]
        else:
            B, L = 1, x.shape[0]
        st = x.stride(0)
    rows = x.numel() // (H * d) if H * d else 0
    sh = x.stride(-2) if H > 1 else d
    st = st if rows > 1 else H * max(sh, d)
    if positions is not None:
        if offsets is not None or cu_seqlens is not None:
            raise ValueError("positions replace offsets and cu_seqlens")
        _check_int(positions, "positions", dev, x.shape[:-2])
        B, L = 1, rows
    if offsets is not None:
        _check_int(offsets, "offsets", dev, (B,))
    if B == 0 or H == 0:
        raise ValueError("x has no sequences or no heads")
    s = _stream(dev)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=dev)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != dev or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like x")
    rc = _attn.lib().attn_rotary_scaled(
        x.data_ptr() or None, out.data_ptr() or None, B, L, H, d, rot, f.data_ptr(), float(amplitude),
        int(bool(interleaved)), int(bool(inverse)), st, sh,
        cu_seqlens.data_ptr() if cu_seqlens is not None else None, total,
        offsets.data_ptr() if offsets is not None else None,
        positions.data_ptr() if positions is not None else None, int(x.dtype == torch.float16), s) if rows else 0
    _check_rc(rc, "attn_rotary_scaled")
    return out


class _RotaryScaledFunction(torch.autograd.Function):
    """The rotation forward, its inverse (times the same amplitude) backward;
    the backward is the same operator turned round, so it has a gradient too."""

    @staticmethod
    def forward(ctx, x, freqs, amplitude, interleaved, cu_seqlens, offsets, positions, inverse):
        # rows outside every sequence are zero, in the output and in the gradient
        out = torch.zeros(x.shape, dtype=x.dtype, device=x.device) if cu_seqlens is not None else None
        y = rotary_scaled(x, freqs, amplitude, interleaved, cu_seqlens, offsets, positions, inverse, out)
        # (freqs too, so that a change of theirs before the backward is an error)
        ctx.save_for_backward(_freqs(freqs, x.shape[-1])[0],
                              *(t for t in (cu_seqlens, offsets, positions) if t is not None))
        ctx.given = [t is not None for t in (cu_seqlens, offsets, positions)]
        ctx.args = (amplitude, interleaved, inverse)
        return y

    @staticmethod
    def backward(ctx, dy):
        freqs, *rest = ctx.saved_tensors
        rest = iter(rest)
        cu, off, pos = (next(rest) if g else None for g in ctx.given)
        amplitude, interleaved, inverse = ctx.args
        return (_RotaryScaledFunction.apply(dy.contiguous(), freqs, amplitude, interleaved, cu, off, pos,
                                            not inverse),) + (None,) * 7


def rotary_scaled_func(x: torch.Tensor, freqs: torch.Tensor, amplitude: float = 1.0, interleaved: bool = False,
                       cu_seqlens: Optional[torch.Tensor] = None, offsets: Optional[torch.Tensor] = None,
                       positions: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``rotary_scaled`` with a gradient for x (the frequencies are constants:
    changing them in place before the backward is an error), on the current
    stream.  With ``cu_seqlens``, rows outside every sequence are zero and get no
    gradient.  A backward that is captured into a CUDA graph needs, as with any
    operator of torch, that no eager graph of the same leaves is alive."""
    return _RotaryScaledFunction.apply(x, freqs, float(amplitude), bool(interleaved), cu_seqlens, offsets, positions,
                                       False)


@_placed
def cache_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 page_table: torch.Tensor, seqlens_k: torch.Tensor, cu_seqlens: torch.Tensor,
                 q: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None, amplitude: float = 1.0,
                 interleaved: bool = False, positions: Optional[torch.Tensor] = None,
                 q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Writes the new tokens' k and v, (total, Hkv, d) with offsets
    ``cu_seqlens`` (int32, B + 1), into the pages; ``seqlens_k`` counts them
    already (they are each sequence's last keys).  With ``freqs`` the keys, and
    the queries q (total, Hq, d), are rotated on the way, as ``rotary_scaled``
    does, at the key index or at ``positions`` (int32 (total)).  k, v and q may
    be slices of one projection's output (contiguous heads, strided tokens).
    Returns the rotated q, in ``q_out`` if given, or None without q.  Rows of q
    outside every sequence are left as they are in q_out.
    """
    c = _cache(k_pages, v_pages, page_table, seqlens_k)
    dev, B = k_pages.device, page_table.shape[0]
    _check_int(cu_seqlens, "cu_seqlens", dev, (B + 1,))
    hkv, d = c.num_kv_heads, c.head_dim
    total = k.shape[0] if k.dim() == 3 else -1
    strides = []
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            strides.append(0)
            continue
        if t.dtype != k_pages.dtype:
            raise TypeError("q, k, v and the cache must share one 16-bit dtype")
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
    rc = _attn.lib().attn_cache_append(
        q.data_ptr() if q is not None else None, k.data_ptr() or None, v.data_ptr() or None,
        q_out.data_ptr() if q is not None else None, *strides, B, q.shape[1] if q is not None else 0, total,
        ctypes.byref(c), cu_seqlens.data_ptr(), rot, f.data_ptr() if f is not None else None, float(amplitude),
        int(bool(interleaved)), positions.data_ptr() if positions is not None else None, s) if total else 0
    _check_rc(rc, "attn_cache_append")
    return q_out


_ws_bytes: dict = {}
_ws_kept = threading.local()
_CHUNK, _DECODE, _WEIGHTS = 0, 1, 2   # ATTN_PAGED_*


def _workspace(device: torch.device, stream: int, d: int, call: int) -> torch.Tensor:
    """Scratch memory of one call (``_scratch``)."""
    n = _ws_bytes.get((device.index, d, call))
    if n is None:
        n = _attn.lib().attn_paged_workspace_bytes(d, call)
        if n < 0:
            raise _attn.AttnError(int(n), "attn_paged_workspace_bytes")
        _ws_bytes[(device.index, d, call)] = n
    return _scratch(device, stream, n)


def _scratch(device: torch.device, stream: int, n: int) -> torch.Tensor:
    """n bytes or more.  Each thread keeps one buffer per stream that it
    has used (its calls on a stream are ordered, whichever they are), for the 8
    streams used last, of up to 41 MB each.  A captured call gets memory of its
    own, which its graph keeps.  Nothing is kept for a stream that torch does not
    own: its handle may come back as another stream's while the last call runs."""
    # (torch names a stream of another owner by its handle, and its own by an index)
    foreign = stream != 0 and torch._C._cuda_getCurrentStream(device.index)[0] == stream
    if foreign or torch.cuda.is_current_stream_capturing():
        return torch.empty(n, dtype=torch.uint8, device=device)
    kept = _ws_kept.__dict__
    key = (device.index, stream)
    ws = kept.pop(key, None)
    if ws is None or ws.numel() < n:
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        if len(kept) >= 8:
            del kept[next(iter(kept))]   # the stream used longest ago
    kept[key] = ws   # last in the dict's order
    return ws


def _outputs(q, out, lse):
    T, Hq, _ = q.shape
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != q.device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor shaped like q")
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    elif lse.shape != (Hq, T) or lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {(Hq, T)}")
    return out, lse


@_placed
def attn_fwd_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                   seqlens_k: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True,
                   scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of a chunk of new tokens over a paged cache: q (total, Hq, d)
    with offsets ``cu_seqlens`` (int32, B + 1) against the ``seqlens_k`` keys of
    each sequence; causal aligns bottom-right (the queries are the last
    positions).  Returns O like q and lse (Hq, total) float32; a query that sees
    no key gives 0 and -inf, rows outside every sequence are left as they are."""
    c = _cache(k_pages, v_pages, page_table, seqlens_k)
    _check_q(q, c, k_pages)
    B = page_table.shape[0]
    _check_int(cu_seqlens, "cu_seqlens", q.device, (B + 1,))
    if scale is None:
        scale = 1.0 / math.sqrt(c.head_dim)
    s = _stream(q.device)
    out, lse = _outputs(q, out, lse)
    ws = _workspace(q.device, s, c.head_dim, _CHUNK)
    rc = _attn.lib().attn_fwd_paged(q.data_ptr(), out.data_ptr(), lse.data_ptr(), B, q.shape[1], q.shape[0],
                                    ctypes.byref(c), cu_seqlens.data_ptr(), int(bool(causal)), float(scale),
                                    ws.data_ptr(), ws.numel(), s) if q.shape[0] else 0
    _check_rc(rc, "attn_fwd_paged")
    return out, lse


@_placed
def attn_decode_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                      seqlens_k: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One decoding step over a paged cache: q (B, Hq, d) holds one query per
    sequence, which sees all of its seqlens_k[b] keys.  Returns O (B, Hq, d)
    and lse (Hq, B) float32."""
    c = _cache(k_pages, v_pages, page_table, seqlens_k)
    _check_q(q, c, k_pages)
    if q.shape[0] != page_table.shape[0]:
        raise ValueError("q holds one row per sequence of page_table")
    if scale is None:
        scale = 1.0 / math.sqrt(c.head_dim)
    s = _stream(q.device)
    out, lse = _outputs(q, out, lse)
    ws = _workspace(q.device, s, c.head_dim, _DECODE)
    rc = _attn.lib().attn_decode_paged(q.data_ptr(), out.data_ptr(), lse.data_ptr(), q.shape[0], q.shape[1],
                                       ctypes.byref(c), float(scale), ws.data_ptr(), ws.numel(), s)
    _check_rc(rc, "attn_decode_paged")
    return out, lse


@_placed
def key_weights(q: torch.Tensor, k_pages: torch.Tensor, lse: torch.Tensor, page_table: torch.Tensor,
                seqlens_k: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True, scale: Optional[float] = None,
                decay: float = 1.0, weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Adds the attention weight that each cached key receives from the queries
    q to ``weights`` (B, Hkv, n) float32, summed over the queries and over the
    query heads of the key's head: weights = decay * weights + added.  q,
    cu_seqlens, causal and scale as the attention call had them, lse (Hq, total)
    as it returned it; after ``attn_decode_paged`` cu_seqlens is 0, 1, ..., B.
    A query whose lse is infinite is left out, whatever it holds.
    Entries past seqlens_k[b] are left as they are.  Without ``weights`` a new
    zeroed (B, Hkv, max_pages * page_size) tensor is returned."""
    c = _cache(k_pages, None, page_table, seqlens_k)
    _check_q(q, c, k_pages)
    B, dev = page_table.shape[0], q.device
    _check_int(cu_seqlens, "cu_seqlens", dev, (B + 1,))
    T, Hq, d = q.shape
    if lse.shape != (Hq, T) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor of shape {(Hq, T)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    s = _stream(dev)
    if weights is None:
        weights = torch.zeros((B, c.num_kv_heads, c.max_pages * c.page_size), dtype=torch.float32, device=dev)
    if weights.dim() != 3 or weights.shape[:2] != (B, c.num_kv_heads) or weights.dtype != torch.float32 or \
            weights.device != dev or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous float32 tensor (B, Hkv, n)")
    ws = _workspace(dev, s, d, _WEIGHTS)
    rc = _attn.lib().attn_key_weights(q.data_ptr() or None, lse.data_ptr() or None, weights.data_ptr() or None,
                                      weights.shape[2], B, Hq, T, ctypes.byref(c), cu_seqlens.data_ptr(),
                                      int(bool(causal)), float(scale), float(decay), ws.data_ptr(), ws.numel(), s)
    _check_rc(rc, "attn_key_weights")
    return weights


@_placed
def cache_evict(weights: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                seqlens_k: torch.Tensor, budget: int, recent: int = 0, dst_page_table: Optional[torch.Tensor] = None,
                weights_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Cuts every sequence back to ``budget`` keys per key/value head: its last
    ``recent`` keys and the heaviest others by ``weights`` (B, Hkv, n) float32,
    ties to the lower index, in the order of the cache.  The kept rows move to
    the front of the sequence's pages, or of the pages of ``dst_page_table``
    (int32 (B, m)), whose entries are the sequence's own page at the same place
    or pages that nothing else in the call uses.  Returns (kept (B, Hkv, budget)
    int32, -1 past the end; the new seqlens (B) int32; the kept keys' weights
    (B, Hkv, budget), 0 past the end, or ``weights_out``, which may be weights
    itself)."""
    c = _cache(k_pages, v_pages, page_table, seqlens_k)
    B, dev, hkv = page_table.shape[0], k_pages.device, c.num_kv_heads
    if not 1 <= budget <= 1 << 30 or not 0 <= recent <= budget:
        raise ValueError("budget >= 1 and 0 <= recent <= budget")
    for t in (weights, weights_out):
        if t is not None and (t.dim() != 3 or t.shape[:2] != (B, hkv) or t.dtype != torch.float32 or t.device != dev
                              or not t.is_contiguous()):
            raise ValueError("weights must be contiguous float32 tensors (B, Hkv, n)")
    if weights_out is not None and weights_out.shape[2] < budget:
        raise ValueError("weights_out must hold budget entries")
    dst, ds, dm = None, 0, 0
    if dst_page_table is not None:
        if dst_page_table.dtype != torch.int32 or dst_page_table.device != dev or dst_page_table.dim() != 2 or \
                dst_page_table.shape[0] != B or dst_page_table.stride(1) != 1:
            raise ValueError("dst_page_table must be an int32 CUDA tensor (B, m) with contiguous rows")
        dst, dm = dst_page_table.data_ptr(), dst_page_table.shape[1]
        ds = dst_page_table.stride(0) if B > 1 else dm
    s = _stream(dev)
    kept = torch.empty((B, hkv, budget), dtype=torch.int32, device=dev)
    seqlens = torch.empty(B, dtype=torch.int32, device=dev)
    if weights_out is None:
        weights_out = torch.empty((B, hkv, budget), dtype=torch.float32, device=dev)
    rc = _attn.lib().attn_cache_evict(weights.data_ptr() or None, weights.shape[2], kept.data_ptr(),
                                      seqlens.data_ptr(), weights_out.data_ptr(), weights_out.shape[2], B,
                                      ctypes.byref(c), dst, ds, dm, int(budget), int(recent), s)
    _check_rc(rc, "attn_cache_evict")
    return kept, seqlens, weights_out
