"""Norms of the queries' and keys' heads with their rotary embedding, over one or
several axes of positions (include/attn.h, attn_qk_norm_rotary), and the
gradients.

Like the rest of the binding this marshals arguments only.  ``qk_norm_rotary``
and ``qk_norm_rotary_bwd`` take ``stream`` by name (default: the current stream of
their tensors' device); ``qk_norm_rotary_func``, the one with autograd, runs on the
current stream.
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import attn as _attn
from .paged import _HALF, _check_rc, _freqs, _placed, _scratch, _stream


def declare(L) -> None:
    """Argument types of the entry points."""
    vp, i, f, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
    tail = [ll, ll, ll, ll, i, i, i, i, vp, vp, i, f, i, vp, vp, i, f, i, vp, i]
    L.attn_qk_norm_rotary.argtypes = [vp] * 4 + tail + [vp]
    L.attn_qk_norm_rotary_bwd.argtypes = [vp] * 8 + tail + [vp, ll, vp]
    L.attn_qk_norm_workspace_bytes.argtypes = [i]
    L.attn_qk_norm_rotary.restype = L.attn_qk_norm_rotary_bwd.restype = i
    L.attn_qk_norm_workspace_bytes.restype = ll


@functools.lru_cache(maxsize=64)
def _axis_table(axes: Tuple[int, ...], n_axes: int, pairs: int):
    if len(axes) != pairs or not all(0 <= a < n_axes for a in axes):
        raise ValueError(f"axes names one of the {n_axes} axes for each of the {pairs} pairs")
    return (ctypes.c_int * pairs)(*axes)


def _strides(x: torch.Tensor, shape, rows: int, name: str) -> Tuple[int, int]:
    """(token, head) strides of x, (rows, H, d) or (B, L, H, d)."""
    st = x.stride()
    H, d = shape[-2:]
    if d > 1 and st[-1] != 1:
        raise ValueError(f"the features of {name} must be contiguous")
    token = st[-3]
    if len(shape) == 4:
        B, L = shape[:2]
        if B > 1 and L > 1 and st[0] != L * st[1]:
            raise ValueError(f"the tokens of {name} must be evenly strided over batch and length")
        token = st[1] if L > 1 else st[0]
    head = st[-2] if H > 1 else d
    # strides of an axis of one entry address nothing: any valid value serves
    return token if rows > 1 else H * max(head, d), head


def _weight(name: str, w: Optional[torch.Tensor], dtype, dev, d: int) -> Optional[int]:
    if w is None:
        return None
    if w.dtype != dtype and w.dtype != torch.float32:
        raise TypeError(f"{name} must be float32 or of the tensors' dtype")
    if w.device != dev or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {d} entries on {dev}")
    return w.data_ptr()


def _arguments(q, k, q_weight, k_weight, freqs, positions, axes, eps, amplitude, interleaved):
    """The arguments that both directions share, as the library takes them from
    the strides on, and what has to stay alive until the call."""
    dtype, dev, shape = q.dtype, q.device, q.shape
    if dtype not in _HALF or (k is not None and k.dtype != dtype):
        raise TypeError("q and k must share one 16-bit dtype")
    if not q.is_cuda or len(shape) not in (3, 4):
        raise ValueError("q is a CUDA tensor (tokens, Hq, d) or (B, L, Hq, d)")
    lead, (Hq, d) = shape[:-2], shape[-2:]
    if Hq == 0 or d == 0:
        raise ValueError("q has no heads or no features")
    rows = lead.numel()
    if rows >= 1 << 31:
        raise ValueError("q has 2^31 tokens or more")
    sq, sk, Hk = _strides(q, shape, rows, "q"), (0, 0), 0
    if k is not None:
        kshape = k.shape
        if k.device != dev or len(kshape) != len(shape) or kshape[:-2] != lead or kshape[-1] != d or kshape[-2] == 0:
            raise ValueError("k is shaped like q but for its heads, on the same device")
        Hk = kshape[-2]
        sk = _strides(k, kshape, rows, "k")
    wq = _weight("q_weight", q_weight, dtype, dev, d)
    if k_weight is not None and k is None:
        raise ValueError("k_weight without its heads")
    wk = _weight("k_weight", k_weight, dtype, dev, d)
    if wq is not None and wk is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must share one dtype")
    w = q_weight if q_weight is not None else k_weight
    w32 = int(w is not None and w.dtype == torch.float32)
    f, rot, n_axes, table, pos = None, 0, 1, None, None
    if freqs is None:
        if positions is not None or axes is not None:
            raise ValueError("positions and axes without freqs")
    else:
        f, rot = _freqs(freqs, d)
        if positions is None:
            raise ValueError("freqs without positions")
        pshape = positions.shape
        if positions.dtype != torch.int32 or positions.device != dev or not positions.is_contiguous() or \
                (pshape != lead and pshape[1:] != lead):
            raise ValueError("positions must be a contiguous int32 tensor of q's leading shape, or (axes, ...) of it")
        pos = positions.data_ptr()
        if len(pshape) > len(lead):
            n_axes = pshape[0]
        if axes is not None:
            table = _axis_table(tuple(map(int, axes)), n_axes, rot // 2)
        elif n_axes != 1:
            raise ValueError("positions of several axes need axes")
    args = (*sq, *sk, rows, Hq, Hk, d, wq, wk, w32, float(eps), rot, f.data_ptr() if f is not None else None, table, n_axes,
            float(amplitude), int(bool(interleaved)), pos, int(dtype == torch.float16))
    return args, (f, table)


def _output(x, out, name):
    if x is None:
        if out is not None:
            raise ValueError(f"{name} without k")
        return None
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of its input's shape and dtype")
    return out


def _ptr(t):
    return (t.data_ptr() or None) if t is not None else None


@_placed
def qk_norm_rotary(q: torch.Tensor, k: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                   k_weight: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None,
                   positions: Optional[torch.Tensor] = None, axes: Optional[Sequence[int]] = None, eps: float = 1e-6,
                   amplitude: float = 1.0, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                   k_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Every head of q (tokens, Hq, d) or (B, L, Hq, d), and of k beside it (or
    None), divided by the root of its mean square plus ``eps``, times the weights
    (d entries, of q's dtype or float32; None: ones), and rotated by
    ``freqs`` (``rotary_freqs``; None: not rotated) times ``amplitude``.

    ``positions`` int32 of q's leading shape; or (axes, ...) of it, and ``axes``
    names for each pair p of features (rot_dim / 2 entries) the axis whose position
    turns it: [0] * 16 + [1] * 24 + [2] * 24 for time, height and width, or any
    other order.  d and rot_dim multiples of 16.  q and k may be strided (slices of
    one projection's output), with contiguous features; ``q_out`` and ``k_out``
    (contiguous) may be q and k themselves where those are contiguous."""
    args, _keep = _arguments(q, k, q_weight, k_weight, freqs, positions, axes, eps, amplitude, interleaved)
    s = _stream(q.device)
    q_out, k_out = _output(q, q_out, "q_out"), _output(k, k_out, "k_out")
    rc = _attn.lib().attn_qk_norm_rotary(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), *args, s)
    _check_rc(rc, "attn_qk_norm_rotary")
    return q_out, k_out


_ws_bytes: dict = {}


def _workspace(device: torch.device, stream: int, d: int) -> torch.Tensor:
    n = _ws_bytes.get((device.index, d))
    if n is None:
        n = _attn.lib().attn_qk_norm_workspace_bytes(d)
        if n < 0:
            raise _attn.AttnError(int(n), "attn_qk_norm_workspace_bytes")
        _ws_bytes[(device.index, d)] = n
    return _scratch(device, stream, n)


@_placed
def qk_norm_rotary_bwd(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor, k: Optional[torch.Tensor] = None,
                       q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                       freqs: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                       axes: Optional[Sequence[int]] = None, eps: float = 1e-6, amplitude: float = 1.0,
                       interleaved: bool = False, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                       weight_grads: bool = True):
    """Gradients (dq, dk, dq_weight, dk_weight) of ``qk_norm_rotary``, from those of
    its outputs (contiguous) and its arguments.  A weight's gradient has its dtype,
    is summed in float32, in an order that the sizes alone fix, and is None for a
    weight that was, or without ``weight_grads``.  ``dq`` and ``dk`` may be dq_out and
    dk_out themselves."""
    args, _keep = _arguments(q, k, q_weight, k_weight, freqs, positions, axes, eps, amplitude, interleaved)
    if (k is None) != (dk_out is None):
        raise ValueError("dk_out comes with k")
    for name, g, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if x is not None and (g.shape != x.shape or g.dtype != x.dtype or g.device != x.device or not g.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous tensor of its output's shape and dtype")
    s = _stream(q.device)
    dq, dk = _output(q, dq, "dq"), _output(k, dk, "dk")
    dwq, dwk = (torch.empty_like(w) if w is not None and weight_grads else None for w in (q_weight, k_weight))
    ws = _workspace(q.device, s, q.shape[-1]) if dwq is not None or dwk is not None else None
    rc = _attn.lib().attn_qk_norm_rotary_bwd(_ptr(dq_out), _ptr(dk_out), _ptr(q), _ptr(k), _ptr(dq), _ptr(dk), _ptr(dwq),
                                             _ptr(dwk), *args, _ptr(ws), ws.numel() if ws is not None else 0, s)
    _check_rc(rc, "attn_qk_norm_rotary_bwd")
    return dq, dk, dwq, dwk


class _QkNormRotaryFunction(torch.autograd.Function):
    """The forward keeps its inputs alone; the backward forms the norms again."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, freqs, positions, axes, eps, amplitude, interleaved):
        y = qk_norm_rotary(q, k, q_weight, k_weight, freqs, positions, axes, eps, amplitude, interleaved)
        f = _freqs(freqs, q.shape[-1])[0] if freqs is not None else None
        # (freqs and positions too, so that a change of theirs before the backward is an error)
        ctx.save_for_backward(q, k, q_weight, k_weight, f, positions)
        ctx.args = (axes, eps, amplitude, interleaved)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, freqs, positions = ctx.saved_tensors
        grads = qk_norm_rotary_bwd(dq_out.contiguous(), dk_out.contiguous() if k is not None else None, q, k, q_weight,
                                   k_weight, freqs, positions, *ctx.args,
                                   weight_grads=ctx.needs_input_grad[2] or ctx.needs_input_grad[3])
        return (*grads,) + (None,) * 6


def qk_norm_rotary_func(q: torch.Tensor, k: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                        k_weight: Optional[torch.Tensor] = None, freqs: Optional[torch.Tensor] = None,
                        positions: Optional[torch.Tensor] = None, axes: Optional[Sequence[int]] = None, eps: float = 1e-6,
                        amplitude: float = 1.0, interleaved: bool = False):
    """``qk_norm_rotary`` with gradients for q, k and the weights, on the current
    stream (frequencies and positions are constants: changing them in place before
    the backward is an error).  The gradients have none of their own: asking for one
    is an error.  A backward that is captured into a CUDA graph needs,
    as with any operator of torch, that no eager graph of the same leaves is alive."""
    axes = tuple(int(a) for a in axes) if axes is not None else None
    return _QkNormRotaryFunction.apply(q, k, q_weight, k_weight, freqs, positions, axes, float(eps), float(amplitude),
                                       bool(interleaved))
