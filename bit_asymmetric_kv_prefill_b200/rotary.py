"""Rotary positions: the rotation of queries and keys (kivi_rope) and its
frequency tables (kivi_rope_frequencies)."""
from __future__ import annotations

import ctypes

import torch

from . import RopeScaling, RopeTensor, _check, _dtype_code, _on_device, _stream_ptr, lib

PLAIN, LINEAR, BASE, YARN, BANDS = "plain", "linear", "base", "yarn", "bands"
_KINDS = {PLAIN: 0, LINEAR: 1, BASE: 2, YARN: 3, BANDS: 4}


def rope_frequencies(rotary_dim: int, theta: float = 10000.0, scaling: str = PLAIN, factor: float = 1.0,
                     original: float = 0.0, low: float = 1.0, high: float = 32.0, device=None):
    """(inv_freq, scale) for :func:`rope`: fp32 [rotary_dim/2] on ``device``
    (the current GPU unless given) and the factor on the rotated channels.
    ``scaling`` is "plain", "linear", "base", "yarn" or "bands" (see
    kivi_rope_frequencies); ``original`` is the context the model was trained
    on, ``low`` and ``high`` the turns between which "yarn" and "bands" blend."""
    if scaling not in _KINDS:
        raise ValueError(f"scaling must be one of {sorted(_KINDS)}, got {scaling!r}")
    f = (ctypes.c_float * max(1, rotary_dim // 2))()
    m = ctypes.c_float()
    s = RopeScaling(_KINDS[scaling], factor, original, low, high)
    _check(lib().kivi_rope_frequencies(rotary_dim, theta, ctypes.byref(s), f, ctypes.byref(m)),
           "kivi_rope_frequencies")
    t = torch.tensor(list(f), dtype=torch.float32)
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return t.to(device), m.value


def _side(x, y, D, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dim() != 3 or x.shape[2] != D or x.stride(2) != 1:
        raise ValueError(f"{name} must have shape [tokens, heads, {D}] with contiguous channels")
    if y.shape != x.shape or y.dtype != x.dtype or y.device != x.device or y.stride(2) != 1:
        raise ValueError(f"the output of {name} must match its shape, type and device, channels contiguous")
    return RopeTensor(x.data_ptr(), y.data_ptr(), x.shape[1], x.stride(0), x.stride(1), y.stride(0), y.stride(1))


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor,
         rotary_dim: int | None = None, interleaved: bool = False, scale: float = 1.0, inverse: bool = False,
         fp32_angles: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
         stream=None):
    """Rotate q [tokens, heads, D] and k [tokens, kv heads, D] (bf16 or fp16 on
    the GPU, any token and head strides; k may be None) by their positions
    (int32 or int64 [tokens]); see kivi_rope.  ``q_out``/``k_out`` default to
    new contiguous tensors; pass ``q_out=q`` to rotate in place.
    ``inverse=True`` undoes the rotation, and is its gradient.

    Returns (q_out, k_out)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 3:
        raise ValueError("q must be a CUDA tensor [tokens, heads, D]")
    N, _, D = q.shape
    rot = D if rotary_dim is None else rotary_dim
    if positions.dtype not in (torch.int32, torch.int64) or positions.device != q.device \
            or tuple(positions.shape) != (N,) or not positions.is_contiguous():
        raise ValueError(f"positions must be contiguous int32 or int64 [{N}] on {q.device}")
    if inv_freq.dtype != torch.float32 or inv_freq.device != q.device or not inv_freq.is_contiguous() \
            or inv_freq.numel() != rot // 2:
        raise ValueError(f"inv_freq must be contiguous float32 [{rot // 2}] on {q.device}")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k is None:
        t = (RopeTensor * 1)(_side(q, q_out, D, "q"))
    else:
        if not isinstance(k, torch.Tensor) or k.dtype != q.dtype or k.device != q.device or k.dim() != 3 \
                or k.shape[0] != N:
            raise ValueError("k must match q's tokens, type and device")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        t = (RopeTensor * 2)(_side(q, q_out, D, "q"), _side(k, k_out, D, "k"))
    with _on_device(q.device):
        _check(lib().kivi_rope(t, len(t), _dtype_code(q.dtype), N, D, positions.data_ptr(),
                               int(positions.dtype == torch.int64), inv_freq.data_ptr(), rot, int(interleaved),
                               scale, int(inverse), int(fp32_angles), _stream_ptr(stream)), "kivi_rope")
    return q_out, k_out
