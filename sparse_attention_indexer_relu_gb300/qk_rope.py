"""Norm and rotation of query and key heads in one pass: the binding of `include/mqaqk.h`.

What a layer does between its projections and the paged cache: `qk_norm_rope` takes the heads of a (fused) projection,
and `kv_append` and `kv_attention` take its answer.
"""
from __future__ import annotations

import ctypes
from fractions import Fraction

from .kv_cache import _on, _types

QK_EXPORTS = ("mqa_qk_norm_rope",)
QK_HEAD_DIMS = (64, 128, 256)
# 2 pi, to more digits than 64-bit fractions of a turn can tell apart
_TWO_PI = Fraction("6.2831853071795864769252867665590057683943387987502")


class _Heads(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("in_stride", ctypes.c_longlong), ("out_stride", ctypes.c_longlong), ("heads", ctypes.c_int)]


def declare(L):
    """Argument types of the entry (called when the library is loaded)."""
    P, I = ctypes.c_void_p, ctypes.c_int
    H = ctypes.POINTER(_Heads)
    L.mqa_qk_norm_rope.argtypes = [H, H, I, I, I, I, I, I, I, ctypes.c_float, P, P, P]
    L.mqa_qk_norm_rope.restype = I


def _api():
    import sparse_attention_indexer_relu_gb300 as m
    return m


class _Place:
    """Where a call runs, as the cache's calls know it."""

    __slots__ = ("device", "_index")

    def __init__(self, device):
        self.device, self._index = device, device.index


def rope_turns(inv_freq, device=None):
    """A rotation's frequencies (radians per position, [rotary / 2], 32 or 64 bits) as 64-bit fractions of a turn, int64:
    what `qk_norm_rope` multiplies positions with.  Made once, on the host, as weights are."""
    import torch
    if inv_freq.dim() != 1 or inv_freq.dtype not in (torch.float32, torch.float64):
        raise TypeError("inv_freq must be a float32 or float64 tensor of one dimension")
    dev = inv_freq.device if device is None else torch.device(device)
    if dev.type != "cuda":
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else dev
    turns = []
    for f in inv_freq.double().tolist():
        t = round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64
        turns.append(t - 2 ** 64 if t >= 2 ** 63 else t)
    return torch.tensor(turns, dtype=torch.int64, device=dev)


def _heads(t, out, weight, dim, dtype, weight_type, device, name):
    """The struct of q or k; its tensors checked."""
    import torch
    if t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which qk_norm_rope does not have: detach it, or call it under "
                         "torch.no_grad()")
    for x, what in ((t, name), (out, name + "_out")):
        if x.dtype != dtype:
            raise TypeError(f"{what} must be {dtype}, got {x.dtype}")
        if x.shape != t.shape or x.dim() != 3 or x.shape[2] != dim:
            raise ValueError(f"{what} has shape {tuple(x.shape)}, expected (rows, heads, {dim})")
        if x.device != device or not x.is_cuda or (x.numel() and (x.stride(2) != 1 or
                                                                  (x.shape[1] > 1 and x.stride(1) != dim))):
            raise ValueError(f"{what} must be on {device} with its heads contiguous in a row")
    wp = None
    if weight is not None:
        if weight.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name}_weight requires a gradient, which qk_norm_rope does not have: detach it, or call it "
                             "under torch.no_grad()")
        if weight.dtype != weight_type:
            raise TypeError(f"{name}_weight must be {weight_type}, got {weight.dtype}")
        if tuple(weight.shape) != (dim,) or weight.device != device or not weight.is_contiguous():
            raise ValueError(f"{name}_weight must be a contiguous tensor ({dim},) on {device}")
        wp = weight.data_ptr()
    width = int(t.shape[1]) * dim
    many = t.shape[0] > 1
    return _Heads(t.data_ptr(), out.data_ptr(), wp, t.stride(0) if many else width, out.stride(0) if many else width,
                  int(t.shape[1]))


def qk_norm_rope(q, k, turns, positions, q_weight=None, k_weight=None, eps: float = 1e-6, norm: bool = True,
                 interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """RMS norm of every head of q [rows, q_heads, dim] and k [rows, kv_heads, dim], times the weights [dim], and the
    rotation by the rows' positions; returns (q_out, k_out).

    q, k       bf16, fp16 or fp32, of one type, dim 64, 128 or 256; rows may be strided (slices of a wider projection)
    turns      int64 [rotary / 2] (`rope_turns`), rotary a multiple of 16 up to dim: the first `rotary` components are
               turned, as pairs (i, i + rotary / 2), or (2i, 2i + 1) where interleaved; None: no rotation
    positions  int32 [rows] (None without turns)
    weights    of one type (the rows', or another of the three); None: ones.  norm=False leaves the norm out
    q_out, k_out  may be q and k themselves; other overlaps are not allowed

    Computed in 32 bits (positions times frequencies in 64), rounded once."""
    import torch
    m, types = _api(), _types()
    if q.dtype not in types:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {q.dtype}")
    if q.dim() != 3 or k.dim() != 3 or q.shape[0] != k.shape[0] or q.shape[2] not in QK_HEAD_DIMS:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)}: (rows, heads, {QK_HEAD_DIMS}) are expected")
    rows, dim, dev = int(q.shape[0]), int(q.shape[2]), q.device
    w = q_weight if q_weight is not None else k_weight
    wt = q.dtype if w is None else w.dtype
    if wt not in types:
        raise TypeError(f"weights must be bfloat16, float16 or float32, got {wt}")
    rotary = 0
    if (turns is None) != (positions is None):
        raise ValueError("turns and positions go together")
    if turns is not None:
        rotary = 2 * int(turns.shape[0])
        for t, dt, shape, name in ((turns, torch.int64, (rotary // 2,), "turns"),
                                   (positions, torch.int32, (rows,), "positions")):
            if t.dtype != dt:
                raise TypeError(f"{name} must be {dt}, got {t.dtype}")
            if tuple(t.shape) != shape or t.device != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous tensor {shape} on {dev}")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    hq = _heads(q, q if q_out is None else q_out, q_weight, dim, q.dtype, wt, dev, "q")
    hk = _heads(k, k if k_out is None else k_out, k_weight, dim, q.dtype, wt, dev, "k")
    with _on(_Place(dev), stream) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            hq.out, hq.out_stride = q_out.data_ptr(), hq.heads * dim
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=dev)
            hk.out, hk.out_stride = k_out.data_ptr(), hk.heads * dim
        m._check(m.lib().mqa_qk_norm_rope(ctypes.byref(hq), ctypes.byref(hk), rows, types[q.dtype], types[wt], dim, rotary,
                                          int(bool(interleaved)), int(bool(norm)), float(eps),
                                          turns.data_ptr() if rotary else None, positions.data_ptr() if rotary else None,
                                          s), "mqa_qk_norm_rope")
    return q_out, k_out
