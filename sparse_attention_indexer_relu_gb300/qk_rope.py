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


def _entry(*args):
    """The C entry; loads the library at the first call."""
    global _entry
    _entry = _api().lib().mqa_qk_norm_rope
    return _entry(*args)


class _Place:
    """Where a call runs, as the cache's calls know it."""

    __slots__ = ("_index",)

    def __init__(self, index):
        self._index = index

    @property
    def device(self):
        import torch
        return torch.device("cuda", self._index)


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


def _layout(t, dtype, shape, where, name):
    """Row stride of a tensor [rows, heads, dim] on device `where` whose heads lie side by side in a row."""
    rows, heads, dim = shape
    across, beside, within = t.stride()
    if t.get_device() != where or (rows and heads and (within != 1 or (heads > 1 and beside != dim))):
        raise ValueError(f"{name} must be on cuda:{where} with its heads contiguous in a row")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return across if rows > 1 else heads * dim


def _no_gradient(t, name):
    if t.requires_grad and _api()._torch().is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, which qk_norm_rope does not have: detach it, or call it under "
                         "torch.no_grad()")


def _heads(t, shape, out, weight, dtype, weight_type, where, name):
    """The struct of q or k; its tensors checked (out is None: made by the caller)."""
    _no_gradient(t, name)
    stride = _layout(t, dtype, shape, where, name)
    _, heads, dim = shape
    op, os, wp = None, heads * dim, None
    if out is not None:
        if out.shape != shape:
            raise ValueError(f"{name}_out has shape {tuple(out.shape)}, expected {tuple(shape)}")
        os = _layout(out, dtype, shape, where, name + "_out")
        op = out.data_ptr()
    if weight is not None:
        _no_gradient(weight, name + "_weight")
        if weight.dtype != weight_type:
            raise TypeError(f"{name}_weight must be {weight_type}, got {weight.dtype}")
        if weight.shape != (dim,) or weight.get_device() != where or not weight.is_contiguous():
            raise ValueError(f"{name}_weight must be a contiguous tensor ({dim},) on cuda:{where}")
        wp = weight.data_ptr()
    return _Heads(t.data_ptr(), op, wp, stride, os, heads)


def _list(t, dtype, n, where, name):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or t.get_device() != where or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor ({n},) on cuda:{where}")
    return t.data_ptr()


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
    dtype, where, qs, ks = q.dtype, q.get_device(), q.shape, k.shape
    if dtype not in types:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dtype}")
    if where < 0:
        raise ValueError("q must be a CUDA tensor")
    if len(qs) != 3 or len(ks) != 3 or qs[0] != ks[0] or qs[2] != ks[2] or qs[2] not in QK_HEAD_DIMS:
        raise ValueError(f"q {tuple(qs)} and k {tuple(ks)}: (rows, heads, {QK_HEAD_DIMS}) are expected")
    weight = k_weight if q_weight is None else q_weight
    weight_type = dtype if weight is None else weight.dtype
    if weight_type not in types:
        raise TypeError(f"weights must be bfloat16, float16 or float32, got {weight_type}")
    rotary, tp, pp = 0, None, None
    if (turns is None) != (positions is None):
        raise ValueError("turns and positions go together")
    if turns is not None:
        half = turns.shape[0]
        rotary = 2 * half
        tp, pp = _list(turns, torch.int64, half, where, "turns"), _list(positions, torch.int32, qs[0], where, "positions")
        if not rotary:
            tp = pp = None
    hq = _heads(q, qs, q_out, q_weight, dtype, weight_type, where, "q")
    hk = _heads(k, ks, k_out, k_weight, dtype, weight_type, where, "k")
    with _on(_Place(where), stream) as s:
        if q_out is None:
            q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
            hq.out = q_out.data_ptr()
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            hk.out = k_out.data_ptr()
        rc = _entry(hq, hk, qs[0], types[dtype], types[weight_type], qs[2], rotary, 1 if interleaved else 0,
                    1 if norm else 0, eps, tp, pp, s)
    if rc:
        m._check(rc, "mqa_qk_norm_rope")
    return q_out, k_out
