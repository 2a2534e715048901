"""Rotary positions (kvc_rotary_rotate): queries and keys turned by their
positions, along one axis (text) or several (images and video)."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib as L
from .cache import HEAD_DIM, _current_device, _need, _stream_ptr


def _rows(t, name, device, batch, n, heads, out):
    """A KvcRows of bf16 rows [batch, heads, n, 128], strided or packed."""
    if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor of dtype {torch.bfloat16}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.shape != (batch, heads, n, HEAD_DIM):
        raise ValueError(f"{name} must be [batch, heads, n, 128] = {(batch, heads, n, HEAD_DIM)}, not {tuple(t.shape)}")
    sb, sh, st, sd = t.stride()
    ptr = t.data_ptr()
    if (sd != 1 or ptr % 16 or (sb % 8 and batch > 1) or (sh % 8 and heads > 1) or (st % 8 and n > 1)):
        raise ValueError(f"the rows of {name} must be of 128 adjacent values and start on 16-byte boundaries")
    return L.KvcRows(ptr, None if out is None else out.data_ptr(), heads, sb, sh, st)


def _first(first):
    if not -1 << 31 <= first < 1 << 31:
        raise ValueError("first must be a 32-bit position")
    return first


def _out(out, t, name):
    """The packed output of rows t: `out`, or a new tensor."""
    if out is None:
        return torch.empty_like(t, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
    _need(out, torch.bfloat16, name, t.device, t.shape)
    return out


class Rotary:
    """The rotation of a model: pair i of a row, (x, y), becomes (x cos t - y sin t,
    y cos t + x sin t) with t = freqs[i] times the position on the pair's axis.  Set
    up once; needs no GPU."""

    def __init__(self, rotary_dim: int = HEAD_DIM, base: float = 10000.0, freqs=None, axes=None,
                 adjacent: bool = False):
        """rotary_dim: values of a row that turn (a multiple of 16), the others
        pass; adjacent: pairs (2i, 2i + 1), else (i, i + rotary_dim / 2); freqs:
        rotary_dim / 2 angles per position (base ** (-2i / rotary_dim) without);
        axes: the axis of every pair, 0 to 3 (all 0 without)."""
        if rotary_dim < 16 or rotary_dim > HEAD_DIM or rotary_dim % 16:
            raise ValueError("rotary_dim must be a multiple of 16 up to 128")
        half = rotary_dim // 2
        if freqs is None:
            if not base > 0:
                raise ValueError("base must be positive")
            freqs = [float(base) ** (-i / half) for i in range(half)]
        freqs = [float(f) for f in freqs]
        axes = [0] * half if axes is None else [int(a) for a in axes]
        if len(freqs) != half or len(axes) != half:
            raise ValueError(f"freqs and axes must have rotary_dim / 2 = {half} entries")
        if not all(math.isfinite(f) and abs(f) <= 65536.0 for f in freqs):
            raise ValueError("freqs must be finite and at most 65536 in magnitude")
        if not all(0 <= a < L.KVC_ROTARY_AXES for a in axes):
            raise ValueError("axes must lie in 0 .. 3")
        self.rotary_dim, self.adjacent, self.num_axes = rotary_dim, bool(adjacent), max(axes) + 1
        self.plan = L.KvcRotary(rotary_dim, int(self.adjacent), self.num_axes, (ctypes.c_float * 64)(*freqs),
                                (ctypes.c_uint8 * 64)(*axes))

    def _positions(self, positions, batch, n, device):
        """The positions' pointer: int32 [num_axes, batch, n] ([batch, n] with one axis)."""
        if positions is None:
            return None
        shape = (self.num_axes, batch, n)
        if isinstance(positions, torch.Tensor) and self.num_axes == 1 and positions.dim() == 2:
            shape = (batch, n)
        _need(positions, torch.int32, "positions", device, shape)
        return positions.data_ptr()

    def rotate(self, q: torch.Tensor, k: torch.Tensor | None = None, *, positions: torch.Tensor | None = None,
               first: int = 0, out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
        """q bf16 [batch, Hq, n, 128] and k [batch, Hkv, n, 128] (strided views
        as well), turned: packed bf16 tensors of the same shapes, q alone without
        k.  positions: int32 [num_axes, batch, n], [batch, n] with one axis; None:
        first + i on every axis.  out, k_out: packed, q and k themselves where
        these are packed."""
        if stream is not None:
            with torch.cuda.stream(stream):  # (what is allocated below belongs to that stream)
                return self.rotate(q, k, positions=positions, first=first, out=out, k_out=k_out)
        if not isinstance(q, torch.Tensor) or q.dim() != 4 or not q.numel():
            raise ValueError("q must be [batch, heads, n, 128]")
        if k is not None and (not isinstance(k, torch.Tensor) or k.dim() != 4 or not k.numel()):
            raise ValueError("k must be [batch, heads, n, 128]")
        batch, hq, n, _ = q.shape
        dev = q.device
        if not q.is_cuda:
            raise ValueError("q must be a CUDA tensor")
        pos = self._positions(positions, batch, n, dev)
        out = _out(out, q, "out")
        rq = _rows(q, "q", dev, batch, n, hq, out)
        if out.data_ptr() == q.data_ptr() and not q.is_contiguous():
            raise ValueError("out may be q only where q is packed")
        rk = None
        if k is not None:
            k_out = _out(k_out, k, "k_out")
            rk = _rows(k, "k", dev, batch, n, k.shape[1], k_out)
            if k_out.data_ptr() == k.data_ptr() and not k.is_contiguous():
                raise ValueError("k_out may be k only where k is packed")
        args = (ctypes.byref(self.plan), batch, n, ctypes.byref(rq), ctypes.byref(rk) if rk is not None else None, pos,
                _first(first))
        if _current_device() == dev.index:
            st = L.lib().kvc_rotary_rotate(*args, _stream_ptr())
        else:
            with torch.cuda.device(dev):
                st = L.lib().kvc_rotary_rotate(*args, _stream_ptr())
        L.check(st, "kvc_rotary_rotate")
        return out if k is None else (out, k_out)
