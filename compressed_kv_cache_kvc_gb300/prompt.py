"""Attention of prompts over themselves with score transforms and per-query
runs of keys (kvc_prompt_attention), without a cache."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib as L
from .cache import HEAD_DIM, _current_device, _need, _stream_ptr


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _slopes(slopes, num_q_heads, device):
    if slopes is not None:
        _need(slopes, torch.float32, "slopes", device, (num_q_heads,))
    return slopes


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, status: torch.Tensor, out=None,
                     sm_scale: float | None = None, softcap: float = 0.0, slopes: torch.Tensor | None = None,
                     key_begin: torch.Tensor | None = None, key_end: torch.Tensor | None = None,
                     column_sums: bool | torch.Tensor = False, workspace=None, stream=None):
    """q bf16 [batch, Hq, n, 128], k/v bf16 [batch, Hkv, n, 128] -> bf16
    [batch, Hq, n, 128]; query i sees the keys [key_begin[i], key_end[i])
    (int32 [batch, n]; None: from 0, and up to itself).  Scores are capped at
    `softcap` by a tanh (0: not) and lowered by slopes[head] * distance
    (float32 [Hq]).  column_sums: True, or a float32 [batch, Hkv, n] tensor,
    returns (out, sums) with every key's sum of probabilities.  status: int32
    [1], zeroed by the caller; KVC_DEV_* bits are or'ed into it."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or q.shape[3] != HEAD_DIM:
        raise ValueError("q must be [batch, num_q_heads, n, 128]")
    _need(q, torch.bfloat16, "q")
    dev = q.device
    batch, hq, n = q.shape[0], q.shape[1], q.shape[2]
    _need(k, torch.bfloat16, "k", dev)
    if k.dim() != 4 or k.shape[0] != batch or k.shape[2] != n or k.shape[3] != HEAD_DIM or k.shape[1] < 1 or \
            hq % k.shape[1] != 0:
        raise ValueError("k, v must be [batch, num_kv_heads, n, 128], num_kv_heads a divisor of num_q_heads")
    hkv = k.shape[1]
    _need(v, torch.bfloat16, "v", dev, k.shape)
    _need(status, torch.int32, "status", dev, (1,))
    _slopes(slopes, hq, dev)
    for name, t in (("key_begin", key_begin), ("key_end", key_end)):
        if t is not None:
            _need(t, torch.int32, name, dev, (batch, n))
    sums = None
    if column_sums is not False:
        sums = torch.empty(batch, hkv, n, dtype=torch.float32, device=dev) if column_sums is True else column_sums
        _need(sums, torch.float32, "column_sums", dev, (batch, hkv, n))
    if out is None:
        out = torch.empty_like(q)
    _need(out, torch.bfloat16, "out", dev, q.shape)
    lib = L.lib()
    if workspace is None:
        # (the caching allocator's blocks are 512-byte aligned)
        nbytes = lib.kvc_prompt_workspace_bytes(batch, hq, hkv, n, sums is not None)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _need(workspace, torch.uint8, "workspace", dev)
    scale = 1.0 / math.sqrt(HEAD_DIM) if sm_scale is None else sm_scale
    params = L.KvcPromptParams(batch, hq, hkv, n, scale, softcap, _ptr(slopes), _ptr(key_begin), _ptr(key_end))

    def call():
        L.check(lib.kvc_prompt_attention(ctypes.byref(params), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                         _ptr(sums), status.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                         _stream_ptr(stream)), "kvc_prompt_attention")

    if _current_device() == dev.index:
        call()
    else:
        with torch.cuda.device(dev):
            call()
    return out if sums is None else (out, sums)


def document_runs(lengths, prefix=0, device=None):
    """(key_begin, key_end), int32 [1, n], of documents of the given lengths
    packed end to end: causal inside each document, the first `prefix` tokens
    of each seeing each other both ways."""
    begin, end, at = [], [], 0
    for m in lengths:
        if m < 0 or prefix < 0:
            raise ValueError("lengths and prefix must not be negative")
        two_way = at + min(prefix, m)
        begin += [at] * m
        end += [max(i + 1, two_way) if i < two_way else i + 1 for i in range(at, at + m)]
        at += m
    return (torch.tensor([begin], dtype=torch.int32, device=device),
            torch.tensor([end], dtype=torch.int32, device=device))
