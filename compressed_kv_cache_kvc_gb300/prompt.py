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
    if stream is not None:
        # what is allocated below then belongs to that stream, as the kernels do
        with torch.cuda.stream(stream):
            return prompt_attention(q, k, v, status=status, out=out, sm_scale=sm_scale, softcap=softcap, slopes=slopes,
                                    key_begin=key_begin, key_end=key_end, column_sums=column_sums,
                                    workspace=workspace)
    bf16 = torch.bfloat16
    _need(q, bf16, "q")
    if q.dim() != 4 or q.shape[3] != HEAD_DIM:
        raise ValueError("q must be [batch, num_q_heads, n, 128]")
    dev = q.device
    batch, hq, n, _ = q.shape
    _need(k, bf16, "k", dev)
    hkv = k.shape[1] if k.dim() == 4 else 0
    if hkv < 1 or hq % hkv != 0 or k.shape != (batch, hkv, n, HEAD_DIM):
        raise ValueError("k, v must be [batch, num_kv_heads, n, 128], num_kv_heads a divisor of num_q_heads")
    _need(v, bf16, "v", dev, k.shape)
    _need(status, torch.int32, "status", dev, (1,))
    if slopes is not None:
        _slopes(slopes, hq, dev)
    if key_begin is not None:
        _need(key_begin, torch.int32, "key_begin", dev, (batch, n))
    if key_end is not None:
        _need(key_end, torch.int32, "key_end", dev, (batch, n))
    sums = None
    if column_sums is True:
        sums = torch.empty(batch, hkv, n, dtype=torch.float32, device=dev)
    elif column_sums is not False:
        sums = column_sums
        _need(sums, torch.float32, "column_sums", dev, (batch, hkv, n))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, bf16, "out", dev, q.shape)
    lib = L.lib()
    if workspace is None:
        # (the caching allocator's blocks are 512-byte aligned)
        ws_bytes = lib.kvc_prompt_workspace_bytes(batch, hq, hkv, n, sums is not None)
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, torch.uint8, "workspace", dev)
        ws_bytes = workspace.numel()
    scale = 1.0 / math.sqrt(HEAD_DIM) if sm_scale is None else sm_scale
    params = L.KvcPromptParams(batch, hq, hkv, n, scale, softcap, _ptr(slopes), _ptr(key_begin), _ptr(key_end))
    args = (ctypes.byref(params), q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), _ptr(sums),
            status.data_ptr(), workspace.data_ptr(), ws_bytes)
    if _current_device() == dev.index:
        st = lib.kvc_prompt_attention(*args, _stream_ptr())
    else:
        with torch.cuda.device(dev):
            st = lib.kvc_prompt_attention(*args, _stream_ptr())
    L.check(st, "kvc_prompt_attention")
    return out if sums is None else (out, sums)


def document_runs(lengths, prefix=0, device=None):
    """(key_begin, key_end), int32 [1, n], of documents of the given lengths
    packed end to end: causal inside each document, the first `prefix` tokens
    of each seeing each other both ways.  One row; rows of a batch are
    concatenated (or repeated) by the caller."""
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
