"""Thin Python binding of the block-scaled cache (kvc_block_*): 8-bit codes with
one scale per block of tokens and KV head, the sinks and the open block in
bf16."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib as L
from .cache import HEAD_DIM, _current_device, _need, _stream_ptr
from .prompt import _ptr, _slopes, prompt_attention
from .rotary import Rotary, _first, _out, _rows


class BlockScaledCache:
    """One layer's block-scaled cache on a CUDA device."""

    def __init__(self, num_q_heads: int, num_kv_heads: int, num_blocks: int, max_batch: int, max_blocks_per_seq: int,
                 block_tokens: int = 16, codes: str = "int8", device=None, key_bounds: bool = False):
        """codes: "int8" or "e4m3"; key_bounds: keep the bounds of every block's
        keys, which `selected_attention` chooses by."""
        if codes not in ("int8", "e4m3"):
            raise ValueError('codes must be "int8" or "e4m3"')
        self.handle = None
        self.lib = L.lib()
        self.cfg = L.KvcBlockConfig(num_q_heads, num_kv_heads, HEAD_DIM, block_tokens, num_blocks, max_batch,
                                    max_blocks_per_seq, L.KVC_CODES_E4M3 if codes == "e4m3" else L.KVC_CODES_INT)
        nbytes = self.lib.kvc_block_state_bytes(ctypes.byref(self.cfg))
        if nbytes == 0:
            raise L.KvcError(L.KVC_ERR_UNSUPPORTED, "kvc_block_state_bytes")
        self.num_q_heads, self.num_kv_heads, self.block_tokens, self.codes = (num_q_heads, num_kv_heads, block_tokens,
                                                                              codes)
        self.num_blocks, self.max_batch, self.max_blocks_per_seq = num_blocks, max_batch, max_blocks_per_seq
        self.device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        if self.device.type != "cuda":
            raise ValueError("device must be a CUDA device")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        # (the caching allocator's blocks are 512-byte aligned)
        self.state = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        h = ctypes.c_void_p()
        L.check(self.lib.kvc_block_cache_create(ctypes.byref(self.cfg), _ptr(self.state), nbytes, ctypes.byref(h)),
                "kvc_block_cache_create")
        self.handle = h
        self._ws = {}
        self._ws_sized, self._ws_of = {}, {}  # buffers by size; those of recent calls' arguments
        self.bounds = None
        if key_bounds:
            nbytes = self.lib.kvc_block_key_bounds_bytes(h)
            self.bounds = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            L.check(self.lib.kvc_block_set_key_bounds(h, _ptr(self.bounds), nbytes), "kvc_block_set_key_bounds")
        self.reset()

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            self.lib.kvc_block_cache_destroy(h)
            self.handle = None

    def _call(self, name, *args, stream=None):
        if _current_device() == self.device.index:
            L.check(getattr(self.lib, name)(self.handle, *args, _stream_ptr(stream)), name)
            return
        with torch.cuda.device(self.device):
            L.check(getattr(self.lib, name)(self.handle, *args, _stream_ptr(stream)), name)

    # -- state ---------------------------------------------------------------
    def reset(self, stream=None):
        self._call("kvc_block_cache_reset", stream=stream)

    def release(self, seq_begin: int = 0, batch: int = 1, stream=None):
        """Free the sequences [seq_begin, seq_begin + batch) (idempotent)."""
        self._call("kvc_block_release", seq_begin, batch, stream=stream)

    def sync_host(self, stream=None):
        self._call("kvc_block_sync_host", stream=stream)

    def buffer(self, name: str) -> torch.Tensor:
        """Device view of one state buffer (uint8, reinterpret with .view)."""
        ptr, nb = ctypes.c_void_p(), ctypes.c_size_t()
        L.check(self.lib.kvc_block_buffer(self.handle, L.BLOCK_BUF[name], ctypes.byref(ptr), ctypes.byref(nb)),
                "kvc_block_buffer")
        off = ptr.value - self.state.data_ptr()
        return self.state[off:off + nb.value]

    def lengths(self, seq_begin: int, batch: int):
        """Tokens held: (least, most) of the sequences."""
        lo, hi = ctypes.c_int32(), ctypes.c_int32()
        L.check(self.lib.kvc_block_lengths(self.handle, seq_begin, batch, ctypes.byref(lo), ctypes.byref(hi)),
                "kvc_block_lengths")
        return lo.value, hi.value

    def length(self, seq: int) -> int:
        return self.lengths(seq, 1)[0]

    def read_status(self, stream=None) -> int:
        v = ctypes.c_int32()
        with torch.cuda.device(self.device):
            st = self.lib.kvc_block_read_status(self.handle, ctypes.byref(v), ctypes.c_void_p(_stream_ptr(stream)))
        if st not in (L.KVC_OK, L.KVC_ERR_DEVICE):
            L.check(st, "kvc_block_read_status")
        return v.value

    def last_launch_count(self) -> int:
        return int(self.lib.kvc_block_last_launch_count(self.handle))

    def workspace_bytes(self, batch: int) -> int:
        return int(self.lib.kvc_block_workspace_bytes(self.handle, batch))

    def workspace(self, batch: int) -> torch.Tensor:
        ws = self._ws.get(batch)
        if ws is None:
            ws = self._ws[batch] = torch.empty(max(self.workspace_bytes(batch), 1), dtype=torch.uint8,
                                               device=self.device)
        return ws

    # -- operators -----------------------------------------------------------
    def append(self, k: torch.Tensor, v: torch.Tensor, seq_begin: int = 0, stream=None):
        """k, v: bf16 [batch, Hkv, n_new, 128]."""
        _need(k, torch.bfloat16, "k", self.device)
        if k.dim() != 4 or k.shape[1] != self.num_kv_heads or k.shape[3] != HEAD_DIM:
            raise ValueError("k, v must be [batch, num_kv_heads, n_new, 128]")
        _need(v, torch.bfloat16, "v", self.device, k.shape)
        self._call("kvc_block_append", seq_begin, k.shape[0], k.shape[2], _ptr(k), _ptr(v), stream=stream)

    def append_rotary(self, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, rotary: Rotary, *,
                      positions: torch.Tensor | None = None, first: int = 0, seq_begin: int = 0,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
        """Append k, v (bf16 [batch, Hkv, n_new, 128]) with the keys turned on
        the way, and return the queries q (bf16 [batch, Hq, n_new, 128], or None)
        turned, packed.  All three may be strided views.  positions: int32
        [num_axes, batch, n_new], [batch, n_new] with one axis; None: first +
        the token's index in its sequence on every axis."""
        if stream is not None:
            with torch.cuda.stream(stream):  # (what is allocated below belongs to that stream)
                return self.append_rotary(q, k, v, rotary, positions=positions, first=first, seq_begin=seq_begin,
                                          out=out)
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k, v must be [batch, num_kv_heads, n_new, 128]")
        batch, n = k.shape[0], k.shape[2]
        rk = _rows(k, "k", self.device, batch, n, self.num_kv_heads, None)
        rv = _rows(v, "v", self.device, batch, n, self.num_kv_heads, None)
        pos = rotary._positions(positions, batch, n, self.device)
        rq = None
        if q is not None:
            rq = _rows(q, "q", self.device, batch, n, self.num_q_heads, None)
            out = _out(out, q, "out")
            rq.d_out = out.data_ptr()
            if rq.d_out == rq.d_in and not q.is_contiguous():
                raise ValueError("out may be q only where q is packed")
        self._call("kvc_block_append_rotary", seq_begin, batch, n, ctypes.byref(rotary.plan),
                   ctypes.byref(rq) if rq is not None else None, ctypes.byref(rk), ctypes.byref(rv), pos,
                   _first(first))
        return out if q is not None else None

    def _attention_args(self, q, out, slopes, sm_scale):
        """(out, scale) of a single-query attention, its arguments checked."""
        _need(q, torch.bfloat16, "q", self.device)
        if q.dim() != 3 or q.shape[1] != self.num_q_heads or q.shape[2] != HEAD_DIM:
            raise ValueError("q must be [batch, num_q_heads, 128]")
        if slopes is not None:
            _slopes(slopes, self.num_q_heads, self.device)
        if out is None:
            out = torch.empty_like(q)
        else:
            _need(out, torch.bfloat16, "out", self.device, q.shape)
        return out, 1.0 / math.sqrt(HEAD_DIM) if sm_scale is None else sm_scale

    def _workspace_of(self, workspace, key, nbytes):
        """`workspace`, or the cache's own for the calls of `key`.  Calls on one cache
        run one after another, so those of one size class (powers of two) share a
        buffer, whatever they ask for; it lives as long as the cache, since captured
        calls go on using it."""
        if workspace is not None:
            _need(workspace, torch.uint8, "workspace", self.device)
            return workspace
        ws = self._ws_of.get(key)
        if ws is None:
            size = 1 << max(int(nbytes()) - 1, (1 << 16) - 1).bit_length()
            ws = self._ws_sized.get(size)
            if ws is None:
                ws = self._ws_sized[size] = torch.empty(size, dtype=torch.uint8, device=self.device)
            if len(self._ws_of) >= 256:
                self._ws_of.clear()
            self._ws_of[key] = ws
        return ws

    def decode_attention(self, q: torch.Tensor, out: torch.Tensor | None = None, seq_begin: int = 0,
                         sm_scale: float | None = None, softcap: float = 0.0, slopes: torch.Tensor | None = None,
                         workspace=None, stream=None) -> torch.Tensor:
        """q: bf16 [batch, Hq, 128], at the newest position -> bf16 [batch,
        Hq, 128]; scores transformed as in `prompt_attention`."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.decode_attention(q, out, seq_begin, sm_scale, softcap, slopes, workspace)
        out, scale = self._attention_args(q, out, slopes, sm_scale)
        if workspace is None:
            ws = self.workspace(q.shape[0])
        else:
            ws = workspace
            _need(ws, torch.uint8, "workspace", self.device)
        self._call("kvc_block_attention", seq_begin, q.shape[0], _ptr(q), _ptr(out), scale,
                   softcap, _ptr(slopes), _ptr(ws), ws.numel())
        return out

    def selected_attention(self, q: torch.Tensor, top_blocks: int, *, recent_blocks: int = 1,
                           out: torch.Tensor | None = None, seq_begin: int = 0, sm_scale: float | None = None,
                           softcap: float = 0.0, slopes: torch.Tensor | None = None,
                           return_blocks: bool | torch.Tensor = False, workspace=None, stream=None):
        """`decode_attention` to the sinks, the open block, the `recent_blocks`
        newest closed blocks and, of the others, the `top_blocks` that score
        highest: an estimate of a block's largest product with the query heads of
        the KV head from its keys' bounds (a cache made with key_bounds).  return_blocks: True, or an int32 tensor
        [batch, Hkv, top_blocks + recent_blocks], returns (out, blocks) with the
        chosen blocks, ascending, -1 behind the last."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.selected_attention(q, top_blocks, recent_blocks=recent_blocks, out=out,
                                               seq_begin=seq_begin, sm_scale=sm_scale, softcap=softcap, slopes=slopes,
                                               return_blocks=return_blocks, workspace=workspace)
        if self.bounds is None:
            raise ValueError("selected_attention needs a cache made with key_bounds=True")
        if top_blocks < 1 or recent_blocks < 0 or top_blocks + recent_blocks > 1 << 20:
            raise ValueError("top_blocks must be positive, recent_blocks not negative, both together at most 2^20")
        out, scale = self._attention_args(q, out, slopes, sm_scale)
        batch = q.shape[0]
        blocks = None
        if return_blocks is not False:
            shape = (batch, self.num_kv_heads, top_blocks + recent_blocks)
            if return_blocks is True:
                blocks = torch.empty(shape, dtype=torch.int32, device=self.device)
            else:
                blocks = return_blocks
                _need(blocks, torch.int32, "return_blocks", self.device, shape)
        ws = self._workspace_of(workspace, ("selected", batch, top_blocks, recent_blocks),
                                lambda: self.lib.kvc_block_selected_workspace_bytes(self.handle, batch, top_blocks,
                                                                                    recent_blocks))
        self._call("kvc_block_selected_attention", seq_begin, batch, top_blocks, recent_blocks, _ptr(q), _ptr(out),
                   _ptr(blocks), scale, softcap, _ptr(slopes), _ptr(ws), ws.numel())
        return out if blocks is None else (out, blocks)

    def prefix_attention(self, q: torch.Tensor, prefix: int, *, out: torch.Tensor | None = None, seq_begin: int = 0,
                         sm_scale: float | None = None, softcap: float = 0.0, slopes: torch.Tensor | None = None,
                         workspace=None, stream=None) -> torch.Tensor:
        """`decode_attention` of sequences that share a prefix, held once as the
        sequence `prefix`: each query sees the prefix and then its own sequence
        (appended with first = the prefix's length where keys are rotated)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.prefix_attention(q, prefix, out=out, seq_begin=seq_begin, sm_scale=sm_scale,
                                             softcap=softcap, slopes=slopes, workspace=workspace)
        out, scale = self._attention_args(q, out, slopes, sm_scale)
        batch = q.shape[0]
        ws = self._workspace_of(workspace, ("prefix", batch),
                                lambda: self.lib.kvc_block_prefix_workspace_bytes(self.handle, batch))
        self._call("kvc_block_prefix_attention", prefix, seq_begin, batch, _ptr(q), _ptr(out), scale, softcap,
                   _ptr(slopes), _ptr(ws), ws.numel())
        return out

    def prefill(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, status: torch.Tensor, seq_begin: int = 0,
                stream=None, **attention) -> torch.Tensor:
        """A fresh prompt: append it and return `prompt_attention` of it (over
        its exact bf16 keys and values; `attention` goes to it unchanged).  A
        refused call leaves the cache, the outputs and `status` as they were."""
        _need(q, torch.bfloat16, "q", self.device)
        if q.dim() != 4 or q.shape[1] != self.num_q_heads or q.shape[3] != HEAD_DIM:
            raise ValueError("q must be [batch, num_q_heads, n, 128]")
        batch = q.shape[0]
        _need(k, torch.bfloat16, "k", self.device, (batch, self.num_kv_heads, q.shape[2], HEAD_DIM))
        if self.lengths(seq_begin, batch)[1] != 0:
            raise L.KvcError(L.KVC_ERR_STATE, "prefill")
        # the append asks for room before it writes; where the attention then
        # refuses its arguments the (so far empty) sequences are given up again
        self.append(k, v, seq_begin=seq_begin, stream=stream)
        try:
            return prompt_attention(q, k, v, status=status, stream=stream, **attention)
        except Exception:
            self.release(seq_begin, batch, stream=stream)
            raise

    def read(self, seq_begin: int = 0, batch: int = 1, pos_begin: int = 0, n: int | None = None, out=None,
             stream=None):
        """Positions [pos_begin, pos_begin + n) of the sequences as dense
        bf16 (k, v), [batch, Hkv, n, 128] each, as the attention sees them; rows
        at or past a sequence's length are left as they are in `out` (zero
        without `out`)."""
        if stream is not None:
            with torch.cuda.stream(stream):  # (the zeros too)
                return self.read(seq_begin, batch, pos_begin, n, out)
        least, most = self.lengths(seq_begin, batch)
        if n is None:
            n = most - pos_begin
        shape = (batch, self.num_kv_heads, n, HEAD_DIM)
        if out is None:
            if batch < 1 or n < 1:
                raise ValueError("batch and n must be positive")
            make = torch.empty if pos_begin + n <= least else torch.zeros
            k = make(shape, dtype=torch.bfloat16, device=self.device)
            v = make(shape, dtype=torch.bfloat16, device=self.device)
        else:
            k, v = out
            _need(k, torch.bfloat16, "k", self.device, shape)
            _need(v, torch.bfloat16, "v", self.device, shape)
        self._call("kvc_block_read", seq_begin, batch, pos_begin, n, k.data_ptr(), v.data_ptr())
        return k, v
