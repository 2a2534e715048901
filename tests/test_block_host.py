"""CPU-only: the host-side checks of the block-scaled cache, the prompt
attention and the score transform refuse bad calls before anything reaches a
GPU; the plain 64-bit forms that the GPU tests use are checked against closed
cases."""
import ctypes

import numpy as np
import pytest

from tests import ops64 as R


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()
    from compressed_kv_cache_kvc_gb300 import _lib as L
    return L


class _Buffer:
    """Aligned host memory standing in for device memory that no call below may touch."""

    def __init__(self, n):
        self.n = n
        self.raw = ctypes.create_string_buffer(n + 512)
        addr = ctypes.addressof(self.raw)
        self.addr = addr + (-addr) % 256
        self.ptr = ctypes.c_void_p(self.addr)


def _cfg(lib, **kw):
    d = dict(num_q_heads=8, num_kv_heads=2, head_dim=128, block_tokens=16, num_blocks=3, max_batch=2,
             max_blocks_per_seq=2, codes=0)
    d.update(kw)
    return lib.KvcBlockConfig(**d)


def test_block_config(lib):
    L = lib.lib()
    n = L.kvc_block_state_bytes(ctypes.byref(_cfg(lib)))
    assert n % 256 == 0 and n >= 2 * 3 * 2 * 16 * 128 + 2 * 2 * 2 * 20 * 128 * 2
    assert n == L.kvc_block_state_bytes(ctypes.byref(_cfg(lib, codes=lib.KVC_CODES_E4M3)))
    for bad in (dict(head_dim=64), dict(block_tokens=8), dict(block_tokens=48), dict(block_tokens=256),
                dict(num_q_heads=7), dict(num_q_heads=32), dict(num_blocks=0), dict(codes=2), dict(max_batch=1025),
                dict(max_batch=0), dict(max_blocks_per_seq=1 << 28), dict(num_blocks=1 << 28)):
        assert L.kvc_block_state_bytes(ctypes.byref(_cfg(lib, **bad))) == 0, bad
    h = ctypes.c_void_p()
    buf = _Buffer(n)
    mk = lambda p, m: L.kvc_block_cache_create(ctypes.byref(_cfg(lib)), p, m, ctypes.byref(h))  # noqa: E731
    assert mk(buf.ptr, n - 1) == lib.KVC_ERR_INVALID_ARG and not h.value
    assert mk(ctypes.c_void_p(buf.addr + 16), n) == lib.KVC_ERR_INVALID_ARG
    assert mk(None, n) == lib.KVC_ERR_INVALID_ARG
    assert L.kvc_block_cache_create(None, buf.ptr, n, ctypes.byref(h)) == lib.KVC_ERR_INVALID_ARG
    L.kvc_block_cache_destroy(None)


def test_block_calls(lib):
    L = lib.lib()
    n = L.kvc_block_state_bytes(ctypes.byref(_cfg(lib)))
    buf, h = _Buffer(n), ctypes.c_void_p()
    assert L.kvc_block_cache_create(ctypes.byref(_cfg(lib)), buf.ptr, n, ctypes.byref(h)) == lib.KVC_OK
    p = buf.ptr
    ptr, nb, v = ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_int32()
    assert L.kvc_block_buffer(h, 0, ctypes.byref(ptr), ctypes.byref(nb)) == lib.KVC_OK
    assert ptr.value == buf.addr and nb.value == 3 * 2 * 16 * 128
    assert L.kvc_block_buffer(h, 11, ctypes.byref(ptr), ctypes.byref(nb)) == lib.KVC_ERR_INVALID_ARG
    assert L.kvc_block_lengths(h, 1, 1, ctypes.byref(v), None) == lib.KVC_OK and v.value == 0
    assert L.kvc_block_lengths(h, 1, 2, ctypes.byref(v), None) == lib.KVC_ERR_INVALID_ARG
    bad = lib.KVC_ERR_INVALID_ARG
    assert L.kvc_block_append(None, 0, 1, 1, p, p, None) == bad
    for args, want in [((1, 2, 1), bad), ((0, 1, -1), bad), ((-1, 1, 1), bad), ((0, 0, 1), bad),
                       ((0, 1, 52), lib.KVC_ERR_CAPACITY), ((0, 2, 36), lib.KVC_ERR_CAPACITY),
                       ((0, 1, 2000000001), lib.KVC_ERR_CAPACITY), ((0, 1, 0), lib.KVC_OK)]:
        assert L.kvc_block_append(h, *args, p, p, None) == want, args
    mis = ctypes.c_void_p(buf.addr + 8)
    assert L.kvc_block_append(h, 0, 1, 1, mis, p, None) == bad
    assert L.kvc_block_append(h, 0, 1, 1, p, None, None) == bad
    ws = L.kvc_block_workspace_bytes(h, 2)
    assert ws > L.kvc_block_workspace_bytes(h, 1) > 0
    assert L.kvc_block_workspace_bytes(h, 3) == 0 and L.kvc_block_workspace_bytes(h, 0) == 0
    att = lambda sc=0.1, cap=0.0, s=0, b=1, q=p, w=p, m=ws: L.kvc_block_attention(  # noqa: E731
        h, s, b, q, p, ctypes.c_float(sc), ctypes.c_float(cap), None, w, m, None)
    for kw in [dict(), dict(sc=0.0), dict(sc=float("inf")), dict(cap=-1.0), dict(cap=float("nan")), dict(s=2),
               dict(b=3), dict(q=mis), dict(w=mis), dict(m=16), dict(w=None)]:  # (the first: an empty sequence)
        assert att(**kw) == bad, kw
    for args in [(0, 3, 0, 1), (0, 1, -1, 1), (0, 1, 0, 0), (2, 1, 0, 1), (0, 1, 2000000000, 1)]:
        assert L.kvc_block_read(h, *args, p, p, None) == bad, args
    assert L.kvc_block_read(h, 0, 1, 0, 1, mis, p, None) == bad
    assert L.kvc_block_release(h, 0, 3, None) == bad
    assert L.kvc_block_release(h, 0, 2, None) == lib.KVC_OK  # empty: nothing to launch
    assert L.kvc_block_last_launch_count(h) == 0
    L.kvc_block_cache_destroy(h)


def test_prompt_calls(lib):
    L = lib.lib()
    assert L.kvc_prompt_workspace_bytes(1, 8, 2, 100, 1) > L.kvc_prompt_workspace_bytes(1, 8, 2, 100, 0) >= \
        100 * 2 * 256
    for a in [(0, 8, 2, 100), (1, 0, 2, 100), (1, 8, 0, 100), (1, 8, 2, 0), (1, 7, 2, 10)]:
        assert L.kvc_prompt_workspace_bytes(*a, 0) == 0
    buf = _Buffer(1 << 20)
    p, mis = buf.ptr, ctypes.c_void_p(buf.addr + 8)

    def call(q=p, k=p, v=p, o=p, sums=None, status=p, ws=p, nbytes=1 << 20, **kw):
        d = dict(batch=1, num_q_heads=8, num_kv_heads=2, n=10, sm_scale=0.1, softcap=0.0, d_slopes=None,
                 d_key_begin=None, d_key_end=None)
        d.update(kw)
        prm = lib.KvcPromptParams(**d)
        return L.kvc_prompt_attention(ctypes.byref(prm), q, k, v, o, sums, status, ws, nbytes, None)

    for kw in [dict(batch=0), dict(n=0), dict(n=-5), dict(num_kv_heads=3), dict(num_q_heads=0), dict(q=mis),
               dict(k=None), dict(v=mis), dict(o=None), dict(status=None), dict(sums=ctypes.c_void_p(buf.addr + 2)),
               dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(softcap=-0.5), dict(softcap=float("inf")),
               dict(ws=mis), dict(ws=None), dict(nbytes=100), dict(d_slopes=ctypes.c_void_p(buf.addr + 1)),
               dict(d_key_begin=ctypes.c_void_p(buf.addr + 2)), dict(d_key_end=ctypes.c_void_p(buf.addr + 1))]:
        assert call(**kw) == lib.KVC_ERR_INVALID_ARG, kw
    assert L.kvc_prompt_attention(None, p, p, p, p, None, p, p, 1 << 20, None) == lib.KVC_ERR_INVALID_ARG
    for kw in [dict(batch=70000), dict(num_q_heads=70000, num_kv_heads=70000), dict(n=0x7FFFFFFF),
               dict(batch=60000, num_q_heads=60000, num_kv_heads=60000)]:
        assert call(**kw) == lib.KVC_ERR_UNSUPPORTED, kw


def test_transform_and_masked_prefill_calls(lib):
    L = lib.lib()
    cfg = lib.KvcConfig(num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=16, bits=8, num_blocks=8, max_batch=2,
                        max_blocks_per_seq=4)
    n = L.kvc_state_bytes(ctypes.byref(cfg))
    buf, h = _Buffer(max(n, 1 << 20)), ctypes.c_void_p()
    assert L.kvc_cache_create(ctypes.byref(cfg), buf.ptr, n, ctypes.byref(h)) == lib.KVC_OK
    p = buf.ptr
    for cap in (-1.0, float("nan"), float("inf")):
        assert L.kvc_set_score_transform(h, ctypes.c_float(cap), None) == lib.KVC_ERR_INVALID_ARG
    assert L.kvc_set_score_transform(h, ctypes.c_float(1.0), ctypes.c_void_p(buf.addr + 2)) == lib.KVC_ERR_INVALID_ARG
    assert L.kvc_set_score_transform(None, ctypes.c_float(1.0), None) == lib.KVC_ERR_INVALID_ARG
    plain = L.kvc_prefill_workspace_bytes(h, 1, 50)
    assert L.kvc_set_score_transform(h, ctypes.c_float(30.0), p) == lib.KVC_OK
    grown = L.kvc_prefill_workspace_bytes(h, 1, 50)
    assert grown == L.kvc_prefill_masked_workspace_bytes(h, 1, 50) > plain
    assert L.kvc_set_score_transform(h, ctypes.c_float(0.0), None) == lib.KVC_OK
    assert L.kvc_prefill_workspace_bytes(h, 1, 50) == plain
    call = lambda s=0, b=1, m=50, sc=0.1, fl=1, kb=None, nb=1 << 20: L.kvc_prefill_attention_masked(  # noqa: E731
        h, s, b, m, p, p, p, p, ctypes.c_float(sc), fl, kb, None, p, nb, None)
    for kw in [dict(s=2), dict(m=0), dict(fl=2), dict(sc=-1.0), dict(kb=ctypes.c_void_p(buf.addr + 1)), dict(nb=64)]:
        assert call(**kw) == lib.KVC_ERR_INVALID_ARG, kw
    assert call(m=70) == lib.KVC_ERR_CAPACITY
    assert L.kvc_last_launch_count(h) == 0
    L.kvc_cache_destroy(h)


def test_plain_forms():
    """The 64-bit forms against cases one can do by hand."""
    x = np.zeros((4 + 16 + 3, 128), np.float32)
    x[4, 0], x[5, 1], x[6, 2] = 127.0, 2.5, -3.5   # scale 1: halves round to even
    x[20:] = 0.3
    held = R.held_block(x, 16, False)
    assert held[4, 0] == 127 and held[5, 1] == 2 and held[6, 2] == -4 and (held[20:] == np.float32(0.3)).all()
    x[4, 0], x[5, 1], x[6, 2] = 448.0, 17.0, 0.0029296875  # E4M3, scale 1: 17 -> 16 (even), 1.5 * 2^-9 -> 2 * 2^-9
    held = R.held_block(x, 16, True)
    assert held[4, 0] == 448 and held[5, 1] == 16 and held[6, 2] == 2.0 ** -8
    p = R.softmax_rows(np.array([[0.0, -np.inf, 0.0], [-np.inf] * 3]))
    assert np.array_equal(p, [[0.5, 0, 0.5], [0, 0, 0]])
    z = R.scores(np.ones((1, 2)), np.ones((2, 2)), 1.0, 4.0, 0.5, [3], [3, 1])
    assert np.allclose(z, [[4 * np.tanh(0.5), 4 * np.tanh(0.5) - 1.0]])


def test_document_runs():
    from compressed_kv_cache_kvc_gb300 import document_runs
    begin, end = document_runs([3, 0, 2], prefix=2)
    assert begin.tolist() == [[0, 0, 0, 3, 3]] and end.tolist() == [[2, 2, 3, 5, 5]]
    with pytest.raises(ValueError):
        document_runs([3, -1])
