"""CPU-only: what the rotary positions refuse before anything reaches a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()
    from compressed_kv_cache_kvc_gb300 import _lib as L
    return L


def _memory(n):
    raw = ctypes.create_string_buffer(n + 512)
    addr = ctypes.addressof(raw)
    return raw, addr + (-addr) % 256


def test_plan():
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(64, base=100.0, axes=[0] * 8 + [1] * 12 + [2] * 12)
    assert rot.num_axes == 3 and rot.plan.axes == 3 and rot.plan.rotary_dim == 64
    assert rot.plan.freq[0] == 1.0 and abs(rot.plan.freq[16] - 0.1) < 1e-8 and rot.plan.freq[32] == 0.0
    for bad in (dict(rotary_dim=8), dict(rotary_dim=144), dict(rotary_dim=40), dict(base=0.0), dict(base=float("nan")),
                dict(freqs=[1.0] * 63), dict(freqs=[float("inf")] * 64), dict(freqs=[1e6] * 64), dict(axes=[4] * 64),
                dict(axes=[-1] * 64), dict(axes=[0] * 32)):
        with pytest.raises(ValueError):
            Rotary(**bad)


def test_rotate_refuses(lib):
    from compressed_kv_cache_kvc_gb300 import Rotary
    L = lib.lib()
    raw, at = _memory(1 << 16)
    plan = Rotary(64, axes=[0] * 16 + [1] * 16).plan

    def rows(**kw):
        d = dict(d_in=at, d_out=at + 8192, heads=2, stride_batch=2048, stride_head=1024, stride_token=128)
        d.update(kw)
        return lib.KvcRows(d["d_in"], d["d_out"], d["heads"], d["stride_batch"], d["stride_head"], d["stride_token"])

    def call(p=plan, batch=2, n=8, q=rows(), k=None, pos=None):
        return L.kvc_rotary_rotate(ctypes.byref(p) if p is not None else None, batch, n,
                                   ctypes.byref(q) if q is not None else None,
                                   ctypes.byref(k) if k is not None else None, pos, 0, None)

    bad = lib.KVC_ERR_INVALID_ARG
    for kw in (dict(p=None), dict(batch=0), dict(n=0), dict(n=-1), dict(q=None), dict(pos=at + 2)):
        assert call(**kw) == bad, kw
    for r in (dict(d_in=None), dict(d_in=at + 8), dict(d_out=None), dict(d_out=at + 8200), dict(heads=0),
              dict(stride_batch=2047), dict(stride_head=1), dict(stride_token=129),
              dict(d_out=at, stride_token=256), dict(d_out=at, stride_batch=4096)):
        assert call(q=rows(**r)) == bad, r
        assert call(k=rows(**r)) == bad, r
    for field, value, want in (("rotary_dim", 8, lib.KVC_ERR_UNSUPPORTED), ("rotary_dim", 144, lib.KVC_ERR_UNSUPPORTED),
                               ("rotary_dim", 60, lib.KVC_ERR_UNSUPPORTED), ("adjacent", 2, bad), ("axes", 0, bad),
                               ("axes", 5, bad), ("axes", 1, bad)):
        p = lib.KvcRotary.from_buffer_copy(plan)
        setattr(p, field, value)
        assert call(p=p) == want, field
    for value in (float("nan"), float("inf"), 65537.0, -1e9):
        p = lib.KvcRotary.from_buffer_copy(plan)
        p.freq[31] = value
        assert call(p=p) == bad
    del raw


def test_append_rotary_refuses(lib):
    from compressed_kv_cache_kvc_gb300 import Rotary
    L = lib.lib()
    cfg = lib.KvcBlockConfig(4, 2, 128, 16, 3, 2, 2, 0)
    n = L.kvc_block_state_bytes(ctypes.byref(cfg))
    raw, at = _memory(n + (1 << 16))
    h = ctypes.c_void_p()
    assert L.kvc_block_cache_create(ctypes.byref(cfg), at, n, ctypes.byref(h)) == lib.KVC_OK
    room = at + n
    plan = Rotary().plan

    def call(begin=0, batch=2, n_new=8, p=plan, heads=(4, 2, 2), q=True, k_in=room):
        r = [lib.KvcRows(k_in if i == 1 else room, room + 32768 if i == 0 else None, m, 8192, 1024, 128)
             for i, m in enumerate(heads)]
        return L.kvc_block_append_rotary(h, begin, batch, n_new, ctypes.byref(p) if p is not None else None,
                                         ctypes.byref(r[0]) if q else None, ctypes.byref(r[1]), ctypes.byref(r[2]),
                                         None, 0, None)

    bad = lib.KVC_ERR_INVALID_ARG
    for kw in (dict(begin=-1), dict(begin=1), dict(batch=0), dict(n_new=-1), dict(p=None), dict(heads=(2, 2, 2)),
               dict(heads=(4, 1, 2)), dict(heads=(4, 2, 4)), dict(k_in=None), dict(k_in=room + 2)):
        assert call(**kw) == bad, kw
    for first in (2 ** 31 - 8, 2 ** 31 - 1):  # the last of eight positions has 32 bits at most
        r = [lib.KvcRows(room, room + 32768, m, 8192, 1024, 128) for m in (4, 2, 2)]
        got = L.kvc_block_append_rotary(h, 0, 1, 9, ctypes.byref(plan), None, ctypes.byref(r[1]), ctypes.byref(r[2]), None,
                                        first, None)
        assert got == bad
        assert L.kvc_rotary_rotate(ctypes.byref(plan), 2, 9, ctypes.byref(r[0]), None, None, first, None) == bad
    assert call(n_new=36) == lib.KVC_ERR_CAPACITY and call(batch=1, n_new=52) == lib.KVC_ERR_CAPACITY
    assert call(n_new=0) == lib.KVC_OK
    assert L.kvc_block_append_rotary(None, 0, 1, 1, None, None, None, None, None, 0, None) == bad
    # the keys' bounds
    nb = L.kvc_block_key_bounds_bytes(h)
    assert nb == 3 * 2 * 256 + 256 and L.kvc_block_key_bounds_bytes(None) == 0
    assert L.kvc_block_set_key_bounds(None, room, nb) == bad
    assert L.kvc_block_set_key_bounds(h, (room + 255) // 256 * 256 + 16, nb) == bad
    assert L.kvc_block_set_key_bounds(h, (room + 255) // 256 * 256, nb - 1) == bad
    assert L.kvc_block_set_key_bounds(h, (room + 255) // 256 * 256, nb) == lib.KVC_OK
    assert L.kvc_block_set_key_bounds(h, None, 0) == lib.KVC_OK
    L.kvc_block_cache_destroy(h)
    del raw
