"""CPU-only: what the block-scaled cache's attentions ask for as workspaces."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()
    from compressed_kv_cache_kvc_gb300 import _lib as L
    return L


@pytest.mark.parametrize("max_blocks", [1, 37, 4096])
def test_a_choice_of_more_blocks_than_a_sequence_has(lib, max_blocks):
    """top_blocks and recent_blocks may be any large numbers ("all"): the lists hold
    no more places than a sequence has blocks."""
    L = lib.lib()
    cfg = lib.KvcBlockConfig(64, 8, 128, 16, 8, 64, max_blocks, 0)
    n = L.kvc_block_state_bytes(ctypes.byref(cfg))
    raw = ctypes.create_string_buffer(n + 512)
    at = ctypes.addressof(raw)
    h = ctypes.c_void_p()
    assert L.kvc_block_cache_create(ctypes.byref(cfg), at + (-at) % 256, n, ctypes.byref(h)) == lib.KVC_OK
    size = lambda top, recent: L.kvc_block_selected_workspace_bytes(h, 64, top, recent)  # noqa: E731
    all_of_them = size(max_blocks, 0)
    for top, recent in ((1 << 20, 0), (1, (1 << 20) - 1), (1 << 19, 1 << 19), (max_blocks, 5)):
        assert size(top, recent) == all_of_them
    # the partials, the keys of every block, list and ids
    assert all_of_them <= L.kvc_block_workspace_bytes(h, 64) + 3 * (64 * 8 * max_blocks * 4 + 256)
    assert size(1, 0) <= all_of_them
    assert size(1 << 20, 1) == 0 and size(0, 1) == 0 and size(1, -1) == 0
    L.kvc_block_cache_destroy(h)
