"""Workspaces of the block-scaled cache's attentions: choices larger than a
sequence, and what a cache keeps over many kinds of calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _cache(lengths, hq=8, hkv=2, block=16, bounds=True):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    g = torch.Generator(device="cuda")
    g.manual_seed(len(lengths))
    counts = [max(n - 4, 0) // block for n in lengths]
    c = BlockScaledCache(hq, hkv, max(sum(counts), 1), len(lengths), max(max(counts), 1), block_tokens=block,
                         key_bounds=bounds)
    for b, n in enumerate(lengths):
        k, v = (torch.randn(1, hkv, n, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        c.append(k, v, seq_begin=b)
    return c, torch.randn(len(lengths), hq, 128, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("top,recent", [(1 << 19, 1 << 19), (62, 0), (61, 0), (3, 70), (1, 4)])
@pytest.mark.parametrize("bias", [False, True])
def test_choices_larger_than_a_sequence(top, recent, bias):
    """A workspace of exactly the bytes asked for, with a guard behind it; the blocks
    given back in rows of top_blocks + recent_blocks all the same."""
    lengths = [1000, 5, 300]  # 62, 0 and 18 blocks
    c, q = _cache(lengths)
    slopes = torch.tensor([2.0 ** -j for j in range(8)], device="cuda") if bias else None
    n = c.lib.kvc_block_selected_workspace_bytes(c.handle, 3, top, recent)
    guarded = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    call = lambda **kw: c.selected_attention(q, top, recent_blocks=recent, slopes=slopes, **kw)  # noqa: E731
    out = call(workspace=guarded[:n])
    again, blocks = call(workspace=guarded[:n], return_blocks=True)
    assert (guarded[n:] == 0xA5).all() and torch.equal(out, again) and torch.equal(out, call())
    whole = c.decode_attention(q, slopes=slopes)
    for b, m in enumerate(lengths):
        closed = max(m - 4, 0) // 16
        kept = blocks[b] if top + recent < 4096 else blocks[b, :, :4096]
        assert (blocks[b, :, kept.shape[1]:] == -1).all()
        for h in range(2):
            got = kept[h].tolist()
            taken = [x for x in got if x >= 0]
            assert len(taken) == min(closed, top + recent) and taken == sorted(set(taken))
            assert got[len(taken):] == [-1] * (len(got) - len(taken))
        if closed <= top + recent:
            torch.testing.assert_close(out[b].float(), whole[b].float(), rtol=2 ** -7, atol=1e-3)
    assert c.read_status() == 0


def test_a_cache_keeps_few_workspaces():
    """Calls of many batches and choices share a few buffers; the results are those of
    workspaces of their own, also of calls captured before the buffers were shared."""
    lengths = [900] + [40 + 7 * b for b in range(12)]
    c, q = _cache(lengths)
    lib, h = c.lib, c.handle
    kinds = [(b, top, recent) for b in (1, 2, 5, 12) for top in range(1, 60) for recent in (0, 3)]
    largest = max(max(lib.kvc_block_selected_workspace_bytes(h, *k) for k in kinds),
                  max(lib.kvc_block_prefix_workspace_bytes(h, b) for b in range(1, 13)))
    c.prefix_attention(q[1:6], 0, seq_begin=1)
    held = torch.empty_like(q[1:6])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.prefix_attention(q[1:6], 0, seq_begin=1, out=held)
    before = torch.cuda.memory_allocated()
    for k in kinds:
        got = c.selected_attention(q[:k[0]], k[1], recent_blocks=k[2])
        if k[1] % 19 == 1:
            own = torch.empty(lib.kvc_block_selected_workspace_bytes(h, *k), dtype=torch.uint8, device="cuda")
            assert torch.equal(got, c.selected_attention(q[:k[0]], k[1], recent_blocks=k[2], workspace=own))
    for b in range(1, 13):
        got = c.prefix_attention(q[1:1 + b], 0, seq_begin=1)
        own = torch.empty(lib.kvc_block_prefix_workspace_bytes(h, b), dtype=torch.uint8, device="cuda")
        assert torch.equal(got, c.prefix_attention(q[1:1 + b], 0, seq_begin=1, workspace=own))
    own = got = None
    # size classes are powers of two: all buffers together are below four times the largest need
    assert torch.cuda.memory_allocated() - before <= 4 * largest + (1 << 20)
    graph.replay()
    assert torch.equal(held, c.prefix_attention(q[1:6], 0, seq_begin=1)) and c.read_status() == 0
