"""Attentions captured into a graph at long sequences and replayed at short
ones: the captured grid then has more CTAs than there are pages, and those
without one must count for nothing."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R
from tests import test_gpu_block_cache as B

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _check_block(out, q, k, v, lengths, block, codes, cap):
    """Rows of `out` against the formula on what the cache holds of k, v."""
    got = T.bf16_tensor_to_f32(out)
    hq, hkv = q.shape[1], k[0].shape[0]
    for b, m in enumerate(lengths):
        for j in range(hq):
            h = j * hkv // hq
            kd, vd = B._held(k[b][h], m, block, codes), B._held(v[b][h], m, block, codes)
            z = R.scores(O.bf16_bits_to_f32(q[b, j:j + 1]), kd, SCALE, cap, 0.0, [m - 1], np.arange(m))
            p = R.softmax_rows(z)
            ref = p @ vd
            bound = R.output_bound(ref, p, vd, R.score_error(z, cap, np.ones_like(z, bool)))
            err = np.abs(got[b, j] - ref[0])
            assert (err <= bound[0]).all(), (m, b, j, float((err / bound[0]).max()))


@pytest.mark.parametrize("codes,block,batch,first,then", [
    ("int8", 16, 1, 8000, [100, 20, 1, 500]),
    ("e4m3", 16, 1, 4000, [100, 4]),
    ("int8", 16, 1, 1000, [20]),
    ("e4m3", 32, 2, 5000, [37, 900]),  # several sequences of one length: equal runs of units
])
def test_block_attention_at_fewer_tokens(codes, block, batch, first, then):
    """Replayed at every length of `then`, each after a release, then eager
    calls that join partial results: the tickets are zero between calls and the
    outputs those of the formula."""
    rng = np.random.default_rng(first + batch)
    hq, hkv, cap = 16, 8, 6.0
    cache = B._cache(hq, hkv, [first] * batch, block, codes)
    draw = lambda n: B._bits(rng, (batch, hkv, n, 128))  # noqa: E731
    k, v = draw(first), draw(first)
    cache.append(T.to_dev_bf16(k), T.to_dev_bf16(v))
    qb = B._bits(rng, (batch, hq, 128), 1.5)
    q = T.to_dev_bf16(qb)
    out, ws = torch.empty_like(q), torch.empty_like(cache.workspace(batch))
    cache.decode_attention(q, out=out, workspace=ws, softcap=cap)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention(q, out=out, workspace=ws, softcap=cap)
    for n in then:
        cache.release(0, batch)
        k, v = draw(n), draw(n)
        cache.append(T.to_dev_bf16(k), T.to_dev_bf16(v))
        for _ in range(2):
            out.fill_(7.0)
            ws.fill_(255)  # (NaN in every partial result)
            graph.replay()
            torch.cuda.synchronize()
            assert (cache.buffer("TICKETS").view(torch.int32) == 0).all(), n
            _check_block(out, qb, k, v, [n] * batch, block, codes, cap)
    more_k, more_v = draw(first - n), draw(first - n)
    cache.append(T.to_dev_bf16(more_k), T.to_dev_bf16(more_v))
    k, v = np.concatenate([k, more_k], 2), np.concatenate([v, more_v], 2)
    for call in (graph.replay, lambda: cache.decode_attention(q, out=out, workspace=ws, softcap=cap)):
        out.fill_(7.0)
        call()
        torch.cuda.synchronize()
        _check_block(out, qb, k, v, [first] * batch, block, codes, cap)
    assert (cache.buffer("TICKETS").view(torch.int32) == 0).all() and cache.read_status() == 0


def _token_cache(hq, hkv, bits, codes, first, window):
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    pages = first // 16 + 4
    return KVCache(hq, hkv, bits, 2 * pages, 2, pages, bf16_window=window, codes=codes)


@pytest.mark.parametrize("bits,codes,first,then,window,cap", [
    (8, "int", 4000, [60, 5, 400], 0, 0.0),
    (4, "int", 3000, [40, 17], 0, 8.0),
    (8, "e4m3", 2500, [90], 32, 8.0),
])
def test_token_attention_at_fewer_tokens(bits, codes, first, then, window, cap):
    """The per-token cache: outputs and H2O scores of a replay at shorter
    lengths equal an eager call's on the same state (another grid's order of
    sums), whatever the workspace held."""
    rng = np.random.default_rng(first)
    hq, hkv = 16, 8
    cache, twin = (_token_cache(hq, hkv, bits, codes, first, window) for _ in range(2))
    for c in (cache, twin):
        c.set_score_transform(softcap=cap)
    draw = lambda n: T.to_dev_bf16(B._bits(rng, (2, hkv, n, 128)))  # noqa: E731
    k, v = draw(first), draw(first)
    cache.quantize_append(k, v)
    q = T.to_dev_bf16(B._bits(rng, (2, hq, 128), 1.5))
    out, ws = torch.empty_like(q), torch.empty_like(cache.workspace(2))
    cache.decode_attention(q, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention(q, out=out, workspace=ws)
    for n in then:
        k, v = draw(n), draw(n)
        for c in (cache, twin):
            c.release(0, 2)
            c.quantize_append(k, v)
        out.fill_(7.0)
        ws.fill_(255)
        graph.replay()
        want = twin.decode_attention(q)
        torch.cuda.synchronize()
        torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
        a, b = T.StateView(cache), T.StateView(twin)
        for s in range(2):
            for h in range(hkv):
                ns = min(n, 4)
                np.testing.assert_allclose(a.sink_score[s, h, :ns], b.sink_score[s, h, :ns], rtol=1e-4, atol=1e-6)
                np.testing.assert_allclose(a.head(s, h)[5], b.head(s, h)[5], rtol=1e-4, atol=1e-6)
                if window:
                    np.testing.assert_allclose(a.ring_head(s, h)[3], b.ring_head(s, h)[3], rtol=1e-4, atol=1e-6)
    assert cache.read_status() == 0 and twin.read_status() == 0


@pytest.mark.parametrize("bits,window", [(8, 0), (4, 0), (8, 24)])
def test_token_step_at_fewer_tokens(bits, window):
    """A whole decode step captured at 3,000 tokens, replayed at 50: the same
    outputs, kept positions and scores as the step called eagerly."""
    rng = np.random.default_rng(bits)
    hq, hkv, first, n = 16, 8, 3000, 50
    cache, twin = (_token_cache(hq, hkv, bits, "int", first, window) for _ in range(2))
    draw = lambda h, n: T.to_dev_bf16(B._bits(rng, (2, h, n, 128)))  # noqa: E731
    k, v = draw(hkv, first), draw(hkv, first)
    cache.quantize_append(k, v)
    q = T.to_dev_bf16(B._bits(rng, (2, hq, 128), 1.5))
    kn, vn = draw(hkv, 1), draw(hkv, 1)
    out, ws = torch.empty_like(q), torch.empty_like(cache.workspace(2))
    # (the recent tokens cover the window)
    keep = dict(mode="h2o", budget=36 + window // 2, recent=8 + window)
    step = lambda c, **kw: c.decode_step(q, kn, vn, **keep, **kw)  # noqa: E731
    twin.quantize_append(k[:, :, :n].contiguous(), v[:, :, :n].contiguous())
    step(twin)  # (the first call, outside a capture)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out=out, workspace=ws)
    cache.sync_host()
    k, v = draw(hkv, n), draw(hkv, n)
    for c in (cache, twin):
        c.release(0, 2)
        c.quantize_append(k, v)
    ws.fill_(255)
    graph.replay()
    want = step(twin)
    torch.cuda.synchronize()
    cache.sync_host()
    torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
    a, b = T.StateView(cache), T.StateView(twin)
    assert np.array_equal(a.slots, b.slots) and np.array_equal(a.seen, b.seen)
    for s in range(2):
        for h in range(hkv):
            pa, pb = a.head(s, h)[0], b.head(s, h)[0]
            assert sorted(pa.tolist()) == sorted(pb.tolist())
            np.testing.assert_allclose(a.head(s, h)[5][np.argsort(pa)], b.head(s, h)[5][np.argsort(pb)], rtol=1e-4,
                                       atol=1e-6)
    assert cache.read_status() == 0 and twin.read_status() == 0
