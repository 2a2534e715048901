"""Edges of the transformed and block-scaled operators: values that are not
finite, caps at the ends of fp32, sequences a replayed graph finds empty, joins
of every query-group size, appends larger than one wave of CTAs, calls on a
stream that is not the current one, one workspace used call after call."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R
from tests import test_gpu_block_cache as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_blocks_with_values_that_are_not_finite(codes):
    """A NaN gets code 0 and counts for nothing; an infinity makes the scale
    infinite and every code 0; the blocks beside them are as ever."""
    rng = np.random.default_rng(3)
    block, n = 32, 4 + 4 * 32
    k = B._bits(rng, (1, 1, n, 128))
    f = O.bf16_bits_to_f32(k[0, 0])
    k[0, 0, 4 + 5, 7::16], k[0, 0, 4 + 9] = 0x7FC0, 0xFFC0      # NaN in block 0
    k[0, 0, 4 + 2 * block + 3, 100] = 0xFF80                     # -inf in block 2
    cache = B._cache(1, 1, [n], block, codes)
    dk = T.to_dev_bf16(k)
    cache.append(dk, dk)
    raw = cache.buffer("K_CODES").view(-1, block, 128)
    raw = (raw.view(torch.float8_e4m3fn) if codes == "e4m3" else raw.view(torch.int8)).cpu().double().numpy()
    scales = cache.buffer("K_SCALE").view(torch.float32).cpu().numpy()
    table = cache.buffer("TABLE").view(torch.int32).cpu()
    g = O.bf16_bits_to_f32(k[0, 0])
    f = np.where(np.isnan(g), np.float32(0), f)
    for c in range(4):
        blk = int(table[c])
        if c == 2:
            assert np.isinf(scales[blk]) and (raw[blk] == 0).all()
            continue
        want, scale = R.quantise_block(f[4 + c * block:4 + (c + 1) * block], codes == "e4m3")
        assert scales[blk] == scale and np.array_equal(raw[blk], want), c


@pytest.mark.parametrize("group", range(1, 9))
def test_joins_of_every_group_size(group):
    B.test_attention_against_formula(group, 1, [2000, 37, 700], 16, "int8", 8.0, group % 2 == 0, 2.0)


def test_a_replay_finds_a_sequence_empty():
    rng = np.random.default_rng(4)
    cache = B._cache(8, 2, [100] * 3, 16, "int8")
    k = T.to_dev_bf16(B._bits(rng, (3, 2, 100, 128)))
    cache.append(k, k)
    q = T.to_dev_bf16(B._bits(rng, (3, 8, 128)))
    out = torch.empty_like(q)
    want = cache.decode_attention(q).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention(q, out=out)
    for empty in ([], [1], [0, 1], [0, 1, 2]):
        for b in empty:
            cache.release(b)
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            if b in empty:
                assert (out[b] == 0).all()
            else:  # (the same values; another grid's order of sums)
                torch.testing.assert_close(out[b].float(), want[b].float(), rtol=2 ** -7, atol=1e-3)
    assert cache.read_status() == 0


@pytest.mark.parametrize("hkv,lengths", [(2, [2000, 37, 700]), (1, [4000, 16, 1, 900, 20]), (8, [60, 3000])])
def test_a_replay_of_unequal_lengths_at_others(hkv, lengths):
    """Captured where the grid was cut to the pairs of these lengths, replayed
    after a release and appends that turn them round."""
    rng = np.random.default_rng(9)
    nb, block = len(lengths), 16
    cache = B._cache(4 * hkv, hkv, [8000] * nb, block, "int8")
    draw = lambda b, n: T.to_dev_bf16(B._bits(rng, (b, hkv, n, 128)))  # noqa: E731
    for b, n in enumerate(lengths):
        cache.append(draw(1, n), draw(1, n), seq_begin=b)
    q = T.to_dev_bf16(B._bits(rng, (nb, 4 * hkv, 128)))
    out = torch.empty_like(q)
    cache.decode_attention(q, softcap=5.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention(q, out=out, softcap=5.0)

    def check():
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        held = [b for b in range(nb) if cache.length(b)]
        for b in range(nb):
            if b not in held:
                assert (got[b] == 0).all()
                continue
            want = cache.decode_attention(q[b:b + 1].contiguous(), seq_begin=b, softcap=5.0)
            # (the same values; another grid's order of sums)
            torch.testing.assert_close(got[b:b + 1].float(), want.float(), rtol=2 ** -7, atol=1e-3)

    check()
    cache.release(0)
    check()
    for b in range(1, nb):
        n = 3000 // b
        cache.append(draw(1, n), draw(1, n), seq_begin=b)
    check()
    cache.append(draw(1, 5), draw(1, 5))
    check()
    assert cache.read_status() == 0


@pytest.mark.parametrize("cap", [1e-45, 1e-38, 3.4e38])
def test_caps_at_the_ends_of_fp32(cap):
    """A cap near 0 leaves every score (and a zero product) at 0: the plain mean
    of the values.  The largest finite cap keeps everything finite."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    rng = np.random.default_rng(5)
    n, hq, hkv = 300, 4, 2
    kb, vb = B._bits(rng, (1, hkv, n, 128)), B._bits(rng, (1, hkv, n, 128))
    qb = B._bits(rng, (1, hq, n, 128))
    qb[:, 1] = 0  # products of exactly 0
    k, v, q = T.to_dev_bf16(kb), T.to_dev_bf16(vb), T.to_dev_bf16(qb)
    vf = O.bf16_bits_to_f32(vb).astype(np.float64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = prompt_attention(q, k, v, status=status, softcap=cap)
    block = B._cache(hq, hkv, [n], 16, "int8")
    block.append(k, v)
    token = KVCache(hq, hkv, 8, 32, 1, 32)
    token.quantize_append(k, v)
    token.set_score_transform(softcap=cap)
    q1 = q[:, :, -1].contiguous()
    ones = [block.decode_attention(q1, softcap=cap), token.decode_attention(q1)]
    assert status.item() == 0 and block.read_status() == 0 and token.read_status() == 0
    assert out.isfinite().all() and all(o.isfinite().all() for o in ones)
    if cap > 1:
        return
    got = T.bf16_tensor_to_f32(out)
    held = {}
    for h in range(hkv):
        held[h] = R.held_block(O.bf16_bits_to_f32(vb[0, h]), 16, False)
    for j in range(hq):
        h = j * hkv // hq
        p = np.tril(np.ones((n, n))) / np.arange(1, n + 1)[:, None]
        ref = p @ vf[0, h]
        bound = R.output_bound(ref, p, vf[0, h], 0.0)
        assert (np.abs(got[0, j] - ref) <= bound).all(), j
        ref = p[-1:] @ held[h]
        err = np.abs(T.bf16_tensor_to_f32(ones[0])[0, j] - ref[0])
        assert (err <= R.output_bound(ref, p[-1:], held[h], 0.0)[0]).all(), j


def test_an_append_of_many_waves():
    """More tiles than resident CTAs, runs that cross heads, K and V and
    sequences: the same state as the same tokens in three appends."""
    rng = np.random.default_rng(6)
    n = 30011
    k, v = (T.to_dev_bf16(B._bits(rng, (2, 2, n, 128))) for _ in range(2))
    for block, codes in ((16, "int8"), (128, "e4m3")):
        one, three = (B._cache(2, 2, [n, n], block, codes) for _ in range(2))
        one.append(k, v)
        for a, b in ((0, 131), (131, 20000), (20000, n)):
            three.append(k[:, :, a:b].contiguous(), v[:, :, a:b].contiguous())
        assert all(torch.equal(x, y) for x, y in zip(one.read(0, 2), three.read(0, 2)))
        # against the definition, on a sample of blocks
        got = one.read(0, 2)[0]
        f = k.float().cpu().numpy()
        for b, h, c in ((0, 0, 0), (1, 1, (n - 4) // block - 1), (0, 1, 77), (1, 0, 150)):
            s = slice(4 + c * block, 4 + (c + 1) * block)
            codes64, scale = R.quantise_block(f[b, h, s], codes == "e4m3")
            want = torch.from_numpy((codes64 * np.float64(scale)).astype(np.float32)).bfloat16()
            assert torch.equal(got[b, h, s].cpu(), want), (b, h, c)
        assert one.read_status() == 0 and one.lengths(0, 2) == (n, n)


def test_reads_on_another_stream():
    """What a call allocates and clears belongs to the stream of the call, not
    to the current one, which is busy meanwhile."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(7)
    n = 90
    cache = B._cache(4, 2, [n], 16, "int8")
    k, v = (T.to_dev_bf16(B._bits(rng, (1, 2, n, 128))) for _ in range(2))
    q = T.to_dev_bf16(B._bits(rng, (1, 4, n, 128)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.append(k, v)
    want = cache.read(0, 1)
    want_p = prompt_attention(q, k, v, status=status)
    want_a = cache.decode_attention(q[:, :, 0].contiguous())
    q0 = q[:, :, 0].contiguous()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(100_000_000)  # (about 50 ms on the current stream)
    got = cache.read(0, 1, 0, n + 20, stream=side)
    got_p = prompt_attention(q, k, v, status=status, stream=side)
    got_a = cache.decode_attention(q0, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x[:, :, :n], y) and (x[:, :, n:] == 0).all()
    assert torch.equal(got_p, want_p) and torch.equal(got_a, want_a)


def test_prefills_on_another_stream():
    """A prefill's workspace is given up on return: it has to belong to the
    stream that still uses it.  Prefills queued on a side stream, while the
    current one allocates and fills blocks of the workspace's size, give what
    they give alone."""
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    rng = np.random.default_rng(10)
    n, hq, hkv, count = 1100, 8, 2, 6
    q, k, v = (T.to_dev_bf16(B._bits(rng, (1, h, n, 128))) for h in (hq, hkv, hkv))
    begin = (torch.arange(n, device="cuda", dtype=torch.int32) // 300 * 300).view(1, n)
    caches = [KVCache(hq, hkv, 8, 72, 1, 72) for _ in range(count + 1)]
    for c in caches:
        c.set_score_transform(softcap=20.0)
    want = caches[-1].prefill(q, k, v, key_begin=begin)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for c in caches[:count]:
        outs.append(c.prefill(q, k, v, key_begin=begin, stream=side))
        nbytes = c.lib.kvc_prefill_masked_workspace_bytes(c.handle, 1, n) + 256
        for _ in range(3):
            torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for c, o in zip(caches, outs):
        assert torch.equal(o, want) and c.read_status() == 0


def test_one_workspace_call_after_call():
    """Prompts of different values through one workspace, one right behind
    another: no call reads what the one before or after it prepared."""
    from compressed_kv_cache_kvc_gb300 import _lib as L
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(8)
    n, hq, hkv = 700, 8, 2
    sets = [[T.to_dev_bf16(B._bits(rng, (2, h, n, 128))) for h in (hq, hkv, hkv)] for _ in range(4)]
    sets[2][2][0, 0, 5, 5] = float("inf")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = [prompt_attention(*s, status=status, softcap=20.0, column_sums=True) for s in sets]
    ws = torch.empty(L.lib().kvc_prompt_workspace_bytes(2, hq, hkv, n, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = [prompt_attention(*sets[i % 4], status=status, softcap=20.0, column_sums=True, workspace=ws)
           for i in range(24)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, want[i % 4]):
            assert torch.equal(x.nan_to_num(123.0), y.nan_to_num(123.0)), i


@pytest.mark.parametrize("batch,hq,hkv,n", [(1, 7, 1, 900), (2, 12, 2, 300), (1, 3, 1, 5), (1, 8, 8, 700)])
def test_column_sums_shared_by_several_ctas(batch, hq, hkv, n):
    """Few key tiles and KV heads: a key tile's sums come from several CTAs.  They
    are the sum of the calls of one query head a KV head each, within the order
    of the additions, and the same from call to call."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(11)
    q, k, v = (T.to_dev_bf16(B._bits(rng, (batch, h, n, 128))) for h in (hq, hkv, hkv))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, sums = prompt_attention(q, k, v, status=status, softcap=15.0, column_sums=True)
    for _ in range(3):
        o, s = prompt_attention(q, k, v, status=status, softcap=15.0, column_sums=True)
        assert torch.equal(o, out) and torch.equal(s, sums)
    group = hq // hkv
    want = torch.zeros_like(sums, dtype=torch.float64)
    for g in range(group):
        heads = q[:, g::group].contiguous()
        o, s = prompt_attention(heads, k, v, status=status, softcap=15.0, column_sums=True)
        assert torch.equal(o, out[:, g::group])
        want += s.double()
    # both sides add up to n fp32 terms in [0, 1] a head: n 2^-24 of the sum each
    assert ((sums.double() - want).abs() <= 2 * (n + group) * 2.0 ** -24 * want).all()
    np.testing.assert_allclose(sums.sum().item(), batch * hq * n, rtol=1e-5)
    assert status.item() == 0


def test_traced_decode_eager_and_captured():
    """Trace events stand between the split and the merge: the merge is then
    launched in order, and the results are the untraced ones."""
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    rng = np.random.default_rng(12)
    hq, hkv, n = 8, 2, 900
    cache = KVCache(hq, hkv, 8, 64, 1, 64)
    k = T.to_dev_bf16(B._bits(rng, (1, hkv, n, 128)))
    cache.quantize_append(k, k)
    cache.set_score_transform(softcap=12.0)
    q = T.to_dev_bf16(B._bits(rng, (1, hq, 128)))
    want = cache.decode_attention(q, accumulate_h2o=False)
    a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    a.record(), b.record()
    cache.set_trace_events(a, b)
    assert torch.equal(cache.decode_attention(q, accumulate_h2o=False), want)
    torch.cuda.synchronize()
    assert a.elapsed_time(b) > 0
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.decode_attention(q, out=out, accumulate_h2o=False)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    cache.set_trace_events(None, None)
    assert torch.equal(cache.decode_attention(q, accumulate_h2o=False), want)
