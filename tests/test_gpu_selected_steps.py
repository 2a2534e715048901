"""Selected blocks where a CTA scores several steps of 64 blocks, against the
definition; the shared prefix on both sides of the rule between its two forms."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _cache(hq, hkv, lengths, block, codes="int8", bounds=False):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    counts = [m // block + 1 for m in lengths]
    return BlockScaledCache(hq, hkv, sum(counts), len(lengths), max(counts), block_tokens=block, codes=codes,
                            key_bounds=bounds)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)


def _eights(x, amax):
    """(INT8 codes of rows x as fp32, scale): IEEE fp32 quotients, half to even."""
    scale = (amax / np.float32(127.0)).astype(np.float32)
    with np.errstate(invalid="ignore", divide="ignore"):
        y = np.where(scale > 0, x / scale, np.float32(0.0)).astype(np.float32)
    return np.clip(np.rint(y), -127, 127).astype(np.float32), scale


def _choice(q, k, block, top, recent):
    """The definition for one KV head: q fp32 [group, 128], k fp32 [tokens, 128]."""
    closed = (len(k) - 4) // block
    spare = closed - recent
    if spare <= top:
        return list(range(closed))
    body = k[4:4 + spare * block].reshape(spare, block, 128)
    amax = np.abs(body).max((1, 2))[:, None]
    lo, t = _eights(body.min(1), amax)
    hi, _ = _eights(body.max(1), amax)
    best = np.full(spare, -np.inf, np.float32)
    for row in q:
        code, s = _eights(row, np.abs(row).max())
        dot = np.maximum(code * lo, code * hi).sum(1, dtype=np.float64).astype(np.float32)  # (exact below 2^24)
        best = np.maximum(best, (dot * s).astype(np.float32) * t[:, 0])
    order = np.argsort(-best.astype(np.float64), kind="stable")[:top]
    return sorted(order.tolist()) + list(range(spare, closed))


@pytest.mark.parametrize("hq,hkv,block,codes,top,recent,lengths", [
    (32, 16, 16, "int8", 100, 4, [20000, 3111, 16004, 9999, 19005, 1700, 12345, 17777]),  # seven chunks, up to three steps
    (32, 32, 16, "e4m3", 30, 1, [8000 - 611 * i for i in range(10)]),                     # two chunks, up to four
    (8, 8, 32, "int8", 9, 0, [6000 - 17 * i for i in range(120)]),                        # one chunk, three
    (6, 2, 16, "int8", 500, 9, [140004, 66000]),                                          # many chunks, a step
])
def test_choice_of_several_steps(hq, hkv, block, codes, top, recent, lengths):
    rand = _gen(hq + len(lengths))
    cache = _cache(hq, hkv, lengths, block, codes, bounds=True)
    kept = {}
    for b, n in enumerate(lengths):
        k, v = rand(1, hkv, n, 128), rand(1, hkv, n, 128)
        cache.append(k, v, seq_begin=b)
        if b in (0, 1, len(lengths) // 2, len(lengths) - 1):
            kept[b] = k[0].float()
    q = rand(len(lengths), hq, 128)
    out, blocks = cache.selected_attention(q, top, recent_blocks=recent, return_blocks=True)
    again, same = cache.selected_attention(q, top, recent_blocks=recent, return_blocks=True)
    assert torch.equal(blocks, same) and torch.equal(out, again) and out.isfinite().all()
    blocks, group = blocks.cpu().numpy(), hq // hkv
    for b, k in kept.items():
        for h in sorted({0, hkv // 2, hkv - 1}):
            qf = q[b, h * group:(h + 1) * group].float().cpu().numpy()
            want = _choice(qf, k[h].cpu().numpy(), block, top, recent)
            assert blocks[b, h].tolist() == want + [-1] * (top + recent - len(want)), (b, h)
    assert cache.read_status() == 0


def test_choice_of_a_graph_captured_while_short():
    """Captured with nothing to choose (one CTA a pair), replayed past several steps
    of 64 blocks, at lengths that end inside one."""
    hq, hkv, block, top, recent, n, steps = 4, 2, 16, 20, 3, 331, 16
    rand = _gen(3)
    lengths = [40 + n * steps, 40 + n * steps]
    caches = [_cache(hq, hkv, lengths, block, bounds=True) for _ in range(2)]
    k, v = rand(2, hkv, 40, 128), rand(2, hkv, 40, 128)
    for c in caches:
        c.append(k, v)
    kn, vn, q = rand(2, hkv, n, 128), rand(2, hkv, n, 128), rand(2, hq, 128)
    out, blocks = torch.empty_like(q), torch.empty(2, hkv, top + recent, dtype=torch.int32, device="cuda")
    c = caches[0]
    ws = torch.empty(c.lib.kvc_block_selected_workspace_bytes(c.handle, 2, top, recent), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.selected_attention(q, top, recent_blocks=recent, out=out, return_blocks=blocks, workspace=ws)
        c.append(kn, vn)
    c.sync_host()
    keys = [k]
    for step in range(steps):
        x, y, z = rand(*kn.shape), rand(*vn.shape), rand(*q.shape)
        kn.copy_(x), vn.copy_(y), q.copy_(z)
        graph.replay()
        want, chosen = caches[1].selected_attention(z, top, recent_blocks=recent, return_blocks=True)
        assert torch.equal(blocks, chosen), step
        torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
        held = torch.cat(keys, dim=2).float().cpu().numpy()
        for b in range(2):
            for h in range(hkv):
                got = [i for i in blocks[b, h].tolist() if i >= 0]
                assert got == _choice(z[b, 2 * h:2 * h + 2].float().cpu().numpy(), held[b, h], block, top, recent), step
        caches[1].append(x, y)
        keys.append(x)
    assert c.read_status() == 0


@pytest.mark.parametrize("codes,cap,bias", [("int8", 0.0, False), ("e4m3", 20.0, True)])
@pytest.mark.parametrize("batch,prefix,product", [(8, 4 + 4096, False), (8, 4 + 4096 + 16, True), (2, 4 + 16 * 1400, False),
                                                  (3, 4 + 85 * 128, False), (3, 4 + 85 * 128 + 33, True)])
def test_prefix_on_both_sides_of_its_rule(batch, prefix, product, codes, cap, bias):
    """Up to 2,048 (sequence, tile, KV head)s, or two sequences, directly; above, as a
    product: the same formula, and a captured call keeps its form across the border."""
    hq, hkv, block = 16, 8, 16
    rand = _gen(batch + prefix)
    own = [5 + 9 * b for b in range(batch)]
    cache = _cache(hq, hkv, [prefix + 32] + own, block, codes)
    kv = []
    for s, n in enumerate([prefix] + own):
        k, v = rand(1, hkv, n, 128), rand(1, hkv, n, 128)
        cache.append(k, v, seq_begin=s)
        kv.append([x[0].float().cpu().numpy() for x in (k, v)])
    q = rand(batch, hq, 128)
    slopes = torch.tensor([2.0 ** (-8.0 * (j + 1) / hq) for j in range(hq)], device="cuda") if bias else None
    call = lambda **kw: cache.prefix_attention(q, 0, seq_begin=1, softcap=cap, slopes=slopes, **kw)  # noqa: E731
    out = call()
    assert cache.last_launch_count() == (2 if product else 1)
    got, qf = T.bf16_tensor_to_f32(out), q.float().cpu().numpy()
    for b, j in ((0, 0), (batch - 1, hq - 1), (1, 7)):
        h = j * hkv // hq
        kd, vd = (np.concatenate([R.held_block(kv[s][i][h], block, codes == "e4m3") for s in (0, 1 + b)]) for i in (0, 1))
        n = prefix + own[b]
        z = R.scores(qf[b, j:j + 1], kd, SCALE, cap, float(slopes[j]) if bias else 0.0, [n - 1], np.arange(n))
        p = R.softmax_rows(z)
        ref = p @ vd
        bound = R.output_bound(ref, p, vd, R.score_error(z, cap, np.ones_like(z, bool)))
        assert (np.abs(got[b, j] - ref[0]) <= bound[0]).all()
    held = torch.empty_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=held)
    graph.replay()
    assert torch.equal(held, out)
    k, v = rand(1, hkv, 32, 128), rand(1, hkv, 32, 128)
    cache.append(k, v, seq_begin=0)  # (over the border, where the prefix lay just below it)
    graph.replay()
    torch.testing.assert_close(held.float(), call().float(), rtol=2 ** -7, atol=1e-3)
    assert cache.read_status() == 0


def _formula(got, qf, kd, vd, newest, at):
    z = R.scores(qf, kd, SCALE, 0.0, 0.0, [newest], at)
    p = R.softmax_rows(z)
    ref = p @ vd
    bound = R.output_bound(ref, p, vd, R.score_error(z, 0.0, np.ones_like(z, bool)))
    assert (np.abs(got - ref[0]) <= bound[0]).all()


@pytest.mark.parametrize("prefix", [3, 100, 900])
def test_more_pairs_than_places(prefix):
    """700 sequences of 4 KV heads: more pairs than an attention has places for parts."""
    hq, hkv, block, B, top, recent = 8, 4, 16, 700, 3, 2
    rand = _gen(prefix)
    own = [1 + 7 * b % 211 for b in range(B)]
    cache = _cache(hq, hkv, [prefix] + own, block, bounds=True)
    kv = {}
    for s, n in enumerate([prefix] + own):
        k, v = rand(1, hkv, n, 128), rand(1, hkv, n, 128)
        cache.append(k, v, seq_begin=s)
        if s in (0, 1, 330, 700):
            kv[s] = [x[0].float().cpu().numpy() for x in (k, v)]
    q = rand(B, hq, 128)
    out = T.bf16_tensor_to_f32(cache.prefix_attention(q, 0, seq_begin=1))
    few, blocks = cache.selected_attention(q, top, recent_blocks=recent, seq_begin=1, return_blocks=True)
    few, blocks, qf = T.bf16_tensor_to_f32(few), blocks.cpu().numpy(), q.float().cpu().numpy()
    for s in (1, 330, 700):
        n, closed = own[s - 1], max(own[s - 1] - 4, 0) // block
        for j in (0, 3, 7):
            h = j * hkv // hq
            front, mine = ([R.held_block(x[h], block, False) for x in kv[i]] for i in (0, s))
            _formula(out[s - 1, j], qf[s - 1, j:j + 1], *(np.concatenate(x) for x in zip(front, mine)), 0, np.zeros(prefix + n))
            want = _choice(qf[s - 1, 2 * h:2 * h + 2], kv[s][0][h], block, top, recent) if closed else []
            assert blocks[s - 1, h].tolist() == want + [-1] * (top + recent - len(want))
            at = np.concatenate([np.arange(min(n, 4))] + [4 + c * block + np.arange(block) for c in want]
                                + [np.arange(4 + closed * block, n)]).astype(int)
            _formula(few[s - 1, j], qf[s - 1, j:j + 1], mine[0][at], mine[1][at], n - 1, at)
    # slices of the same cache make the same choice
    part, chosen = cache.selected_attention(q[200:203], top, recent_blocks=recent, seq_begin=201, return_blocks=True)
    assert np.array_equal(chosen.cpu().numpy(), blocks[200:203])
    torch.testing.assert_close(part.float().cpu(), torch.from_numpy(few[200:203]), rtol=2 ** -7, atol=1e-3)
    part = cache.prefix_attention(q[200:203], 0, seq_begin=201)
    torch.testing.assert_close(part.float().cpu(), torch.from_numpy(out[200:203]), rtol=2 ** -7, atol=1e-3)
    assert cache.read_status() == 0 and (cache.buffer("TICKETS").view(torch.int32) == 0).all()
