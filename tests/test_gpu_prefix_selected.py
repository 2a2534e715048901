"""Attention over a shared prefix and over selected blocks of the block-scaled
cache: outputs against the formula in 64 bits on what the cache holds, the chosen
blocks against their definition (equal), replays, streams, refusals, and a run of
rotated appends with both."""
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


def _bits(rng, shape, mult=1.0):
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    return bf16_bits((rng.standard_normal(shape) * mult).astype(np.float32))


def _cache(hq, hkv, lengths, block, codes, bounds=False, extra=64):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    counts = [(m + extra) // block + 1 for m in lengths]
    return BlockScaledCache(hq, hkv, sum(counts), len(lengths), max(counts), block_tokens=block, codes=codes,
                            key_bounds=bounds)


def _fill(cache, kv):
    """kv: (k, v) bf16 bits [hkv, n, 128] of every sequence."""
    for b in reversed(range(len(kv))):  # blocks of the sequences interleave out of order
        if kv[b][0].shape[1]:
            cache.append(T.to_dev_bf16(kv[b][0][None]), T.to_dev_bf16(kv[b][1][None]), seq_begin=b)


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / hq) for j in range(hq)], dtype=torch.float32, device="cuda")


def _held(x, block, codes):
    return R.held_block(O.bf16_bits_to_f32(x), block, codes == "e4m3")


def _check(got, q, kd, vd, cap, slope, newest, at):
    """One output row against the formula over keys kd, vd at positions `at`."""
    z = R.scores(O.bf16_bits_to_f32(q[None]), kd, SCALE, cap, slope, [newest], at)
    p = R.softmax_rows(z)
    ref = p @ vd
    bound = R.output_bound(ref, p, vd, R.score_error(z, cap, np.ones_like(z, bool)))
    err = np.abs(got - ref[0])
    assert (err <= bound[0]).all(), float((err / bound[0]).max())


# ------------------------------------------------------------------ prefix

PREFIX = [
    # hq, hkv, prefix, own lengths, block, codes, cap, bias, size of K
    (8, 8, 1, [1], 16, "int8", 0.0, False, 1.0),
    (8, 2, 3, [0, 1, 5, 300], 16, "int8", 10.0, True, 1.0),
    (4, 4, 0, [1, 20, 133], 32, "e4m3", 0.0, True, 1.0),
    (4, 1, 20, [0, 0], 16, "int8", 0.0, True, 1.0),
    (8, 8, 517, [37, 37, 37, 37], 16, "int8", 0.0, False, 1.0),
    (10, 2, 1300, [33, 2, 90], 32, "int8", 20.0, True, 2.0),
    (64, 8, 700, [70, 4], 64, "e4m3", 3.0, False, 6.0),
    (3, 1, 3000, [1] * 9, 16, "e4m3", 0.0, True, 1.0),
    (8, 1, 2117, [150] * 20, 128, "int8", 4.0, True, 3.0),
    (7, 1, 4100, list(range(0, 40)), 64, "int8", 0.0, False, 2.0),
    (8, 2, 6000, [5 + 13 * i for i in range(33)], 16, "e4m3", 30.0, True, 1.0),
    (8, 1, 900, [3 * i for i in range(70)], 16, "int8", 0.0, True, 1.0),
    # (many rows of much: the prefix as a product)
    (7, 1, 8200, list(range(0, 40)), 64, "int8", 0.0, False, 2.0),
    (8, 1, 4100, [3 * i for i in range(70)], 16, "int8", 0.0, True, 1.0),
    (10, 2, 6000, [33, 2, 90] * 8, 32, "int8", 20.0, True, 2.0),
    (16, 16, 2117, [150] * 20, 128, "int8", 4.0, True, 3.0),
    (12, 6, 1501, [5, 0, 31] * 15, 64, "e4m3", 3.0, False, 6.0),
    (3, 1, 40000, [1] * 9, 16, "e4m3", 0.0, True, 1.0),
    (16, 8, 900, [3 * i for i in range(40)], 16, "e4m3", 0.0, False, 1.0),
]


@pytest.mark.parametrize("hq,hkv,prefix,own,block,codes,cap,bias,mult", PREFIX)
def test_prefix_against_formula(hq, hkv, prefix, own, block, codes, cap, bias, mult):
    rng = np.random.default_rng(hq + prefix + len(own))
    B = len(own)
    at, first, lengths = (0, 1, [prefix] + own) if prefix % 2 == 0 else (B, 0, own + [prefix])
    kv = [(_bits(rng, (hkv, n, 128), mult), _bits(rng, (hkv, n, 128))) for n in lengths]
    q = _bits(rng, (B, hq, 128), 1.5)
    cache = _cache(hq, hkv, lengths, block, codes)
    _fill(cache, kv)
    slopes = _slopes(hq) if bias else None
    dq = T.to_dev_bf16(q)
    call = lambda **kw: cache.prefix_attention(dq, at, seq_begin=first, softcap=cap, slopes=slopes, **kw)  # noqa: E731
    out = call()
    assert torch.equal(out, call())
    n = cache.lib.kvc_block_prefix_workspace_bytes(cache.handle, B)
    assert torch.equal(out, call(workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda")))
    got = T.bf16_tensor_to_f32(out)
    for h in range(hkv):
        front = [_held(x[h], block, codes) for x in kv[at]]
        for b in range(B):
            mine = [_held(x[h], block, codes) for x in kv[first + b]]
            kd, vd = (np.concatenate(x) for x in zip(front, mine))
            for j in range(h * hq // hkv, (h + 1) * hq // hkv):
                _check(got[b, j], q[b, j], kd, vd, cap, float(slopes[j]) if bias else 0.0, prefix + own[b] - 1,
                       np.arange(prefix + own[b]))
    assert cache.read_status() == 0
    assert (cache.buffer("TICKETS").view(torch.int32) == 0).all()


@pytest.mark.parametrize("hq,hkv,batch,prefix", [(32, 32, 5, 9000), (8, 1, 3, 150000), (128, 16, 17, 9000),
                                                 (32, 16, 13, 15669), (96, 32, 5, 7035), (24, 8, 33, 36883)])
def test_prefix_long_runs(hq, hkv, batch, prefix):
    """Many tiles for every CTA, in one stream of rows and in two, call after call."""
    rng = np.random.default_rng(hq + batch)
    own = [7 + b for b in range(batch)]
    cache = _cache(hq, hkv, [prefix] + own, 32, "int8")
    kv = [(_bits(rng, (hkv, n, 128)), _bits(rng, (hkv, n, 128))) for n in [prefix] + own]
    _fill(cache, kv)
    q = _bits(rng, (batch, hq, 128), 1.5)
    dq = T.to_dev_bf16(q)
    slopes = _slopes(hq)
    for bias in (slopes, None):  # (the two streams of a CTA do not keep step)
        first = cache.prefix_attention(dq, 0, seq_begin=1, slopes=bias)
        outs = [cache.prefix_attention(dq, 0, seq_begin=1, slopes=bias) for _ in range(300)]
        assert all(torch.equal(first, o) for o in outs)
        assert cache.read_status() == 0
    got = T.bf16_tensor_to_f32(first)
    for b, j in ((0, 0), (batch - 1, hq - 1), (1, hq // 2)):
        h = j * hkv // hq
        kd, vd = (np.concatenate([_held(kv[0][i][h], 32, "int8"), _held(kv[1 + b][i][h], 32, "int8")]) for i in (0, 1))
        _check(got[b, j], q[b, j], kd, vd, 0.0, 0.0, prefix + own[b] - 1, np.arange(prefix + own[b]))


@pytest.mark.parametrize("prefix", [4 + 16 * 40 + 9, 4 + 16 * 480 + 9])
def test_prefix_values_of_any_size(prefix):
    """V of very different sizes in the prefix's blocks, its exact rows and the
    sequences' own: every value keeps its bits relative to the largest that counts."""
    rng = np.random.default_rng(8)
    hq, hkv, block, own = 8, 1, 16, [50, 2, 21] * 12
    for big, small in ((1e30, 1e-30), (3e37, 1.0), (1e-30, 1e-36), (1.0, 1e-9)):
        mult = np.full((hkv, prefix, 1), small)
        mult[:, 20:52] = big
        kv = [(_bits(rng, (hkv, prefix, 128)), _bits(rng, (hkv, prefix, 128), mult))]
        kv += [(_bits(rng, (hkv, n, 128)), _bits(rng, (hkv, n, 128), small)) for n in own]
        kv[0][0][:, 20:52] = _bits(rng, (hkv, 32, 128), 1e-3)  # scores near 0, so that the others can outweigh them
        cache = _cache(hq, hkv, [prefix] + own, block, "int8")
        _fill(cache, kv)
        q = _bits(rng, (len(own), hq, 128), 1.5)
        got = T.bf16_tensor_to_f32(cache.prefix_attention(T.to_dev_bf16(q), 0, seq_begin=1))
        front = [_held(x[0], block, "int8") for x in kv[0]]
        for b in range(0, len(own), 5):
            kd, vd = (np.concatenate([x, _held(y[0], block, "int8")]) for x, y in zip(front, kv[1 + b]))
            for j in range(hq):
                z = R.scores(O.bf16_bits_to_f32(q[b, j][None]), kd, SCALE, 0.0, 0.0, [0], np.zeros(len(kd)))
                p = R.softmax_rows(z)
                ref = (p @ vd)[0]
                # (the bound's own last term is absolute, for values near 1)
                a = (p @ np.abs(vd))[0]
                bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * R.score_error(z, 0.0, np.ones_like(z, bool))
                                                   + len(kd) * 2.0 ** -24) * a
                         + len(kd) * 2.0 ** -24 * np.abs(vd).max())
                assert (np.abs(got[b, j] - ref) <= bound).all(), (big, small, b, j)
        assert cache.read_status() == 0


@pytest.mark.parametrize("hkv,B", [(2, 5), (8, 90)])
def test_prefix_replays_streams_and_slices(hkv, B):
    """A captured step (append, attention) replayed while the sequences and the
    prefix grow equals the eager calls; another stream; two graphs that share a
    workspace, one after the other."""
    rng = np.random.default_rng(5)
    hq, block, few = 8, 16, B // 2
    caches = [_cache(hq, hkv, [2000] + [200] * B, block, "e4m3") for _ in range(2)]
    k, v = (T.to_dev_bf16(_bits(rng, (1, hkv, 1000, 128))) for _ in range(2))
    for c in caches:
        c.append(k, v, seq_begin=0)
    kn, vn, q = (torch.zeros(B, h, *x, 128, device="cuda", dtype=torch.bfloat16)
                 for h, x in ((hkv, (1,)), (hkv, (1,)), (hq, ())))
    out, other = torch.empty_like(q), torch.empty_like(q[:few])
    c = caches[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.append(kn, vn, seq_begin=1, stream=side)
    c.prefix_attention(q, 0, seq_begin=1, out=out, stream=side)
    side.synchronize()
    caches[1].append(kn, vn, seq_begin=1)
    ws = torch.zeros(c.lib.kvc_block_prefix_workspace_bytes(c.handle, B), dtype=torch.uint8, device="cuda")
    graphs = []
    for step in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            if step == 0:
                c.append(kn, vn, seq_begin=1)
                c.prefix_attention(q, 0, seq_begin=1, out=out, workspace=ws)
            else:
                c.prefix_attention(q[1:1 + few], 0, seq_begin=2, out=other, workspace=ws)
        graphs.append(g)
    c.sync_host()
    for step in range(45):
        x, y, z = (T.to_dev_bf16(_bits(rng, t.shape)) for t in (kn, vn, q))
        kn.copy_(x), vn.copy_(y), q.copy_(z)
        graphs[0].replay()
        graphs[1].replay()
        caches[1].append(x, y, seq_begin=1)
        if step in (20, 30):  # a longer prefix, and a much longer one
            m = 50 if step == 20 else 900
            for d in caches:
                d.append(k[:, :, :m].contiguous(), v[:, :, :m].contiguous(), seq_begin=0)
        want = caches[1].prefix_attention(z, 0, seq_begin=1) if step not in (20, 30) else None
        if want is not None:
            torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
            torch.testing.assert_close(other.float(), want[1:1 + few].float(), rtol=2 ** -7, atol=1e-3)
    # nothing left: rows of 0
    c.sync_host()
    c.release(0, B + 1)
    graphs[1].replay()
    assert (other == 0).all() and c.read_status() == 0


# ---------------------------------------------------------------- selected

def _choice(q, k, closed, block, top, recent):
    """The definition: q fp32 [group, 128], k fp32 [tokens, 128]."""
    spare = max(closed - recent, 0)
    if spare <= top:
        return list(range(closed))
    best = np.full(spare, -np.inf, np.float32)
    ends = []
    for c in range(spare):
        code, t = R.quantise_block(k[4 + c * block:4 + (c + 1) * block], False)
        ends.append((code.min(0), code.max(0), t))
    for row in q:
        code, s = R.quantise_block(row, False)
        for c, (lo, hi, t) in enumerate(ends):
            dot = np.maximum(code * lo, code * hi).sum()
            assert abs(dot) < 2 ** 24 and dot == int(dot)
            best[c] = max(best[c], np.float32(np.float32(dot) * s) * t)
    order = np.argsort(-best.astype(np.float64), kind="stable")[:top]
    return sorted(order.tolist()) + list(range(spare, closed))


SELECTED = [
    # hq, hkv, lengths, block, codes, top, recent, cap, bias
    (8, 8, [1], 16, "int8", 1, 0, 0.0, False),
    (8, 2, [4, 5, 19, 20, 21, 200], 16, "int8", 2, 1, 10.0, True),
    (4, 4, [700, 131, 900], 128, "e4m3", 3, 0, 0.0, True),
    (40, 8, [333, 1090], 32, "int8", 7, 2, 20.0, True),
    (64, 8, [2000], 64, "e4m3", 11, 0, 3.0, False),
    (3, 1, [3000], 16, "e4m3", 1, 0, 0.0, True),
    (16, 16, [1257, 12, 1000], 16, "int8", 50, 5, 50.0, False),
    (7, 1, [2117], 16, "int8", 100, 31, 0.0, True),
    (5, 1, [70000], 16, "int8", 60, 4, 0.0, False),
    (4, 2, [300, 301], 32, "int8", 100, 100, 0.0, True),
]


@pytest.mark.parametrize("hq,hkv,lengths,block,codes,top,recent,cap,bias", SELECTED)
def test_selected_against_definition(hq, hkv, lengths, block, codes, top, recent, cap, bias):
    rng = np.random.default_rng(hq + sum(lengths))
    B = len(lengths)
    kv = [(_bits(rng, (hkv, n, 128), rng.choice([0.3, 1.0, 2.0], size=(hkv, n, 1))), _bits(rng, (hkv, n, 128)))
          for n in lengths]
    q = _bits(rng, (B, hq, 128), 1.5)
    if lengths[0] >= 4 + 6 * block:  # equal scores: blocks twice, a query of zeros
        for x in kv[0]:
            x[:, 4 + 5 * block:4 + 6 * block] = x[:, 4 + block:4 + 2 * block]
        q[0, 0] = 0
    cache = _cache(hq, hkv, lengths, block, codes, bounds=True)
    _fill(cache, kv)
    slopes = _slopes(hq) if bias else None
    dq = T.to_dev_bf16(q)
    call = lambda **kw: cache.selected_attention(dq, top, recent_blocks=recent, softcap=cap, slopes=slopes, **kw)  # noqa: E731
    out, blocks = call(return_blocks=True)
    assert torch.equal(out, call())
    n = cache.lib.kvc_block_selected_workspace_bytes(cache.handle, B, top, recent)
    again, same = call(return_blocks=torch.full_like(blocks, 77),
                       workspace=torch.full((n,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out, again) and torch.equal(blocks, same)
    got, blocks = T.bf16_tensor_to_f32(out), blocks.cpu().numpy()
    for b, m in enumerate(lengths):
        closed = max(m - 4, 0) // block
        for h in range(hkv):
            heads = range(h * hq // hkv, (h + 1) * hq // hkv)
            kf = O.bf16_bits_to_f32(kv[b][0][h])
            want = _choice(O.bf16_bits_to_f32(q[b, heads.start:heads.stop]), kf, closed, block, top, recent)
            assert blocks[b, h].tolist() == want + [-1] * (top + recent - len(want)), (b, h)
            at = np.concatenate([np.arange(min(m, 4))] + [4 + c * block + np.arange(block) for c in want]
                                + [np.arange(4 + closed * block, m)])
            kd, vd = (_held(x[h], block, codes)[at] for x in kv[b])
            for j in heads:
                _check(got[b, j], q[b, j], kd, vd, cap, float(slopes[j]) if bias else 0.0, m - 1, at)
    assert cache.read_status() == 0
    assert (cache.buffer("TICKETS").view(torch.int32) == 0).all()
    if all(max(m - 4, 0) // block <= top + recent for m in lengths):  # nothing is left out
        whole = cache.decode_attention(dq, softcap=cap, slopes=slopes)
        torch.testing.assert_close(out.float(), whole.float(), rtol=2 ** -7, atol=1e-3)


def test_selected_replays():
    """A captured step replayed while the sequences grow from none left out to
    many, and after they were released."""
    rng = np.random.default_rng(6)
    hq, hkv, block, B = 4, 2, 16, 3
    caches = [_cache(hq, hkv, [1200] * B, block, "int8", bounds=True) for _ in range(2)]
    k, v = (T.to_dev_bf16(_bits(rng, (B, hkv, 40, 128))) for _ in range(2))
    for c in caches:
        c.append(k, v)
    kn, vn = (torch.zeros(B, hkv, 17, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    q = torch.zeros(B, hq, 128, device="cuda", dtype=torch.bfloat16)
    out, blocks = torch.empty_like(q), torch.empty(B, hkv, 7, dtype=torch.int32, device="cuda")
    c = caches[0]
    c.selected_attention(q, 5, recent_blocks=2, out=out, return_blocks=blocks)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append(kn, vn)
        c.selected_attention(q, 5, recent_blocks=2, out=out, return_blocks=blocks)
    c.sync_host()
    for step in range(60):
        x, y, z = (T.to_dev_bf16(_bits(rng, t.shape)) for t in (kn, vn, q))
        kn.copy_(x), vn.copy_(y), q.copy_(z)
        g.replay()
        caches[1].append(x, y)
        want, chosen = caches[1].selected_attention(z, 5, recent_blocks=2, return_blocks=True)
        assert torch.equal(blocks, chosen), step
        torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
    c.sync_host()
    c.release(0, B)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.append(k, v, stream=side)
    got = c.selected_attention(q, 5, recent_blocks=2, stream=side)
    side.synchronize()
    caches[1].release(0, B)
    caches[1].append(k, v)
    torch.testing.assert_close(got.float(), caches[1].decode_attention(q).float(), rtol=2 ** -7, atol=1e-3)
    assert c.read_status() == 0


def test_bad_block_ids_are_flagged():
    rng = np.random.default_rng(6)
    cache = _cache(4, 2, [400, 30], 16, "int8", bounds=True)
    _fill(cache, [(_bits(rng, (2, n, 128)), _bits(rng, (2, n, 128))) for n in (400, 30)])
    cache.buffer("TABLE").view(torch.int32)[2] = 1 << 20
    cache.buffer("TABLE").view(torch.int32)[3] = -5
    q = T.to_dev_bf16(_bits(rng, (1, 4, 128)))
    out, blocks = cache.selected_attention(q, 20, recent_blocks=1, return_blocks=True)
    assert out.isfinite().all() and not ((blocks == 2) | (blocks == 3)).any() and cache.read_status() == 0
    assert cache.selected_attention(q, 100).isfinite().all() and cache.read_status() == 0x2
    assert cache.prefix_attention(q, 0, seq_begin=1).isfinite().all() and cache.read_status() == 0x2
    cache = _cache(8, 8, [2000] + [30] * 20, 16, "int8")
    kv = [(_bits(rng, (8, n, 128)), _bits(rng, (8, n, 128))) for n in [2000] + [30] * 20]
    _fill(cache, kv)
    table = cache.buffer("TABLE").view(torch.int32)
    kept = table[2:4].clone()
    table[2], table[3] = 1 << 20, -5
    q = _bits(rng, (20, 8, 128))
    out = cache.prefix_attention(T.to_dev_bf16(q), 0, seq_begin=1)
    assert out.isfinite().all() and cache.read_status() == 0x2
    table[2:4] = kept
    cut = np.r_[0:4 + 32, 4 + 64:2000]  # the two blocks left out
    kd, vd = (np.concatenate([_held(kv[0][i][3], 16, "int8")[cut], _held(kv[2][i][3], 16, "int8")]) for i in (0, 1))
    _check(T.bf16_tensor_to_f32(out)[1, 3], q[1, 3], kd, vd, 0.0, 0.0, 0, np.zeros(len(kd)))


def test_refusals():
    from compressed_kv_cache_kvc_gb300 import _lib as L
    cache, plain = _cache(4, 2, [40, 40], 16, "int8", bounds=True), _cache(4, 2, [40, 40], 16, "int8")
    z = lambda *s: torch.zeros(*s, 128, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    q = z(1, 4)
    for call in (lambda: cache.selected_attention(q, 1), lambda: cache.prefix_attention(q, 0, seq_begin=1)):
        with pytest.raises(L.KvcError):  # nothing to attend to
            call()
    cache.append(z(2, 2, 20), z(2, 2, 20))
    plain.append(z(2, 2, 20), z(2, 2, 20))
    for call in (lambda: plain.selected_attention(q, 1), lambda: cache.selected_attention(q, 0),
                 lambda: cache.selected_attention(q, 1, recent_blocks=-1), lambda: cache.selected_attention(q, 1 << 20),
                 lambda: cache.selected_attention(q.float(), 1), lambda: cache.selected_attention(z(1, 3), 1),
                 lambda: cache.selected_attention(q, 1, return_blocks=torch.zeros(1, 2, 1, device="cuda")),
                 lambda: cache.selected_attention(q, 1, slopes=torch.zeros(3, device="cuda")),
                 lambda: cache.prefix_attention(z(1, 3), 0, seq_begin=1), lambda: cache.prefix_attention(q.cpu(), 0),
                 lambda: cache.prefix_attention(q, 0, seq_begin=1, out=z(2, 4))):
        with pytest.raises(ValueError):
            call()
    short = torch.zeros(8, dtype=torch.uint8, device="cuda")
    for call in (lambda: cache.prefix_attention(q, 0, seq_begin=0), lambda: cache.prefix_attention(q, 2, seq_begin=1),
                 lambda: cache.prefix_attention(q, -1, seq_begin=1), lambda: cache.prefix_attention(z(2, 4), 0, seq_begin=1),
                 lambda: cache.prefix_attention(q, 0, seq_begin=1, softcap=-1.0),
                 lambda: cache.prefix_attention(q, 0, seq_begin=1, workspace=short),
                 lambda: cache.selected_attention(q, 1, seq_begin=2), lambda: cache.selected_attention(q, 1, sm_scale=0.0),
                 lambda: cache.selected_attention(q, 1, workspace=short)):
        with pytest.raises(L.KvcError) as e:
            call()
        assert e.value.status == L.KVC_ERR_INVALID_ARG
    assert cache.read_status() == 0


# ------------------------------------------------------------- in one run

@pytest.mark.parametrize("codes,block", [("int8", 16), ("e4m3", 32)])
def test_a_server_of_shared_prompts(codes, block):
    """A system prompt is appended once, rotated; turns of several sequences follow
    at their positions; decode steps attend to both.  Beside it, each sequence
    alone with the whole prompt, which the selected form reads.  Every step against
    the formula on what the caches hold of the turned keys."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rng = np.random.default_rng(11)
    rot = Rotary(96, axes=[0] * 16 + [1] * 16 + [2] * 16)
    hq, hkv, B, prefix, n = 8, 2, 3, 411, 53
    cache = _cache(hq, hkv, [prefix] + [n + 3] * B, block, codes)
    alone = [_cache(hq, hkv, [prefix + n + 3], block, codes, bounds=True) for _ in range(B)]
    rows = lambda b, m: [T.to_dev_bf16(_bits(rng, (b, m, h, 128))).transpose(1, 2) for h in (hq, hkv, hkv)]  # noqa: E731
    bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    q, k, v = rows(1, prefix)
    image = torch.randint(0, 60, (3, 1, prefix), dtype=torch.int32, device="cuda")
    first = cache.append_rotary(q, k, v, rot, positions=image)
    for c in alone:
        assert torch.equal(c.append_rotary(q, k, v, rot, positions=image), first)
    front = [bits(rot.rotate(k, positions=image))[0], bits(v)[0]]
    own = [[np.zeros((hkv, 0, 128), np.uint16)] * 2 for _ in range(B)]
    for step in range(4):
        m, at = (n, 0) if step == 0 else (1, n + step - 1)
        q, k, v = rows(B, m)
        qr = cache.append_rotary(q, k, v, rot, first=prefix, seq_begin=1)
        kr = rot.rotate(k, first=prefix + at)
        for b, c in enumerate(alone):
            assert torch.equal(c.append_rotary(q[b:b + 1], k[b:b + 1], v[b:b + 1], rot), qr[b:b + 1])
            own[b] = [np.concatenate([x, bits(y)[b]], axis=1) for x, y in zip(own[b], (kr, v))]
        qr = qr[:, :, -1].contiguous()
        out = T.bf16_tensor_to_f32(cache.prefix_attention(qr, 0, seq_begin=1, softcap=25.0))
        total = prefix + at + m
        for b, c in enumerate(alone):
            few, blocks = c.selected_attention(qr[b:b + 1], 5, recent_blocks=2, softcap=25.0, return_blocks=True)
            few, blocks = T.bf16_tensor_to_f32(few)[0], blocks[0].tolist()
            for h in range(hkv):
                kd, vd = (np.concatenate([_held(x[h], block, codes), _held(y[h], block, codes)])
                          for x, y in zip(front, own[b]))
                closed = (total - 4) // block
                assert blocks[h][-2:] == [closed - 2, closed - 1] and len(set(blocks[h])) == 7
                seen = np.concatenate([np.arange(4)] + [4 + x * block + np.arange(block) for x in blocks[h]]
                                      + [np.arange(4 + closed * block, total)])
                ka, va = (_held(np.concatenate([x[h], y[h]]), block, codes)[seen] for x, y in zip(front, own[b]))
                for j in range(4 * h, 4 * h + 4):
                    row = bits(qr)[b, j]
                    _check(out[b, j], row, kd, vd, 25.0, 0.0, total - 1, np.arange(total))
                    _check(few[j], row, ka, va, 25.0, 0.0, total - 1, seen)
    assert cache.read_status() == 0 and all(c.read_status() == 0 for c in alone)
