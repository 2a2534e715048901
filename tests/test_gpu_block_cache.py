"""The block-scaled cache: codes and scales bit for bit, however the tokens are
split into appends; attention against the formula in 64 bits on what the cache
holds; read-back, release, graphs and refusals."""
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


def _cache(hq, hkv, lengths, block, codes, extra=64):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    per_seq = (max(lengths) + extra) // block + 1
    return BlockScaledCache(hq, hkv, len(lengths) * per_seq, len(lengths), per_seq, block_tokens=block, codes=codes)


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / hq) for j in range(hq)], dtype=torch.float32, device="cuda")


def _held(x, n, block, codes):
    return R.held_block(O.bf16_bits_to_f32(x[:n]), block, codes == "e4m3")


def _bf16(x):
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


APPENDS = [
    # block, codes, appends
    (16, "int8", [1]),
    (16, "int8", [3, 1, 1, 15, 1, 40]),
    (16, "e4m3", [20, 0, 300, 7]),
    (32, "int8", [4, 31, 1, 1, 200]),
    (64, "e4m3", [2, 66, 130, 64]),
    (128, "int8", [131, 1, 127, 260]),
    (128, "e4m3", [700]),
]


@pytest.mark.parametrize("block,codes,parts", APPENDS)
def test_append_and_read(block, codes, parts):
    """What the cache holds equals the definition (bf16 of code * scale, exact
    where exact), equals the same tokens appended one at a time, and reads back
    from any position."""
    rng = np.random.default_rng(block + len(parts))
    B, hkv, n = 3, 2, sum(parts)
    mult = rng.choice([1e-3, 1.0, 30.0], size=(B, hkv, n, 1))
    k, v = _bits(rng, (B, hkv, n, 128), mult), _bits(rng, (B, hkv, n, 128))
    k[1, 0, 5:70] = 0  # whole blocks of zeros
    dk, dv = T.to_dev_bf16(k), T.to_dev_bf16(v)
    cache, single = _cache(4, hkv, [n] * B, block, codes), _cache(4, hkv, [n] * B, block, codes)
    at = 0
    for m in parts:
        cache.append(dk[:, :, at:at + m].contiguous(), dv[:, :, at:at + m].contiguous())
        assert cache.last_launch_count() == (1 if m else 0)
        at += m
    for i in range(n):
        single.append(dk[:, :, i:i + 1].contiguous(), dv[:, :, i:i + 1].contiguous())
    ko, vo = cache.read(0, B)
    for b in range(B):
        assert cache.length(b) == n
        for h in range(hkv):
            for got, x in ((ko, k), (vo, v)):
                assert torch.equal(got[b, h].cpu(), _bf16(_held(x[b, h], n, block, codes))), (b, h)
    assert all(torch.equal(x, y) for x, y in zip(single.read(0, B), (ko, vo)))
    p0 = n // 3
    part = cache.read(1, 2, p0, n - p0)
    assert torch.equal(part[0], ko[1:, :, p0:]) and torch.equal(part[1], vo[1:, :, p0:])
    # rows past a sequence's end are left as they were
    out = tuple(torch.full((1, hkv, 20, 128), 7.0, device="cuda").bfloat16() for _ in range(2))
    cache.read(0, 1, n - 1, 20, out=out)
    assert torch.equal(out[0][:, :, 0], ko[:1, :, n - 1]) and (out[0][:, :, 1:] == 7).all()
    assert cache.read_status() == 0 and single.read_status() == 0


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_rounding_borders(codes):
    """Quotients on and around the rounding borders: every bf16 value of one
    binade against several scales, tiny and huge ones among them."""
    from compressed_kv_cache_kvc_gb300.workloads import bf16_to_f32
    block, hkv = 128, 1
    tops = [1.0, 127.0, 448.0, 1.5, 3e-39, 1e-37, 2.0 ** -120, 3e38, 0.0078125]
    pats = np.arange(2 ** 15, dtype=np.uint32)
    vals = bf16_to_f32(pats.astype(np.uint16))
    rows = []
    for t in tops:
        usable = vals[np.isfinite(vals) & (vals <= np.float32(t))]
        x = np.zeros(block * 128, np.float32)
        x[:min(usable.size, x.size - 1)] = usable[-(x.size - 1):]
        x[1::2] *= -1
        x[-1] = t
        rows.append(x.reshape(block, 128))
    x = np.concatenate([np.zeros((4, 128), np.float32)] + rows)[None, None]
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    bits = bf16_bits(x)
    n = x.shape[2]
    cache = _cache(1, hkv, [n], block, codes)
    d = T.to_dev_bf16(bits)
    cache.append(d, d)
    raw = cache.buffer("K_CODES").view(-1, block, 128).cpu()
    table = cache.buffer("TABLE").view(torch.int32).cpu()
    scales = cache.buffer("K_SCALE").view(torch.float32).cpu().numpy()
    f = O.bf16_bits_to_f32(bits[0, 0])
    with np.errstate(all="ignore"):
        for c in range(len(tops)):
            want, scale = R.quantise_block(f[4 + c * block:4 + (c + 1) * block], codes == "e4m3")
            blk = int(table[c])
            got = raw[blk].view(torch.float8_e4m3fn).double() if codes == "e4m3" else raw[blk].view(torch.int8).double()
            assert scales[blk] == scale, tops[c]
            assert np.array_equal(got.numpy(), want), (tops[c], int((got.numpy() != want).sum()))


ATTEND = [
    # hq, hkv, lengths, block, codes, cap, bias, size of K
    (8, 8, [1], 16, "int8", 0.0, False, 1.0),
    (8, 2, [4, 5, 19, 20, 21], 16, "int8", 10.0, True, 1.0),
    (4, 4, [130, 131, 132, 133], 128, "e4m3", 0.0, True, 1.0),
    (40, 8, [333, 90], 32, "int8", 20.0, True, 2.0),
    (64, 8, [700], 64, "e4m3", 3.0, False, 6.0),
    (3, 1, [3000], 16, "e4m3", 0.0, True, 1.0),
    (16, 16, [257, 12, 1000], 64, "int8", 50.0, False, 1.0),
    (5, 1, [2117], 128, "int8", 4.0, True, 6.0),
]


@pytest.mark.parametrize("hq,hkv,lengths,block,codes,cap,bias,mult", ATTEND)
def test_attention_against_formula(hq, hkv, lengths, block, codes, cap, bias, mult):
    rng = np.random.default_rng(hq + sum(lengths))
    B, n = len(lengths), max(lengths)
    k, v, q = _bits(rng, (B, hkv, n, 128), mult), _bits(rng, (B, hkv, n, 128)), _bits(rng, (B, hq, 128), 1.5)
    cache = _cache(hq, hkv, lengths, block, codes)
    for b in reversed(range(B)):  # blocks of the sequences interleave out of order
        m = lengths[b]
        cache.append(T.to_dev_bf16(np.ascontiguousarray(k[b:b + 1, :, :m])),
                     T.to_dev_bf16(np.ascontiguousarray(v[b:b + 1, :, :m])), seq_begin=b)
    slopes = _slopes(hq) if bias else None
    dq = T.to_dev_bf16(q)
    out = cache.decode_attention(dq, softcap=cap, slopes=slopes)
    assert cache.last_launch_count() == 1
    assert torch.equal(out, cache.decode_attention(dq, softcap=cap, slopes=slopes))
    # a slice gives the same rows up to the order of its sums; a dirty workspace changes nothing
    ws = torch.full_like(cache.workspace(B), 255)
    assert torch.equal(out, cache.decode_attention(dq, softcap=cap, slopes=slopes, workspace=ws))
    got = T.bf16_tensor_to_f32(out)
    for b, m in enumerate(lengths):
        for j in range(hq):
            h = j * hkv // hq
            kd, vd = _held(k[b, h], m, block, codes), _held(v[b, h], m, block, codes)
            z = R.scores(O.bf16_bits_to_f32(q[b, j:j + 1]), kd, SCALE, cap, float(slopes[j]) if bias else 0.0,
                         [m - 1], np.arange(m))
            p = R.softmax_rows(z)
            ref = p @ vd
            bound = R.output_bound(ref, p, vd, R.score_error(z, cap, np.ones_like(z, bool)))
            err = np.abs(got[b, j] - ref[0])
            assert (err <= bound[0]).all(), (b, j, float((err / bound[0]).max()))
    assert cache.read_status() == 0
    assert (cache.buffer("TICKETS").view(torch.int32) == 0).all()


def test_decode_loop_matches_dense_reads():
    """Prefill, then steps of append and attention as a server runs them, with
    a release in between; every step against the formula on what read() gives."""
    rng = np.random.default_rng(4)
    hq, hkv, block, B = 8, 4, 16, 2
    cache = _cache(hq, hkv, [120, 120], block, "int8")
    slopes, status = _slopes(hq), torch.zeros(1, dtype=torch.int32, device="cuda")
    held = [np.zeros((2, hkv, 0, 128), np.uint16) for _ in range(B)]

    def grow(b, k, v):
        held[b] = np.concatenate([held[b], np.stack([k, v])], axis=2)

    q, k, v = (_bits(rng, (B, h, 37, 128)) for h in (hq, hkv, hkv))
    out = cache.prefill(*[T.to_dev_bf16(x) for x in (q, k, v)], status=status, softcap=12.0, slopes=slopes)
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    assert torch.equal(out, prompt_attention(*[T.to_dev_bf16(x) for x in (q, k, v)], status=status, softcap=12.0,
                                             slopes=slopes))
    for b in range(B):
        grow(b, k[b], v[b])
    for step in range(24):
        if step == 10:
            free = cache.buffer("COUNTERS").view(torch.int32)[0].item()
            cache.release(1, 1)
            torch.cuda.synchronize()
            assert cache.buffer("COUNTERS").view(torch.int32)[0].item() == free + (37 + 10 - 4) // block
            held[1] = held[1][:, :, :0]
            cache.release(1, 1)
            assert cache.last_launch_count() == 0
        k, v, q = _bits(rng, (B, hkv, 1, 128)), _bits(rng, (B, hkv, 1, 128)), _bits(rng, (B, hq, 128))
        cache.append(T.to_dev_bf16(k), T.to_dev_bf16(v))
        got = T.bf16_tensor_to_f32(cache.decode_attention(T.to_dev_bf16(q), softcap=12.0, slopes=slopes))
        for b in range(B):
            grow(b, k[b], v[b])
            m = held[b].shape[2]
            for j in range(hq):
                kd, vd = (_held(held[b][i, j // 2], m, block, "int8") for i in range(2))
                z = R.scores(O.bf16_bits_to_f32(q[b, j:j + 1]), kd, SCALE, 12.0, float(slopes[j]), [m - 1],
                             np.arange(m))
                p = R.softmax_rows(z)
                bound = R.output_bound(p @ vd, p, vd, R.score_error(z, 12.0, np.ones_like(z, bool)))
                assert (np.abs(got[b, j] - (p @ vd)[0]) <= bound[0]).all(), (step, b, j)
    assert cache.read_status() == 0 and status.item() == 0


def test_graph_replays_at_other_lengths():
    """A captured append + attention replayed many times (through several block
    completions) equals the eager calls."""
    rng = np.random.default_rng(5)
    hq, hkv, block = 8, 2, 16
    caches = [_cache(hq, hkv, [200, 200], block, "e4m3") for _ in range(2)]
    k, v = (T.to_dev_bf16(_bits(rng, (2, hkv, 30, 128))) for _ in range(2))
    for c in caches:
        c.append(k, v)
    kn, vn, q = (torch.zeros(2, h, *x, 128, device="cuda", dtype=torch.bfloat16)
                 for h, x in ((hkv, (1,)), (hkv, (1,)), (hq, ())))
    out = torch.empty_like(q)
    ws = caches[0].workspace(2)
    snap = caches[0].state.clone()
    caches[0].append(kn, vn)          # (warm: the launches are captured at this length)
    caches[0].decode_attention(q, out=out, workspace=ws)
    torch.cuda.synchronize()
    caches[0].state.copy_(snap)
    caches[0].sync_host()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        caches[0].append(kn, vn)
        caches[0].decode_attention(q, out=out, workspace=ws)
    for step in range(60):
        a, b, c = (T.to_dev_bf16(_bits(rng, t.shape)) for t in (kn, vn, q))
        kn.copy_(a), vn.copy_(b), q.copy_(c)
        g.replay()
        caches[1].append(a, b)
        want = caches[1].decode_attention(c)
        # the same values; a grid chosen at another length sums in another order
        torch.testing.assert_close(out.float(), want.float(), rtol=2 ** -7, atol=1e-3)
    caches[0].sync_host()
    assert caches[0].length(0) == 90 == caches[1].length(0)
    assert all(torch.equal(x, y) for x, y in zip(caches[0].read(0, 2), caches[1].read(0, 2)))


def test_bad_block_ids_and_stack_are_flagged():
    """A table entry outside the pool is flagged and left out; an empty device
    stack (state bytes behind the host's back) is flagged and nothing is
    appended."""
    rng = np.random.default_rng(6)
    cache = _cache(4, 2, [100], 16, "int8")
    k = T.to_dev_bf16(_bits(rng, (1, 2, 100, 128)))
    cache.append(k, k)
    cache.buffer("TABLE").view(torch.int32)[2] = 1 << 20
    out = cache.decode_attention(T.to_dev_bf16(_bits(rng, (1, 4, 128))))
    assert out.isfinite().all() and cache.read_status() == 0x2
    cache.read(0, 1)
    assert cache.read_status() == 0x2
    cache.reset()
    cache.buffer("COUNTERS").view(torch.int32)[0] = 1
    cache.append(k, k)
    assert cache.read_status() == 0x1
    cache.sync_host()
    assert cache.length(0) == 0


def test_refusals():
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    from compressed_kv_cache_kvc_gb300 import _lib as L
    cache = BlockScaledCache(4, 2, 3, 2, 2, block_tokens=16)
    z = lambda *s: torch.zeros(*s, 128, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    for bad in [z(1, 3, 5), z(1, 2, 5).float(), z(1, 5, 2).transpose(1, 2), z(2, 5)]:
        with pytest.raises(ValueError):
            cache.append(bad, bad)
    for args, status in [((z(1, 2, 52), z(1, 2, 52)), L.KVC_ERR_CAPACITY),     # 3 blocks, 2 per sequence
                         ((z(2, 2, 36), z(2, 2, 36)), L.KVC_ERR_CAPACITY),     # 4 blocks, 3 in the pool
                         ((z(3, 2, 1), z(3, 2, 1)), L.KVC_ERR_INVALID_ARG)]:
        with pytest.raises(L.KvcError) as e:
            cache.append(*args)
        assert e.value.status == status and cache.length(0) == 0
    q = z(1, 4)
    with pytest.raises(L.KvcError):  # nothing to attend to
        cache.decode_attention(q)
    cache.append(z(1, 2, 20), z(1, 2, 20))
    for kw in [dict(softcap=-1.0), dict(softcap=float("nan")), dict(sm_scale=0.0), dict(seq_begin=1),
               dict(seq_begin=-1), dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(L.KvcError) as e:
            cache.decode_attention(q, **kw)
        assert e.value.status == L.KVC_ERR_INVALID_ARG, kw
    for bad in [z(1, 3), q.float(), z(4)]:
        with pytest.raises(ValueError):
            cache.decode_attention(bad)
    with pytest.raises(ValueError):
        cache.decode_attention(q, slopes=torch.zeros(4))
    for a in [(0, 3, 0, 5), (0, 1, -1, 5), (0, 1, 0, 0)]:
        with pytest.raises((L.KvcError, ValueError)):
            cache.read(*a)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(L.KvcError) as e:  # a prompt starts a sequence
        cache.prefill(z(1, 4, 2), z(1, 2, 2), z(1, 2, 2), status=st)
    assert e.value.status == L.KVC_ERR_STATE and cache.length(0) == 20
    with pytest.raises(ValueError):
        BlockScaledCache(4, 2, 3, 2, 2, codes="int4")
    with pytest.raises(L.KvcError):
        BlockScaledCache(4, 2, 3, 2, 2, block_tokens=24)
