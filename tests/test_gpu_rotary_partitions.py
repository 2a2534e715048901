"""Appends with the rotation large enough for every part of their partition: shares
of the KV heads (also uneven ones), several units a CTA, units without rows, groups of
one to eight warps, sequences whose open blocks are at different places; the
queries' own launch with positions of several axes.  Equal, bit for bit, to the
rotation followed by the plain append."""
import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _rows(seed, b, n, *heads):
    """Views [b, heads, n, 128] of one projection's output."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((b, n, sum(heads), D), generator=g, device="cuda").to(torch.bfloat16)
    return [y.transpose(1, 2) for y in x.split(list(heads), dim=2)]


def _cache(hq, hkv, b, most, block, codes, bounds):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    per_seq = most // block + 1
    c = BlockScaledCache(hq, hkv, b * per_seq, b, per_seq, block_tokens=block, codes=codes, key_bounds=bounds)
    if bounds:
        c.bounds.zero_()
    return c


def _same(a, b):
    for name in ("SEQ_POS", "TABLE", "COUNTERS", "TICKETS", "K_SCALE", "V_SCALE", "K_CODES", "V_CODES", "K_EXACT", "V_EXACT"):
        assert torch.equal(a.buffer(name), b.buffer(name)), name
    if a.bounds is not None:
        assert torch.equal(a.bounds, b.bounds)
    assert a.read_status() == 0


CASES = [
    # batch, hkv, tokens, block, codes, bounds, axes, held by the sequences before (in turn)
    (4, 8, 8000, 32, "int8", True, 1, [0]),            # 3 shares of 8 heads, 5 units a CTA
    (4, 5, 7000, 16, "e4m3", False, 3, [0]),           # 2 shares of 5 heads
    (1, 8, 20000, 16, "int8", False, 1, [0]),          # 4 shares
    (6, 8, 4001, 64, "e4m3", True, 2, [0, 3, 67, 20]),
    (5, 8, 3969, 128, "int8", True, 3, [0, 4, 131, 4 + 127, 50]),  # some last units without rows
    (200, 3, 41, 16, "int8", False, 1, [0, 1, 4, 5, 19, 20, 33]),  # groups of four warps
    (300, 8, 9, 16, "e4m3", True, 1, [0, 3, 11, 12, 18]),          # of one warp
    (90, 7, 70, 32, "int8", True, 4, [5, 35, 4, 20]),              # of eight, more than half without rows
]


@pytest.mark.parametrize("queries", [False, True])
@pytest.mark.parametrize("b,hkv,n,block,codes,bounds,axes,held", CASES)
def test_partitions(b, hkv, n, block, codes, bounds, axes, held, queries):
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(96, axes=[i * axes // 48 for i in range(48)], adjacent=b % 2 == 0)
    hq, most = 2 * hkv, n + max(held)
    both, plain = (_cache(hq, hkv, b, most, block, codes, bounds) for _ in range(2))
    before = [held[i % len(held)] for i in range(b)]
    for i, m in enumerate(before):
        if m:
            k, v = (x.contiguous() for x in _rows(1000 + i, 1, m, hkv, hkv))
            both.append(k, v, seq_begin=i)
            plain.append(k, v, seq_begin=i)
    q, k, v = _rows(n, b, n, hq, hkv, hkv)
    if axes > 1:
        pos = torch.randint(-1000, 100000, (axes, b, n), dtype=torch.int32, device="cuda")
        where = dict(positions=pos)
        turned = rot.rotate(q, k, **where)
    else:  # counted from what each sequence holds
        where = dict(first=-7)
        at = torch.tensor(before, device="cuda", dtype=torch.int32)[:, None] + torch.arange(n, device="cuda", dtype=torch.int32) - 7
        turned = rot.rotate(q, k, positions=at.contiguous())
    got = both.append_rotary(q if queries else None, k, v, rot, **where)
    apart = queries and b * n * hq >= 1 << 15
    assert both.last_launch_count() == (2 if apart else 1)
    plain.append(turned[1], v.contiguous())
    _same(both, plain)
    assert got is None if not queries else torch.equal(got, turned[0])


@pytest.mark.parametrize("queries", [False, True])
def test_replays_of_several_units(queries):
    """Captured, and replayed while the sequences' open blocks move on."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(64, axes=[0] * 16 + [1] * 16)
    b, hkv, n, block = 4, 8, 2503, 64
    both, plain = (_cache(16, hkv, b, 4 * n + 60, block, "int8", True) for _ in range(2))
    for i in range(1, b):
        k, v = (x.contiguous() for x in _rows(i, 1, 20 * i, hkv, hkv))
        both.append(k, v, seq_begin=i)
        plain.append(k, v, seq_begin=i)
    q, k, v = _rows(9, b, n, 16, hkv, hkv)
    pos = torch.zeros(2, b, n, dtype=torch.int32, device="cuda")
    out = torch.empty(b, 16, n, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both.append_rotary(q if queries else None, k, v, rot, positions=pos, out=out if queries else None)
    both.sync_host()
    for step in range(4):
        pos.copy_(torch.randint(0, 1 << 30, pos.shape, dtype=torch.int32, device="cuda"))
        graph.replay()
        qr, kr = rot.rotate(q, k, positions=pos)
        plain.append(kr, v.contiguous())
        _same(both, plain)
        assert not queries or torch.equal(out, qr)


@pytest.mark.parametrize("n", [5, 3000])
def test_in_place_broadcast_and_streams(n):
    """Queries turned in place, keys and values broadcast over the batch, a call on
    another stream."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(32, adjacent=True)
    b, hkv, block = 3, 4, 16
    both, plain = (_cache(16, hkv, b, n, block, "int8", False) for _ in range(2))
    q = _rows(1, b, n, 16)[0].contiguous()
    k, v = (x.expand(b, -1, -1, -1) for x in _rows(2, 1, n, hkv, hkv))
    qr, kr = rot.rotate(q, k, first=11)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert both.append_rotary(q, k, v, rot, first=11, out=q, stream=side) is q
    side.synchronize()
    assert torch.equal(q, qr)
    plain.append(kr, v.contiguous())
    _same(both, plain)
