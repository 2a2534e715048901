"""Rotary positions: rows against the formula in 64 bits or more at any position,
layout and number of axes; appends with the rotation equal, bit for bit, to the
rotation followed by the plain append; the bounds of every block's keys."""
import numpy as np
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


def _rows(seed, *shape, mult=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * mult).to(torch.bfloat16)


def _fused(seed, b, n, *heads):
    """Views [b, heads, n, 128] of one projection's output."""
    return [x.transpose(1, 2) for x in _rows(seed, b, n, sum(heads), D).split(list(heads), dim=2)]


def _axes(half, count):
    return [i * count // half for i in range(half)]


def _formula(x, rot, positions):
    """(turned, sum of the pair's magnitudes) of x [b, h, n, 128] in long double;
    positions int64 [axes, b, n]."""
    half = rot.rotary_dim // 2
    x = x.float().cpu().numpy().astype(np.longdouble)
    freq = np.array(list(rot.plan.freq)[:half], dtype=np.float32).astype(np.longdouble)
    axis = np.array(list(rot.plan.axis)[:half])
    t = positions[axis].astype(np.longdouble).transpose(1, 2, 0)[:, None] * freq  # [b, 1, n, half]
    c, s = np.cos(t), np.sin(t)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if rot.adjacent else (i, i + half)
    out, size = x.copy(), np.zeros_like(x)
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, size


def _check(got, x, rot, positions):
    """bf16's half step 2^-8 of the value; cos and sin off by at most 1.5e-7, a
    product and a multiply-add round by 2^-24 each: 3e-7 of |x| + |y| in all."""
    want, size = _formula(x, rot, positions)
    far = np.abs(got.float().cpu().numpy().astype(np.longdouble) - want)
    assert np.all(far <= 2.0 ** -8 * np.abs(want) + 3e-7 * size + 1e-38), float(far.max())


CASES = [
    # batch, hq, hkv, n, rotary_dim, adjacent, axes, fused
    (1, 8, 8, 1, 128, False, 1, False),
    (1, 1, 1, 1, 16, True, 1, True),
    (3, 6, 2, 5, 128, True, 3, True),
    (2, 5, 1, 67, 96, False, 3, True),
    (5, 12, 4, 3, 48, False, 4, False),
    (2, 64, 8, 33, 64, True, 2, True),
    (1, 28, 4, 1003, 112, False, 1, True),
]


@pytest.mark.parametrize("b,hq,hkv,n,dim,adjacent,axes,fused", CASES)
def test_rotate(b, hq, hkv, n, dim, adjacent, axes, fused):
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(dim, base=5e5, axes=_axes(dim // 2, axes), adjacent=adjacent)
    assert rot.num_axes == axes
    q, k = _fused(n, b, n, hq, hkv) if fused else (_rows(1, b, hq, n, D), _rows(2, b, hkv, n, D))
    rng = np.random.default_rng(n)
    pos = rng.integers(-5000, 200000, size=(axes, b, n))
    pos[:, 0, 0] = 0
    dev = torch.from_numpy(pos.astype(np.int32)).cuda()
    qo, ko = rot.rotate(q, k, positions=dev)
    _check(qo, q, rot, pos)
    _check(ko, k, rot, pos)
    assert torch.equal(qo[0, :, 0], q[0, :, 0])  # position 0
    assert torch.equal(qo[..., dim:], q[..., dim:])
    # without positions: counted from `first` on every axis
    line = np.broadcast_to(np.arange(n) + 77, (axes, b, n))
    alone = rot.rotate(q, first=77)
    _check(alone, q, rot, line)
    assert torch.equal(alone, rot.rotate(q, positions=torch.from_numpy(line.astype(np.int32)).cuda().contiguous()))
    # in place, and into a given tensor
    x = q.contiguous().clone()
    assert rot.rotate(x, first=77, out=x) is x and torch.equal(x, alone)
    if axes == 1:
        assert torch.equal(rot.rotate(q, positions=dev[0]), qo)


def test_far_positions_and_frequencies():
    """Positions over the whole of 32 bits, frequencies from 65536 down to ones
    whose turn is below the fixed point's last place."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    freqs = [65536.0, -3.0, 1.0, 2.0 ** -24 * 3, 1e-12, 1e-30, 0.0, 6.2831855] + [10000.0 ** (-i / 24) for i in range(24)]
    rot = Rotary(64, freqs=freqs)
    rng = np.random.default_rng(0)
    pos = rng.integers(-2 ** 31, 2 ** 31, size=(1, 2, 300))
    pos[0, 0, :6] = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 << 30]
    q = _rows(3, 2, 3, 300, D)
    got = rot.rotate(q, positions=torch.from_numpy(pos.astype(np.int32)).cuda())
    # (exact angles: 31 and 24 bits in the long double's 64, its own 2 pi to 2^-64)
    _check(got, q, rot, pos)


def test_values_that_are_not_finite_stay_in_their_pairs():
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(32)
    q = _rows(4, 1, 2, 9, D)
    clean = rot.rotate(q, first=5)
    q[0, 0, 3, 2], q[0, 1, 4, 20], q[0, 1, 4, 100] = float("inf"), float("nan"), float("inf")
    got = rot.rotate(q, first=5)
    hit = torch.zeros_like(q, dtype=torch.bool)
    hit[0, 0, 3, [2, 18]] = hit[0, 1, 4, [4, 20]] = hit[0, 1, 4, 100] = True
    assert not torch.isfinite(got[hit]).any() and torch.equal(got[~hit], clean[~hit])


def _cache(hq, hkv, lengths, block, codes, bounds=False):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    per_seq = max(lengths) // block + 1
    return BlockScaledCache(hq, hkv, len(lengths) * per_seq, len(lengths), per_seq, block_tokens=block, codes=codes,
                            key_bounds=bounds)


def _same_state(a, b, bounds=False):
    """Equal lengths, tables, scales, codes and exact rows of what is held."""
    for name in ("SEQ_POS", "TABLE", "COUNTERS", "K_SCALE", "V_SCALE", "K_CODES", "V_CODES", "K_EXACT", "V_EXACT"):
        assert torch.equal(a.buffer(name), b.buffer(name)), name


APPENDS = [
    # block, codes, parts, rotary_dim, adjacent, axes, fused, bounds
    (16, "int8", [1, 1, 1, 1, 1, 15, 1, 1], 128, False, 1, True, False),
    (16, "e4m3", [20, 0, 300, 7], 64, True, 3, True, True),
    (32, "int8", [4, 31, 1, 1, 200, 30], 96, False, 3, False, True),
    (64, "int8", [700], 16, True, 1, True, True),
    (64, "e4m3", [2, 66, 130, 64], 128, False, 1, False, False),
    (128, "int8", [131, 1, 127, 260], 128, True, 3, True, True),
    (128, "e4m3", [1000, 5], 80, False, 2, True, True),
]


@pytest.mark.parametrize("block,codes,parts,dim,adjacent,axes,fused,bounds", APPENDS)
def test_append_rotary(block, codes, parts, dim, adjacent, axes, fused, bounds):
    """The same state and queries as the rotation and then the plain append, also
    for open rows that a later append quantises."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(dim, axes=_axes(dim // 2, axes), adjacent=adjacent)
    b, hq, hkv, n = 3, 6, 2, sum(parts)
    both, plain = _cache(hq, hkv, [n] * b, block, codes, bounds), _cache(hq, hkv, [n] * b, block, codes)
    q, k, v = _fused(n, b, n, hq, hkv, hkv)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, 100000, (axes, b, n), dtype=torch.int32, device="cuda")
    at, turned = 0, []
    for i, m in enumerate(parts):
        part = [x[:, :, at:at + m] for x in (q, k, v)]
        given = i % 2 == 1 or axes > 1
        where = dict(positions=pos[:, :, at:at + m].contiguous()) if given else dict(first=9)
        got = both.append_rotary(*part, rot, **where)
        assert both.last_launch_count() == (1 if m else 0)
        if m:
            if not given:
                where["first"] += at
            qr, kr = rot.rotate(part[0], part[1], **where)
            assert torch.equal(got, qr)
            plain.append(kr, part[2].contiguous())
            turned.append(kr)
        at += m
    _same_state(both, plain)
    assert both.read_status() == 0
    if bounds:
        _check_bounds(both, torch.cat(turned, dim=2).float().cpu().numpy())


def _check_bounds(cache, keys):
    """Least and largest INT8 codes of every closed block's keys [b, hkv, n, 128]."""
    from tests import ops64 as R
    b, hkv, n, _ = keys.shape
    block, nb = cache.block_tokens, cache.num_blocks
    got = cache.bounds[:nb * hkv * 256].view(torch.int8).view(nb, hkv, 2, D).cpu().numpy()
    scale = cache.bounds[nb * hkv * 256:][:nb * hkv * 4].view(torch.float32).view(nb, hkv).cpu().numpy()
    table = cache.buffer("TABLE").view(torch.int32).view(b, -1).cpu().numpy()
    for s in range(b):
        for h in range(hkv):
            for c in range((n - 4) // block):
                code, t = R.quantise_block(keys[s, h, 4 + c * block:4 + (c + 1) * block], False)
                assert scale[table[s, c], h] == t
                assert np.array_equal(got[table[s, c], h], np.stack([code.min(0), code.max(0)]))


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("codes", ["int8", "e4m3"])
def test_key_bounds(block, codes):
    """Bounds kept by the plain append: INT8 codes whatever the cache's are, the
    same however the tokens are split; the cache itself as without them."""
    from compressed_kv_cache_kvc_gb300 import _lib as L
    b, hkv, n = 2, 3, 4 + 5 * block + 3
    k, v = _rows(block, b, hkv, n, D), _rows(block + 1, b, hkv, n, D)
    k[..., 7] *= 9
    k[1, 0, 4:4 + block] = 0
    k[0, 1, :, 20:40] = k[0, 1, :, 20:40].abs() + 1  # channels of one sign
    whole, split, plain = (_cache(6, hkv, [n] * b, block, codes, x) for x in (True, True, False))
    whole.append(k, v)
    plain.append(k, v)
    for i in range(0, n, 11):
        split.append(k[:, :, i:i + 11].contiguous(), v[:, :, i:i + 11].contiguous())
    _same_state(whole, plain)
    for c in (whole, split):
        _check_bounds(c, k.float().cpu().numpy())
    # a state with sequences in it has blocks without bounds
    assert whole.lib.kvc_block_set_key_bounds(whole.handle, None, 0) == L.KVC_ERR_STATE


def test_replays_and_streams():
    """A captured append goes on counting; a call on another stream."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary()
    b, hq, hkv, n = 2, 4, 2, 40
    a, ref = _cache(hq, hkv, [n + 8] * b, 16, "int8"), _cache(hq, hkv, [n + 8] * b, 16, "int8")
    q, k, v = _fused(5, b, n, hq, hkv, hkv)
    part = [x[:, :, :1].clone() for x in (q, k, v)]
    out = torch.empty_like(part[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.append_rotary(*part, rot, first=100, out=out, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.append_rotary(*part, rot, first=100, out=out)
    for i in range(1, n):
        for x, y in zip(part, (q, k, v)):
            x.copy_(y[:, :, i:i + 1])
        graph.replay()
        if i in (1, 20, n - 1):
            assert torch.equal(out, rot.rotate(q[:, :, i:i + 1], first=100 + i))
    kr = rot.rotate(k, first=100)
    ref.append(kr, v.contiguous())
    a.sync_host()
    assert a.lengths(0, b) == (n, n)
    for x, y in zip(a.read(0, b, 0, n), ref.read(0, b, 0, n)):
        assert torch.equal(x, y)


def test_replays_of_long_appends():
    """Queries of many rows, turned by a launch of their own that also advances the
    lengths: captured, replayed, and replayed once more than there is room for."""
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot = Rotary(64, adjacent=True)
    b, hq, hkv, n, block = 2, 16, 2, 1100, 32
    a, ref = (_cache(hq, hkv, [3 * n] * b, block, "e4m3") for _ in range(2))
    q, k, v = _fused(6, b, n, hq, hkv, hkv)
    out = torch.empty(b, hq, n, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.append_rotary(q, k, v, rot, first=7, out=out)
    assert a.lib.kvc_block_last_launch_count(a.handle) == 2
    for i in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, rot.rotate(q, first=7 + i * n))
        ref.append(rot.rotate(k, first=7 + i * n), v.contiguous())
    a.sync_host()
    assert a.lengths(0, b) == (3 * n, 3 * n) and a.read_status() == 0
    for x, y in zip(a.read(0, b, 0, 3 * n), ref.read(0, b, 0, 3 * n)):
        assert torch.equal(x, y)
    graph.replay()  # no room: flagged, nothing appended
    assert a.read_status() != 0
    a.sync_host()
    assert a.lengths(0, b) == (3 * n, 3 * n)
    assert (a.buffer("TICKETS").view(torch.int32) == 0).all()
    for x, y in zip(a.read(0, b, 0, 3 * n), ref.read(0, b, 0, 3 * n)):
        assert torch.equal(x, y)


def test_refused():
    from compressed_kv_cache_kvc_gb300 import Rotary
    rot, two = Rotary(), Rotary(axes=_axes(64, 2))
    q = _rows(0, 2, 4, 8, D)
    pos = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    for call in (lambda: rot.rotate(q.float()), lambda: rot.rotate(q[0]), lambda: rot.rotate(q[..., :64]),
                 lambda: rot.rotate(q.transpose(2, 3)), lambda: rot.rotate(q, positions=pos.long()),
                 lambda: rot.rotate(q, positions=pos[:, :4].contiguous()), lambda: two.rotate(q, positions=pos),
                 lambda: rot.rotate(q, out=q[:1]), lambda: rot.rotate(q.cpu()), lambda: rot.rotate(q[:0]),
                 lambda: rot.rotate(q, q[:1]), lambda: rot.rotate(_rows(0, 2, 4, 8, 132)[..., :128]),
                 lambda: rot.rotate(q.transpose(0, 1), out=q.transpose(0, 1)), lambda: rot.rotate(q, first=1 << 31),
                 lambda: rot.rotate(q, first=-(1 << 31) - 1)):
        with pytest.raises(ValueError):
            call()
    c = _cache(4, 2, [20] * 2, 16, "int8")
    k = _rows(1, 2, 2, 8, D)
    for call in (lambda: c.append_rotary(q, q, q, rot), lambda: c.append_rotary(k, k, k, rot),
                 lambda: c.append_rotary(q, k, k[:1], rot), lambda: c.append_rotary(q, k, k.float(), rot),
                 lambda: c.append_rotary(q, k, k, two, positions=pos), lambda: c.append_rotary(q[:, :, :4], k, k, rot)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(RuntimeError):
        c.append_rotary(None, _rows(1, 2, 2, 100, D), _rows(1, 2, 2, 100, D), rot)  # no room
    assert c.lengths(0, 2) == (0, 0)
    assert c.append_rotary(None, k, k, rot) is None and c.lengths(0, 2) == (8, 8)
