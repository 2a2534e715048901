"""Prompt attention with runs of keys, caps, distance biases and column sums
(kvc_prompt_attention) against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)
# column sums: every p off by 2 ln 2 dz relative, dz <= 100 (2^-22 + 7.2e-7) (log2
# units, |z| <= 100 and cap <= 50 in these cases): 1.4e-4; 2e-4 leaves the fp32
# sums their part
SUM_RTOL = 2e-4


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _bits(rng, shape, mult=1.0):
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    return bf16_bits((rng.standard_normal(shape) * mult).astype(np.float32))


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / hq) for j in range(hq)], dtype=torch.float32, device="cuda")


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _runs(kind, n, rng):
    """(begin, end) int arrays [n], or None for the causal default."""
    at = np.arange(n)
    if kind == "causal":
        return None, None
    if kind == "window":
        return np.maximum(0, at - 40), at + 1
    if kind == "prefix":
        m = n // 3
        return np.zeros(n, int), np.where(at < m, m, at + 1)
    if kind == "full":
        return np.zeros(n, int), np.full(n, n)
    if kind == "documents":
        cuts = np.unique(np.concatenate([[0], rng.integers(0, n, max(1, n // 50))]))
        begin = cuts[np.searchsorted(cuts, at, side="right") - 1]
        return begin, at + 1
    if kind == "pads":  # the first and last rows, and some in between, see nothing
        begin, end = np.zeros(n, int), at + 1
        for rows in (at < 3, at >= n - 5, at % 97 == 50):
            begin[rows], end[rows] = 7, 7
        return begin, end
    if kind == "future":  # only keys after the query: the last rows see nothing
        return at + 1, np.minimum(n, at + 30)
    if kind == "outside":  # values outside [0, n) are clamped
        return at - 1000, np.where(at % 2 == 0, n + 1000, at + 1)
    raise AssertionError(kind)


def _reference(q, k, v, begin, end, cap, slopes):
    """(out, bound, sums) in fp64 of one sequence: q [hq, n, 128]."""
    hq, n = q.shape[:2]
    hkv = k.shape[0]
    at = np.arange(n)
    lo = np.zeros(n, int) if begin is None else np.clip(begin, 0, None)
    hi = at + 1 if end is None else np.clip(end, None, n)
    see = (at[None, :] >= lo[:, None]) & (at[None, :] < hi[:, None])
    out, bound, sums = np.empty(q.shape), np.empty(q.shape), np.zeros((hkv, n))
    for j in range(hq):
        h = j * hkv // hq
        z = R.scores(q[j], k[h], SCALE, cap, slopes[j] if slopes is not None else 0.0, at, at)
        p = R.softmax_rows(np.where(see, z, -np.inf))
        vd = v[h].astype(np.float64)
        out[j] = p @ vd
        bound[j] = R.output_bound(out[j], p, vd, R.score_error(z, cap, see))
        sums[h] += p.sum(0)
    return out, bound, sums


def _dev_runs(begin, end, batch):
    mk = lambda x: None if x is None else torch.tensor(np.tile(x, (batch, 1)).astype(np.int32)).cuda()  # noqa: E731
    return mk(begin), mk(end)


CASES = [
    # hq, hkv, batch, n, runs, cap, bias
    (8, 8, 1, 1, "causal", 10.0, True),
    (4, 2, 3, 7, "pads", 0.0, False),
    (8, 2, 2, 100, "documents", 20.0, True),
    (8, 1, 1, 128, "full", 0.0, True),
    (6, 2, 1, 129, "prefix", 3.0, True),
    (5, 1, 2, 255, "pads", 30.0, False),
    (4, 4, 1, 257, "future", 30.0, True),
    (4, 1, 2, 383, "window", 0.0, False),
    (16, 2, 1, 520, "documents", 0.0, True),
    (4, 2, 1, 700, "outside", 2.0, False),
    (2, 1, 1, 1500, "causal", 8.0, True),
    (2, 2, 1, 1411, "documents", 50.0, False),
    (2, 1, 1, 1100, "prefix", 0.0, False),
]


@pytest.mark.parametrize("hq,hkv,batch,n,runs,cap,bias", CASES)
def test_prompt_against_formula(hq, hkv, batch, n, runs, cap, bias):
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(n + hq)
    q, k, v = _bits(rng, (batch, hq, n, 128), 1.5), _bits(rng, (batch, hkv, n, 128), 1.5), \
        _bits(rng, (batch, hkv, n, 128))
    begin, end = _runs(runs, n, rng)
    db, de = _dev_runs(begin, end, batch)
    slopes = _slopes(hq) if bias else None
    status = _status()
    args = [T.to_dev_bf16(x) for x in (q, k, v)]
    kw = dict(status=status, softcap=cap, slopes=slopes, key_begin=db, key_end=de)
    out, sums = prompt_attention(*args, column_sums=True, **kw)
    alone = prompt_attention(*args, **kw)
    assert torch.equal(out, alone) and status.item() == 0
    again, sums2 = prompt_attention(*args, column_sums=True, **kw)
    assert torch.equal(out, again) and torch.equal(sums, sums2)
    got, gsum = T.bf16_tensor_to_f32(out), sums.cpu().numpy()
    f = O.bf16_bits_to_f32
    for b in range(batch):
        ref, bound, rsum = _reference(f(q[b]), f(k[b]), f(v[b]), begin, end, cap,
                                      slopes.double().cpu().numpy() if bias else None)
        err = np.abs(got[b] - ref)
        assert (err <= bound).all(), (b, float((err / bound).max()))
        np.testing.assert_allclose(gsum[b], rsum, rtol=SUM_RTOL, atol=1e-6)


def test_masked_places_do_not_leak():
    """NaN and infinities in K and V at masked places change nothing; a row
    that sees a V row that is not finite is NaN, the others keep their bits."""
    from compressed_kv_cache_kvc_gb300 import document_runs, prompt_attention
    rng = np.random.default_rng(2)
    hq, hkv, n = 4, 2, 300
    q, k, v = (torch.randn(1, h, n, 128, generator=torch.Generator().manual_seed(i)).cuda().bfloat16()
               for i, h in enumerate((hq, hkv, hkv)))
    begin, end = document_runs([100, 90, 110], device="cuda")
    kw = dict(key_begin=begin, key_end=end, softcap=10.0)
    clean, csum = prompt_attention(q, k, v, status=_status(), column_sums=True, **kw)
    k2, v2 = k.clone(), v.clone()
    k2[0, :, 150, 5] = float("nan")       # second document: keys 100 .. 189
    v2[0, 0, 120, 7] = float("inf")
    v2[0, 1, 130, 9] = float("nan")
    status = _status()
    out, sums = prompt_attention(q, k2, v2, status=status, column_sums=True, **kw)
    assert status.item() == 0x80  # the range flag
    for h, first in ((0, 120), (1, 130)):
        for j in (2 * h, 2 * h + 1):
            same = torch.ones(n, dtype=torch.bool)
            same[min(first, 150):190] = False  # rows that see the key
            assert torch.equal(out[0, j][same], clean[0, j][same])
            assert out[0, j, first:190].isnan().all()
    keep = torch.ones(n, dtype=torch.bool)
    keep[100:190] = False
    assert torch.equal(sums[0][:, keep], csum[0][:, keep])
    # a row of Q that is not finite spoils itself alone
    q2 = q.clone()
    q2[0, 1, 210, 3] = float("nan")
    out = prompt_attention(q2, k, v, status=_status(), **kw)
    rows = torch.arange(n) != 210
    assert torch.equal(out[0, 1][rows], clean[0, 1][rows]) and out[0, 1, 210].isnan().all()
    assert torch.equal(out[0, [0, 2, 3]], clean[0, [0, 2, 3]])


def test_large_values_saturate_and_flag():
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(1, 2, 50, 128, generator=g).cuda().bfloat16() for _ in range(3))
    v[0, 0, 4, 4] = 65280.0
    status = _status()
    prompt_attention(q, k, v, status=status)
    assert status.item() == 0
    v[0, 0, 4, 4] = 70000.0
    assert prompt_attention(q, k, v, status=status).isfinite().all()
    assert status.item() == 0x80


def test_large_scores():
    """Scores of many hundreds: the running maximum moves from tile to tile and
    no probability overflows."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(8)
    n = 400
    q, k, v = _bits(rng, (1, 2, n, 128), 8.0), _bits(rng, (1, 1, n, 128), 8.0), _bits(rng, (1, 1, n, 128))
    f = O.bf16_bits_to_f32
    out = T.bf16_tensor_to_f32(prompt_attention(*[T.to_dev_bf16(x) for x in (q, k, v)], status=_status()))
    ref, bound, _ = _reference(f(q[0]), f(k[0]), f(v[0]), None, None, 0.0, None)
    assert (np.abs(out[0] - ref) <= bound).all()


def test_steep_slopes():
    """Slopes of either sign far from 0: whole tiles underflow, or the furthest
    key wins."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(9)
    n, hq = 420, 4
    q, k, v = _bits(rng, (1, hq, n, 128)), _bits(rng, (1, 1, n, 128)), _bits(rng, (1, 1, n, 128))
    slopes = torch.tensor([4.0, -1.0, 0.0, 1e-3], device="cuda")
    f = O.bf16_bits_to_f32
    for cap in (0.0, 12.0):
        out, sums = prompt_attention(*[T.to_dev_bf16(x) for x in (q, k, v)], status=_status(), slopes=slopes,
                                     softcap=cap, column_sums=True)
        ref, bound, rsum = _reference(f(q[0]), f(k[0]), f(v[0]), None, None, cap, slopes.cpu().numpy())
        got = T.bf16_tensor_to_f32(out)
        assert (np.abs(got[0] - ref) <= bound).all()
        np.testing.assert_allclose(sums[0].cpu().numpy(), rsum, rtol=5e-4, atol=1e-6)


def test_graph_and_streams():
    """Captured and replayed on new inputs, and on a stream of its own with two
    calls' workspaces in flight, the results are the eager ones."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    g = torch.Generator().manual_seed(6)
    mk = lambda h: torch.randn(2, h, 333, 128, generator=g).cuda().bfloat16()  # noqa: E731
    q, k, v, q2, k2, v2 = mk(4), mk(2), mk(2), mk(4), mk(2), mk(2)
    status = _status()
    kw = dict(status=status, softcap=9.0, column_sums=True)
    want = prompt_attention(q, k, v, **kw)
    want2 = prompt_attention(q2, k2, v2, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = prompt_attention(q, k, v, **kw)
    b = prompt_attention(q2, k2, v2, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + b, want + want2))
    iq, ik, iv = q.clone(), k.clone(), v.clone()
    out, sums = torch.empty_like(q), torch.empty_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        prompt_attention(iq, ik, iv, out=out, status=status, softcap=9.0, column_sums=sums)
    for src, ref in (((q2, k2, v2), want2), ((q, k, v), want)):
        for d, s in zip((iq, ik, iv), src):
            d.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(sums, ref[1])
    assert status.item() == 0


def test_refusals():
    from compressed_kv_cache_kvc_gb300 import _lib as L
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    q = torch.zeros(1, 4, 20, 128, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(1, 2, 20, 128, device="cuda", dtype=torch.bfloat16)
    st = _status()
    for a in [(q.float(), k, k), (q, k.transpose(1, 2), k), (q, k, k[:, :, :10].contiguous()), (q.cpu(), k, k),
              (q[..., :64].contiguous(), k, k), (q, torch.zeros(1, 3, 20, 128, device="cuda").bfloat16(), k),
              (q[0], k, k)]:
        with pytest.raises(ValueError):
            prompt_attention(*a, status=st)
    for kw in [dict(slopes=torch.zeros(3, device="cuda")), dict(key_begin=torch.zeros(1, 20, device="cuda")),
               dict(key_end=torch.zeros(20, device="cuda", dtype=torch.int32)), dict(out=q.float()),
               dict(column_sums=torch.zeros(1, 4, 20, device="cuda"))]:
        with pytest.raises(ValueError):
            prompt_attention(q, k, k, status=st, **kw)
    with pytest.raises(ValueError):
        prompt_attention(q, k, k, status=torch.zeros(1, device="cuda"))
    for kw in [dict(softcap=-1.0), dict(softcap=float("inf")), dict(softcap=float("nan")), dict(sm_scale=0.0),
               dict(sm_scale=float("nan")), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises(L.KvcError) as e:
            prompt_attention(q, k, k, status=st, **kw)
        assert e.value.status == L.KVC_ERR_INVALID_ARG
    with pytest.raises(L.KvcError):
        prompt_attention(q[:, :, :0], k[:, :, :0], k[:, :, :0], status=st)
    assert st.item() == 0
