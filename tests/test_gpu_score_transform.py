"""Capped and distance-biased scores (kvc_set_score_transform) in every
attention on a cache, against the formula in 64 bits on the cache's own device
state: the tokens it holds, at the positions they were appended at."""
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


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (j + 1) / hq) for j in range(hq)], dtype=torch.float32, device="cuda")


def _values(st, codes, kind):
    if kind == "e4m3":
        raw = torch.from_numpy(np.ascontiguousarray(codes).view(np.uint8))
        return raw.view(torch.float8_e4m3fn).double().numpy()
    return codes.astype(np.float64)


def _tokens(st, b, h, kind):
    """(positions, K, V, K scales, V scales) in fp64 of everything (b, h)
    attends to; the scales are 0 where a token is not held in integer codes."""
    pos, kc, ks, vc, vs, _ = st.head(b, h)
    k = _values(st, kc, kind) * ks[:, None].astype(np.float64)
    v = _values(st, vc, kind) * vs[:, None].astype(np.float64)
    ns = min(int(st.seen[b]), 4)
    f = lambda x: O.bf16_bits_to_f32(x).astype(np.float64)  # noqa: E731
    whole = 0.0 if kind == "e4m3" else 1.0
    parts = [(np.arange(ns), f(st.sink_k[b, h, :ns]), f(st.sink_v[b, h, :ns]), np.zeros(ns), np.zeros(ns)),
             (pos, k, v, whole * ks.astype(np.float64), whole * vs.astype(np.float64))]
    if st.W:
        rp, rk, rv, _ = st.ring_head(b, h)
        parts.append((rp, f(rk), f(rv), np.zeros(len(rp)), np.zeros(len(rp))))
    return tuple(np.concatenate([p[i] for p in parts]) for i in range(5))


def _expect(st, q, kind, hq, cap, slopes):
    """[(b, j)] -> (positions, p, output, bound) from the state before."""
    B, G = q.shape[0], hq // st.hkv
    res = {}
    for b in range(B):
        P = int(st.seen[b])
        for j in range(hq):
            pos, k, v, ks, vs = _tokens(st, b, j // G, kind)
            qf = O.bf16_bits_to_f32(q[b, j:j + 1])
            z = R.scores(qf, k, SCALE, cap, slopes[j] if slopes is not None else 0.0,
                         [P - 1], pos)
            p = R.softmax_rows(z)
            ref = p @ v
            dz_codes, more = R.offset_terms(qf, ks, vs, p, SCALE)
            dz = R.score_error(z, cap, np.ones_like(z, dtype=bool)) + dz_codes
            res[b, j] = pos, p[0], ref[0], (R.output_bound(ref, p, v, dz) + more)[0], dz
    return res


def _check_out(out, exp, what=""):
    got = T.bf16_tensor_to_f32(out)
    for (b, j), (_, _, ref, bound, _) in exp.items():
        err = np.abs(got[b, j] - ref)
        assert (err <= bound).all(), (what, b, j, float((err / bound).max()))


def _filled(rng, hq, hkv, bits, kind, lengths, W=0, mult=1.0):
    from compressed_kv_cache_kvc_gb300 import KVCache
    B = len(lengths)
    mbps = (max(lengths) + 40) // 16 + 2
    order = np.random.default_rng(3).permutation(B * mbps).astype(np.int32)
    cache = KVCache(hq, hkv, bits, B * mbps, B, mbps, block_order=order, bf16_window=W,
                    codes="e4m3" if kind == "e4m3" else "int")
    for b, n in enumerate(lengths):
        k, v = _bits(rng, (1, hkv, n, 128), mult), _bits(rng, (1, hkv, n, 128))
        cache.quantize_append(T.to_dev_bf16(k), T.to_dev_bf16(v), seq_begin=b)
    return cache


DECODE = [
    # bits, kind, hq, hkv, lengths, window W, cap, bias, size of K
    (8, "int", 8, 8, [512], 0, 50.0, False, 1.0),
    (8, "int", 8, 2, [300, 41, 5, 1], 0, 0.0, True, 1.0),
    (4, "int", 40, 8, [700, 90], 0, 20.0, True, 2.0),
    (8, "e4m3", 16, 4, [260, 33], 0, 5.0, True, 6.0),      # most scores beyond the polynomial's interval
    (8, "int", 64, 8, [130], 0, 1.5, False, 6.0),          # saturated caps, the largest group
    (8, "int", 4, 4, [20, 70], 100, 30.0, True, 1.0),      # nothing in the pool; the window wraps
    (4, "int", 16, 4, [400, 180], 50, 10.0, True, 3.0),
    (8, "e4m3", 3, 1, [2000], 16, 0.0, True, 1.0),
]


@pytest.mark.parametrize("bits,kind,hq,hkv,lengths,W,cap,bias,mult", DECODE)
def test_decode_attention(bits, kind, hq, hkv, lengths, W, cap, bias, mult):
    """Outputs and the H2O scores of one decode attention; the split, window,
    merge and score passes all see the transform."""
    rng = np.random.default_rng(bits + hq + sum(lengths))
    cache = _filled(rng, hq, hkv, bits, kind, lengths, W, mult)
    slopes = _slopes(hq) if bias else None
    cache.set_score_transform(softcap=cap, slopes=slopes)
    q = _bits(rng, (len(lengths), hq, 128), 1.5)
    st0 = T.StateView(cache)
    exp = _expect(st0, q, kind, hq, cap, slopes.double().cpu().numpy() if bias else None)
    out = cache.decode_attention(T.to_dev_bf16(q), accumulate_h2o=True)
    _check_out(out, exp)
    noalloc = torch.empty_like(out)
    assert cache.lib.kvc_decode_attention_noalloc(
        cache.handle, 0, len(lengths), T.to_dev_bf16(q).data_ptr(), noalloc.data_ptr(), SCALE, 0,
        torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, noalloc)
    st = T.StateView(cache)
    G = hq // hkv
    for b in range(len(lengths)):
        for h in range(hkv):
            want = sum(exp[b, h * G + g][1] for g in range(G))
            ns = min(int(st.seen[b]), 4)
            got = np.concatenate([st.sink_score[b, h, :ns], st.head(b, h)[5]] +
                                 ([st.ring_head(b, h)[3]] if W else []))
            # relative: 2 ln 2 dz, and fp32 sums
            dz = max(exp[b, h * G + g][4] for g in range(G))
            np.testing.assert_allclose(got, want, rtol=2 * np.log(2) * dz + 1e-5, atol=1e-7)
    assert cache.read_status() == 0


def test_positions_after_evictions():
    """After H2O evictions slots are not in position order: the bias goes by the
    positions the tokens were appended at.  Several one-call steps against the
    formula on the state that the append left (rebuilt by a twin cache)."""
    from compressed_kv_cache_kvc_gb300 import KVCache
    rng = np.random.default_rng(9)
    hq, hkv, n, budget, recent = 16, 4, 300, 90, 20
    caches = [KVCache(hq, hkv, 8, 40, 1, 40) for _ in range(2)]
    slopes = _slopes(hq)
    k, v = _bits(rng, (1, hkv, n, 128)), _bits(rng, (1, hkv, n, 128))
    for c in caches:
        c.set_score_transform(softcap=15.0, slopes=slopes)
        c.quantize_append(T.to_dev_bf16(k), T.to_dev_bf16(v))
    for step in range(6):
        q = _bits(rng, (1, hq, 128), 1.5)
        kn, vn = _bits(rng, (1, hkv, 1, 128)), _bits(rng, (1, hkv, 1, 128))
        d = [T.to_dev_bf16(x) for x in (q, kn, vn)]
        one = caches[0].decode_step(*d, mode="h2o", budget=budget, recent=recent)
        caches[1].quantize_append(d[1], d[2])
        st = T.StateView(caches[1])
        if step > 1:
            assert (np.diff(st.head(0, 0)[0]) < 0).any()  # slots out of position order
        exp = _expect(st, q, "int", hq, 15.0, slopes.double().cpu().numpy())
        _check_out(one, exp, f"step {step}")
        out = caches[1].decode_attention(d[0])
        assert torch.equal(one, out)
        mask = caches[1].h2o_select_evict(1, mode="h2o", budget=budget, recent=recent)
        caches[1].compact_blocks(mask, 1)
        a, b = T.StateView(caches[0]), T.StateView(caches[1])
        for h in range(hkv):
            for x, y in zip(a.head(0, h), b.head(0, h)):
                assert np.array_equal(np.asarray(x).view(np.uint8), np.asarray(y).view(np.uint8))


def test_overlapped_step_and_graph():
    """The overlapped step equals the one-call step bit for bit; a captured
    transformed attention replays at a longer length; clearing the transform
    gives the plain attention's bits back."""
    rng = np.random.default_rng(10)
    hq, hkv = 8, 2
    slopes = _slopes(hq)
    pair = []
    for _ in range(2):
        r = np.random.default_rng(11)
        pair.append(_filled(r, hq, hkv, 4, "int", [200, 77]))
        pair[-1].set_score_transform(softcap=8.0, slopes=slopes)
    side = torch.cuda.Stream()
    for _ in range(3):
        d = [T.to_dev_bf16(_bits(rng, s)) for s in ((2, hq, 128), (2, hkv, 1, 128), (2, hkv, 1, 128))]
        a = pair[0].decode_step(*d, mode="h2o", budget=80, recent=16)
        b = pair[1].decode_step_overlap(*d, side, mode="h2o", budget=80, recent=16)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    cache = pair[0]
    q = T.to_dev_bf16(_bits(rng, (2, hq, 128)))
    out = torch.empty_like(q)
    ws = cache.workspace(2)
    cache.decode_attention(q, out=out, workspace=ws, accumulate_h2o=False)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.decode_attention(q, out=out, workspace=ws, accumulate_h2o=False)
    cache.quantize_append(T.to_dev_bf16(_bits(rng, (2, hkv, 60, 128))), T.to_dev_bf16(_bits(rng, (2, hkv, 60, 128))))
    g.replay()
    torch.cuda.synchronize()
    exp = _expect(T.StateView(cache), q.view(torch.int16).cpu().numpy().view(np.uint16), "int", hq, 8.0,
                  slopes.double().cpu().numpy())
    _check_out(out, exp, "replayed")
    cache.set_score_transform()
    plain = cache.decode_attention(q, accumulate_h2o=False)
    twin = _filled(np.random.default_rng(11), hq, hkv, 4, "int", [200, 77])
    twin.state_view.copy_(cache.state_view)
    twin.sync_host()
    assert torch.equal(plain, twin.decode_attention(q, accumulate_h2o=False))


@pytest.mark.parametrize("bits,kind,hq,hkv,ctx,n,W,cap,bias", [
    (8, "int", 8, 2, 100, 37, 0, 10.0, True),
    (4, "int", 40, 8, 50, 20, 0, 0.0, True),
    (8, "e4m3", 8, 8, 0, 18, 0, 4.0, False),
    (8, "int", 16, 4, 90, 30, 24, 10.0, True),
    (4, "int", 16, 4, 70, 9, 16, 6.0, False),
])
def test_prefill_context(bits, kind, hq, hkv, ctx, n, W, cap, bias):
    """A prompt over context: query i sees what a decode step at its position
    would, and every held token's score grows by its column sum."""
    rng = np.random.default_rng(bits + hq + ctx)
    cache = _filled(rng, hq, hkv, bits, kind, [ctx], W) if ctx else _filled(rng, hq, hkv, bits, kind, [1], W)
    if not ctx:
        cache.release()
    slopes = _slopes(hq) if bias else None
    cache.set_score_transform(softcap=cap, slopes=slopes)
    q, k, v = _bits(rng, (1, hq, n, 128), 1.5), _bits(rng, (1, hkv, n, 128)), _bits(rng, (1, hkv, n, 128))
    out = T.bf16_tensor_to_f32(cache.prefill_context(T.to_dev_bf16(q), T.to_dev_bf16(k), T.to_dev_bf16(v)))
    st = T.StateView(cache)
    G = hq // hkv
    sums, dz_all = {h: 0.0 for h in range(hkv)}, 0.0
    for j in range(hq):
        pos, kd, vd, ks, vs = _tokens(st, 0, j // G, kind)
        qp = ctx + np.arange(n)
        z = R.scores(O.bf16_bits_to_f32(q[0, j]), kd, SCALE, cap, float(slopes[j]) if bias else 0.0, qp, pos)
        see = pos[None, :] <= qp[:, None]
        p = R.softmax_rows(np.where(see, z, -np.inf))
        ref = p @ vd
        err = np.abs(out[0, j] - ref)
        dz_codes, more = R.offset_terms(O.bf16_bits_to_f32(q[0, j]), ks, vs, p, SCALE)
        dz = R.score_error(z, cap, see) + dz_codes
        dz_all = max(dz_all, dz)
        bound = R.output_bound(ref, p, vd, dz) + more
        assert (err <= bound).all(), (j, float((err / bound).max()))
        sums[j // G] = sums[j // G] + p.sum(0)
    if not ctx:
        for h in range(hkv):
            got = np.concatenate([st.sink_score[0, h], st.head(0, h)[5]])
            np.testing.assert_allclose(got, sums[h], rtol=2 * np.log(2) * dz_all + 1e-5, atol=1e-6)
    assert cache.read_status() == 0


def test_prefill_with_transform_then_step():
    """kvc_prefill_attention honours the transform (outputs and the scores that
    seed the eviction), and its workspace grows with it."""
    from compressed_kv_cache_kvc_gb300 import KVCache
    rng = np.random.default_rng(12)
    hq, hkv, n = 8, 2, 150
    cache = KVCache(hq, hkv, 8, 24, 2, 12)
    plain_ws = cache.lib.kvc_prefill_workspace_bytes(cache.handle, 1, n)
    slopes = _slopes(hq)
    cache.set_score_transform(softcap=6.0, slopes=slopes)
    assert cache.lib.kvc_prefill_workspace_bytes(cache.handle, 1, n) > plain_ws
    q, k, v = _bits(rng, (1, hq, n, 128), 1.5), _bits(rng, (1, hkv, n, 128)), _bits(rng, (1, hkv, n, 128))
    f = O.bf16_bits_to_f32
    # one document after another: query i sees its own document only
    begin = torch.tensor([[0] * 60 + [60] * 90], dtype=torch.int32, device="cuda")
    for seq, kw in ((0, {}), (1, {"key_begin": begin})):
        d = [T.to_dev_bf16(x) for x in (q, k, v)]
        out = T.bf16_tensor_to_f32(cache.prefill(*d, seq_begin=seq, **kw))
        st = T.StateView(cache)
        at = np.arange(n)
        lo = begin[0].cpu().numpy() if kw else np.zeros(n, dtype=int)
        for h in range(hkv):
            total = np.zeros(n)
            for j in range(4 * h, 4 * h + 4):
                z = R.scores(f(q[0, j]), f(k[0, h]), SCALE, 6.0, float(slopes[j]), at, at)
                see = (at[None, :] <= at[:, None]) & (at[None, :] >= lo[:, None])
                p = R.softmax_rows(np.where(see, z, -np.inf))
                vd = f(v[0, h]).astype(np.float64)
                ref = p @ vd
                bound = R.output_bound(ref, p, vd, R.score_error(z, 6.0, see))
                assert (np.abs(out[0, j] - ref) <= bound).all()
                total += p.sum(0)
            pos, *_, score = st.head(seq, h)
            np.testing.assert_allclose(np.concatenate([st.sink_score[seq, h], score]),
                                       total[np.concatenate([np.arange(4), pos])], rtol=2e-4, atol=1e-6)
    step = [T.to_dev_bf16(_bits(rng, s)) for s in ((2, hq, 128), (2, hkv, 1, 128), (2, hkv, 1, 128))]
    cache.decode_step(*step, mode="h2o", budget=60, recent=16)
    assert cache.lengths(0) == (56, n + 1) and cache.read_status() == 0
