"""Later turns' prompts over context with a distance bias where the pool's
slots are not in position order (after H2O evictions), over several rounds of
query rows, and past the staged block ids."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R
from tests import test_gpu_score_transform as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _check(cache, kind, q, out, before, seen, cap, slopes):
    """Outputs and the growth of every held token's score against the formula on
    the state after the call; before: {(head, position): score}."""
    st = T.StateView(cache)
    hq, n = q.shape[1:3]
    G = hq // st.hkv
    for h in range(st.hkv):
        total, dz_all = 0.0, 0.0
        for j in range(h * G, h * G + G):
            pos, kd, vd, ks, vs = S._tokens(st, 0, h, kind)
            qp = seen + np.arange(n)
            qf = O.bf16_bits_to_f32(q[0, j])
            z = R.scores(qf, kd, S.SCALE, cap, slopes[j] if slopes is not None else 0.0, qp, pos)
            see = pos[None, :] <= qp[:, None]
            p = R.softmax_rows(np.where(see, z, -np.inf))
            ref = p @ vd
            dz_codes, more = R.offset_terms(qf, ks, vs, p, S.SCALE)
            dz = R.score_error(z, cap, see) + dz_codes
            err = np.abs(out[0, j] - ref)
            bound = R.output_bound(ref, p, vd, dz) + more
            assert (err <= bound).all(), (j, float((err / bound).max()))
            total, dz_all = total + p.sum(0), max(dz_all, dz)
        got = np.concatenate([st.sink_score[0, h], st.head(0, h)[5]] + ([st.ring_head(0, h)[3]] if st.W else []))
        old = np.array([before.get((h, int(x)), 0.0) for x in pos])
        # (a sum of two fp32 scores: a step of the larger)
        np.testing.assert_allclose(got, old + total, rtol=2 * np.log(2) * dz_all + 1e-5, atol=1e-6 + 2e-7 * old.max())


def _scores(cache):
    st = T.StateView(cache)
    d = {}
    for h in range(st.hkv):
        for x, y in zip(range(4), st.sink_score[0, h]):
            d[h, x] = float(y)
        pos, *_, sc = st.head(0, h)
        d.update({(h, int(x)): float(y) for x, y in zip(pos, sc)})
        if st.W:
            rp, _, _, rs = st.ring_head(0, h)
            d.update({(h, int(x)): float(y) for x, y in zip(rp, rs)})
    return d


@pytest.mark.parametrize("bits,kind,hq,hkv,ctx,budget,n,W,cap,bias", [
    (8, "int", 8, 2, 700, 300, 60, 0, 12.0, True),
    (4, "int", 10, 2, 500, 200, 90, 0, 0.0, True),
    (8, "e4m3", 4, 4, 400, 150, 33, 0, 5.0, True),
    (8, "int", 8, 2, 600, 250, 40, 32, 12.0, True),
    (4, "int", 8, 1, 300, 120, 40, 24, 0.0, True),
    (8, "int", 8, 1, 200, 100, 700, 0, 9.0, True),      # 5,600 rows: two rounds of CTAs
    (8, "int", 2, 1, 33500, 0, 20, 0, 9.0, True),        # 2,094 pages: past the staged block ids
])
def test_after_evictions(bits, kind, hq, hkv, ctx, budget, n, W, cap, bias):
    rng = np.random.default_rng(ctx + n)
    from compressed_kv_cache_kvc_gb300 import KVCache
    pages = (ctx + n + 60) // 16 + 2
    cache = KVCache(hq, hkv, bits, pages, 1, pages, bf16_window=W, codes="e4m3" if kind == "e4m3" else "int")
    slopes = S._slopes(hq) if bias else None
    cache.set_score_transform(softcap=cap, slopes=slopes)
    draw = lambda h, m, size=1.0: S._bits(rng, (1, h, m, 128), size)  # noqa: E731
    cache.quantize_append(T.to_dev_bf16(draw(hkv, ctx)), T.to_dev_bf16(draw(hkv, ctx)))
    if budget:
        for _ in range(4):
            cache.decode_step(T.to_dev_bf16(S._bits(rng, (1, hq, 128), 1.5)), T.to_dev_bf16(draw(hkv, 1)),
                              T.to_dev_bf16(draw(hkv, 1)), mode="h2o", budget=budget, recent=16 + W)
        st = T.StateView(cache)
        assert any((np.diff(st.head(0, h)[0]) < 0).any() for h in range(hkv))  # slots out of position order
    before, seen = _scores(cache), ctx + (4 if budget else 0)
    q = draw(hq, n, 1.5)
    out = cache.prefill_context(T.to_dev_bf16(q), T.to_dev_bf16(draw(hkv, n)), T.to_dev_bf16(draw(hkv, n)))
    _check(cache, kind, q, T.bf16_tensor_to_f32(out), before, seen, cap,
           slopes.double().cpu().numpy() if bias else None)
    assert cache.read_status() == 0


@pytest.mark.parametrize("bits,kind", [(8, "int"), (4, "int"), (8, "e4m3")])
@pytest.mark.parametrize("pool,window", [(1e35, 1.0), (1e35, 1e35), (1.0, 1e35), (1e-30, 1.0), (1e-30, 1e-30)])
def test_value_range_with_a_window(bits, kind, pool, window):
    """A prompt over a pool and a bf16 window of very different V."""
    from compressed_kv_cache_kvc_gb300 import KVCache
    rng = np.random.default_rng(bits)
    hq, hkv, ctx, W, n = 4, 2, 200, 32, 20
    cache = KVCache(hq, hkv, bits, 40, 1, 40, bf16_window=W, codes="e4m3" if kind == "e4m3" else "int")
    size = np.where(np.arange(ctx) < ctx + n - W, pool, window)[:, None]
    draw = lambda h, m: S._bits(rng, (1, h, m, 128))  # noqa: E731
    cache.quantize_append(T.to_dev_bf16(draw(hkv, ctx)), T.to_dev_bf16(S._bits(rng, (1, hkv, ctx, 128), size)))
    q = draw(hq, n)
    out = T.bf16_tensor_to_f32(cache.prefill_context(T.to_dev_bf16(q), T.to_dev_bf16(draw(hkv, n)),
                                                     T.to_dev_bf16(S._bits(rng, (1, hkv, n, 128), window))))
    st = T.StateView(cache)
    for j in range(hq):
        pos, kd, vd, ks, vs = S._tokens(st, 0, j // 2, kind)
        qp = ctx + np.arange(n)
        qf = O.bf16_bits_to_f32(q[0, j])
        z = R.scores(qf, kd, S.SCALE, 0.0, 0.0, qp, pos)
        see = pos[None, :] <= qp[:, None]
        p = R.softmax_rows(np.where(see, z, -np.inf))
        ref = p @ vd
        dz_codes, more = R.offset_terms(qf, ks, vs, p, S.SCALE)
        dz = R.score_error(z, 0.0, see) + dz_codes
        m = p.shape[-1]
        # ops64's bound without its absolute terms, all of them relative to V
        bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * np.log(2) * dz + m * 2.0 ** -24) * (p @ np.abs(vd))
                 + m * 2.0 ** -24 * np.abs(vd).max() + more)
        err = np.abs(out[0, j] - ref)
        assert (err <= bound).all(), (j, float((err / bound).max()))
    assert cache.read_status() == 0


@pytest.mark.parametrize("bits,kind,hq,hkv,ctx,n,W,bias", [
    (8, "int", 56, 8, 66, 38, 40, True),
    (8, "int", 16, 2, 300, 90, 100, True),
    (4, "int", 40, 8, 200, 33, 130, False),
    (8, "e4m3", 28, 4, 150, 70, 64, True),
    (4, "int", 8, 1, 700, 100, 512, True),
])
def test_windows_of_several_tiles(bits, kind, hq, hkv, ctx, n, W, bias):
    """More tiles of the bf16 window than stages for them, the warps of a CTA at
    different tiles: the formula's outputs and scores, call after call."""
    from compressed_kv_cache_kvc_gb300 import KVCache
    rng = np.random.default_rng(W + n)
    pages = (ctx + n) // 16 + 4
    cache = KVCache(hq, hkv, bits, pages, 1, pages, bf16_window=W, codes="e4m3" if kind == "e4m3" else "int")
    slopes = S._slopes(hq) if bias else None
    cache.set_score_transform(softcap=20.0, slopes=slopes)
    draw = lambda h, m, size=1.0: S._bits(rng, (1, h, m, 128), size)  # noqa: E731
    k0, v0, k, v = (T.to_dev_bf16(draw(hkv, m)) for m in (ctx, ctx, n, n))
    q = draw(hq, n, 1.5)
    first = None
    for _ in range(20):
        cache.release()
        cache.quantize_append(k0, v0)
        before = _scores(cache) if first is None else None
        out = cache.prefill_context(T.to_dev_bf16(q), k, v)
        if first is None:
            first = out
            _check(cache, kind, q, T.bf16_tensor_to_f32(out), before, ctx, 20.0,
                   slopes.double().cpu().numpy() if bias else None)
        assert torch.equal(out, first)
    assert cache.read_status() == 0
