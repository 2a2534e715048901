"""Prompt attention where V is small: V enters its product in fp16, brought into
range by a power of two where a (sequence, KV head) holds small values only."""
import math

import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R
from tests import test_gpu_prompt as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _check(q, k, v, begin, end, cap, slopes, out, sums):
    """Against the formula, with a bound whose every term is relative to V: that
    of ops64 with, in place of its absolute terms,
      * V in fp16: 2^-25 where the KV head's largest |v|, M, is 2^-6 or more, so
        2^-19 M, less where the power of two applies, for each unit of p;
      * P below fp16's normal range: 2^-25 of at most M for each of n keys;
      * a bf16 output below bf16's normal range: half its step there, 2^-134."""
    n = q.shape[1]
    ref, _, rsum = P._reference(q, k, v, begin, end, cap, slopes)
    at = np.arange(n)
    lo = np.zeros(n, int) if begin is None else np.clip(begin, 0, None)
    hi = at + 1 if end is None else np.clip(end, None, n)
    see = (at[None, :] >= lo[:, None]) & (at[None, :] < hi[:, None])
    for j in range(q.shape[0]):
        h = j * k.shape[0] // q.shape[0]
        vd = v[h].astype(np.float64)
        z = R.scores(q[j], k[h], P.SCALE, cap, slopes[j] if slopes is not None else 0.0, at, at)
        p = R.softmax_rows(np.where(see, z, -np.inf))
        dz = R.score_error(z, cap, see)
        bound = (2.0 ** -8 * np.abs(ref[j]) + (2.0 ** -11 + 2 * math.log(2) * dz + n * 2.0 ** -24) * (p @ np.abs(vd))
                 + (2.0 ** -19 + n * 2.0 ** -25) * np.abs(vd).max() + 2.0 ** -134)
        err = np.abs(out[j] - ref[j])
        assert (err <= bound).all(), (j, float((err / bound).max()))
    np.testing.assert_allclose(sums, rsum, rtol=P.SUM_RTOL, atol=1e-6)


CASES = [
    # hq, hkv, n, runs, cap, bias, V's size per 100 keys (in turn)
    (4, 2, 300, "causal", 0.0, False, [1e-7]),
    (4, 2, 300, "causal", 20.0, True, [1e-9]),
    (2, 1, 700, "documents", 15.0, False, [1e-30]),
    (2, 2, 129, "full", 0.0, True, [1e-37]),
    (4, 1, 520, "prefix", 0.0, False, [1.0, 1e-5]),
    (2, 1, 900, "causal", 10.0, False, [1e-6, 1e-3, 1e-9, 1e2]),
    (2, 1, 900, "causal", 0.0, True, [1e4, 1e-12, 1e-2]),
    (2, 1, 650, "window", 10.0, True, [1e-3, 0.0, 1e-8]),
    (2, 1, 400, "pads", 5.0, True, [0.0]),
    (2, 1, 1500, "documents", 5.0, True, [1e-10, 3.0, 1e-2, 1e-25]),
    (2, 1, 1700, "causal", 0.0, False, [1e-3] * 15 + [2.0]),  # a large tile far from the small ones
    (2, 2, 1100, "window", 0.0, True, [0.0, 0.0, 1e-12, 1e-5]),
]


@pytest.mark.parametrize("hq,hkv,n,runs,cap,bias,sizes", CASES)
def test_small_values(hq, hkv, n, runs, cap, bias, sizes):
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    rng = np.random.default_rng(n + hq)
    size = np.array(sizes)[(np.arange(n) // 100) % len(sizes)][:, None]
    q, k = P._bits(rng, (1, hq, n, 128), 1.5), P._bits(rng, (1, hkv, n, 128), 1.5)
    v = bf16_bits((rng.standard_normal((1, hkv, n, 128)) * size).astype(np.float32))
    begin, end = P._runs(runs, n, rng)
    db, de = P._dev_runs(begin, end, 1)
    slopes = P._slopes(hq) if bias else None
    status = P._status()
    out, sums = prompt_attention(*[T.to_dev_bf16(x) for x in (q, k, v)], status=status, softcap=cap, slopes=slopes,
                                 key_begin=db, key_end=de, column_sums=True)
    assert status.item() == 0
    f = O.bf16_bits_to_f32
    _check(f(q[0]), f(k[0]), f(v[0]), begin, end, cap, slopes.double().cpu().numpy() if bias else None,
           T.bf16_tensor_to_f32(out)[0], sums[0].cpu().numpy())


def test_values_scaled_by_a_power_of_two():
    """V times a power of two gives the output times that power, bit for bit (V
    and the outputs are normal numbers)."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(3)
    n = 700
    q, k = (T.to_dev_bf16(P._bits(rng, (2, h, n, 128))) for h in (4, 2))
    v = torch.rand(2, 2, n, 128, generator=torch.Generator().manual_seed(1)).cuda().mul(0.5).add(0.5).bfloat16()
    kw = dict(softcap=12.0, slopes=P._slopes(4))
    want = prompt_attention(q, k, v, status=P._status(), **kw).float()
    for e in (-3, -30, -90):
        got = prompt_attention(q, k, (v.float() * 2.0 ** e).bfloat16(), status=P._status(), **kw).float()
        assert torch.equal(got, want * 2.0 ** e), e


def test_prefill_of_small_values():
    """The cache's prompts with a transform take the same kernels."""
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    rng = np.random.default_rng(4)
    hq, hkv, n = 4, 2, 333
    q, k = P._bits(rng, (1, hq, n, 128)), P._bits(rng, (1, hkv, n, 128))
    v = bf16_bits((rng.standard_normal((1, hkv, n, 128)) * 1e-8).astype(np.float32))
    cache = KVCache(hq, hkv, 8, 24, 1, 24)
    cache.set_score_transform(softcap=20.0)
    out = T.bf16_tensor_to_f32(cache.prefill(*[T.to_dev_bf16(x) for x in (q, k, v)]))[0]
    assert cache.read_status() == 0
    f = O.bf16_bits_to_f32
    sums = P._reference(f(q[0]), f(k[0]), f(v[0]), None, None, 20.0, None)[2]
    _check(f(q[0]), f(k[0]), f(v[0]), None, None, 20.0, None, out, sums)


@pytest.mark.parametrize("scale,cap,size", [(5e32, 1e30, 2e-33), (1e34, 3e31, 1e-34)])
def test_scales_and_caps_far_from_one(scale, cap, size):
    """Caps and scales whose polynomials' coefficients leave fp32's range: the
    scores are as for any others.  The polynomials are off by 2^-22 of a score
    (their fits by 2e-7 and a step's rounding), all scores lie in their
    interval: |z| (2^-22 + 2e-7) in place of the cap's absolute bound."""
    from compressed_kv_cache_kvc_gb300 import prompt_attention
    rng = np.random.default_rng(5)
    n = 200
    q, k, v = P._bits(rng, (1, 2, n, 128), size), P._bits(rng, (1, 1, n, 128), 0.1), P._bits(rng, (1, 1, n, 128))
    out = T.bf16_tensor_to_f32(prompt_attention(*[T.to_dev_bf16(x) for x in (q, k, v)], status=P._status(),
                                                sm_scale=scale, softcap=cap))[0]
    f = O.bf16_bits_to_f32
    at = np.arange(n)
    see = at[None, :] <= at[:, None]
    vd = f(v[0, 0]).astype(np.float64)
    for j in range(2):
        z = R.scores(f(q[0, j]), f(k[0, 0]), scale, cap, 0.0, at, at)
        assert 0.1 < np.abs(z).max() < 100
        p = R.softmax_rows(np.where(see, z, -np.inf))
        dz = R.score_error(z, 0.0, see) + np.abs(z).max() * R.LOG2E * (2.0 ** -22 + 2e-7)
        ref = p @ vd
        assert (np.abs(out[j] - ref) <= R.output_bound(ref, p, vd, dz)).all()
