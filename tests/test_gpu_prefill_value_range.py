"""kvc_prefill_attention (no transform) where V is small: its P V product takes V in
fp16, times a power of two where a block's keys hold small values only."""
import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import test_gpu_prompt as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


@pytest.mark.parametrize("hq,hkv,n,sizes", [
    (4, 2, 300, [1e-7]), (2, 1, 1, [1e-9]), (8, 1, 700, [1e-30]), (2, 2, 129, [1e-37]), (2, 1, 520, [0.0]),
    (4, 1, 900, [1e-3, 1e-6]), (2, 1, 1300, [1e-8] * 9 + [1.0]), (2, 1, 800, [1e4, 1e-12, 1e-2]),
    (2, 2, 650, [0.0, 0.0, 1e-5]),
])
def test_small_values(hq, hkv, n, sizes):
    """Against the oracle, with a bound whose terms are relative to V: bf16's half
    step; P in fp16, 2^-11, and 2^-14 for the scores (fp32 products of 128 terms
    and ex2: |z| 2^-20 with |z| below 30 here) of sum p |v|; V in fp16 2^-19 of
    the KV head's largest |v|, P below fp16's normal range 2^-25 of it for each of
    n keys; half a step of a bf16 below its normal range, 2^-134."""
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    rng = np.random.default_rng(n)
    size = np.array(sizes)[(np.arange(n) // 100) % len(sizes)][:, None]
    q, k = P._bits(rng, (1, hq, n, 128)), P._bits(rng, (1, hkv, n, 128))
    v = bf16_bits((rng.standard_normal((1, hkv, n, 128)) * size).astype(np.float32))
    pages = n // 16 + 2
    f = O.bf16_bits_to_f32
    ref, _ = O.prefill_attention(f(q[0]), f(k[0]), f(v[0]), T.sm_scale())
    mag, _ = O.prefill_attention(f(q[0]), f(k[0]), np.abs(f(v[0])), T.sm_scale())
    top = np.abs(f(v[0])).max(axis=(1, 2))[np.arange(hq) * hkv // hq][:, None, None]
    bound = (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14) * mag + (2.0 ** -19 + n * 2.0 ** -25) * top
             + 2.0 ** -134)
    for scores in (True, False):
        cache = KVCache(hq, hkv, 8, pages, 1, pages)
        out = T.bf16_tensor_to_f32(cache.prefill(*[T.to_dev_bf16(x) for x in (q, k, v)], accumulate_h2o=scores))
        assert cache.read_status() == 0
        err = np.abs(out[0].astype(np.float64) - ref)
        assert (err <= bound).all(), float((err / bound).max())


def test_values_scaled_by_a_power_of_two():
    """V times a power of two gives the output times that power, bit for bit, and
    the same scores."""
    from compressed_kv_cache_kvc_gb300.cache import KVCache
    rng = np.random.default_rng(3)
    n = 700
    q, k = (T.to_dev_bf16(P._bits(rng, (1, h, n, 128))) for h in (4, 2))
    v = torch.rand(1, 2, n, 128, generator=torch.Generator().manual_seed(1)).cuda().mul(0.5).add(0.5).bfloat16()
    got = []
    for e in (0, -3, -30, -90):
        cache = KVCache(4, 2, 8, 48, 1, 48)
        out = cache.prefill(q, k, (v.float() * 2.0 ** e).bfloat16())
        got.append((out.float() * 2.0 ** -e, cache.buffer("SCORE").clone(), cache.buffer("SINK_SCORE").clone()))
        assert cache.read_status() == 0
    for g in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(g, got[0]))
