"""Attention over the block-scaled cache where V is very large or very small:
closed blocks at either end of bf16's range beside exact rows (sinks and open
block) of ordinary size and the other way round.  Every finite V is admitted."""
import math

import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R
from tests import test_gpu_block_cache as B

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)
TOP = 3.3895313892515355e38  # the largest bf16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _bound(ref, p, v, dz, more):
    """As ops64.output_bound, with its absolute terms relative to the values: V
    enters exactly, as codes c <= 448 times 2^E or as bf16.  P below fp16's normal
    range is off by 2^-25 of the unit 2^E, which is at most the largest V scale or
    1/128 of the largest exact |v|, but never below 2^-126: 2^-25 c 2^E <= 2^-25
    max(3.5 max|v|, 448 2^-126) for each of n terms.  A bf16 output below bf16's
    normal range: half its step there, 2^-134."""
    n = p.shape[-1]
    return (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * math.log(2) * dz + n * 2.0 ** -24) * (p @ np.abs(v))
            + n * 2.0 ** -25 * max(3.5 * np.abs(v).max(), 448 * 2.0 ** -126) + 2.0 ** -134 + more)


CASES = [
    # closed blocks, sinks, open rows: the size of V
    (1e34, 1.0, 1.0), (1e35, 1.0, 1e3), (3e38, 1.0, 1.0), (1e-37, 1.0, 1.0), (1.0, 1.0, 3e38), (1.0, 3e38, 1.0),
    (3e38, 3e38, 3e38), (1e-37, 1e-37, 1e-37), (0.0, 1.0, 1.0), (0.0, 1e-37, 1e38), (0.0, 0.0, 0.0), (1e33, 1e-30, 1e-30),
]


@pytest.mark.parametrize("codes", ["int8", "e4m3"])
@pytest.mark.parametrize("group,n", [(4, 4 + 5 * 16 + 7), (1, 3001), (8, 40), (3, 1200)])
@pytest.mark.parametrize("closed,sinks,rows", CASES)
def test_ends_of_the_value_range(closed, sinks, rows, group, n, codes):
    rng = np.random.default_rng(n + group)
    hkv, block = 2, 16
    end = 4 + (n - 4) // block * block
    size = np.full((1, 1, n, 1), closed)
    size[:, :, :4], size[:, :, end:] = sinks, rows
    k = B._bits(rng, (1, hkv, n, 128))
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    # magnitudes in [1/8, 1] of the size, so that nothing leaves bf16's range
    x = rng.uniform(0.125, 1.0, (1, hkv, n, 128)) * rng.choice([-1.0, 1.0], (1, hkv, n, 128))
    v = bf16_bits((x * np.minimum(size, TOP * 0.99)).astype(np.float32))
    q = B._bits(rng, (1, group * hkv, 128), 2.0)
    cache = B._cache(group * hkv, hkv, [n], block, codes)
    cache.append(T.to_dev_bf16(k), T.to_dev_bf16(v))
    got = T.bf16_tensor_to_f32(cache.decode_attention(T.to_dev_bf16(q))).astype(np.float64)
    assert cache.read_status() == 0
    f = O.bf16_bits_to_f32
    for j in range(group * hkv):
        h = j // group
        kd, vd = B._held(k[0, h], n, block, codes), B._held(v[0, h], n, block, codes)
        z = R.scores(f(q[0, j:j + 1]), kd, SCALE, 0.0, 0.0, [n - 1], np.arange(n))
        p = R.softmax_rows(z)
        ref = p @ vd
        ks, vs = np.zeros(n), np.zeros(n)
        if codes == "int8":
            for c in range(4, end, block):
                ks[c:c + block] = np.abs(f(k[0, h, c:c + block])).max() / 127
                vs[c:c + block] = np.abs(f(v[0, h, c:c + block])).max() / 127
        dz_codes, more = R.offset_terms(f(q[0, j:j + 1]), ks, vs, p, SCALE)
        bound = _bound(ref, p, vd, R.score_error(z, 0.0, np.ones_like(z, bool)) + dz_codes, more)
        err = np.abs(got[0, j] - ref[0])
        assert (err <= bound[0]).all(), (j, float((err - bound[0]).max()), float(np.abs(ref).max()))
