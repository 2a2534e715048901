"""BlockScaledCache.prefill refuses before it writes: no output, no tokens."""
import numpy as np
import pytest
import torch

from tests import kvc_testlib as T
from tests import test_gpu_block_cache as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def test_refused_prefills_leave_everything_as_it_was():
    from compressed_kv_cache_kvc_gb300 import _lib as L
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    rng = np.random.default_rng(1)
    draw = lambda h, n, b=1: T.to_dev_bf16(B._bits(rng, (b, h, n, 128)))  # noqa: E731
    hq, hkv = 4, 2
    cache = BlockScaledCache(hq, hkv, 3, 2, 2, block_tokens=16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = cache.state.clone()

    def refused(error, q, k, v, status=status, code=None, **kw):
        out = torch.full_like(q, 7.0) if q.dtype == torch.bfloat16 else None
        with pytest.raises(error) as e:
            cache.prefill(q, k, v, status=status, out=out, **kw)
        torch.cuda.synchronize()
        assert code is None or e.value.status == code
        assert out is None or (out == 7.0).all()
        assert cache.lengths(0, 2) == (0, 0) and status.abs().sum() == 0

    refused(L.KvcError, draw(hq, 60), draw(hkv, 60), draw(hkv, 60), code=L.KVC_ERR_CAPACITY)
    refused(L.KvcError, draw(hq, 36, 2), draw(hkv, 36, 2), draw(hkv, 36, 2), code=L.KVC_ERR_CAPACITY)
    refused(ValueError, draw(8, 20), draw(hkv, 20), draw(hkv, 20))   # another number of query heads
    refused(ValueError, draw(hq, 20), draw(1, 20), draw(1, 20))      # of KV heads
    refused(ValueError, draw(hq, 20), draw(hkv, 20), draw(hkv, 19))
    refused(ValueError, draw(hq, 20).float(), draw(hkv, 20), draw(hkv, 20))
    refused(ValueError, draw(hq, 20)[0], draw(hkv, 20), draw(hkv, 20))
    refused(ValueError, draw(hq, 20), draw(hkv, 20), draw(hkv, 20), status=torch.zeros(1, device="cuda"))
    refused(ValueError, draw(hq, 20), draw(hkv, 20), draw(hkv, 20), slopes=torch.zeros(3, device="cuda"))
    refused(L.KvcError, draw(hq, 20), draw(hkv, 20), draw(hkv, 20), softcap=-1.0, code=L.KVC_ERR_INVALID_ARG)
    refused(L.KvcError, draw(hq, 20), draw(hkv, 20), draw(hkv, 20), sm_scale=0.0, code=L.KVC_ERR_INVALID_ARG)
    refused(TypeError, draw(hq, 20), draw(hkv, 20), draw(hkv, 20), unknown=1)
    assert torch.equal(cache.buffer("COUNTERS"), before[cache.buffer("COUNTERS").data_ptr() - cache.state.data_ptr():]
                       [:cache.buffer("COUNTERS").numel()])
    q, k, v = draw(hq, 20), draw(hkv, 20), draw(hkv, 20)
    out = cache.prefill(q, k, v, status=status, seq_begin=1)
    assert out.isfinite().all() and cache.lengths(0, 2) == (0, 20) and cache.read_status() == 0
