"""Attention over the block-scaled cache where V differ by more than fp16 holds and
the largest may have no weight: small V that carry an output keep their bits beside
large ones that do not, for every query head of a group by itself, in every form
(whole sequences, selected blocks, a shared prefix directly and as a product)."""
import math

import numpy as np
import pytest
import torch

from oracle import kvc_oracle as O
from tests import kvc_testlib as T
from tests import ops64 as R

pytestmark = pytest.mark.gpu

SCALE = 1.0 / np.sqrt(128.0)
BLOCK = 16
DIR = np.where(np.arange(128) % 3 == 0, -1.0, 1.0) / np.sqrt(128.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from compressed_kv_cache_kvc_gb300.build import build_library
    build_library()


def _f(x):
    return O.bf16_bits_to_f32(x).astype(np.float64)


def _bits(x):
    from compressed_kv_cache_kvc_gb300.workloads import bf16_bits
    return bf16_bits(x.astype(np.float32))


def _scales(x, qmax):
    """fp64 [tokens]: the scale of every token's block, 0 for rows held in bf16."""
    out = np.zeros(len(x))
    for c in range(max(len(x) - 4, 0) // BLOCK):
        rows = slice(4 + c * BLOCK, 4 + (c + 1) * BLOCK)
        out[rows] = np.abs(x[rows]).max() / qmax
    return out


def _bound(ref, p, v, vs, ks, q, z, int8):
    """o = sum p v, A = sum p |v|, as ops64 derives them, but nothing relative to a V
    beyond its weight:
      * 2^-8 |o| for the bf16 output, 2^-134 below its normal range;
      * (2^-11 + 2 ln 2 dz + n 2^-24) A: P in fp16, scores off by dz, fp32 sums;
      * P below fp16's normal range is off by 2^-25 of the head's unit.  That is at most
        2^4 times the power of two below the largest product of p and V scale (of exact
        rows |v| / 128) so far, or 2^-126, and a code is at most 448: n 2^-25 max(2^4
        3.5 max_j p_j max|v_j|, 448 2^-126 max_j p_j) (what is rounded is then divided by
        the sum of exp2(z - m), at least the sum of exp2(z - max z) = 1 / max_j p_j);
      * INT8 codes as offset subnormals: ops64.offset_terms, the keys' scales of tokens
        that have weight; what a step of 16 products drops of the accumulator, which holds
        sums of p v_scale (code + 128) <= 256 p v_scale: n / 16 2^-23 256 sum p v_scale."""
    n = len(p)
    dz, more = R.score_error(z, 0.0, np.ones_like(z, bool)), 0.0
    if int8:
        codes, drop = R.offset_terms(q, np.where(p > 2.0 ** -40, ks, 0.0), vs, p[None], SCALE)
        dz, more = dz + codes, float(drop[0, 0]) + n / 16 * 2.0 ** -15 * float(p @ vs)
    top = (p * np.abs(v).max(-1)).max()
    return (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * math.log(2) * dz + n * 2.0 ** -24) * (p @ np.abs(v))
            + n * 2.0 ** -25 * max(2.0 ** 4 * 3.5 * top, 448 * 2.0 ** -126 * p.max()) + 2.0 ** -134 + more)


def _marked(where, n):
    """Which of a sequence's n tokens have the large V."""
    at, end = np.zeros(n, bool), 4 + (n - 4) // BLOCK * BLOCK
    if where == "blocks":
        at[4 + 3 * BLOCK:4 + 5 * BLOCK] = True
    elif where == "newest":
        at[end - 9 * BLOCK:end] = True
    elif where == "every other":
        for c in range(0, (end - 4) // BLOCK, 2):
            at[4 + c * BLOCK:4 + (c + 1) * BLOCK] = True
    elif where == "sinks":
        at[:3] = True
    elif where == "open":
        at[end + 1:] = True
    elif where == "a sink and a block":
        at[1] = at[4 + 7 * BLOCK:4 + 8 * BLOCK] = True
    return at


# large V, the others, by how much (natural log) the large ones' scores lie below the
# others'; a head in three has the sign turned, and so sees nothing but the large V
SIZES = [(2.0 ** 24, 1.0, 250.0), (1.0, 2.0 ** -45, 250.0), (3e37, 1e-30, 250.0), (2.0 ** 40, 1.0, 28.0),
         (2.0 ** 18, 1.0, 12.0), (2.0 ** 30, 1.0, 0.0), (1e-33, 1e-37, 250.0)]
FORMS = {  # sequences, tokens of the first and of the others
    "whole": (2, 1493, 900), "selected": (2, 1493, 900), "direct": (3, 1493, 95), "product": (40, 3853, 95),
    "product, one stream": (15, 9997, 95),
}
WHERE = ["blocks", "newest", "every other", "sinks", "open", "a sink and a block", "own"]


@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("form", list(FORMS))
def test_large_values_without_weight(form, where):
    from compressed_kv_cache_kvc_gb300 import BlockScaledCache
    codes = "int8" if (list(FORMS).index(form) + WHERE.index(where)) % 2 else "e4m3"
    count, long, short = FORMS[form]
    prefix = form in ("direct", "product", "product, one stream")
    if where == "own" and not prefix:
        where = "every other"  # (of the shorter sequence too)
    rng = np.random.default_rng(len(form) + len(where))
    hkv, group = 2, 3
    hq = hkv * group
    lengths = [long] + [short + b % 20 for b in range(count)] if prefix else [long, short][:count]
    counts = [(n - 4) // BLOCK for n in lengths]
    cache = BlockScaledCache(hq, hkv, sum(counts), len(lengths), max(counts), block_tokens=BLOCK, codes=codes,
                             key_bounds=form == "selected")
    first, B = (1, count) if prefix else (0, count)
    for big, small, gap in SIZES:
        sign = np.where(np.arange(hq) % 3 == 2, -1.0, 1.0)[:, None]
        q = _bits(rng.standard_normal((B, hq, 128)) + 12.0 * sign * DIR)
        kv = []
        cache.release(0, len(lengths))
        for s, n in enumerate(lengths):
            large = _marked("blocks" if where == "own" else where, n)
            if prefix and (s > 0) != (where == "own"):
                large[:] = False
            k = rng.standard_normal((hkv, n, 128))
            k[:, large] -= gap / 12.0 / SCALE * DIR
            # magnitudes in [1/8, 1] of the size
            v = rng.uniform(0.125, 1.0, (hkv, n, 128)) * rng.choice([-1.0, 1.0], (hkv, n, 128))
            v *= np.where(large, big, small)[None, :, None]
            k, v = _bits(k), _bits(v)
            kv.append((k, v))
            cache.append(T.to_dev_bf16(k[None]), T.to_dev_bf16(v[None]), seq_begin=s)
        dq = T.to_dev_bf16(q)
        if prefix:
            out = cache.prefix_attention(dq, 0, seq_begin=1)
            assert cache.last_launch_count() == (1 if form == "direct" else 2)
        elif form == "selected":
            out = cache.selected_attention(dq, 4096)
        else:
            out = cache.decode_attention(dq)
        assert cache.read_status() == 0
        got = T.bf16_tensor_to_f32(out).astype(np.float64)
        held, beyond, seen = {}, 0, 0
        for b in sorted({0, 1, B // 2, B - 1}):
            for j in range(hq):
                h = j // group
                parts = []
                for s in ([0, 1 + b] if prefix else [b]):
                    if (s, h) not in held:
                        k, v = (_f(x[h]) for x in kv[s])
                        e4 = codes == "e4m3"
                        held[s, h] = (R.held_block(k, BLOCK, e4), R.held_block(v, BLOCK, e4), _scales(k, 127), _scales(v, 127))
                    parts.append(held[s, h])
                kd, vd, ks, vs = (np.concatenate(x) for x in zip(*parts))
                qf = _f(q[b, j:j + 1])
                z = R.scores(qf, kd, SCALE, 0.0, 0.0, [0], np.zeros(len(kd)))
                p = R.softmax_rows(z)[0]
                ref = p @ vd
                bound = _bound(ref, p, vd, vs, ks, qf, z, codes == "int8")
                err = np.abs(got[b, j] - ref)
                assert (err <= bound).all(), (big, small, gap, b, j, float((err / bound).max()))
                beyond += int((np.abs(ref) > bound).sum())
                seen += ref.size
        assert beyond > 0.9 * seen, (big, small, gap, beyond / seen)  # (rows of 0 would fail)
