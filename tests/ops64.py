"""Plain 64-bit forms of the transformed attentions and of the block-scaled
cache's quantisation, for the GPU tests, with the bounds those tests use.

Bounds of an attention output o = sum_j p_j v_j against its 64-bit value, A =
sum_j p_j |v_j| (all products and sums in fp32):
  * the bf16 output: half a step, 2^-8 |o|;
  * P enters its product in fp16 (half a step, 2^-11 p) or, where it is two
    bf16 parts, less: 2^-11 A;
  * scores z (log2 units, |z| <= Z) off by at most dz: the fp32 rounding of the
    product, scale and bias and of z itself, 4 steps of 2^-24 Z, and the cap's
    7.2e-7 of the cap (ex2 2^-22 twice, rcp 2^-23 and two roundings of 2^-24):
    every p off by dz ln 2 relative, both in the numerator and in the sum: 2 ln 2
    dz A;
  * fp32 sums of n terms: n 2^-24 A covers any order;
  * P below fp16's normal range: an absolute 2^-25 of the largest p scaled by up
    to 2^5, for each of n terms: n 2^-20 max|v| is 2^-24 n max|v| with the
    running maximum within 2^4 of the final one; V below 2^-14 in fp16
    (prompts): 2^-25 per unit of p;
  * integer codes in the per-token cache (`offset`): a code c enters the tensor
    core as the fp16 subnormal (c + O) 2^-24.  The core adds a step's 16 products
    and the accumulator aligned to the largest exponent, dropping what lies 23
    bits below it; a subnormal's exponent counts as that of 2^-14, so with the
    other operand at 2^e the dropped unit is 2^(e - 14 - 23) = 2^(e - 37), in
    units of a code (2^e 2^-24) 2^-13.  17 terms a step drop at most 17 2^-13
    codes times that operand's largest magnitude.  Q K^T: 8 steps, so 8 17 2^-13
    max|q| k_scale per score; P V: per page of 16 tokens at most 17 2^-13 max(p
    v_scale) <= 17 2^-13 sum(p v_scale) over the page.
"""
import math

import numpy as np

LOG2E = 1.4426950408889634


def softmax_rows(z):
    """z [..., keys] (natural log units, -inf masked) -> probabilities, rows of
    nothing but -inf being 0."""
    m = np.max(z, axis=-1, keepdims=True)
    m = np.where(np.isfinite(m), m, 0.0)
    p = np.exp(z - m)
    s = p.sum(-1, keepdims=True)
    return p / np.where(s > 0, s, 1.0)


def scores(q, k, scale, cap, slope, q_pos, k_pos):
    """fp64 scores [rows, keys] of q [rows, 128] at q_pos, k [keys, 128] at k_pos."""
    s = (q.astype(np.float64) @ k.astype(np.float64).T) * scale
    if cap:
        s = cap * np.tanh(s / cap)
    if slope:
        s = s - slope * np.abs(np.asarray(q_pos)[:, None] - np.asarray(k_pos)[None, :])
    return s


def score_error(z, cap, visible):
    """dz (log2 units): see the module's docstring."""
    big = np.abs(np.where(visible, z, 0.0)).max() * LOG2E if visible.any() else 0.0
    return big * 4 * 2.0 ** -24 + 7.2e-7 * cap * LOG2E + 2.0 ** -24


def offset_terms(q, k_scale, v_scale, p, scale):
    """(added dz, added output bound [rows, 1]) of integer codes, see above;
    k_scale, v_scale [keys], 0 for tokens held in bf16."""
    unit = 17 * 2.0 ** -13
    return 8 * unit * np.abs(q).max() * k_scale.max(initial=0.0) * scale * LOG2E, unit * (p @ v_scale)[:, None]


def output_bound(ref, p, v, dz):
    """The bound of an output [rows, 128] from p [rows, keys], v [keys, 128]."""
    a = p @ np.abs(v)
    n = p.shape[-1]
    return (2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2 * math.log(2) * dz + n * 2.0 ** -24) * a
            + n * 2.0 ** -24 * np.abs(v).max() + 2.0 ** -25)


def quantise_block(x, e4m3):
    """(codes as fp64 values, fp32 scale) of a block's fp32 values."""
    amax = np.abs(x).max()
    scale = np.float32(amax) / np.float32(448.0 if e4m3 else 127.0)
    if scale == 0:
        return np.zeros(x.shape), scale
    y = (x / scale).astype(np.float32).astype(np.float64)  # IEEE fp32 quotients
    if not e4m3:
        return np.clip(np.rint(y), -127, 127), scale
    # E4M3: 4 significant bits from 2^-6 up, steps of 2^-9 below, at most 448
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    return np.clip(np.rint(y / step) * step, -448, 448), scale


def held_block(x, block, e4m3):
    """fp64 [tokens, 128] that the block-scaled cache holds of x (fp32)."""
    out = x.astype(np.float64).copy()
    closed = max(0, x.shape[0] - 4) // block
    for c in range(closed):
        rows = slice(4 + c * block, 4 + (c + 1) * block)
        code, scale = quantise_block(x[rows], e4m3)
        out[rows] = code * np.float64(scale)
    return out
