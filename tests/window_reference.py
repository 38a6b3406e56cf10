"""Plain 64-bit forms of the 4-bit cache and of attention with a sliding window.

Written from the definitions in ``include/gqa_attn.h``; shares no code with the
library.
"""

import numpy as np

from cache_reference import E4M3

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode_rows(rows, D):
    """Values of 4-bit rows [..., 9 D / 16], in units of the tensor's scale."""
    rows = np.asarray(rows)
    codes = np.stack([rows[..., : D // 2] & 15, rows[..., : D // 2] >> 4], -1)
    codes = codes.reshape(*rows.shape[:-1], D)
    value = np.where(codes & 8, -E2M1[codes & 7], E2M1[codes & 7])
    return value * np.repeat(E4M3[rows[..., D // 2:]], 16, -1)


def nearest_even(x, values):
    """Index of the nearest of ascending values >= 0, ties to the even index, for x >= 0
    up to any size."""
    i = np.clip(np.searchsorted(values, x), 1, len(values) - 1)
    lo, hi = values[i - 1], values[i]
    below, above = x - lo, hi - x
    up = (above < below) | ((above == below) & (i % 2 == 0))
    return np.where(x >= values[-1], len(values) - 1, np.where(up, i, i - 1))


def encode_rows(u):
    """4-bit rows of fp32 values u [..., D] (no NaN), by the header's formulas in 32 bits."""
    u = np.asarray(u, np.float32)
    block = u.reshape(*u.shape[:-1], -1, 16)
    scale = nearest_even((np.abs(block).max(-1) / np.float32(6)).astype(np.float64),
                         E4M3[:127]).astype(np.uint8)
    s = E4M3[scale].astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        x = np.where(s > 0, block / s, np.float32(0))
    codes = nearest_even(np.abs(x).astype(np.float64), E2M1).astype(np.uint8)
    codes = np.where((s > 0) & np.signbit(x), codes | 8, codes).reshape(u.shape)
    return np.concatenate([codes[..., 0::2] | codes[..., 1::2] << 4, scale], -1).astype(np.uint8)


def visible(pos, keys, window, sinks):
    """[rows, keys]: which keys the rows at positions pos see."""
    j = np.arange(keys)
    p = np.asarray(pos)[:, None]
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    return see


def attend(q, k, v, see, scale):
    """(out, bound) of rows q [n, D] over k, v [keys, D]; rows that see nothing are zeros.

    bound: what a kernel with 32-bit sums, fp16 weights P and an fp16 result may be off
    by.  P has 2^-11 of itself, or 2^-25 where it is subnormal (in units where some
    weight of the row is 1); scores in log2 units hold to 2^-19 of the magnitudes that
    enter them (products of fp16 values are exact in 32 bits, sums of at most 256 lose
    2^-20 of them even where every addition is cut off) and the exponential to 2^-21;
    the result rounds by 2^-11 of itself, or 2^-25.
    """
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, keys = see.shape
    out = np.zeros((n, v.shape[1]))
    bound = np.zeros_like(out)
    for i in range(n):
        at = np.nonzero(see[i])[0]
        if not len(at):
            continue
        s = scale * (k[at] @ q[i])
        w = np.exp(s - s.max())
        w /= w.sum()
        off = 2.0 ** -11 + 2.0 ** -20 + 2.0 ** -19 * scale * (np.abs(k[at]) @ np.abs(q[i]))
        out[i] = w @ v[at]
        # Twice: the weights' sum is off as they are.
        bound[i] = 2 * ((w * off + 2.0 ** -25) @ np.abs(v[at])) + 2.0 ** -11 * np.abs(out[i]) \
            + 2.0 ** -25
    return out, bound
