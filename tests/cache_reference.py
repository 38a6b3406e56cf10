"""Plain 64-bit forms of the cache write, read, block index and selection.

Written from the definitions in ``include/gqa_attn.h`` with numpy, row by row;
it shares no code with the library.
"""

import numpy as np
import torch


def e4m3_table():
    """Value of every E4M3 code (OCP e4m3fn), in 64 bits."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


E4M3 = e4m3_table()


def decode(x):
    """A cache tensor's values in 64 bits (codes of uint8, or 16-bit floats)."""
    if x.dtype == torch.uint8:
        return E4M3[x.cpu().numpy()]
    return x.cpu().double().numpy()


def rows_of(starts, ctx_lens, tables, page):
    """[(row, sequence, position, physical token)] of a launch's rows."""
    got = []
    for b in range(len(ctx_lens)):
        n = starts[b + 1] - starts[b]
        for j in range(n):
            p = ctx_lens[b] - n + j
            got.append((starts[b] + j, b, p, int(tables[b][p // page]) * page + p % page))
    return got


def norm_rotate(x, weight, eps, inv_freq, interleaved, pos):
    """One token's heads [H, D]: (values, magnitude each value's error scales with)."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    mag = np.abs(x)
    n = len(inv_freq)
    if n:
        a = pos * inv_freq.astype(np.float64)
        c, s = np.cos(a), np.sin(a)
        i = np.arange(n)
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        y = x.copy()
        y[:, lo] = x[:, lo] * c - x[:, hi] * s
        y[:, hi] = x[:, hi] * c + x[:, lo] * s
        mag[:, lo] = mag[:, hi] = np.abs(x[:, lo]) + np.abs(x[:, hi])
        x = y
    return x, mag


def block_sums(keys):
    """fp32 sums (k0 + k1) + (k2 + k3) of [4, width] keys, as the header states them."""
    k = keys.astype(np.float32)
    return (k[0] + k[1]) + (k[2] + k[3])


def summary(s, scale):
    """(codes, scale) of one block's fp32 sums."""
    most = np.float32(np.abs(s).max()) if np.isfinite(s).all() else np.float32(np.inf)
    if not np.isfinite(most) or most == 0:
        return np.zeros(s.shape, np.int8), np.float32(0)
    inv = np.float32(127) / most
    codes = np.rint(s * inv).astype(np.int8)
    return codes, most * (np.float32(scale) / np.float32(508))


def select(q, index, index_scale, table, page, ctx, max_sel, n_first, n_last):
    """sel_idx, sel_cnt of gqa_select_blocks: whole-number dots, one fp32 product."""
    q = q.cpu().numpy().astype(np.float64)
    rows, Hq, D = q.shape
    Hkv = index.shape[2]
    nb = (ctx + 3) // 4
    b = np.arange(nb)
    table = table.cpu().numpy()
    at = table[b * 4 // page], b % (page // 4)
    codes = index.cpu().numpy()[at].reshape(nb, Hkv * D).astype(np.int64)
    scale = index_scale.cpu().numpy()[at]
    with np.errstate(invalid="ignore"):
        total = q.reshape(rows, Hkv, Hq // Hkv, D).sum(2).reshape(rows, Hkv * D)
    sel = np.full((rows, max_sel), -1, np.int32)
    cnt = np.zeros(rows, np.int32)
    for i in range(rows):
        s = total[i].astype(np.float32)
        most = np.abs(s).max() if np.isfinite(q[i]).all() else np.float32(0)
        c = np.rint(s * (np.float32(127) / most)) if most > 0 else np.zeros_like(s)
        score = (codes @ c.astype(np.int64)).astype(np.float32) * scale
        own = (ctx - rows + i) // 4
        n = min(max_sel, own + 1)
        always = [x for x in range(own + 1) if x < n_first or x > own - n_last]
        if n == own + 1:
            pick = list(range(own + 1))
        else:
            others = np.arange(n_first, own - n_last + 1)
            key = np.where(np.isnan(score[others]), -np.inf, score[others])
            order = np.lexsort((others, np.isnan(score[others]), -key))
            pick = sorted(always + list(others[order][: n - len(always)]))
        sel[i, :n] = pick
        cnt[i] = n
    return sel, cnt
