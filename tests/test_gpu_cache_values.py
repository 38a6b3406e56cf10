"""GPU tests of the cache write's values: what padding rows hold, values beyond
fp16, infinities and NaN in the queries and keys, far positions.

Errors of the 32-bit steps in units of 2^-24 of the magnitudes that enter a value.
Norm: 13 of the sum of squares' 8 fused terms and 5 shuffled additions and 2 of the
mean and eps, halved by the root; rsqrt 4 (2 units in the last place); its two
products 2.  Rotation: 2 of a product and the fused one.  15.5 together.  cos and sin:
the functions' 2^-21.19 (7), the angle's 2 pi and its product (4.6), the fraction of
a turn's last addition, 2^-25 turns (3.2) below position 2^24; beyond, its five
additions of up to 2^-23, 5 2^-24 turns together (31.5).  The frequency's turns are
held to 1.5 2^-47, as are the two roundings behind their product with the position:
2^-45 of position * frequency, in radians.  Storing K multiplies by a rounded
reciprocal: 2.  Then one rounding: fp16 2^-11 (2^-25 among subnormals), E4M3 2^-4
(2^-10)."""

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -24


def bound(m, pos, freq, rot, interleaved):
    """The 32-bit error of one token's heads, m: what enters each value [H, D]."""
    units = np.full(m.shape[-1], 17.5)
    if rot:
        i = np.arange(rot // 2)
        turn = (14.8 if pos < 1 << 24 else 43.1) + abs(pos) * freq * 2.0 ** -45 / UNIT
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        units[lo] += turn
        units[hi] += turn
    # (products of these errors are far below a unit)
    return m * (units + 0.1) * UNIT


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("ctx", [5000, (1 << 24) + 3, (1 << 26) + 5])
def test_far_positions(cuda_lib, ctx, interleaved):
    dev = torch.device("cuda")
    page, D, rows, rot = 256, 128, 8, 128
    stride = -(-ctx // page)
    kc = torch.empty(stride, page, 1, D, dtype=torch.uint8, device=dev)
    vc = torch.empty_like(kc)
    g = torch.Generator().manual_seed(ctx)
    qkv = torch.randn(rows, 5, D, generator=g).half().to(dev)
    q, k, v = qkv[:, :3], qkv[:, 3:4], qkv[:, 4:]
    w = (1 + 0.3 * torch.randn(D, generator=g)).half().to(dev)
    freq = (1e6 ** (-torch.arange(rot // 2) / (rot // 2))).float().to(dev)
    s = torch.tensor([0.01], device=dev)
    tables = torch.arange(stride, dtype=torch.int32, device=dev).view(1, -1)
    lens = torch.tensor([ctx], dtype=torch.int32, device=dev)
    q_out = cuda_lib.cache_write_e4m3(q, k, v, kc, vc, s, s, tables, lens, ctx, q_weight=w,
                                      k_weight=w, eps=1e-6, inv_freq=freq,
                                      interleaved=interleaved)
    assert cuda_lib.device_error() == 0
    f64, fr = (lambda x: x.cpu().double().numpy()), freq.cpu().numpy()
    for j in range(rows):
        pos = ctx - rows + j
        y, m = ref.norm_rotate(f64(q[j]), f64(w), 1e-6, fr, interleaved, pos)
        tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + bound(m, pos, fr, rot, interleaved)
        assert (np.abs(f64(q_out[j]) - y) <= tol).all()
        y, m = ref.norm_rotate(f64(k[j]), f64(w), 1e-6, fr, interleaved, pos)
        y, m = y / float(s), m / float(s)
        got = ref.decode(kc.view(-1, 1, D)[pos])
        tol = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 + bound(m, pos, fr, rot, interleaved)
        assert (np.abs(got - np.clip(y, -448, 448)) <= tol).all()


@pytest.mark.parametrize("e4m3", [True, False])
def test_what_padding_rows_hold_has_no_effect(cuda_lib, e4m3):
    """Rows in front of the first sequence and behind the last, and those of a
    sequence with a bad context: NaN in them changes nothing, outputs stay."""
    dev = torch.device("cuda")
    T, D, page, pages = 23, 256, 16, 8
    starts = torch.tensor([2, 9, 14, 20], dtype=torch.int32, device=dev)
    lens = torch.tensor([30, 4, 17], dtype=torch.int32, device=dev)      # 4 < its 5 rows
    tables = torch.tensor([[0, 5], [1, 2], [7, 3]], dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(T, 8, D, generator=g).half().to(dev)
    w = torch.ones(D, dtype=torch.float16, device=dev)
    freq = (1e4 ** (-torch.arange(64) / 64)).float().to(dev)
    s = torch.tensor([0.02], device=dev)
    got = []
    for bad in (False, True):
        x = qkv.clone()
        if bad:
            x[:2] = x[9:14] = x[20:] = float("nan")
        kc = torch.full((pages, page, 1, D), 9, dtype=torch.uint8 if e4m3 else torch.float16,
                        device=dev)
        vc = kc.clone()
        q_out = torch.full((T, 6, D), 7.0, dtype=torch.float16, device=dev)
        args = (x[:, :6], x[:, 6:7], x[:, 7:], kc, vc) + ((s, s) if e4m3 else ())
        write = cuda_lib.cache_write_e4m3 if e4m3 else cuda_lib.cache_write
        write(*args, tables, lens, 32, q_weight=w, k_weight=w, inv_freq=freq, row_starts=starts,
              q_out=q_out)
        assert cuda_lib.device_error() == cuda_lib.DEVERR_BAD_CTX_LEN
        assert (q_out[:2] == 7).all() and (q_out[9:14] == 7).all() and (q_out[20:] == 7).all()
        assert torch.isfinite(q_out).all() and (q_out[2:9] != 7).any()
        got.append((q_out, kc, vc))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_values_beyond_fp16(cuda_lib):
    """bf16 values past 65504, and normed ones, become infinities in q_out and in an
    fp16 cache, and the largest code in an E4M3 one."""
    dev = torch.device("cuda")
    D = 128
    x = torch.ones(4, 3, D, dtype=torch.bfloat16, device=dev)
    x[0, :, 0], x[0, :, 1], x[1, :, 2], x[2, :, 3] = 1e5, -3e38, 65280.0, 65536.0
    at = (torch.zeros(1, 1, dtype=torch.int32, device=dev),
          torch.tensor([4], dtype=torch.int32, device=dev), 4)
    kc, vc = (torch.zeros(1, 8, 1, D, dtype=torch.float16, device=dev) for _ in "kv")
    q_out = cuda_lib.cache_write(x[:, :1], x[:, 1:2], x[:, 2:], kc, vc, *at)
    inf = float("inf")
    want = torch.ones(4, 1, D, dtype=torch.float16, device=dev)
    want[0, 0, 0], want[0, 0, 1], want[1, 0, 2], want[2, 0, 3] = inf, -inf, 65280.0, inf
    for got in (q_out, kc[0, :4], vc[0, :4]):
        assert torch.equal(got, want)
    # Weights take a normed value to the largest number, and past it.
    y = torch.ones(4, 1, D, dtype=torch.float16, device=dev)
    w = torch.full((D,), 65504.0, dtype=torch.float16, device=dev)
    q_out = cuda_lib.cache_write(y, y, y, kc, vc, *at, q_weight=w, k_weight=w, eps=0.0)
    assert (q_out == 65504).all() and (kc[0, :4] == 65504).all()
    w[:] = 32768.0
    y[:, :, 0] = 3.0       # 3 / sqrt(136 / 128) * 32768 = 95364
    q_out = cuda_lib.cache_write(y, y, y, kc, vc, *at, q_weight=w, k_weight=w, eps=0.0)
    assert (q_out[:, :, 0] == inf).all() and (kc[0, :4, :, 0] == inf).all()
    assert torch.isfinite(q_out[:, :, 1:]).all()
    k8, v8 = (torch.zeros(1, 8, 1, D, dtype=torch.uint8, device=dev) for _ in "kv")
    s = torch.ones(1, device=dev)
    cuda_lib.cache_write_e4m3(None, x[:, 1:2], x[:, 2:], k8, v8, s, s, *at)
    assert k8[0, 0, 0, 0] == 0x7E and k8[0, 0, 0, 1] == 0xFE and k8[0, 1, 0, 2] == 0x7E
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_and_nan(cuda_lib, interleaved):
    """They go where the formulas take them, in the row and head that hold them:
    a NaN, and an infinity in a normed head, to the whole head (of an infinity's
    head the other values go to zero); in a head that is only turned, to the pair."""
    dev = torch.device("cuda")
    D, rows, rot = 128, 6, 64
    x = torch.randn(rows, 4, D, generator=torch.Generator().manual_seed(2)).half().to(dev)
    x[1, 0, 3], x[2, 1, 70], x[3, 2, 9] = float("inf"), float("-inf"), float("nan")
    x[4, 0, 40], x[4, 2, 127] = float("nan"), float("inf")
    at = (torch.zeros(1, 1, dtype=torch.int32, device=dev),
          torch.tensor([9], dtype=torch.int32, device=dev), 9)
    freq = (1e2 ** (-torch.arange(rot // 2) / (rot // 2))).float().to(dev)
    for weight in (None, torch.ones(D, dtype=torch.float16, device=dev)):
        kc, vc = (torch.zeros(1, 16, 1, D, dtype=torch.float16, device=dev) for _ in "kv")
        q_out = cuda_lib.cache_write(x[:, :2], x[:, 2:3], x[:, 3:], kc, vc, *at, q_weight=weight,
                                     k_weight=weight, inv_freq=freq, interleaved=interleaved)
        assert cuda_lib.device_error() == 0
        w = None if weight is None else weight.cpu().double().numpy()
        for j in range(rows):
            for got, src in ((q_out[j], x[j, :2]), (kc[0, 3 + j], x[j, 2:3])):
                with np.errstate(invalid="ignore"):
                    y, m = ref.norm_rotate(src.cpu().double().numpy(), w, 1e-6,
                                           freq.cpu().numpy(), interleaved, 3 + j)
                g = got.cpu().double().numpy()
                assert np.array_equal(np.isnan(g), np.isnan(y))
                assert np.array_equal(g[np.isinf(y)], y[np.isinf(y)])
                fine = np.isfinite(y)
                assert np.isfinite(g[fine]).all()
                # (a pair's magnitude may be infinite only where its values are not finite)
                tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + bound(m, 3 + j, freq.cpu().numpy(),
                                                                  rot, interleaved)
                assert (np.abs(g - y)[fine] <= tol[fine]).all()


def test_index_of_the_most_rows(cuda_lib):
    """2^31 - 2 rows: 1023 sequences that share their pages."""
    dev = torch.device("cuda")
    batch, ctx, page, D = 1023, 2099202, 256, 128
    pages = -(-ctx // page)
    assert batch * ctx == 2 ** 31 - 2
    kc = torch.randint(0, 120, (pages, page, 1, D), dtype=torch.uint8, device=dev)
    s = torch.tensor([0.02], device=dev)
    tables = torch.arange(pages, dtype=torch.int32, device=dev).repeat(batch, 1)
    lens = torch.full((batch,), ctx, dtype=torch.int32, device=dev)
    got = []
    for n in (1, batch):
        index = torch.zeros(pages, page // 4, 1, D, dtype=torch.int8, device=dev)
        scale = torch.zeros(pages, page // 4, device=dev)
        cuda_lib.block_index_e4m3(kc, s, tables[:n].contiguous(), lens[:n].contiguous(), ctx,
                                  n * ctx, index, scale)
        got.append((index, scale))
    assert cuda_lib.device_error() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert int((got[1][1] > 0).sum()) == ctx // 4
