"""GPU tests of the 4-bit cache's write and read against the plain forms.

Without norm and rotation every step of the write is one 32-bit operation the header
names, so codes and scales are compared for equality.  With them the values hold to
2 * 2^-19 of the magnitudes that enter (see test_gpu_cache_ops.py); the stored scale is
then within half a step (2^-4, 2^-10 among subnormals) of a sixth of the block's
magnitude, and a code within half a step of the value over the stored scale.
"""

import numpy as np
import pytest
import torch

import cache_reference as cref
import window_reference as ref
from test_gpu_cache_ops import CHAIN, WRITES, device_rows, make_case

pytestmark = pytest.mark.gpu


def fp4_case(seed, batch, rows, ctx, page, Hkv, D, pad=0, ragged=True):
    """make_case with 4-bit caches of random codes and scales (no NaN)."""
    c = make_case(seed, batch, rows, ctx, page, Hkv, D, True, pad, ragged)
    g = torch.Generator().manual_seed(seed + 5)
    caches = []
    for _ in range(2):
        x = torch.randint(0, 256, (c["pages"], Hkv, page, 9 * D // 16), generator=g,
                          dtype=torch.uint8)
        x[..., D // 2:][(x[..., D // 2:] & 127) == 127] = 3
        caches.append(x)
    c["caches"] = caches
    return c


def places(c):
    """[(row, position, page, place in the page)] of the rows that belong to a sequence."""
    page = c["page"]
    return [(r, p, slot // page, slot % page)
            for r, _, p, slot in cref.rows_of(c["starts"], c["lens"], c["tables"].numpy(), page)]


def half_step(x):
    """Half the distance of neighbouring codes around |x| (up to 6 and what rounds to it)."""
    return np.where(x <= 2, 0.25, np.where(x <= 4, 0.5, 1.0))


def check_rows(rows, want, mag, D):
    """Rows as stored, of values `want` that hold to 2 CHAIN mag."""
    off = 2 * CHAIN * mag
    s = cref.E4M3[rows[..., D // 2:]]
    most = np.abs(want).reshape(*want.shape[:-1], -1, 16).max(-1)
    slack = off.reshape(*off.shape[:-1], -1, 16).max(-1)
    aim = np.minimum(most / 6, 448)
    assert (np.abs(s - aim) <= aim * 2.0 ** -4 + 2.0 ** -10 + slack).all(), "scales"
    wide = np.repeat(s, 16, -1)
    got = ref.decode_rows(rows, D)
    x = np.clip(want, -6 * wide, 6 * wide)
    with np.errstate(invalid="ignore", divide="ignore"):
        step = np.where(wide > 0, half_step(np.abs(x) / wide), 0) * wide
    fine = wide > 0
    assert (np.abs(got - x)[fine] <= (step + off)[fine] * (1 + 2.0 ** -20)).all(), "codes"
    assert (got[~fine] == 0).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", WRITES)
def test_cache_write_fp4(cuda_lib, case, bf16):
    batch, rows, ctx, page, Hq, Hkv, D, rot, inter, pad, ragged = case
    dev = torch.device("cuda")
    seed = batch * 137 + rows + Hq
    c = fp4_case(seed, batch, rows, ctx, page, Hkv, D, pad, ragged)
    g = torch.Generator().manual_seed(seed + 1)
    dt = torch.bfloat16 if bf16 else torch.float16
    qkv = torch.randn(c["tokens"], Hq + 2 * Hkv, D, generator=g).to(dt).to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    norm = rows % 2 == 1
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(dev) if norm else None
              for _ in range(2))
    freq = (1e4 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float().to(dev) if rot else None
    ks, vs = torch.tensor([0.031], device=dev), torch.tensor([0.0213], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    tables, lens, starts = device_rows(c)
    q_out = torch.full((c["tokens"], Hq, D), 7.0, dtype=torch.float16, device=dev)
    got = cuda_lib.cache_write_fp4(q, k, v, kc, vc, ks, vs, tables, lens, c["max_ctx"],
                                   q_weight=qw, k_weight=kw, eps=1e-5, inv_freq=freq,
                                   interleaved=inter, row_starts=starts, q_out=q_out)
    assert got is q_out and cuda_lib.device_error() == 0
    # The queries are those of the write into an fp16 cache, bit for bit.
    kc16 = torch.zeros(c["pages"], page, Hkv, D, dtype=torch.float16, device=dev)
    want_q = torch.full_like(q_out, 7.0)
    cuda_lib.cache_write(q, k, v, kc16, kc16.clone(), tables, lens, c["max_ctx"], q_weight=qw,
                         k_weight=kw, eps=1e-5, inv_freq=freq, interleaved=inter,
                         row_starts=starts, q_out=want_q)
    assert torch.equal(q_out, want_q)

    at = places(c)
    row, pos, pg, pl = (np.array(x) for x in zip(*at)) if at else ([], [], [], [])
    kc, vc = kc.cpu().numpy(), vc.cpu().numpy()
    # V: equality with the formulas in 32 bits, and nothing else touched.
    want = c["caches"][1].numpy().copy()
    inv = np.float32(1) / np.float32(vs.item())
    if at:
        want[pg, :, pl] = ref.encode_rows(v.float().cpu().numpy()[row] * inv)
    assert np.array_equal(vc, want)
    rest = c["caches"][0].numpy().copy()
    if at:
        rest[pg, :, pl] = kc[pg, :, pl]
    assert np.array_equal(kc, rest)
    if not at:
        return
    kf = k.cpu().double().numpy()
    if not norm and not rot:
        inv = np.float32(1) / np.float32(ks.item())
        assert np.array_equal(kc[pg, :, pl], ref.encode_rows(kf[row].astype(np.float32) * inv))
    fr = np.zeros(0) if freq is None else freq.cpu().double().numpy()
    kwf = None if kw is None else kw.cpu().double().numpy()
    pairs = [cref.norm_rotate(kf[r], kwf, 1e-5, fr, inter, p) for r, p in zip(row, pos)]
    y, m = (np.stack(x) / float(ks) for x in zip(*pairs))
    check_rows(kc[pg, :, pl], y, m, D)


@pytest.mark.parametrize("case", [
    (1, 1, 1, 8, 1, 256, 0, False), (5, 37, 90, 16, 2, 128, 3, True), (3, 40, 64, 256, 1, 256, 8, True),
    (40, 17, 33, 8, 4, 128, 1, True), (2, 3000, 1700, 64, 3, 256, 0, False)])
def test_cache_read_fp4(cuda_lib, case):
    batch, rows, ctx, page, Hkv, D, pad, ragged = case
    dev = torch.device("cuda")
    c = fp4_case(batch + rows, batch, rows, ctx, page, Hkv, D, pad, ragged)
    tables, lens, starts = device_rows(c)
    ks, vs = torch.tensor([0.37], device=dev), torch.tensor([0.0213], device=dev)
    outs = [torch.full((c["tokens"], Hkv, D), 7.0, dtype=torch.float16, device=dev) for _ in "kv"]
    cuda_lib.cache_read_fp4(*(x.to(dev) for x in c["caches"]), ks, vs, tables, lens, c["max_ctx"],
                            c["tokens"], row_starts=starts, k_out=outs[0], v_out=outs[1])
    assert cuda_lib.device_error() == 0
    at = places(c)
    for cache, s, out in zip(c["caches"], (ks, vs), outs):
        want = np.full(out.shape, 7, np.float16)
        if at:
            row, _, pg, pl = (np.array(x) for x in zip(*at))
            x = ref.decode_rows(cache.numpy()[pg, :, pl], D).astype(np.float32)
            with np.errstate(over="ignore"):
                want[row] = (x * np.float32(s.item())).astype(np.float16)
        assert np.array_equal(out.cpu().numpy(), want)


def test_special_values(cuda_lib):
    """Infinities saturate, a NaN makes its block NaN, zeros and what is far below the
    smallest scale become zero; blocks beside them are untouched."""
    dev = torch.device("cuda")
    k = torch.ones(5, 1, 128, dtype=torch.float16, device=dev)
    k[0, 0, 3], k[1, 0, 21], k[2, 0, 127] = float("inf"), float("-inf"), float("nan")
    k[3] = 0
    k[4, 0, :16] = 2.0 ** -14       # a sixth of 2^-13 lies below half the smallest scale
    kc = torch.zeros(2, 1, 8, 72, dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    one = torch.ones(1, dtype=torch.float32, device=dev)
    two = torch.tensor([0.5], device=dev)
    where = (torch.tensor([[1]], dtype=torch.int32, device=dev),
             torch.tensor([5], dtype=torch.int32, device=dev), 8)
    cuda_lib.cache_write_fp4(None, k, k, kc, vc, two, one, *where)
    a, b = cuda_lib.cache_read_fp4(kc, vc, two, one, *where, 5)
    got = a[:, 0].float().cpu().numpy()
    want = np.ones((5, 128))
    want[0, :16], want[1, 16:32], want[2, 112:], want[3], want[4, :16] = 0, 0, np.nan, 0, 0
    want[0, 3], want[1, 21] = 6 * 448 * 0.5, -6 * 448 * 0.5
    # 1 over its scale e4m3(2 / 6 of it) is not a code: 6 * 0.3125 * 0.5.
    want[want == 1] = 6 * 0.34375 * 0.5
    assert np.array_equal(got, want, equal_nan=True), (got[0, :5], got[4, :20])
    assert cuda_lib.device_error() == 0
    # A page outside the cache: nothing stored, zeros read, flagged.
    before = kc.clone()
    bad = (torch.tensor([[2]], dtype=torch.int32, device=dev), *where[1:])
    cuda_lib.cache_write_fp4(None, k, k, kc, vc, two, one, *bad)
    a, b = cuda_lib.cache_read_fp4(kc, vc, two, one, *bad, 5)
    assert torch.equal(kc, before) and not a.any() and not b.any()
    assert cuda_lib.device_error() == cuda_lib.DEVERR_BAD_PAGE_ID


def test_stream_and_graph(cuda_lib):
    """A write and a read on a stream of their own, captured and replayed as the context
    grows: the same rows as eager calls give."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(3)
    k = torch.randn(2, 2, 128, generator=g).half().to(dev)
    s = torch.tensor([0.05], device=dev)
    table = torch.tensor([[3, 0, 2, 1]], dtype=torch.int32, device=dev)
    ctx = torch.tensor([2], dtype=torch.int32, device=dev)
    kc, vc = (torch.zeros(4, 2, 8, 72, dtype=torch.uint8, device=dev) for _ in "kv")
    ko, vo = (torch.zeros(2, 2, 128, dtype=torch.float16, device=dev) for _ in "kv")

    def step(stream=None):
        cuda_lib.cache_write_fp4(None, k, k, kc, vc, s, s, table, ctx, 32, stream=stream)
        cuda_lib.cache_read_fp4(kc, vc, s, s, table, ctx, 32, 2, k_out=ko, v_out=vo,
                                stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (2, 9, 17, 32):
        ctx.fill_(n)
        k.copy_(torch.randn(2, 2, 128, generator=g).half())
        graph.replay()
        got = ko.clone(), vo.clone(), kc.clone()
        kc.zero_()
        step()
        assert torch.equal(ko, got[0]) and torch.equal(vo, got[1])
        pages = [int(table[0, p // 8]) for p in (n - 2, n - 1)]
        for p, pg in zip((n - 2, n - 1), pages):
            assert torch.equal(kc[pg, :, p % 8], got[2][pg, :, p % 8])
    assert cuda_lib.device_error() == 0


def test_quotients_half_way_and_far(cuda_lib):
    """Values half way between two codes go to the even one; blocks beyond 2^100, where
    the kernel divides, and blocks of tiny values give the formula's codes too."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(11)
    T, D = 512, 128
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    # Blocks whose scale is m / 8 * 2^e and whose values are half-way points of it.
    m = torch.randint(8, 16, (T, 1, D // 16, 1), generator=g) / 8
    e = torch.randint(-6, 7, (T, 1, D // 16, 1), generator=g).float()
    x = mids[torch.randint(0, 8, (T, 1, D // 16, 16), generator=g)]
    x[..., 0] = 6.0
    x = x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0) * m * 2.0 ** e
    k = x.reshape(T, 1, D).bfloat16()
    assert torch.equal(k.float(), x.reshape(T, 1, D))
    v = torch.randn(T, 1, D, generator=g).bfloat16()
    v[0::4] *= 2.0 ** 104
    v[1::4] *= 2.0 ** -13
    v[2::4] *= 2.0 ** -126
    pages = T // 8
    kc, vc = (torch.zeros(pages, 1, 8, 72, dtype=torch.uint8, device=dev) for _ in "kv")
    one = torch.ones(1, device=dev)
    table = torch.arange(pages, dtype=torch.int32, device=dev)[None].contiguous()
    lens = torch.tensor([T], dtype=torch.int32, device=dev)
    cuda_lib.cache_write_fp4(None, k.to(dev), v.to(dev), kc, vc, one, one, table, lens, T)
    for cache, y in ((kc, k), (vc, v)):
        want = ref.encode_rows(y.float().numpy()).reshape(cache.shape)
        assert np.array_equal(cache.cpu().numpy(), want)
    assert cuda_lib.device_error() == 0


def test_read_into_odd_addresses(cuda_lib):
    """Outputs 16 bytes past a 32-byte boundary: the same rows, and nothing beside them."""
    dev = torch.device("cuda")
    c = fp4_case(3, 3, 21, 60, 8, 2, 128)
    tables, lens, starts = device_rows(c)
    s = torch.tensor([0.37], device=dev)
    caches = [x.to(dev) for x in c["caches"]]
    args = (*caches, s, s, tables, lens, c["max_ctx"], c["tokens"])
    zeros = [torch.full((c["tokens"], 2, 128), 7.0, dtype=torch.float16, device=dev) for _ in "kv"]
    cuda_lib.cache_read_fp4(*args, row_starts=starts, k_out=zeros[0], v_out=zeros[1])
    n = zeros[0].numel()
    flat = [torch.full((n + 16,), 7.0, dtype=torch.float16, device=dev) for _ in "kv"]
    for at in ((8, 8), (0, 8), (8, 0)):
        outs = [f[a:a + n].view(zeros[0].shape) for f, a in zip(flat, at)]
        cuda_lib.cache_read_fp4(*args, row_starts=starts, k_out=outs[0], v_out=outs[1])
        for f, o, a, want in zip(flat, outs, at, zeros):
            assert torch.equal(o, want)
            assert (f[:a] == 7).all() and (f[a + n:] == 7).all()
            f.fill_(7.0)
    assert cuda_lib.device_error() == 0
