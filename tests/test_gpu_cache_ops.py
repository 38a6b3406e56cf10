"""GPU tests of the cache write, cache read and block index against plain
64-bit forms (tests/cache_reference.py).

Tolerances.  The write computes norm and rotation in 32 bits and rounds once.
Relative errors of the 32-bit steps, in units of 2^-24: the sum of squares adds
at most 13 (8 fused terms, 5 shuffled additions), halved by the square root;
2 each for rsqrt, the two products and the rotation's products and sum; cos and
sin 4: below 2^-19 of the magnitudes that enter a value.  One rounding to fp16
adds 2^-11 of the value (2^-25 among subnormals), one to E4M3 2^-4 (2^-10).
Reads and the as-is copies are exact up to the one fp16 rounding; block codes
follow fixed fp32 operations and are compared for equality.
"""

import random

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu

CHAIN = 2.0 ** -19


def make_case(seed, batch, rows, ctx, page, Hkv, D, e4m3, pad=0, ragged=True, fill=None):
    """Row starts, context lengths, tables and filled caches of a batch."""
    rnd = random.Random(seed)
    if ragged:
        cuts = sorted(rnd.randint(0, rows) for _ in range(batch - 1))
        starts = [0] + cuts + [rows]
    else:
        assert rows % batch == 0
        starts = [rows // batch * b for b in range(batch + 1)]
    n = [starts[b + 1] - starts[b] for b in range(batch)]
    lens = [rnd.randint(max(1, x), max(1, x, ctx)) for x in n]
    stride = -(-max(lens) // page)
    pages = batch * stride + 3
    g = torch.Generator().manual_seed(seed)
    tables = torch.randperm(pages, generator=g)[: batch * stride].view(batch, stride).int()
    caches = []
    for _ in range(2):
        x = torch.randn(pages, page, Hkv, D, generator=g)
        if e4m3:
            x = torch.randint(0, 256, x.shape, generator=g, dtype=torch.uint8)
            x[(x & 127) == 127] = 3   # no NaN codes
        else:
            x = x.half()
        caches.append(x)
    return dict(starts=starts, lens=lens, tables=tables, caches=caches, page=page, Hkv=Hkv, D=D,
                tokens=rows + pad, batch=batch, max_ctx=max(lens), pages=pages, stride=stride,
                e4m3=e4m3, ragged=ragged or pad > 0)


def device_rows(c):
    dev = torch.device("cuda")
    starts = torch.tensor(c["starts"], dtype=torch.int32, device=dev) if c["ragged"] else None
    return c["tables"].to(dev), torch.tensor(c["lens"], dtype=torch.int32, device=dev), starts


def run_write(lib, c, q, k, v, kc, vc, ks, vs, **kw):
    tables, lens, starts = device_rows(c)
    if c["e4m3"]:
        return lib.cache_write_e4m3(q, k, v, kc, vc, ks, vs, tables, lens, c["max_ctx"],
                                    row_starts=starts, **kw)
    return lib.cache_write(q, k, v, kc, vc, tables, lens, c["max_ctx"], row_starts=starts, **kw)


def check_write(c, q, k, v, q_out, q_before, kc, vc, ks, vs, qw, kw, eps, freq, interleaved):
    rows = ref.rows_of(c["starts"], c["lens"], c["tables"].numpy(), c["page"])
    f64 = lambda t: None if t is None else t.cpu().double().numpy()  # noqa: E731
    qn, kn, vn, qwn, kwn = f64(q), f64(k), f64(v), f64(qw), f64(kw)
    fr = np.zeros(0) if freq is None else f64(freq)
    Hkv, D = c["Hkv"], c["D"]
    # Untouched rows and cache tokens keep their bytes.
    want_k = ref.decode(c["caches"][0]).reshape(-1, Hkv, D).copy()
    want_v = ref.decode(c["caches"][1]).reshape(-1, Hkv, D).copy()
    tol_k, tol_v = np.zeros_like(want_k), np.zeros_like(want_v)
    want_q = None if q is None else q_before.cpu().double().numpy().copy()
    tol_q = None if q is None else np.zeros_like(want_q)
    top = 448.0 if c["e4m3"] else 65504.0
    step, sub = (2.0 ** -4, 2.0 ** -10) if c["e4m3"] else (2.0 ** -11, 2.0 ** -25)
    for r, _, p, slot in rows:
        if q is not None:
            y, m = ref.norm_rotate(qn[r], qwn, eps, fr, interleaved, p)
            want_q[r], tol_q[r] = y, 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2 * CHAIN * m
        y, m = ref.norm_rotate(kn[r], kwn, eps, fr, interleaved, p)
        y, m = y / ks, m / ks
        want_k[slot] = np.clip(y, -top, top)
        tol_k[slot] = step * np.abs(y) + sub + 2 * CHAIN * m
        y = vn[r] / vs
        want_v[slot] = np.clip(y, -top, top)
        tol_v[slot] = step * np.abs(y) + sub + 2 * CHAIN * np.abs(y)
    if q is not None:
        got = q_out.cpu().double().numpy()
        assert (np.abs(got - want_q) <= tol_q).all(), "q"
    for name, got, want, tol in (("k", kc, want_k, tol_k), ("v", vc, want_v, tol_v)):
        d = np.abs(ref.decode(got).reshape(want.shape) - want)
        assert (d <= tol).all(), (name, float(np.nanmax(d - tol)))


WRITES = [
    # batch, rows, ctx, page, Hq, Hkv, D, rot, interleaved, pad, ragged
    (1, 1, 1, 8, 6, 1, 256, 256, False, 0, False),
    (8, 8, 500, 16, 6, 1, 256, 64, False, 0, False),
    (5, 33, 90, 16, 6, 2, 256, 256, True, 3, True),
    (7, 61, 200, 32, 16, 4, 128, 128, False, 0, True),
    (3, 40, 64, 256, 8, 1, 128, 96, True, 8, True),
    (40, 17, 33, 8, 4, 4, 128, 16, False, 1, True),     # more sequences than rows
    (1, 1300, 1400, 64, 6, 1, 256, 64, False, 20, True),
    (2, 1026, 700, 128, 12, 4, 256, 208, True, 0, False),
    (1, 37, 50, 16, 64, 64, 128, 0, False, 0, False),
]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", WRITES)
def test_cache_write(cuda_lib, case, bf16, e4m3):
    batch, rows, ctx, page, Hq, Hkv, D, rot, inter, pad, ragged = case
    dev = torch.device("cuda")
    seed = batch * 131 + rows + Hq
    c = make_case(seed, batch, rows, ctx, page, Hkv, D, e4m3, pad, ragged)
    g = torch.Generator().manual_seed(seed + 1)
    dt = torch.bfloat16 if bf16 else torch.float16
    # One fused projection: q, k and v are strided views of it.
    qkv = torch.randn(c["tokens"], Hq + 2 * Hkv, D, generator=g).to(dt).to(dev)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    norm = rows % 2 == 1
    qw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(dev) if norm else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt).to(dev) if norm else None
    freq = (1e4 ** (-torch.arange(rot // 2) / max(1, rot // 2))).float().to(dev) if rot else None
    ks = torch.tensor([0.01 if e4m3 else 1.0], device=dev)
    vs = torch.tensor([0.0113 if e4m3 else 1.0], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    q_out = torch.full((c["tokens"], Hq, D), 7.0, dtype=torch.float16, device=dev)
    before = q_out.clone()
    got = run_write(cuda_lib, c, q, k, v, kc, vc, ks, vs, q_weight=qw, k_weight=kw, eps=1e-5,
                    inv_freq=freq, interleaved=inter, q_out=q_out)
    assert got is q_out
    assert cuda_lib.device_error() == 0
    check_write(c, q, k, v, q_out, before, kc, vc, float(ks), float(vs), qw, kw, 1e-5, freq,
                inter)


def test_cache_write_without_queries_and_other_strides(cuda_lib):
    dev = torch.device("cuda")
    c = make_case(5, 3, 21, 60, 16, 2, 128, True)
    g = torch.Generator().manual_seed(6)
    # Heads twice their size apart, tokens in reverse of the head order.
    k = torch.randn(2, 21, 2, 128, generator=g).half().to(dev)[:, :, 0].transpose(0, 1)
    v = torch.randn(21, 1, 128, generator=g).half().to(dev).expand(21, 2, 128)
    ks, vs = torch.tensor([0.02], device=dev), torch.tensor([0.01], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    assert run_write(cuda_lib, c, None, k, v, kc, vc, ks, vs) is None
    assert cuda_lib.device_error() == 0
    check_write(c, None, k, v, None, None, kc, vc, float(ks), float(vs), None, None, 0.0, None,
                False)


def test_cache_write_special_values(cuda_lib):
    """Infinities saturate, NaN stays NaN, a head of zeros stays zero with eps > 0."""
    dev = torch.device("cuda")
    c = make_case(7, 1, 4, 4, 8, 1, 128, True, ragged=False)
    k = torch.ones(4, 1, 128, dtype=torch.float16, device=dev)
    k[0, 0, 3], k[1, 0, 5], k[2, 0, 7] = float("inf"), float("-inf"), float("nan")
    k[3] = 0
    ks = torch.tensor([0.5], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    run_write(cuda_lib, c, None, k, k, kc, vc, ks, ks)
    rows = ref.rows_of(c["starts"], c["lens"], c["tables"].numpy(), 8)
    got = ref.decode(kc).reshape(-1, 128)[[s for *_, s in rows]]
    want = np.full((4, 128), 2.0)
    want[0, 3], want[1, 5], want[2, 7], want[3] = 448, -448, np.nan, 0
    assert np.array_equal(got, want, equal_nan=True)
    run_write(cuda_lib, c, None, k, k, kc, vc, ks, ks,
              k_weight=torch.ones(128, dtype=torch.float16, device=dev), eps=1e-6)
    got = ref.decode(kc).reshape(-1, 128)[rows[3][3]]
    assert (got == 0).all()


def test_bad_contexts_and_pages_are_left_out(cuda_lib):
    dev = torch.device("cuda")
    c = make_case(9, 4, 20, 40, 8, 1, 128, True, ragged=False)
    c["tables"] = c["tables"].clone()
    n = 5
    c["lens"] = [30, 4, 33, 40]             # 4 < its 5 rows
    c["max_ctx"] = 39                       # 40 is past the bound
    c["tables"] = torch.arange(4 * 5).view(4, 5).int()
    assert c["pages"] >= 20
    good = [r for r in ref.rows_of([0, 5, 10, 15, 20], [30, 5, 33, 40], c["tables"].numpy(), 8)
            if r[1] in (0, 2)]
    c["tables"][2, 4] = c["pages"]          # sequence 2's position 32
    bad = [r for r in good if r[1] == 2 and r[2] >= 32]
    good = [r for r in good if r not in bad]
    assert len(bad) == 1 and len(good) == 2 * n - 1
    g = torch.Generator().manual_seed(3)
    q = torch.randn(20, 2, 128, generator=g).half().to(dev)
    k = torch.randn(20, 1, 128, generator=g).half().to(dev)
    s = torch.tensor([0.01], device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    q_out = torch.full((20, 2, 128), 7.0, dtype=torch.float16, device=dev)
    run_write(cuda_lib, c, q, k, k, kc, vc, s, s, q_out=q_out)
    assert cuda_lib.device_error() == (cuda_lib.DEVERR_BAD_CTX_LEN | cuda_lib.DEVERR_BAD_PAGE_ID)
    written = [r[3] for r in good]
    same = np.ones(c["pages"] * 8, bool)
    same[written] = False
    for now, was in zip((kc, vc), c["caches"]):
        now = now.cpu().view(-1, 128).numpy()
        assert np.array_equal(now[same], was.view(-1, 128).numpy()[same])
        assert not np.array_equal(now[written[0]], was.view(-1, 128).numpy()[written[0]])
    kept = [r for r in range(20) if r not in [x[0] for x in good + bad]]
    assert (q_out[kept] == 7).all()
    assert torch.equal(q_out[[x[0] for x in good + bad]], q[[x[0] for x in good + bad]])
    # The read leaves the same rows out and gives zeros for the bad page.
    tables, lens, _ = device_rows(c)
    outs = [torch.full((20, 1, 128), 7.0, dtype=torch.float16, device=dev) for _ in range(2)]
    cuda_lib.cache_read_e4m3(kc, vc, s, s, tables, lens, c["max_ctx"], 20, k_out=outs[0],
                             v_out=outs[1])
    assert cuda_lib.device_error() == (cuda_lib.DEVERR_BAD_CTX_LEN | cuda_lib.DEVERR_BAD_PAGE_ID)
    for o in outs:
        assert (o[kept] == 7).all() and (o[bad[0][0]] == 0).all()
        assert (o[[x[0] for x in good]] != 7).any()
    # And the index writes no block of them.
    index = torch.full((c["pages"], 2, 1, 128), 99, dtype=torch.int8, device=dev)
    scale = torch.full((c["pages"], 2), 5.0, device=dev)
    cuda_lib.block_index_e4m3(kc, s, tables, lens, c["max_ctx"], 20, index, scale)
    assert cuda_lib.device_error() == (cuda_lib.DEVERR_BAD_CTX_LEN | cuda_lib.DEVERR_BAD_PAGE_ID)
    blocks = sorted(r[3] // 4 for r in good if r[2] % 4 == 3)
    touched = torch.nonzero((scale.view(-1) != 5).cpu())[:, 0].tolist()
    assert touched == blocks


@pytest.mark.parametrize("starts", [[5, 3, 9, 2], [-4, 6, 2, 20], [30, 40, 50, 60],
                                    [0, 0, 0, 0], [0, 2**31 - 1, 5, -2**31]])
def test_row_starts_that_do_not_ascend_stay_in_bounds(cuda_lib, starts):
    """Starts that no batch has: whatever rows they leave, no store outside
    the named tokens' rows (bounds are the kernel's own checks)."""
    dev = torch.device("cuda")
    c = make_case(11, 3, 12, 40, 8, 1, 128, False)
    tables, lens, _ = device_rows(c)
    s = torch.tensor(starts, dtype=torch.int32, device=dev)
    k = torch.ones(12, 1, 128, dtype=torch.float16, device=dev)
    kc, vc = (x.to(dev) for x in c["caches"])
    cuda_lib.cache_write(None, k, k, kc, vc, tables, lens, c["max_ctx"], row_starts=s)
    cuda_lib.cache_read(kc, vc, tables, lens, c["max_ctx"], 12, row_starts=s)
    torch.cuda.synchronize()
    cuda_lib.device_error()
    used = set()
    for b in range(3):
        for p in range(c["lens"][b]):
            used.add(int(c["tables"][b][p // 8]) * 8 + p % 8)
    other = [t for t in range(c["pages"] * 8) if t not in used]
    assert torch.equal(kc.cpu().view(-1, 128)[other], c["caches"][0].view(-1, 128)[other])


READS = [(1, 1, 1, 8, 1, 128, 0, False), (1, 333, 333, 16, 1, 256, 0, False),
         (9, 333, 120, 16, 2, 256, 7, True), (3, 2500, 1500, 64, 2, 128, 33, True),
         (64, 40, 90, 256, 4, 128, 0, True), (2, 50, 60, 32, 64, 128, 0, False)]


@pytest.mark.parametrize("case", READS)
@pytest.mark.parametrize("kind", ["dequant", "codes", "f16"])
def test_cache_read(cuda_lib, case, kind):
    batch, rows, ctx, page, Hkv, D, pad, ragged = case
    dev = torch.device("cuda")
    c = make_case(rows + batch, batch, rows, ctx, page, Hkv, D, kind != "f16", pad, ragged)
    tables, lens, starts = device_rows(c)
    kc, vc = (x.to(dev) for x in c["caches"])
    kept = torch.float16 if kind != "codes" else torch.uint8
    outs = [torch.full((c["tokens"], Hkv, D), 7, dtype=kept, device=dev) for _ in range(2)]
    args = (tables, lens, c["max_ctx"], c["tokens"])
    how = dict(row_starts=starts, k_out=outs[0], v_out=outs[1])
    if kind == "dequant":
        # Every code, NaN among them, and a scale that makes some overflow fp16.
        kc.view(-1)[: min(256, kc.numel())] = torch.arange(256, dtype=torch.uint8, device=dev)
        ks, vs = torch.tensor([0.37], device=dev), torch.tensor([200.0], device=dev)
        cuda_lib.cache_read_e4m3(kc, vc, ks, vs, *args, **how)
    else:
        cuda_lib.cache_read(kc, vc, *args, **how)
    assert cuda_lib.device_error() == 0
    slots = [s for *_, s in ref.rows_of(c["starts"], c["lens"], c["tables"].numpy(), page)]
    for out, cache, scale in ((outs[0], kc, 0.37), (outs[1], vc, 200.0)):
        rest = out[rows:]
        assert (rest == 7).all()
        want = cache.cpu().view(-1, Hkv, D)[slots]
        if kind == "dequant":
            # code * scale is exact in 64 bits (4 + 24 bits): numpy's one rounding to fp16;
            # the kernel rounds to 32 bits first, which moves a value by half a step of 32
            # bits at most and so the fp16 result only where that crosses a tie.
            with np.errstate(over="ignore"):
                w = (ref.decode(want) * np.float64(np.float32(scale))).astype(np.float16)
            got = out[:rows].cpu().numpy()
            same = (got == w) | (np.isnan(got) & np.isnan(w))
            d = np.abs(got.astype(np.float64) - w.astype(np.float64))
            with np.errstate(invalid="ignore"):
                assert (same | (d <= 2.0 ** -10 * np.abs(w.astype(np.float64)))).all()
            assert same.mean() > 0.999
        else:
            assert torch.equal(out[:rows].cpu().view(torch.uint8), want.view(torch.uint8))


def test_sequences_that_share_pages(cuda_lib):
    """Two sequences with the same table read the same tokens and summarise the
    same blocks."""
    dev = torch.device("cuda")
    c = make_case(5, 2, 24, 40, 16, 1, 128, True, ragged=False)
    c["tables"][1] = c["tables"][0]
    c["lens"], c["max_ctx"] = [21, 30], 30
    tables, lens, _ = device_rows(c)
    kc, vc = (x.to(dev) for x in c["caches"])
    k, v = cuda_lib.cache_read(kc, vc, tables, lens, 30, 24)
    assert torch.equal(k[18 - 9:12], k[12:15]) and torch.equal(v[18 - 9:12], v[12:15])
    s = torch.tensor([0.5], device=dev)
    got = []
    for last in (1, 2):     # the second sequence alone, then both
        index = torch.zeros(c["pages"], 4, 1, 128, dtype=torch.int8, device=dev)
        scale = torch.zeros(c["pages"], 4, device=dev)
        cuda_lib.block_index_e4m3(kc, s, tables[2 - last:].contiguous(), lens[2 - last:].contiguous(),
                                  30, 12 * last, index, scale)
        got.append((index, scale))
    assert cuda_lib.device_error() == 0
    both, alone = got[1][1].view(-1), got[0][1].view(-1)
    assert torch.equal(both[alone != 0], alone[alone != 0])
    # Positions 11, 15, 19 of the first; 19, 23, 27 of the second.
    assert int((both != 0).sum()) == 5 and int((alone != 0).sum()) == 3


INDEXES = [(1, 4, 4, 8, 1, 128, 0, False), (16, 64, 200, 16, 1, 256, 0, False),
           (5, 130, 90, 32, 2, 256, 6, True), (3, 4500, 3000, 64, 2, 128, 3, True),
           (6, 100, 300, 256, 4, 256, 0, True), (2, 40, 60, 16, 7, 128, 0, True),
           (2, 40, 60, 8, 3, 128, 0, False), (30, 20, 60, 8, 8, 128, 0, True)]


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("case", INDEXES)
def test_block_index(cuda_lib, case, e4m3):
    batch, rows, ctx, page, Hkv, D, pad, ragged = case
    dev = torch.device("cuda")
    c = make_case(rows + 3 * batch, batch, rows, ctx, page, Hkv, D, e4m3, pad, ragged)
    tables, lens, starts = device_rows(c)
    located = ref.rows_of(c["starts"], c["lens"], c["tables"].numpy(), page)
    blocks = [s // 4 for _, _, p, s in located if p % 4 == 3]
    cache = c["caches"][0]
    flat = cache.view(-1, 4, Hkv * D)
    zero, nan = (0, 0x7F) if e4m3 else (0.0, float("nan"))
    if len(blocks) > 2:
        flat[blocks[0]] = zero            # a block of zeros
        flat[blocks[1], 2, 5] = nan       # one NaN key
        if not e4m3:
            flat[blocks[2], 1, 7] = float("inf")
    kc = cache.to(dev)
    ks = torch.tensor([0.0173], device=dev)
    index = torch.full((c["pages"], page // 4, Hkv, D), 99, dtype=torch.int8, device=dev)
    scale = torch.full((c["pages"], page // 4), 5.0, device=dev)
    args = (tables, lens, c["max_ctx"], c["tokens"], index, scale)
    if e4m3:
        cuda_lib.block_index_e4m3(kc, ks, *args, row_starts=starts)
    else:
        cuda_lib.block_index(kc, *args, row_starts=starts)
    assert cuda_lib.device_error() == 0
    want_i = np.full((c["pages"] * (page // 4), Hkv * D), 99, np.int8)
    want_s = np.full(c["pages"] * (page // 4), 5.0, np.float32)
    keys = ref.decode(cache).reshape(-1, 4, Hkv * D)
    for b in blocks:
        s = ref.block_sums(keys[b])
        want_i[b], want_s[b] = ref.summary(s, ks.cpu().numpy()[0] if e4m3 else 1.0)
        if np.isfinite(keys[b]).all() and keys[b].any():
            # Against the definition in 64 bits: half a code, plus the 32-bit
            # roundings of the sum (2^-23 of the magnitudes summed, at most)
            # and of the quotient and product (2^-22 of 127).
            e = keys[b].sum(0)
            a = np.abs(e).max()
            off = np.abs(want_i[b] - e * 127 / a)
            tol = 0.5 + 127 * 2.0 ** -22 + 2 * 127 * 2.0 ** -23 * np.abs(keys[b]).sum(0).max() / a
            assert (off <= tol).all()
    assert np.array_equal(index.cpu().numpy().reshape(want_i.shape), want_i)
    assert np.array_equal(scale.cpu().numpy().reshape(-1), want_s)


def test_far_positions_and_offsets_past_32_bits(cuda_lib):
    """The last tokens of a context beyond 2^24, in a cache whose byte offsets
    pass 2^32: write, read back and summarise."""
    dev = torch.device("cuda")
    page, Hkv, D, rows = 256, 2, 128, 9
    ctx = (1 << 24) + 1003
    stride = -(-ctx // page)
    pages = stride + 1
    kc = torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    assert kc.numel() > 1 << 32
    tables = (pages - 1 - torch.arange(stride)).int().flip(0).view(1, -1).contiguous()
    c = dict(starts=[0, rows], lens=[ctx], tables=tables, page=page, Hkv=Hkv, D=D, max_ctx=ctx,
             e4m3=True, ragged=False)
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(rows, 6, D, generator=g).half().to(dev)
    q, k, v = qkv[:, :2], qkv[:, 2:4], qkv[:, 4:]
    freq = (1e4 ** (-torch.arange(64) / 64)).float().to(dev)
    s = torch.tensor([0.01], device=dev)
    q_out = run_write(cuda_lib, c, q, k, v, kc, vc, s, s, inv_freq=freq)
    assert cuda_lib.device_error() == 0
    located = ref.rows_of(c["starts"], c["lens"], tables.numpy(), page)
    got_k, got_v = cuda_lib.cache_read(kc, vc, tables.to(dev), torch.tensor(
        [ctx], dtype=torch.int32, device=dev), ctx, rows)
    for r, _, p, slot in located:
        y, m = ref.norm_rotate(q[r].cpu().double().numpy(), None, 0, freq.cpu().numpy(), False, p)
        tol = 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2 * CHAIN * m
        assert (np.abs(q_out[r].cpu().double().numpy() - y) <= tol).all()
        y, m = ref.norm_rotate(k[r].cpu().double().numpy(), None, 0, freq.cpu().numpy(), False, p)
        code = kc.view(-1, Hkv, D)[slot]
        tol = 2.0 ** -4 * np.abs(y) / 0.01 + 2.0 ** -10 + 200 * CHAIN * m
        want = np.clip(y / float(s), -448, 448)
        assert (np.abs(ref.decode(code) - want) <= tol).all()
        assert torch.equal(got_k[r], code) and torch.equal(got_v[r], vc.view(-1, Hkv, D)[slot])
    index = torch.zeros(pages, page // 4, Hkv, D, dtype=torch.int8, device=dev)
    scale = torch.zeros(pages, page // 4, device=dev)
    cuda_lib.block_index_e4m3(kc, s, tables.to(dev), torch.tensor(
        [ctx], dtype=torch.int32, device=dev), ctx, rows, index, scale)
    for r, _, p, slot in located:
        if p % 4 == 3:
            keys = ref.decode(kc.view(-1, 4, Hkv * D)[slot // 4])
            code, sc = ref.summary(ref.block_sums(keys), s.cpu().numpy()[0])
            assert np.array_equal(index.view(-1, Hkv * D)[slot // 4].cpu().numpy(), code)
            assert float(scale.view(-1)[slot // 4]) == float(sc)
    assert int((scale != 0).sum()) == sum(p % 4 == 3 for _, _, p, _ in located)


def test_binding_refuses_mismatched_tensors(cuda_lib):
    dev = torch.device("cuda")
    c = make_case(2, 2, 6, 20, 16, 1, 256, True)
    tables, lens, starts = device_rows(c)
    kc, vc = (x.to(dev) for x in c["caches"])
    k = torch.zeros(6, 1, 256, dtype=torch.float16, device=dev)
    s = torch.ones(1, device=dev)
    ok = dict(q=k, k=k, v=k, kcache=kc, vcache=vc, kscale=s, vscale=s, block_tables=tables,
              ctx_lens_dev=lens, max_ctx_len=c["max_ctx"], row_starts=starts)
    cuda_lib.cache_write_e4m3(**ok)
    for bad in (dict(k=k.float()), dict(v=k.bfloat16()), dict(v=k[:5]), dict(kcache=kc.half()),
                dict(vcache=vc[:-1]), dict(kscale=s.double()), dict(kscale=torch.ones(2, device=dev)),
                dict(vscale=torch.ones(1)), dict(block_tables=tables.long()),
                dict(block_tables=tables[:, :0]), dict(ctx_lens_dev=lens[:1]),
                dict(row_starts=starts[:-1]), dict(row_starts=starts.long()),
                dict(q_out=k.float()), dict(q_out=k[:, :, :128]), dict(q_weight=k.view(-1)[:128]),
                dict(k_weight=torch.ones(256, device=dev)), dict(k=k[:, :, ::2]),
                dict(k=torch.zeros(6, 2, 256, dtype=torch.float16, device=dev)),
                dict(inv_freq=torch.ones(5, device=dev)), dict(inv_freq=torch.ones(136, device=dev)),
                dict(q=None, q_out=k), dict(q=torch.zeros(6, 1, 264, dtype=torch.float16,
                                                          device=dev)[:, :, 4:260])):
        with pytest.raises(cuda_lib.GQAError):
            cuda_lib.cache_write_e4m3(**{**ok, **bad})
    with pytest.raises(cuda_lib.GQAError):
        cuda_lib.cache_read(kc, vc.half(), tables, lens, c["max_ctx"], 6)
    with pytest.raises(cuda_lib.GQAError):
        cuda_lib.cache_read(kc, vc, tables, lens, c["max_ctx"], 6, row_starts=starts,
                            k_out=k)
    with pytest.raises(cuda_lib.GQAError):
        cuda_lib.block_index_e4m3(kc, s, tables, lens, c["max_ctx"], 6,
                                  torch.zeros(c["pages"], 8, 1, 256, dtype=torch.int8, device=dev),
                                  torch.zeros(c["pages"], 8, device=dev), row_starts=starts)
    assert cuda_lib.device_error() == 0
