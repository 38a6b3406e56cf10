"""The cache operators together, as a serving step uses them: write a step's
rows, summarise the blocks they finish, select, attend; read a prefix back for
a prefill.  Attention results against the FP64 oracle on the cached values."""

import numpy as np
import pytest
import torch

import cache_reference as ref
import oracle

pytestmark = pytest.mark.gpu


def _close(got, want):
    g = got.float().cpu().numpy().astype(np.float64)
    err = np.abs(g - want).max()
    rel = np.linalg.norm(g - want) / np.linalg.norm(want)
    assert np.isfinite(g).all() and err <= 1e-3 and rel <= 1e-2, (err, rel)


class Cache:
    """One sequence's paged cache with its block index."""

    def __init__(self, ctx, page, Hkv, D, e4m3, seed=0):
        dev = torch.device("cuda")
        self.page, self.e4m3 = page, e4m3
        used = -(-ctx // page)
        pages = used + 2
        shape = (pages, page, Hkv, D)
        if e4m3:
            self.k = torch.full(shape, 0x7F, dtype=torch.uint8, device=dev)
        else:
            self.k = torch.full(shape, float("nan"), dtype=torch.float16, device=dev)
        self.v = self.k.clone()
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(pages, generator=g)[:used].int().to(dev)
        self.ks = torch.tensor([0.011], device=dev)
        self.vs = torch.tensor([0.009], device=dev)
        self.index = torch.zeros(pages, page // 4, Hkv, D, dtype=torch.int8, device=dev)
        self.index_scale = torch.zeros(pages, page // 4, device=dev)
        self.max_ctx = ctx

    def write(self, lib, qkv, Hq, Hkv, ctx, **kw):
        lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        where = (self.table.view(1, -1), lens, self.max_ctx)
        T = qkv.shape[0]
        if self.e4m3:
            out = lib.cache_write_e4m3(q, k, v, self.k, self.v, self.ks, self.vs, *where, **kw)
            lib.block_index_e4m3(self.k, self.ks, *where, T, self.index, self.index_scale)
        else:
            out = lib.cache_write(q, k, v, self.k, self.v, *where, **kw)
            lib.block_index(self.k, *where, T, self.index, self.index_scale)
        return out


@pytest.mark.parametrize("e4m3", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(6, 1, 256), (8, 2, 128)])
def test_chunked_sparse_prefill_then_decode(cuda_lib, e4m3, Hq, Hkv, D):
    """Chunks of a prompt and two single tokens: write, index, select, attend."""
    dev = torch.device("cuda")
    steps = [700, 333, 2, 1, 1]
    total = sum(steps)
    c = Cache(total, 16, Hkv, D, e4m3)
    g = torch.Generator().manual_seed(9)
    w = (1 + 0.1 * torch.randn(D, generator=g)).half().to(dev)
    freq = (1e4 ** (-torch.arange(32) / 32)).float().to(dev)
    ctx = 0
    for n in steps:
        ctx += n
        qkv = torch.randn(n, Hq + 2 * Hkv, D, generator=g).half().to(dev)
        q = c.write(cuda_lib, qkv, Hq, Hkv, ctx, q_weight=w, k_weight=w, inv_freq=freq)
        sel, cnt = cuda_lib.select_blocks(q, c.index, c.index_scale, c.table, ctx, 32, n_first=1,
                                          n_last=2)
        want_sel, want_cnt = ref.select(q, c.index, c.index_scale, c.table, 16, ctx, 32, 1, 2)
        assert np.array_equal(sel.cpu().numpy(), want_sel)
        assert np.array_equal(cnt.cpu().numpy(), want_cnt)
        if e4m3:
            out = cuda_lib.sparse_blocks_e4m3(q, c.k, c.v, c.ks, c.vs, c.table, sel, cnt, ctx)
            want = oracle.sparse_blocks_e4m3(q.cpu(), c.k.cpu(), c.v.cpu(), float(c.ks),
                                             float(c.vs), c.table.cpu(), sel.cpu(), cnt.cpu(),
                                             ctx, 1 / 16)
        else:
            out = cuda_lib.sparse_blocks(q, c.k, c.v, c.table, sel, cnt, ctx)
            want = oracle.sparse_blocks(q.cpu(), c.k.cpu(), c.v.cpu(), c.table.cpu(), sel.cpu(),
                                        cnt.cpu(), ctx, 1 / 16)
        assert cuda_lib.device_error() == 0
        _close(out, want)


def test_prefix_read_back_feeds_the_prefill(cuda_lib):
    dev = torch.device("cuda")
    Hq, Hkv, D, n = 6, 1, 256, 150
    c = Cache(1000, 32, Hkv, D, True, seed=3)
    g = torch.Generator().manual_seed(4)
    for ctx, rows in ((850, 850), (1000, n)):
        qkv = torch.randn(rows, Hq + 2, D, generator=g).half().to(dev)
        q = c.write(cuda_lib, qkv, Hq, Hkv, ctx)
    where = (c.table.view(1, -1), torch.tensor([1000], dtype=torch.int32, device=dev), 1000, 1000)
    k, v = cuda_lib.cache_read_e4m3(c.k, c.v, c.ks, c.vs, *where)
    out = cuda_lib.prefill(q, k, v)
    _close(out, oracle.dense(q.cpu(), k.cpu(), v.cpu(), 1 / 16))
    kc, vc = cuda_lib.cache_read(c.k, c.v, *where)
    out8 = cuda_lib.prefill_e4m3(q, kc, vc, c.ks, c.vs)
    want = oracle.dense_e4m3(q.cpu(), kc.cpu(), vc.cpu(), float(c.ks), float(c.vs), 1 / 16)
    _close(out8, want)
    tail = cuda_lib.paged_e4m3(q[-4:].contiguous(), c.k, c.v, c.ks, c.vs, c.table, 1000)
    _close(tail, want[-4:])
    assert cuda_lib.device_error() == 0


def test_batched_decode_step_in_a_graph(cuda_lib):
    """Write, index and batched attention captured once, replayed as every
    context grows; padded rows behind the last sequence stay untouched."""
    dev = torch.device("cuda")
    B, R, Hq, Hkv, D, page, top = 3, 2, 6, 1, 256, 16, 160
    stride = top // page
    pages = B * stride + 1
    g = torch.Generator().manual_seed(2)
    tables = torch.randperm(pages, generator=g)[: B * stride].view(B, stride).int().to(dev)
    kc = torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    ks, vs = torch.tensor([0.01], device=dev), torch.tensor([0.01], device=dev)
    index = torch.zeros(pages, page // 4, Hkv, D, dtype=torch.int8, device=dev)
    scale = torch.zeros(pages, page // 4, device=dev)
    freq = (1e4 ** (-torch.arange(32) / 32)).float().to(dev)
    lens = torch.tensor([40, 2, 101], dtype=torch.int32, device=dev)
    starts = (torch.arange(B + 1) * R).int().to(dev)
    # The tokens that are in the cache before the steps.
    first = torch.randn(143, 8, D, generator=g).half().to(dev)
    cuda_lib.cache_write_e4m3(None, first[:, 6:7], first[:, 7:], kc, vc, ks, vs, tables, lens, top,
                              row_starts=torch.tensor([0, 40, 42, 143], dtype=torch.int32,
                                                      device=dev))
    qkv = torch.zeros(B * R + 2, 8, D, dtype=torch.float16, device=dev)
    q_out = torch.full((B * R + 2, Hq, D), 7.0, dtype=torch.float16, device=dev)
    out = torch.zeros(B, R, Hq, D, dtype=torch.float16, device=dev)

    def step():
        cuda_lib.cache_write_e4m3(qkv[:, :6], qkv[:, 6:7], qkv[:, 7:], kc, vc, ks, vs, tables,
                                  lens, top, inv_freq=freq, row_starts=starts, q_out=q_out)
        cuda_lib.block_index_e4m3(kc, ks, tables, lens, top, B * R + 2, index, scale,
                                  row_starts=starts)
        cuda_lib.paged_e4m3_batch(q_out[: B * R].view(B, R, Hq, D), kc, vc, ks, vs, tables, lens,
                                  top, out=out)

    lens += R
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        lens += R
        qkv.copy_(torch.randn(qkv.shape, generator=g).half())
        graph.replay()
        torch.cuda.synchronize()
        assert cuda_lib.device_error() == 0
        assert (q_out[B * R:] == 7).all()
        for b in range(B):
            n = int(lens[b])
            for j in range(R):
                p = n - R + j
                y, m = ref.norm_rotate(qkv[b * R + j, :6].cpu().double().numpy(), None, 0,
                                       freq.cpu().numpy(), False, p)
                d = np.abs(q_out[b * R + j].cpu().double().numpy() - y)
                assert (d <= 2.0 ** -11 * np.abs(y) + 2.0 ** -25 + 2.0 ** -18 * m).all()
                if p % 4 == 3:
                    slot = int(tables[b, p // page]) * page + p % page
                    keys = ref.decode(kc.view(-1, 4, D)[slot // 4])
                    codes, sc = ref.summary(ref.block_sums(keys), ks.cpu().numpy()[0])
                    assert np.array_equal(index.view(-1, D)[slot // 4].cpu().numpy(), codes)
                    assert float(scale.view(-1)[slot // 4]) == float(sc)
            want = oracle.paged_e4m3(q_out[b * R:(b + 1) * R].cpu(), kc.cpu(), vc.cpu(),
                                     float(ks), float(vs), tables[b].cpu(), n, 1 / 16)
            _close(out[b], want)


def test_side_stream_and_eager_order(cuda_lib):
    """The whole step on a stream of its own gives what the default stream gives."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(6)
    qkv = torch.randn(90, 8, 256, generator=g).half().to(dev)
    got = []
    for s in (None, torch.cuda.Stream()):
        c = Cache(90, 16, 1, 256, True, seed=1)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            q = c.write(cuda_lib, qkv, 6, 1, 90)
            sel, cnt = cuda_lib.select_blocks(q, c.index, c.index_scale, c.table, 90, 8)
            out = cuda_lib.sparse_blocks_e4m3(q, c.k, c.v, c.ks, c.vs, c.table, sel, cnt, 90)
        torch.cuda.synchronize()
        got.append((q, c.k, c.v, c.index, c.index_scale, sel, cnt, out))
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once(cuda_lib):
    """Writes, reads and summaries need no workspace: two sequences on two streams
    at once, over one cache, give what they give one after the other."""
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(9)
    qkv = [torch.randn(700, 8, 256, generator=g).half().to(dev) for _ in range(2)]
    got = []
    for together in (False, True):
        c = Cache(1600, 16, 1, 256, True, seed=3)
        tables = [c.table[:50].contiguous().view(1, -1), c.table[50:].contiguous().view(1, -1)]
        lens = [torch.tensor([n], dtype=torch.int32, device=dev) for n in (700, 790)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream() if together else None]
        streams[1] = streams[1] or streams[0]
        outs = [[torch.zeros(700, 1, 256, dtype=torch.float16, device=dev) for _ in range(2)]
                + [torch.zeros(700, 6, 256, dtype=torch.float16, device=dev)] for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(3):
            for x, t, n, s, o in zip(qkv, tables, lens, streams, outs):
                where = (t, n, 800)
                cuda_lib.cache_write_e4m3(x[:, :6], x[:, 6:7], x[:, 7:], c.k, c.v, c.ks, c.vs,
                                          *where, q_out=o[2], stream=s)
                cuda_lib.block_index_e4m3(c.k, c.ks, *where, 700, c.index, c.index_scale, stream=s)
                cuda_lib.cache_read_e4m3(c.k, c.v, c.ks, c.vs, *where, 700, k_out=o[0], v_out=o[1],
                                         stream=s)
        torch.cuda.synchronize()
        assert cuda_lib.device_error() == 0
        got.append([c.k, c.v, c.index, c.index_scale] + outs[0] + outs[1])
    for a, b in zip(*got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
