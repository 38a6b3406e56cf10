"""GPU tests of the block selection: equal, id by id, to the plain form in
tests/cache_reference.py (the scores are whole numbers times one scale, so
there is nothing to tolerate)."""

import numpy as np
import pytest
import torch

import cache_reference as ref

pytestmark = pytest.mark.gpu


def make(seed, rows, ctx, page, Hq, Hkv, D, spare=2):
    g = torch.Generator().manual_seed(seed)
    used = -(-ctx // page)
    pages = used + spare
    q = torch.randn(rows, Hq, D, generator=g).half()
    index = torch.randint(-127, 128, (pages, page // 4, Hkv, D), generator=g, dtype=torch.int8)
    scale = torch.rand(pages, page // 4, generator=g)
    table = torch.randperm(pages, generator=g)[:used].int()
    return q, index, scale, table


def run(lib, q, index, scale, table, ctx, max_sel, first, last, **kw):
    dev = torch.device("cuda")
    got = lib.select_blocks(q.to(dev), index.to(dev), scale.to(dev), table.to(dev), ctx, max_sel,
                            n_first=first, n_last=last, **kw)
    torch.cuda.synchronize()
    return got


def check(lib, q, index, scale, table, page, ctx, max_sel, first, last):
    sel, cnt = run(lib, q, index, scale, table, ctx, max_sel, first, last)
    want_sel, want_cnt = ref.select(q, index, scale, table, page, ctx, max_sel, first, last)
    assert np.array_equal(cnt.cpu().numpy(), want_cnt)
    bad = np.nonzero((sel.cpu().numpy() != want_sel).any(1))[0]
    assert len(bad) == 0, (bad[:5], sel[bad[0]].tolist()[:40], want_sel[bad[0]].tolist()[:40])


CASES = [
    # rows, ctx, page, Hq, Hkv, D, max_sel, first, last
    (1, 1, 16, 6, 1, 256, 1, 0, 1),
    (1, 4, 16, 6, 1, 256, 4, 0, 1),
    (4, 4, 8, 6, 1, 256, 1, 0, 1),
    (5, 41, 8, 6, 1, 256, 3, 1, 1),
    (41, 41, 16, 6, 2, 256, 5, 1, 2),
    (1, 4096, 16, 6, 1, 256, 128, 1, 2),
    (3, 1001, 32, 16, 4, 128, 16, 4, 12),       # only first and last blocks
    (8, 3001, 16, 6, 1, 256, 64, 0, 1),
    (9, 3002, 256, 8, 1, 128, 33, 2, 3),
    (31, 2003, 64, 64, 4, 256, 40, 1, 1),
    (33, 515, 16, 3, 3, 128, 200, 0, 1),        # most rows see fewer than max_sel
    (64, 2048, 16, 6, 1, 256, 16, 0, 1),
    (100, 3001, 16, 6, 1, 256, 128, 1, 4),
    (129, 1030, 16, 6, 6, 128, 7, 0, 2),
    (257, 5003, 128, 7, 7, 128, 100, 3, 5),
    (300, 9999, 16, 8, 8, 128, 512, 1, 1),
    (130, 20011, 16, 5, 1, 128, 64, 0, 1),
    (1, 100003, 16, 6, 1, 256, 2000, 0, 1),
    (700, 700, 16, 6, 1, 256, 12, 1, 3),        # from the first position on
    (32, 9003, 16, 6, 1, 256, 30, 1, 2),        # the most rows of the path for few
    (33, 9003, 16, 6, 1, 256, 30, 1, 2),
    (8, 5001, 32, 8, 8, 128, 70, 0, 1),
    (9, 5001, 32, 8, 8, 128, 70, 0, 1),
    (20, 4999, 16, 4, 4, 128, 25, 2, 2),
    (70, 66001, 16, 2, 1, 128, 1700, 2, 2),     # a row's pick with all scores, long rows
    (330, 18005, 64, 2, 1, 128, 900, 0, 3),     # and many
    (33, 9001, 16, 6, 1, 256, 64, 0, 1),
    (300, 12007, 32, 8, 2, 128, 20, 2, 3),
    (257, 9002, 16, 8, 4, 256, 9, 0, 2),        # width 1024
    (40, 16390, 64, 6, 6, 128, 200, 17, 30),
    (130, 9999, 256, 1, 1, 128, 3, 1, 1),
    (60, 40001, 16, 6, 1, 256, 600, 0, 1),
    (2500, 2500 + 7000, 16, 2, 1, 128, 32, 1, 1),
    # Many scores and many blocks for what is taken: candidates by the bound of a
    # sample, of every block to every eighth.
    (2000, 13001, 16, 6, 1, 128, 32, 1, 1),
    (2700, 6203, 16, 2, 1, 128, 2, 0, 1),       # the fewest blocks, spaced widest
    (33, 98405, 16, 6, 1, 256, 64, 0, 1),
    (257, 98402, 32, 8, 4, 256, 200, 17, 30),   # width 1024
    (40, 99999, 64, 6, 6, 128, 9, 1, 1),
    (64, 110001, 16, 1, 1, 128, 2048, 5, 9),
    (300, 100001, 256, 2, 1, 128, 600, 0, 1),
    (35, 120001, 8, 4, 1, 128, 1, 0, 1),
    (47, 100003, 16, 6, 1, 256, 500, 250, 249),
]


@pytest.mark.parametrize("case", CASES)
def test_select_matches_the_definition(cuda_lib, case):
    rows, ctx, page, Hq, Hkv, D, max_sel, first, last = case
    q, index, scale, table = make(rows + ctx, rows, ctx, page, Hq, Hkv, D)
    check(cuda_lib, q, index, scale, table, page, ctx, max_sel, first, last)
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("rows,ctx", [(1, 4000), (7, 4000), (40, 4000), (200, 4000), (70, 10000), (40, 99000)])
@pytest.mark.parametrize("kind", ["equal", "few", "zero_scale", "zero_query", "two_values"])
def test_ties_go_to_the_lowest_id(cuda_lib, rows, ctx, kind):
    page = 16
    q, index, scale, table = make(rows, rows, ctx, page, 6, 1, 256)
    if kind == "equal":        # every block the same summary
        index[:] = index[0, 0]
        scale[:] = 0.5
    elif kind == "few":        # four distinct blocks over and over
        index[:] = index[:1]
        scale[:] = 0.25
    elif kind == "zero_scale":
        scale[:] = 0           # +0 and -0 are one score
    elif kind == "zero_query":
        q[:] = 0
    else:                      # one block in three beats the rest, more than fit
        index[:] = 1
        scale[:] = 1.0
        scale.view(-1)[::3] = 2.0
        q = q.abs()
    check(cuda_lib, q, index, scale, table, page, ctx, 50, 1, 2)
    check(cuda_lib, q, index, scale, table, page, ctx, 9, 0, 1)   # id 0 among the equal ones


@pytest.mark.parametrize("rows,ctx", [(2, 3000), (150, 3000), (50, 12000), (34, 99000)])
def test_extreme_values(cuda_lib, rows, ctx):
    """Largest codes, huge / tiny / infinite / NaN scales, infinite and NaN queries."""
    page = 16
    q, index, scale, table = make(3, rows, ctx, page, 8, 4, 256)
    index[1] = 127
    index[2] = -127
    index[3] = -128            # not a code the index writes; an int8 all the same
    scale[4] = 1e30
    scale[5] = 1e-38
    scale[6] = float("inf")
    scale[7, 0] = float("nan")
    q[0] = 65504.0
    q[1, 3, 7] = float("inf")
    if rows > 5:
        q[2, 0, 0] = float("nan")
        q[3] = 6e-8            # subnormal queries
        q[4] = -65504.0
        q[5, :, 0] = 60000.0   # one value far above the rest
    check(cuda_lib, q, index, scale, table, page, ctx, 30, 0, 1)


@pytest.mark.parametrize("rows,ctx", [(3, 2002), (200, 2002), (100, 11002), (100, 98502)])
def test_unfinished_and_unused_blocks_do_not_matter(cuda_lib, rows, ctx):
    """What lies at or behind a row's own block, and in pages nobody names,
    changes nothing (a step's later rows write their blocks' summaries first)."""
    page = 16
    q, index, scale, table = make(8, rows, ctx, page, 6, 1, 256)
    a = run(cuda_lib, q, index, scale, table, ctx, 40, 1, 2)
    nb = (ctx + 3) // 4
    first_own = (ctx - rows) // 4
    used = torch.zeros(scale.shape, dtype=torch.bool)
    for b in range(nb):
        used[int(table[b * 4 // page]), b % (page // 4)] = True
    scale2, index2 = scale.clone(), index.clone()
    scale2[~used] = float("nan")
    last = int(table[(nb - 1) * 4 // page]), (nb - 1) % (page // 4)
    scale2[last] = float("inf")       # the last, unfinished block
    index2[last] = 127
    b = run(cuda_lib, q, index2, scale2, table, ctx, 40, 1, 2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # Row by row: a later row's blocks do not reach an earlier one.
    c = run(cuda_lib, q[:1], index, scale, table, ctx - rows + 1, 40, 1, 2)
    assert torch.equal(a[0][:1], c[0]) and first_own + 1 >= int(c[0].max()) + 1


@pytest.mark.parametrize("ctx", [12000, 100000])
@pytest.mark.parametrize("kind", ["most_nan", "clustered", "rising", "walk", "period"])
def test_scores_that_defeat_the_sample(cuda_lib, kind, ctx):
    """Fewer numbers than are taken, all the best in one stretch, scores that
    rise with the position, neighbours that are all but equal: rows whose
    candidates run out or do not fit."""
    rows, page = 64, 16
    q, index, scale, table = make(17, rows, ctx, page, 6, 1, 256)
    b = torch.arange(ctx // 4)
    at = table[b * 4 // page].long(), b % (page // 4)
    if kind == "most_nan":
        scale[at] = torch.where(b % 300 == 5, 1.0, float("nan"))
    elif kind == "clustered":
        q = q.abs()
        index[at[0], at[1]] = torch.where((b >= 1000) & (b < 1500), 100, 1)[:, None, None].to(
            torch.int8).expand(-1, 1, 256)
        scale[at] = 1 + b.float() * 1e-4
    elif kind == "period":     # three of four blocks beat the fourth
        scale[at] = torch.where(b % 4 == 0, 0.1, 1.0) * scale[at]
    elif kind == "walk":
        g = torch.Generator().manual_seed(5)
        walk = torch.randn(len(b), 1, 256, generator=g).cumsum(0) * 2
        index[at] = (walk - walk.mean(0)).clamp(-127, 127).to(torch.int8)
        scale[at] = 1.0
    else:
        q = q.abs()
        index[:] = 3
        scale[at] = 1 + b.float()
    check(cuda_lib, q, index, scale, table, page, ctx, 60, 1, 2)


def test_rows_do_not_depend_on_the_launch(cuda_lib):
    """A row's selection is the same alone, in a small call and in a large one."""
    ctx, page, rows = 6007, 32, 300
    q, index, scale, table = make(21, rows, ctx, page, 6, 2, 128)
    sel, cnt = run(cuda_lib, q, index, scale, table, ctx, 64, 1, 1)
    for r0, n in ((0, 1), (10, 5), (37, 64), (170, 130)):
        end = ctx - rows + r0 + n
        s, c = run(cuda_lib, q[r0:r0 + n], index, scale, table, end, 64, 1, 1)
        assert torch.equal(s, sel[r0:r0 + n]) and torch.equal(c, cnt[r0:r0 + n])


@pytest.mark.parametrize("rows", [4, 200])
def test_bad_pages_read_page_zero(cuda_lib, rows):
    ctx, page = 1500, 16
    q, index, scale, table = make(5, rows, ctx, page, 6, 1, 256)
    bad = table.clone()
    bad[7], bad[20] = -3, index.shape[0]
    mapped = table.clone()
    mapped[7] = mapped[20] = 0
    a = run(cuda_lib, q, index, scale, bad, ctx, 30, 0, 1)
    assert cuda_lib.device_error() == cuda_lib.DEVERR_BAD_PAGE_ID
    b = run(cuda_lib, q, index, scale, mapped, ctx, 30, 0, 1)
    assert cuda_lib.device_error() == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("rows,ctx,Hq,D,max_sel", [
    (4096, 8192, 6, 256, 128), (1000, 65537, 6, 256, 128), (3, 1000001, 6, 256, 128),
    (20000, 20003, 1, 128, 700),     # more scores than are held at once
    (30000, 40001, 1, 128, 1240),    # more maxima
    (13100, 330001, 1, 128, 512),    # more candidates
    (70000, 70001, 1, 128, 128),     # more rows than a launch takes
])
def test_large_calls_sampled_rows(cuda_lib, rows, ctx, Hq, D, max_sel):
    page = 16
    q, index, scale, table = make(rows, rows, ctx, page, Hq, 1, D)
    sel, cnt = run(cuda_lib, q, index, scale, table, ctx, max_sel, 2, 3)
    pick = sorted({0, 1, 2, 63, 64, 127, 128, 6143, 6144, 6400, 11263, 11264, 65535, 65536,
                   rows // 2, rows - 2, rows - 1} & set(range(rows)))
    for r in pick:
        end = ctx - rows + r + 1
        s, c = ref.select(q[r:r + 1], index, scale, table, page, end, max_sel, 2, 3)
        assert np.array_equal(sel[r].cpu().numpy(), s[0]) and int(cnt[r]) == c[0]
    # Every row: ids ascending, distinct and visible.
    d = sel.long()
    pos = torch.arange(rows, device=d.device) + ctx - rows
    live = d >= 0
    assert torch.equal(live.sum(1), cnt.long())
    assert ((d[:, 1:] > d[:, :-1]) | ~live[:, 1:]).all()
    assert (d <= (pos // 4)[:, None]).all()


def test_graph_replay_and_streams(cuda_lib):
    dev = torch.device("cuda")
    ctx, page = 9001, 16
    for rows in (2, 200):
        q, index, scale, table = (x.to(dev) for x in make(4, rows, ctx, page, 6, 1, 256))
        ref_sel, ref_cnt = cuda_lib.select_blocks(q, index, scale, table, ctx, 64)
        sel, cnt = torch.zeros_like(ref_sel), torch.zeros_like(ref_cnt)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cuda_lib.select_blocks(q, index, scale, table, ctx, 64, sel_idx=sel, sel_cnt=cnt)
        for _ in range(3):
            sel.zero_()
            cnt.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(sel, ref_sel) and torch.equal(cnt, ref_cnt)
        s = torch.cuda.Stream()
        sel.zero_()
        torch.cuda.synchronize()
        cuda_lib.select_blocks(q, index, scale, table, ctx, 64, sel_idx=sel, sel_cnt=cnt, stream=s)
        s.synchronize()
        assert torch.equal(sel, ref_sel)
    assert cuda_lib.device_error() == 0


def test_needs_its_workspace(cuda_lib):
    """Through the C entry, a workspace that is too small is refused."""
    dev = torch.device("cuda")
    q, index, scale, table = (x.to(dev) for x in make(4, 64, 9001, 16, 6, 1, 256))
    need = cuda_lib.workspace_bytes(cuda_lib.KIND_SELECT_BLOCKS, 64, 9001)
    assert need > 4096
    keep = cuda_lib._ws.get(0)
    small = torch.empty(4096, dtype=torch.uint8, device=dev)
    cuda_lib.register_workspace(small)
    sel = torch.zeros(64, 8, dtype=torch.int32, device=dev)
    cnt = torch.zeros(64, dtype=torch.int32, device=dev)
    st = cuda_lib.load().gqa_select_blocks(
        q.data_ptr(), index.data_ptr(), scale.data_ptr(), table.data_ptr(), index.shape[0], 16,
        9001, 64, 6, 1, 256, 8, 0, 1, sel.data_ptr(), cnt.data_ptr(), None)
    assert st == cuda_lib.GQA_ERR_WORKSPACE
    if keep is not None:
        cuda_lib.register_workspace(keep)


def test_workspace_of_a_longer_context_is_no_smaller(cuda_lib):
    """A workspace sized for the last block of a context serves every call on it."""
    for rows in (1, 32, 33, 300, 4096):
        sizes = [cuda_lib.workspace_bytes(cuda_lib.KIND_SELECT_BLOCKS, rows, c)
                 for c in sorted({rows, rows + 1, 5000, 8191, 8200, 33000, 98300, 98400, 261888,
                                  3000000}) if c >= rows]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_captured_call_outlives_a_growing_workspace(cuda_lib):
    """A later call that needs a larger workspace leaves a captured one its own."""
    dev = torch.device("cuda")
    ctx = 20001
    q, index, scale, table = (x.to(dev) for x in make(4, 400, ctx, 16, 6, 1, 256))
    want = cuda_lib.select_blocks(q, index, scale, table, ctx, 32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sel, cnt = cuda_lib.select_blocks(q, index, scale, table, ctx, 32)
    before = cuda_lib.ensure_workspace(1)
    cuda_lib.ensure_workspace(before.numel() + 1)
    assert cuda_lib.ensure_workspace(1).data_ptr() != before.data_ptr()
    # What memory the allocator has to give is taken and filled.
    rest = [torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(24)]
    for _ in range(2):
        other = cuda_lib.select_blocks(q, index, scale, table, ctx, 32)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, other, (sel, cnt)):
            assert torch.equal(a, b) and torch.equal(a, c)
    del rest
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("rows,ctx", [(1, 300000), (3, 300004), (8, 300036)])
def test_most_blocks_of_a_long_context(cuda_lib, rows, ctx):
    """The largest max_sel over contexts whose maxima are an odd number or an even
    one: a row's keys, maxima and bits fill its CTA's shared memory."""
    page = 32
    q, index, scale, table = make(ctx, rows, ctx, page, 6, 1, 256)
    check(cuda_lib, q, index, scale, table, page, ctx, 2048, 1, 1)
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("rows,ctx,Hq,Hkv,D,max_sel", [
    (1, 9001, 6, 1, 256, 64), (20, 9001, 8, 1, 128, 64), (32, 70001, 6, 1, 256, 128),
    (300, 9001, 6, 1, 256, 64), (9, 9001, 8, 4, 128, 512), (257, 70001, 12, 2, 128, 128),
    (2500, 40001, 6, 1, 256, 128)])
def test_workspace_goes_by_the_heads_of_the_index(cuda_lib, monkeypatch, rows, ctx, Hq, Hkv, D,
                                                  max_sel):
    """The wrapper asks for what the index's own width takes, and that is enough."""
    q, index, scale, table = make(ctx, rows, ctx, 16, Hq, Hkv, D)
    want, _ = run(cuda_lib, q, index, scale, table, ctx, max_sel, 1, 2)
    keep, asked = cuda_lib.ensure_workspace(1), []
    none = torch.empty(4096, dtype=torch.uint8, device="cuda")

    def ensure(n, device=None):
        asked.append(n)
        cuda_lib.register_workspace(torch.empty(n, dtype=torch.uint8, device="cuda"))

    monkeypatch.setattr(cuda_lib, "ensure_workspace", ensure)
    cuda_lib.register_workspace(none)
    try:
        got, _ = run(cuda_lib, q, index, scale, table, ctx, max_sel, 1, 2)
    finally:
        cuda_lib.register_workspace(keep)
    assert asked == [cuda_lib.workspace_bytes(cuda_lib.KIND_SELECT_BLOCKS, rows, ctx, Hkv, D)]
    assert asked[0] <= cuda_lib.workspace_bytes(cuda_lib.KIND_SELECT_BLOCKS, rows, ctx, Hq, D)
    assert torch.equal(got, want)
    assert cuda_lib.device_error() == 0
