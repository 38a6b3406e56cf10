"""GPU tests of which pages the tails of gqa_attn_paged_fp4 and gqa_attn_paged_e4m3_window
look up: those some row sees, and no others, wherever a tile of the kernels ends."""

import numpy as np
import pytest
import torch

import window_reference as ref
from test_gpu_window import Tails

pytestmark = pytest.mark.gpu

# R, Hq, Hkv, D, lens, window, sinks: up to eight packed rows and more, tiles of 128 and 64
# keys; windows and sinks that begin and end anywhere in a tile, sinks that hold nothing,
# that reach the window, that end with a page; a context shorter than its window, and none.
SHAPES = [
    (1, 6, 1, 256, (1000, 517, 90, 0), 150, 20),
    (2, 4, 2, 128, (1500, 700, 130), 129, 0),
    (3, 6, 1, 256, (1000, 500, 2), 150, 20),
    (5, 6, 1, 256, (1311, 640, 257), 333, 64),
    (8, 6, 1, 256, (1290, 1029), 300, 131),
    (4, 8, 1, 128, (1153, 2049), 7, 1),
    (6, 8, 1, 128, (900, 1301), 500, 380),
]


def unseen_pages(t, b, window, sinks):
    """Logical pages of sequence b, in front of the context's end, without a key that some
    row sees."""
    n = t.lens[b]
    seen = ref.visible(range(n - t.R, n), n, window, sinks).any(0)
    return [p for p in range(-(-n // t.page)) if not seen[p * t.page:(p + 1) * t.page].any()]


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("shape", SHAPES)
def test_pages_no_row_sees_are_not_looked_up(cuda_lib, shape, page, fp4):
    """Their entries may be out of range, and so may those behind the context: nothing is
    flagged and the result is the same."""
    R, Hq, Hkv, D, lens, window, sinks = shape
    t = Tails(fp4, R, Hq, Hkv, D, page, lens, seed=page + R, max_ctx=max(lens) + 300)
    args = t.args()
    clean = t.run(cuda_lib, window, sinks, 0.0625, args)
    t.check(clean, window, sinks, 0.0625)
    assert cuda_lib.device_error() == 0
    table = t.tables.copy()
    spoiled = 0
    for b, n in enumerate(lens):
        for p in unseen_pages(t, b, window, sinks):
            table[b, p] = (-1, t.pages, 10 ** 6, -2 ** 31)[p % 4]
            spoiled += 1
        table[b, -(-n // page):] = -1
    assert spoiled
    args[5] = torch.tensor(table, dtype=torch.int32, device="cuda")
    assert torch.equal(t.run(cuda_lib, window, sinks, 0.0625, args), clean)
    assert cuda_lib.device_error() == 0


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("R", [1, 3, 8])
def test_every_page_some_row_sees_is_looked_up(cuda_lib, R, page, fp4):
    """One bad entry, for the first and the last page that the window and the sinks touch,
    is flagged each time; the pages beside them are not."""
    n, window, sinks = 1100, 205, 70
    t = Tails(fp4, R, 6, 1, 256, page, [n], seed=page)
    lo = n - R + 1 - window                       # the first row's first key
    touched = {0, (sinks - 1) // page, lo // page, (n - 1) // page}
    beside = set(unseen_pages(t, 0, window, sinks)) & {(sinks - 1) // page + 1, lo // page - 1}
    assert beside
    for p in sorted(touched | beside):
        args = t.args()
        args[5][0, p] = -1
        out = t.run(cuda_lib, window, sinks, 0.0625, args)
        assert cuda_lib.device_error() == (cuda_lib.DEVERR_BAD_PAGE_ID if p in touched else 0), p
        if p in beside:
            t.check(out, window, sinks, 0.0625)


@pytest.mark.parametrize("fp4", [True, False])
def test_pages_are_given_back_while_a_graph_replays(cuda_lib, fp4):
    """A sequence grows under one captured graph, and its pages' entries go to -1 as they
    leave the window."""
    t = Tails(fp4, 2, 6, 1, 256, 16, [900], seed=17)
    window, sinks = 100, 4
    args = t.args()
    out = torch.zeros(t.q.shape, dtype=torch.float16, device="cuda")
    t.run(cuda_lib, window, sinks, 0.0625, args, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.run(cuda_lib, window, sinks, 0.0625, args, out=out)
    table = t.tables.copy()
    for n in (2, 50, 101, 118, 119, 300, 513, 900):
        t.lens = [n]
        for p in unseen_pages(t, 0, window, sinks):
            table[0, p] = -1
        args[5].copy_(torch.from_numpy(table))
        args[6].copy_(torch.tensor([n]))
        g.replay()
        t.check(out, window, sinks, 0.0625)
        assert cuda_lib.device_error() == 0, n
    assert (table == -1).sum() == len(unseen_pages(t, 0, window, sinks)) > 40
    assert np.isfinite(out.cpu().numpy()).all()
