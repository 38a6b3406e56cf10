"""GPU tests of the tails over the 4-bit and the windowed E4M3 cache at every number of
packed rows (R * Hq / Hkv) that a kernel of its own serves: up to 8, 16, 24, 32 and 48, for
both head sizes and both caches."""

import random

import pytest

from test_gpu_window import Tails

pytestmark = pytest.mark.gpu

# R, Hq, Hkv by head size: the packed rows of each kernel, full and not.
ROWS = {
    256: [(1, 6, 1), (1, 16, 2), (2, 6, 1), (8, 4, 2), (3, 6, 1), (6, 8, 2), (5, 6, 1), (4, 8, 1),
          (31, 1, 1), (6, 6, 1), (7, 6, 1), (8, 6, 1), (48, 2, 2)],
    128: [(1, 8, 1), (7, 2, 2), (3, 4, 1), (2, 16, 2), (3, 6, 1), (3, 16, 2), (5, 6, 1), (4, 8, 1),
          (2, 32, 2), (11, 3, 1), (5, 8, 1), (6, 16, 2), (3, 16, 1)],
}
SHAPES = [(R, Hq, Hkv, D) for D, rows in ROWS.items() for R, Hq, Hkv in rows]
PACKED = {(D, R * Hq // Hkv) for R, Hq, Hkv, D in SHAPES}


def test_every_kernel_is_met():
    """Of each head size and each number of eights, a full and another one."""
    for D in (256, 128):
        for low, high in ((1, 8), (9, 16), (17, 24), (25, 32), (33, 48)):
            assert len([n for d, n in PACKED if d == D and low <= n <= high]) >= 2, (D, high)
            assert (D, high) in PACKED


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged_batch(cuda_lib, shape, fp4):
    """Lengths of no whole tile and page, shorter than the rows, and zero; with a window and
    sinks, and over the whole context."""
    R, Hq, Hkv, D = shape
    t = Tails(fp4, R, Hq, Hkv, D, 16, [517, 64, R - 1, 0, 193, 1, 130], seed=R * Hq + D)
    args = t.args()
    for window, sinks in ((150, 20), (0, 0)):
        if window or fp4:
            out = t.run(cuda_lib, window, sinks, D ** -0.5, args)
            assert cuda_lib.device_error() == 0
            t.check(out, window, sinks, D ** -0.5)


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("page", [8, 256])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in (4, 5, 8, 3)])
def test_shortest_and_longest_pages(cuda_lib, shape, page, fp4):
    R, Hq, Hkv, D = shape
    t = Tails(fp4, R, Hq, Hkv, D, page, [1001, 333, 65], seed=R + page)
    out = t.run(cuda_lib, 301, 67, D ** -0.5)
    assert cuda_lib.device_error() == 0
    t.check(out, 301, 67, D ** -0.5)


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("R,Hq,Hkv,D", [(5, 6, 1, 256), (4, 8, 1, 128), (3, 6, 1, 128),
                                        (8, 6, 1, 256), (6, 8, 1, 128)])
def test_more_sequences_than_a_warp_has_lanes(cuda_lib, R, Hq, Hkv, D, fp4):
    rnd = random.Random(R * D)
    lens = [rnd.choice([0, 1, 2, 700, rnd.randint(1, 1500)]) for _ in range(70)]
    t = Tails(fp4, R, Hq, Hkv, D, 16, lens, seed=R)
    out = t.run(cuda_lib, 900, 5, 0.07)
    assert cuda_lib.device_error() == 0
    t.check(out, 900, 5, 0.07, only=range(0, 70, 3))


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("R,Hq,Hkv,D", [(5, 6, 1, 256), (4, 8, 1, 128), (3, 6, 1, 128),
                                        (8, 6, 1, 256)])
def test_one_context_in_many_pieces(cuda_lib, R, Hq, Hkv, D, fp4):
    t = Tails(fp4, R, Hq, Hkv, D, 16, [11003], seed=R + 1)
    out = t.run(cuda_lib, 9500, 70, D ** -0.5)
    assert cuda_lib.device_error() == 0
    t.check(out, 9500, 70, D ** -0.5)
