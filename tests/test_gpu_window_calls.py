"""GPU tests of how the calls of the 4-bit cache and of the windows are made: the workspace
they ask for, other streams, captures behind other work."""

import pytest
import torch

from test_gpu_streams import SLEEP, outputs
from test_gpu_window import Tails

pytestmark = pytest.mark.gpu


def test_workspace_of_tails_does_not_ask_for_a_context(cuda_lib):
    """ctx_or_kv is unused: any value gives the same bytes, and they are enough."""
    lib = cuda_lib
    for R, Hq, D in ((1, 6, 256), (8, 6, 256), (4, 64, 128)):
        want = lib.workspace_bytes(lib.KIND_TAILS, R, 1, Hq, D)
        assert want > 0
        for ctx in (0, -1, R - 1, 10 ** 6, 2 ** 31 - 1, -2 ** 31):
            assert lib.workspace_bytes(lib.KIND_TAILS, R, ctx, Hq, D) == want
    for kind in (lib.KIND_PREFILL, lib.KIND_PAGED_E4M3, lib.KIND_PAGED_E4M3_BATCH,
                 lib.KIND_SPARSE, lib.KIND_SELECT_BLOCKS):
        assert lib.workspace_bytes(kind, 1, 0, 6, 256) == 0


def calls(lib):
    """The entry points of the 4-bit cache and of the windows, as functions of the stream."""
    dev = torch.device("cuda")
    n, page, D = 64, 16, 256
    q, k, v = (torch.zeros(n, h, D, dtype=torch.float16, device=dev) for h in (6, 1, 1))
    k8 = torch.zeros(n, 1, D, dtype=torch.uint8, device=dev)
    c8 = torch.zeros(n // page, page, 1, D, dtype=torch.uint8, device=dev)
    c4 = torch.zeros(n // page, 1, page, 9 * D // 16, dtype=torch.uint8, device=dev)
    s = torch.ones(1, device=dev)
    tables = torch.arange(n // page, dtype=torch.int32, device=dev).view(1, -1)
    at = (tables, torch.tensor([n], dtype=torch.int32, device=dev), n)
    tail = q[None, :2].contiguous()
    return {
        "write_fp4": lambda st: lib.cache_write_fp4(q, k, v, c4, c4.clone(), s, s, *at, stream=st),
        "read_fp4": lambda st: lib.cache_read_fp4(c4, c4, s, s, *at, n, stream=st),
        "paged_fp4": lambda st: lib.paged_fp4(tail, c4, c4, s, s, *at, window=9, stream=st),
        "paged_e4m3_window": lambda st: lib.paged_e4m3_window(tail, c8, c8, s, s, *at, 9,
                                                              stream=st),
        "prefill_window": lambda st: lib.prefill_window(q, k, v, 9, stream=st),
        "prefill_e4m3_window": lambda st: lib.prefill_e4m3_window(q, k8, k8, s, s, 9, stream=st),
    }


@pytest.mark.parametrize("name", ["write_fp4", "read_fp4", "paged_fp4", "paged_e4m3_window",
                                  "prefill_window", "prefill_e4m3_window"])
def test_outputs_are_the_streams_own(cuda_lib, name):
    """An output that the binding allocates for another stream is not handed out again while
    the current stream's work on it is under way."""
    call = calls(cuda_lib)[name]
    call(None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = outputs(call(side))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(1)        # (its first call loads it)
    torch.cuda._sleep(SLEEP)
    sizes = [(x.shape, x.dtype, x.data_ptr()) for x in got]
    copies = [x + 1 for x in got]
    del got
    with torch.cuda.stream(side):
        again = [torch.full(shape, 9, dtype=dtype, device="cuda") for shape, dtype, _ in sizes]
    torch.cuda.synchronize()
    assert all((c == 1).all() for c in copies) and all((x == 9).all() for x in again)


@pytest.mark.parametrize("fp4", [True, False])
def test_capture_behind_other_work(cuda_lib, fp4):
    """Calls captured behind a copy, behind a fill, and behind work of two joined streams:
    what they are launched behind is no kernel that they could overlap, or not the only one."""
    t = Tails(fp4, 2, 6, 1, 256, 16, [700, 333], seed=23)
    args = t.args()
    dev = torch.device("cuda")
    q0, lens0 = args[0].clone(), args[6].clone()
    k, v = (torch.randn(600, 1, 256, dtype=torch.float16, device=dev) for _ in "kv")
    rows = torch.randn(70, 6, 256, dtype=torch.float16, device=dev)
    out, pre = torch.zeros_like(q0), torch.zeros_like(rows)
    k1, v1, rows1 = (torch.zeros_like(x) for x in (k, v, rows))

    def step(fork):
        here = torch.cuda.current_stream()
        args[0].zero_()
        args[6].copy_(lens0)
        if fork is not None:
            fork.wait_stream(here)
            with torch.cuda.stream(fork):
                torch.mul(q0, 1, out=args[0])
            here.wait_stream(fork)
        else:
            args[0].copy_(q0)
        t.run(cuda_lib, 150, 3, 0.0625, args, out=out)
        k1.copy_(k)
        v1.copy_(v)
        if fork is not None:
            fork.wait_stream(here)
            with torch.cuda.stream(fork):
                rows1.copy_(rows)
            here.wait_stream(fork)
        else:
            torch.mul(rows, 1, out=rows1)
        cuda_lib.prefill_window(rows1, k1, v1, 200, sinks=4, out=pre)

    step(None)
    want, want_pre = out.clone(), pre.clone()
    t.check(want, 150, 3, 0.0625)
    for fork in (None, torch.cuda.Stream()):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(fork)
        for x in (out, pre, k1, v1, rows1, args[0], args[6]):
            x.zero_()
        for _ in range(3):
            g.replay()
        assert torch.equal(out, want) and torch.equal(pre, want_pre)
    assert cuda_lib.device_error() == 0
