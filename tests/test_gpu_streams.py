"""GPU tests of the outputs that the binding allocates for a call on another
stream than the current one: their memory is that stream's, and what the current
stream does with them holds it back."""

import pytest
import torch

pytestmark = pytest.mark.gpu

SLEEP = 200_000_000     # clock cycles, about a tenth of a second


def calls(lib):
    """Every entry point that allocates its outputs, as functions of the stream."""
    dev = torch.device("cuda")
    n, page, D = 64, 16, 256
    half = torch.float16
    q, k, v = (torch.zeros(n, h, D, dtype=half, device=dev) for h in (6, 1, 1))
    k8 = torch.zeros(n, 1, D, dtype=torch.uint8, device=dev)
    c16 = torch.zeros(n // page, page, 1, D, dtype=half, device=dev)
    c8 = c16.to(torch.uint8)
    s = torch.ones(1, device=dev)
    table = torch.arange(n // page, dtype=torch.int32, device=dev)
    tables, lens = table.view(1, -1), torch.tensor([n], dtype=torch.int32, device=dev)
    index = torch.zeros(n // page, page // 4, 1, D, dtype=torch.int8, device=dev)
    scale = torch.zeros(n // page, page // 4, device=dev)
    sel = torch.zeros(n, 2, dtype=torch.int32, device=dev)
    cnt = torch.ones(n, dtype=torch.int32, device=dev)
    tail = q[:2].contiguous()
    at = (tables, lens, n)
    return {
        "prefill": lambda st: lib.prefill(q, k, v, stream=st),
        "prefill_e4m3": lambda st: lib.prefill_e4m3(q, k8, k8, s, s, stream=st),
        "paged": lambda st: lib.paged_e4m3(tail, c8, c8, s, s, table, n, stream=st),
        "paged_devctx": lambda st: lib.paged_e4m3_devctx(tail, c8, c8, s, s, table, lens, n,
                                                         stream=st),
        "paged_batch": lambda st: lib.paged_e4m3_batch(tail.view(1, 2, 6, D), c8, c8, s, s,
                                                       tables, lens, n, stream=st),
        "sparse": lambda st: lib.sparse_blocks(q, c16, c16, table, sel, cnt, n, stream=st),
        "sparse_e4m3": lambda st: lib.sparse_blocks_e4m3(q, c8, c8, s, s, table, sel, cnt, n,
                                                         stream=st),
        "write": lambda st: lib.cache_write(q, k, v, c16, c16, *at, stream=st),
        "write_e4m3": lambda st: lib.cache_write_e4m3(q, k, v, c8, c8, s, s, *at, stream=st),
        "read": lambda st: lib.cache_read(c16, c16, *at, n, stream=st),
        "read_codes": lambda st: lib.cache_read(c8, c8, *at, n, stream=st),
        "read_e4m3": lambda st: lib.cache_read_e4m3(c8, c8, s, s, *at, n, stream=st),
        "select": lambda st: lib.select_blocks(q, index, scale, table, n, 2, stream=st),
    }


NAMES = ("prefill", "prefill_e4m3", "paged", "paged_devctx", "paged_batch", "sparse",
         "sparse_e4m3", "write", "write_e4m3", "read", "read_codes", "read_e4m3", "select")


def outputs(got):
    return got if isinstance(got, tuple) else (got,)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_the_streams_own(cuda_lib, name):
    call = calls(cuda_lib)[name]
    side = torch.cuda.Stream()
    like = outputs(call(None))
    torch.cuda.synchronize()
    # Blocks of these sizes are free on the current stream, whose work may still
    # use them.
    freed = [torch.empty_like(x) for x in like for _ in range(8)]
    places = {x.data_ptr() for x in freed}
    del freed
    got = outputs(call(side))
    assert not places & {x.data_ptr() for x in got}
    # The current stream is still at work on the outputs when they are freed.
    side.synchronize()
    for x in got:
        x.add_(1)
    torch.cuda._sleep(1)        # (its first call loads it)
    torch.cuda._sleep(SLEEP)
    held = {x.data_ptr() for x in got}
    del got, x
    again = outputs(call(side))
    assert not held & {x.data_ptr() for x in again}
    torch.cuda.synchronize()
    for a, b in zip(outputs(call(None)), again):
        assert torch.equal(a, b)
    assert cuda_lib.device_error() == 0


def test_a_stream_that_is_only_a_handle(cuda_lib):
    class Handle:
        def __init__(self, stream):
            self.cuda_stream = stream.cuda_stream

    call = calls(cuda_lib)["read"]
    side = torch.cuda.Stream()
    got = outputs(call(Handle(side)))
    torch.cuda.synchronize()
    for a, b in zip(outputs(call(None)), got):
        assert torch.equal(a, b)
