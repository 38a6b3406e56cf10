"""How many keys a call of the batched 4-bit and windowed E4M3 tails may name, as the header
says: batch * Hkv * max_ctx_len < 2^35 (nothing here reaches a GPU: the window is refused
behind the limits)."""

import pytest

from long_context_causal_gqa_gb300 import binding, build_lib
from test_cache_ops_host import FAKE, INVALID, UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("batch,Hkv,max_ctx,want", [
    (1024, 64, 2 ** 19, UNSUPPORTED),
    (1024, 64, 2 ** 19 - 1, INVALID),         # (more whole tiles of 64 keys than 2^29 - 1)
    (1024, 64, 2 ** 19 + 129, UNSUPPORTED),
    (1, 64, 2 ** 29, UNSUPPORTED),
    (1, 64, 2 ** 29 - 65, INVALID),
    (1024, 1, 2 ** 25, UNSUPPORTED),
    (1023, 1, 2 ** 25, INVALID),
    (16, 1, 2 ** 31 - 256, INVALID),
    (17, 1, 2 ** 31 - 256, UNSUPPORTED),
])
@pytest.mark.parametrize("D,group", [(256, 1), (128, 1), (128, 33)])
def test_keys_of_a_call(lib, D, group, batch, Hkv, max_ctx, want, fp4):
    if group > 1 and Hkv > 1:
        group = 1
    page = 256
    pages = -(-max_ctx // page)
    fn = lib.gqa_attn_paged_fp4 if fp4 else lib.gqa_attn_paged_e4m3_window
    assert fn(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, pages, pages, page, FAKE, max_ctx, batch, 1,
              Hkv * group, Hkv, D, 0.0625, -1, 0, FAKE, None) == want
