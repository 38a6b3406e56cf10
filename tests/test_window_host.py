"""Refusals of the 4-bit cache's and the windowed entry points, and the plain forms'
own values: nothing here reaches a GPU."""


import numpy as np
import pytest
import torch

import window_reference as ref
from long_context_causal_gqa_gb300 import binding, build_lib
from test_cache_ops_host import FAKE, INVALID, ODD2, ODD8, P, ROW_REFUSALS, UNSUPPORTED, WriteArgs


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


TAIL_REFUSALS = [
    (dict(q=P(0)), INVALID), (dict(kc=P(0)), INVALID), (dict(vc=P(0)), INVALID),
    (dict(ks=P(0)), INVALID), (dict(vs=P(0)), INVALID), (dict(bt=P(0)), INVALID),
    (dict(ctx=P(0)), INVALID), (dict(out=P(0)), INVALID), (dict(q=ODD8), INVALID),
    (dict(kc=ODD8), INVALID), (dict(vc=ODD8), INVALID), (dict(out=ODD8), INVALID),
    (dict(ks=ODD2), INVALID), (dict(vs=ODD2), INVALID), (dict(bt=ODD2), INVALID),
    (dict(ctx=ODD2), INVALID), (dict(rows=0), INVALID), (dict(max_ctx=0), INVALID),
    (dict(pages=0), INVALID), (dict(batch=0), INVALID), (dict(stride=0), INVALID),
    (dict(max_ctx=129), INVALID), (dict(max_ctx=100, stride=6), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(sinks=-1), INVALID),
    (dict(rows=9), UNSUPPORTED), (dict(batch=1025), UNSUPPORTED), (dict(page=12), UNSUPPORTED),
    (dict(page=4), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(Hq=7, Hkv=2), UNSUPPORTED), (dict(Hq=65), UNSUPPORTED), (dict(Hkv=0), UNSUPPORTED),
    (dict(pages=1 << 27, page=16), UNSUPPORTED),
]


@pytest.mark.parametrize("fp4", [True, False])
@pytest.mark.parametrize("kw,want", TAIL_REFUSALS)
def test_windowed_tails_refuse(lib, kw, want, fp4):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, stride=8, pages=8, page=16,
             ctx=FAKE, max_ctx=100, batch=2, rows=2, Hq=6, Hkv=1, D=256, scale=0.0625, window=64,
             sinks=4, out=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    fn = lib.gqa_attn_paged_fp4 if fp4 else lib.gqa_attn_paged_e4m3_window
    assert fn(*a.values(), None) == want


def test_e4m3_tails_need_a_window(lib):
    args = [FAKE] * 6 + [8, 8, 16, FAKE, 100, 2, 2, 6, 1, 256, 0.0625, 0, 0, FAKE, None]
    assert lib.gqa_attn_paged_e4m3_window(*args) == INVALID


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(q=P(0)), INVALID), (dict(k=P(0)), INVALID), (dict(v=P(0)), INVALID),
    (dict(out=P(0)), INVALID), (dict(q=ODD8), INVALID), (dict(k=ODD8), INVALID),
    (dict(v=ODD8), INVALID), (dict(out=ODD8), INVALID), (dict(Q=0), INVALID),
    (dict(Q=17), INVALID), (dict(KV=0), INVALID), (dict(scale=-1.0), INVALID),
    (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(sinks=-1), INVALID),
    (dict(D=192), UNSUPPORTED), (dict(Hq=6, Hkv=4), UNSUPPORTED), (dict(Hq=66), UNSUPPORTED),
    (dict(Q=1 << 28, KV=1 << 28, Hq=8), INVALID)])
def test_windowed_prefills_refuse(lib, kw, want, e4m3):
    a = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, Q=8, KV=16, Hq=6, Hkv=1, D=256, scale=0.0625,
             window=4, sinks=1)
    assert not set(kw) - set(a)
    a.update(kw)
    first, rest = [a["q"], a["k"], a["v"]], list(a.values())[3:]
    if e4m3:
        assert lib.gqa_attn_prefill_e4m3_window(*first, FAKE, FAKE, *rest, None) == want
        assert lib.gqa_attn_prefill_e4m3_window(*first, P(0), FAKE, *rest, None) == INVALID
        assert lib.gqa_attn_prefill_e4m3_window(*first, FAKE, ODD2, *rest, None) == INVALID
    else:
        assert lib.gqa_attn_prefill_window(*first, *rest, None) == want


def _write4(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, qt=2048, qh=256, kt=2048, kh=256, vt=2048, vh=256,
             qw=FAKE, kw=FAKE, eps=1e-6, freq=FAKE, rot=64, inter=0, ks=FAKE, vs=FAKE, bt=FAKE,
             stride=8, pages=8, page=16, starts=P(0), ctx=FAKE, max_ctx=100, batch=2, tokens=4,
             Hq=6, Hkv=1, D=256, out=FAKE, kc=FAKE, vc=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    args = WriteArgs()
    for name, x in a.items():
        setattr(args, name, x)
    return lib.gqa_cache_write_fp4(bytes(args), None)


@pytest.mark.parametrize("kw,want", ROW_REFUSALS + [
    (dict(k=P(0)), INVALID), (dict(q=P(0)), INVALID), (dict(kc=ODD8), INVALID),
    (dict(vc=P(0)), INVALID), (dict(ks=P(0)), INVALID), (dict(vs=P(0)), INVALID),
    (dict(vs=ODD2), INVALID), (dict(kt=100), INVALID), (dict(eps=-1.0), INVALID),
    (dict(rot=8), UNSUPPORTED), (dict(rot=272), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED)])
def test_cache_write_fp4_refuses(lib, kw, want):
    assert _write4(lib, **kw) == want
    assert lib.gqa_cache_write_fp4(None, None) == INVALID


@pytest.mark.parametrize("kw,want", ROW_REFUSALS + [
    (dict(kc=P(0)), INVALID), (dict(vc=ODD8), INVALID), (dict(ko=P(0)), INVALID),
    (dict(vo=ODD8), INVALID), (dict(ks=P(0)), INVALID), (dict(vs=ODD2), INVALID)])
def test_cache_read_fp4_refuses(lib, kw, want):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, stride=8, pages=8, page=16,
             starts=P(0), ctx=FAKE, max_ctx=100, batch=2, tokens=4, Hkv=1, D=256, ko=FAKE, vo=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    assert lib.gqa_cache_read_fp4(*a.values(), None) == want


def test_workspace_bytes_refuse():
    lib = binding.load()
    assert lib.gqa_workspace_bytes(binding.KIND_TAILS, 49, 1, 6, 256) == 0
    assert lib.gqa_workspace_bytes(binding.KIND_TAILS, 0, 1, 6, 256) == 0
    assert lib.gqa_workspace_bytes(binding.KIND_TAILS, 1, 1, 6, 64) == 0


def test_binding_refuses_cpu_tensors():
    q3 = torch.zeros(4, 6, 256, dtype=torch.float16)
    q4 = torch.zeros(1, 4, 6, 256, dtype=torch.float16)
    c = torch.zeros(8, 1, 16, 144, dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.ones(1)
    for call in (lambda: binding.cache_write_fp4(q3, q3, q3, c, c, f, f, i, i, 64),
                 lambda: binding.cache_read_fp4(c, c, f, f, i, i, 64, 4),
                 lambda: binding.paged_fp4(q4, c, c, f, f, i, i, 64),
                 lambda: binding.paged_e4m3_window(q4, c, c, f, f, i, i, 64, 16),
                 lambda: binding.prefill_window(q3, q3, q3, 16),
                 lambda: binding.prefill_e4m3_window(q3, c, c, f, f, 16)):
        with pytest.raises(binding.GQAError) as e:
            call()
        assert e.value.status == INVALID


def test_plain_codes_round_to_even():
    half = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 7.0])
    assert ref.E2M1[ref.nearest_even(half, ref.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 6]
    u = np.linspace(-6, 6, 16).astype(np.float32)
    row = ref.encode_rows(u)
    assert row.shape == (9,) and row[8] == 0x38   # 6 / 6 = 1
    assert np.abs(ref.decode_rows(row, 16) - u).max() <= 1.0
    assert not ref.encode_rows(np.zeros(16, np.float32)).any()
    t = torch.tensor(ref.E4M3[:127])
    assert torch.equal(t.to(torch.float8_e4m3fn).view(torch.uint8), torch.arange(127).byte())


def test_plain_mask_and_empty_rows():
    see = ref.visible([-1, 0, 5], 6, 2, 1)
    assert see.tolist() == [[False] * 6, [True] + [False] * 5,
                            [True, False, False, False, True, True]]
    out, bound = ref.attend(np.ones((3, 4)), np.ones((6, 4)), np.ones((6, 4)), see, 1.0)
    assert (out[0] == 0).all() and np.allclose(out[1:], 1) and (bound[0] == 0).all()
