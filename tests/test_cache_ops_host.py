"""Refusals of the cache write, cache read, block index and block selection
entry points: all before anything reaches a GPU (no GPU needed)."""

import ctypes

import pytest
import torch

from long_context_causal_gqa_gb300 import binding, build_lib

P = ctypes.c_void_p
FAKE = P(0x10000)        # aligned non-null stand-in; never dereferenced
ODD8 = P(0x10008)
ODD2 = P(0x10002)
INVALID, UNSUPPORTED = binding.GQA_ERR_INVALID_ARG, binding.GQA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return binding.load()


WRITE_FIELDS = [(n, ctypes.c_void_p) for n in
                ("q", "k", "v", "qw", "kw", "freq", "ks", "vs", "bt", "starts", "ctx", "out", "kc",
                 "vc")] + \
               [(n, ctypes.c_int64) for n in ("qt", "qh", "kt", "kh", "vt", "vh")] + \
               [("dtype", ctypes.c_int32), ("rot", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("eps", ctypes.c_float)] + \
               [(n, ctypes.c_int32) for n in
                ("stride", "pages", "page", "max_ctx", "batch", "tokens", "Hq", "Hkv", "D")]


class WriteArgs(ctypes.Structure):
    """gqa_cache_write_args."""
    _fields_ = WRITE_FIELDS


def _write(lib, e4m3=True, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, qt=2048, qh=256, kt=2048, kh=256, vt=2048, vh=256,
             qw=FAKE, kw=FAKE, eps=1e-6, freq=FAKE, rot=64, inter=0, ks=FAKE, vs=FAKE, bt=FAKE,
             stride=8, pages=8, page=16, starts=P(0), ctx=FAKE, max_ctx=100, batch=2, tokens=4,
             Hq=6, Hkv=1, D=256, out=FAKE, kc=FAKE, vc=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    args = WriteArgs()
    for name, x in a.items():
        setattr(args, name, x)
    fn = lib.gqa_cache_write_e4m3 if e4m3 else lib.gqa_cache_write
    return fn(bytes(args), None)


def test_write_arguments_have_the_c_layout(lib):
    """The binding packs gqa_cache_write_args itself: same size as the structure
    the C compiler lays out."""
    assert binding._WRITE_ARGS.size == ctypes.sizeof(WriteArgs)
    packed = binding._WRITE_ARGS.pack(*range(1, 24), 0.5, *range(30, 39))
    args = WriteArgs.from_buffer_copy(packed)
    assert args.q == 1 and args.vc == 14 and args.vh == 20 and args.inter == 23
    assert args.eps == 0.5 and args.stride == 30 and args.D == 38
    assert lib.gqa_cache_write_e4m3(None, None) == INVALID
    assert lib.gqa_cache_write(None, None) == INVALID


ROW_REFUSALS = [
    (dict(bt=P(0)), INVALID), (dict(bt=ODD2), INVALID), (dict(ctx=P(0)), INVALID),
    (dict(ctx=ODD2), INVALID), (dict(starts=ODD2), INVALID), (dict(tokens=0), INVALID),
    (dict(batch=0), INVALID), (dict(pages=0), INVALID), (dict(max_ctx=0), INVALID),
    (dict(stride=0), INVALID), (dict(max_ctx=129), INVALID),
    (dict(max_ctx=100, stride=6), INVALID), (dict(tokens=5), INVALID),
    (dict(batch=1025, tokens=1025), UNSUPPORTED), (dict(page=12), UNSUPPORTED),
    (dict(page=4), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(D=64), UNSUPPORTED),
    (dict(D=192), UNSUPPORTED), (dict(pages=1 << 27, page=16), UNSUPPORTED),
    (dict(Hkv=0), UNSUPPORTED), (dict(Hkv=65), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", ROW_REFUSALS + [
    (dict(k=P(0)), INVALID), (dict(v=P(0)), INVALID), (dict(kc=P(0)), INVALID),
    (dict(vc=P(0)), INVALID), (dict(q=P(0)), INVALID), (dict(out=P(0)), INVALID),
    (dict(q=ODD8), INVALID), (dict(k=ODD8), INVALID), (dict(v=ODD8), INVALID),
    (dict(out=ODD8), INVALID), (dict(kc=ODD8), INVALID), (dict(vc=ODD8), INVALID),
    (dict(qw=ODD8), INVALID), (dict(kw=ODD8), INVALID), (dict(ks=P(0)), INVALID),
    (dict(vs=ODD2), INVALID), (dict(qt=2044), INVALID), (dict(kh=100), INVALID),
    (dict(vt=1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(freq=P(0)), INVALID), (dict(freq=ODD2), INVALID),
    (dict(rot=-16), INVALID), (dict(rot=8), UNSUPPORTED), (dict(rot=72), UNSUPPORTED),
    (dict(rot=272), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(Hq=7, Hkv=2), UNSUPPORTED),
    (dict(Hq=65), UNSUPPORTED),
])
def test_cache_write_refuses(lib, kw, want):
    assert _write(lib, **kw) == want
    if "ks" not in kw and "vs" not in kw:
        assert _write(lib, e4m3=False, **kw) == want


def _read(lib, kw, e4m3):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, eb=2, bt=FAKE, stride=8, pages=8, page=16,
             starts=P(0), ctx=FAKE, max_ctx=100, batch=2, tokens=4, Hkv=1, D=256, ko=FAKE, vo=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    tail = [a[x] for x in ("bt", "stride", "pages", "page", "starts", "ctx", "max_ctx", "batch",
                           "tokens", "Hkv", "D", "ko", "vo")]
    if e4m3:
        return lib.gqa_cache_read_e4m3(a["kc"], a["vc"], a["ks"], a["vs"], *tail, None)
    return lib.gqa_cache_read(a["kc"], a["vc"], a["eb"], *tail, None)


@pytest.mark.parametrize("kw,want", ROW_REFUSALS + [
    (dict(kc=P(0)), INVALID), (dict(vc=ODD8), INVALID), (dict(ko=P(0)), INVALID),
    (dict(vo=ODD8), INVALID)])
def test_cache_read_refuses(lib, kw, want):
    assert _read(lib, kw, True) == want
    assert _read(lib, kw, False) == want


def test_cache_read_refuses_scales_and_types(lib):
    assert _read(lib, dict(ks=P(0)), True) == INVALID
    assert _read(lib, dict(vs=ODD2), True) == INVALID
    assert _read(lib, dict(eb=4), False) == UNSUPPORTED
    assert _read(lib, dict(eb=0), False) == UNSUPPORTED


def _index(lib, kw, e4m3):
    a = dict(kc=FAKE, ks=FAKE, bt=FAKE, stride=8, pages=8, page=16, starts=P(0), ctx=FAKE,
             max_ctx=100, batch=2, tokens=4, Hkv=1, D=256, ix=FAKE, sc=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    tail = [a[x] for x in ("bt", "stride", "pages", "page", "starts", "ctx", "max_ctx", "batch",
                           "tokens", "Hkv", "D", "ix", "sc")]
    if e4m3:
        return lib.gqa_block_index_e4m3(a["kc"], a["ks"], *tail, None)
    return lib.gqa_block_index(a["kc"], *tail, None)


@pytest.mark.parametrize("kw,want", ROW_REFUSALS + [
    (dict(kc=P(0)), INVALID), (dict(kc=ODD8), INVALID), (dict(ix=P(0)), INVALID),
    (dict(ix=ODD8), INVALID), (dict(sc=P(0)), INVALID), (dict(sc=ODD2), INVALID),
    (dict(Hkv=5), UNSUPPORTED), (dict(Hkv=9, D=128), UNSUPPORTED)])
def test_block_index_refuses(lib, kw, want):
    assert _index(lib, kw, True) == want
    assert _index(lib, kw, False) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=P(0)), INVALID), (dict(q=ODD8), INVALID), (dict(ix=P(0)), INVALID),
    (dict(ix=ODD8), INVALID), (dict(sc=P(0)), INVALID), (dict(sc=ODD2), INVALID),
    (dict(bt=P(0)), INVALID), (dict(bt=ODD2), INVALID), (dict(si=P(0)), INVALID),
    (dict(si=ODD2), INVALID), (dict(ct=P(0)), INVALID), (dict(ct=ODD2), INVALID),
    (dict(rows=0), INVALID), (dict(rows=101), INVALID), (dict(pages=0), INVALID),
    (dict(max_sel=0), INVALID), (dict(first=-1), INVALID), (dict(last=0), INVALID),
    (dict(first=7, last=2), INVALID), (dict(first=2**31 - 1, last=2**31 - 1), INVALID),
    (dict(ctx=129, rows=1), INVALID), (dict(max_sel=2049), UNSUPPORTED),
    (dict(D=64), UNSUPPORTED), (dict(Hq=7, Hkv=2), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(Hq=10, Hkv=5), UNSUPPORTED), (dict(Hq=9, Hkv=9, D=128), UNSUPPORTED),
    (dict(pages=1 << 27), UNSUPPORTED)])
def test_select_blocks_refuses(lib, kw, want):
    a = dict(q=FAKE, ix=FAKE, sc=FAKE, bt=FAKE, pages=8, page=16, ctx=100, rows=4, Hq=6, Hkv=1,
             D=256, max_sel=8, first=0, last=1, si=FAKE, ct=FAKE)
    assert not set(kw) - set(a)
    a.update(kw)
    assert lib.gqa_select_blocks(*a.values(), None) == want


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 1, 256, dtype=torch.float16)
    c = torch.zeros(8, 16, 1, 256, dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    calls = [
        lambda: binding.cache_write_e4m3(x, x, x, c, c, i, i, i, i, 64),
        lambda: binding.cache_write(x, x, x, c, c, i, i, 64),
        lambda: binding.cache_read_e4m3(c, c, i, i, i, i, 64, 4),
        lambda: binding.cache_read(c, c, i, i, 64, 4),
        lambda: binding.block_index_e4m3(c, i, i, i, 64, 4, c, i),
        lambda: binding.block_index(c, i, i, 64, 4, c, i),
        lambda: binding.select_blocks(x, c, i, i, 64, 4),
    ]
    for call in calls:
        with pytest.raises(binding.GQAError) as e:
            call()
        assert e.value.status == INVALID
