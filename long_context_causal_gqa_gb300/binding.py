"""Python binding of libgqa_attn.so (ctypes; argument marshalling only).

Every function here forwards torch tensors' device pointers, shapes and the
current CUDA stream to the C ABI declared in ``include/gqa_attn.h``; all of the
attention runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or a call fails, a ``GQAError`` is raised.

Workspace: the prefill, paged-E4M3 and block-selection entry points keep what
they need in between in a workspace registered per device.  ``ensure_workspace``
allocates it with torch (outside the C calls) and registers it; the wrappers call
it for you.  Calls that share it must not overlap on the GPU.

Streams: a call runs on ``stream`` (a torch stream), or on the current one.
Outputs that a call allocates belong to the stream it runs on.
"""

from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgqa_attn.so")

GQA_OK = 0
GQA_ERR_INVALID_ARG = 1
GQA_ERR_UNSUPPORTED = 2
GQA_ERR_WORKSPACE = 3
GQA_ERR_CUDA = 4
KIND_PREFILL = 0
KIND_PAGED_E4M3 = 1
KIND_SPARSE = 2
KIND_PAGED_E4M3_BATCH = 3
KIND_SELECT_BLOCKS = 4
KIND_TAILS = 5
DTYPE_F16 = 0
DTYPE_BF16 = 1
DEVERR_WAIT_TIMEOUT = 0x1
DEVERR_BAD_BLOCK_ID = 0x2
DEVERR_BAD_PAGE_ID = 0x4
DEVERR_BAD_CTX_LEN = 0x8
DEVERR_DUP_BLOCK_ID = 0x10

# Every symbol include/gqa_attn.h declares.
EXPORTED = ("gqa_attn_prefill", "gqa_attn_prefill_e4m3", "gqa_attn_paged_e4m3", "gqa_attn_paged_e4m3_devctx",
            "gqa_attn_paged_e4m3_batch",
            "gqa_attn_paged_e4m3_noalloc",
            "gqa_attn_sparse_blocks", "gqa_attn_sparse_blocks_e4m3",
            "gqa_cache_write_e4m3", "gqa_cache_write", "gqa_cache_read_e4m3", "gqa_cache_read",
            "gqa_block_index_e4m3", "gqa_block_index", "gqa_select_blocks",
            "gqa_cache_write_fp4", "gqa_cache_read_fp4", "gqa_attn_paged_fp4",
            "gqa_attn_paged_e4m3_window", "gqa_attn_prefill_window",
            "gqa_attn_prefill_e4m3_window",
            "gqa_workspace_bytes", "gqa_set_workspace", "gqa_get_device_error",
            "gqa_check_wait_limit", "gqa_prefill_sm_pairs", "gqa_status_string")


class GQAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lock = threading.Lock()
_lib = None
_ws = {}  # device index -> torch.uint8 tensor registered as workspace
_outgrown = []  # workspaces replaced by larger ones: captured graphs may still use them


def load():
    """Load libgqa_attn.so (it must have been built; see build_lib.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise GQAError(GQA_ERR_CUDA, f"{LIB_PATH} not built")
            lib = ctypes.CDLL(LIB_PATH)
            P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.gqa_attn_prefill.argtypes = [P, P, P, P, I, I, I, I, I, F, P]
            lib.gqa_attn_prefill.restype = I
            lib.gqa_attn_prefill_e4m3.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, P]
            lib.gqa_attn_prefill_e4m3.restype = I
            lib.gqa_attn_paged_e4m3.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, F, P, P]
            lib.gqa_attn_paged_e4m3.restype = I
            lib.gqa_attn_paged_e4m3_devctx.argtypes = [P, P, P, P, P, P, I, I, P, I, I, I, I, I,
                                                       F, P, P]
            lib.gqa_attn_paged_e4m3_devctx.restype = I
            lib.gqa_attn_paged_e4m3_batch.argtypes = [P, P, P, P, P, P, I, I, I, P, I, I, I, I, I,
                                                      I, F, P, P]
            lib.gqa_attn_paged_e4m3_batch.restype = I
            lib.gqa_attn_paged_e4m3_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I,
                                                        F, P, P]
            lib.gqa_attn_paged_e4m3_noalloc.restype = I
            lib.gqa_attn_sparse_blocks.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F,
                                                   P, P]
            lib.gqa_attn_sparse_blocks.restype = I
            lib.gqa_attn_sparse_blocks_e4m3.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I,
                                                        I, I, I, F, P, P]
            lib.gqa_attn_sparse_blocks_e4m3.restype = I
            for f in (lib.gqa_cache_write_e4m3, lib.gqa_cache_write, lib.gqa_cache_write_fp4):
                f.argtypes = [ctypes.c_char_p, P]
                f.restype = I
            lib.gqa_cache_read_e4m3.argtypes = [P, P, P, P, P, I, I, I, P, P, I, I, I, I, I, P,
                                                P, P]
            lib.gqa_cache_read_e4m3.restype = I
            lib.gqa_cache_read_fp4.argtypes = lib.gqa_cache_read_e4m3.argtypes
            lib.gqa_cache_read_fp4.restype = I
            lib.gqa_attn_paged_fp4.argtypes = [P, P, P, P, P, P, I, I, I, P, I, I, I, I, I, I, F,
                                               I, I, P, P]
            lib.gqa_attn_paged_fp4.restype = I
            lib.gqa_attn_paged_e4m3_window.argtypes = lib.gqa_attn_paged_fp4.argtypes
            lib.gqa_attn_paged_e4m3_window.restype = I
            lib.gqa_attn_prefill_window.argtypes = [P, P, P, P, I, I, I, I, I, F, I, I, P]
            lib.gqa_attn_prefill_window.restype = I
            lib.gqa_attn_prefill_e4m3_window.argtypes = [P, P, P, P, P, P, I, I, I, I, I, F, I, I,
                                                         P]
            lib.gqa_attn_prefill_e4m3_window.restype = I
            lib.gqa_cache_read.argtypes = [P, P, I, P, I, I, I, P, P, I, I, I, I, I, P, P, P]
            lib.gqa_cache_read.restype = I
            lib.gqa_block_index_e4m3.argtypes = [P, P, P, I, I, I, P, P, I, I, I, I, I, P, P, P]
            lib.gqa_block_index_e4m3.restype = I
            lib.gqa_block_index.argtypes = [P, P, I, I, I, P, P, I, I, I, I, I, P, P, P]
            lib.gqa_block_index.restype = I
            lib.gqa_select_blocks.argtypes = [P, P, P, P, I, I, I, I, I, I, I, I, I, I, P, P, P]
            lib.gqa_select_blocks.restype = I
            lib.gqa_workspace_bytes.argtypes = [I, I, I, I, I]
            lib.gqa_workspace_bytes.restype = Z
            lib.gqa_set_workspace.argtypes = [I, P, Z]
            lib.gqa_set_workspace.restype = I
            lib.gqa_get_device_error.argtypes = [P]
            lib.gqa_get_device_error.restype = I
            lib.gqa_check_wait_limit.argtypes = [P]
            lib.gqa_check_wait_limit.restype = I
            lib.gqa_prefill_sm_pairs.argtypes = []
            lib.gqa_prefill_sm_pairs.restype = I
            lib.gqa_status_string.argtypes = [I]
            lib.gqa_status_string.restype = ctypes.c_char_p
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().gqa_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != GQA_OK:
        raise GQAError(status, what)


def _stream_ptr(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: torch.Tensor):
    return ctypes.c_void_p(t.data_ptr())


def _empty(shape, dtype, device, stream):
    """Memory of an output, from the stream that writes it.  (From the current
    stream's it could still be in use by that stream's earlier work.)  Freed, it is
    not given out again before what the current stream does with it until then."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(device))
    return out


def _need_cuda(*ts):
    dev = None
    for t in ts:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise GQAError(GQA_ERR_INVALID_ARG, "tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise GQAError(GQA_ERR_INVALID_ARG, "tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise GQAError(GQA_ERR_INVALID_ARG, "tensors on different devices")
    return dev


def workspace_bytes(kind: int, query_rows: int, ctx_or_kv: int, Hq: int = 6, D: int = 256) -> int:
    return int(load().gqa_workspace_bytes(kind, query_rows, ctx_or_kv, Hq, D))


def ensure_workspace(nbytes: int, device=None) -> torch.Tensor:
    """Make sure the device's registered workspace holds at least nbytes.  A
    workspace that a larger one replaces is kept, for graphs captured with it
    (see release_outgrown)."""
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    cur = _ws.get(idx)
    if cur is None or cur.numel() < nbytes:
        torch.cuda.synchronize(idx)
        need = size = max(int(nbytes), 4096)
        if cur is not None:
            # Half as much again at least, so that the ones kept stay few.
            size = max(need, cur.numel() * 3 // 2)
        try:
            buf = torch.empty(size, dtype=torch.uint8, device=f"cuda:{idx}")
        except torch.cuda.OutOfMemoryError:
            if size == need:
                raise
            buf = torch.empty(need, dtype=torch.uint8, device=f"cuda:{idx}")
        _check(load().gqa_set_workspace(idx, _ptr(buf), buf.numel()), "gqa_set_workspace")
        if cur is not None:
            _outgrown.append(cur)
        _ws[idx] = buf
        cur = buf
    return cur


def release_outgrown(device=None) -> int:
    """Free the workspaces of a device that larger ones have replaced, and
    return their bytes.  A graph captured with one of them must not be replayed
    afterwards: capture it again, or keep them."""
    dev = torch.device(device if device is not None else "cuda")
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    torch.cuda.synchronize(idx)
    mine = [b for b in _outgrown if b.device.index == idx]
    _outgrown[:] = [b for b in _outgrown if b.device.index != idx]
    return sum(b.numel() for b in mine)


def register_workspace(buf: torch.Tensor):
    """Register a caller-provided uint8 CUDA buffer as its device's workspace."""
    _need_cuda(buf)
    idx = buf.device.index
    _check(load().gqa_set_workspace(idx, _ptr(buf), buf.numel()), "gqa_set_workspace")
    _ws[idx] = buf


def device_error(stream=None) -> int:
    """Synchronise the stream and read-and-clear the device error word."""
    v = load().gqa_get_device_error(_stream_ptr(stream))
    if v < 0:
        raise GQAError(GQA_ERR_CUDA, "gqa_get_device_error")
    return v


def check_wait_limit(stream=None) -> None:
    """Queue the bounded-wait diagnostic (gqa_check_wait_limit): a wait on an
    mbarrier nothing arrives on, which gives up after its limit and sets
    DEVERR_WAIT_TIMEOUT; read it with device_error()."""
    st = load().gqa_check_wait_limit(_stream_ptr(stream))
    if st != GQA_OK:
        raise GQAError(st, "gqa_check_wait_limit")


def prefill_sm_pairs() -> int:
    """SM pairs the dense prefill kernel runs on (co-resident two-CTA clusters)."""
    v = load().gqa_prefill_sm_pairs()
    if v < 0:
        raise GQAError(GQA_ERR_CUDA, "gqa_prefill_sm_pairs")
    return v


def prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, scale: float = 1.0 / 16,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Dense causal GQA prefill: q [Q,Hq,D], k/v [KV,Hkv,D] fp16 -> out [Q,Hq,D]."""
    dev = _need_cuda(q, k, v)
    Q, Hq, D = q.shape
    KV, Hkv, _ = k.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        ensure_workspace(workspace_bytes(KIND_PREFILL, Q, KV, Hq, D), dev)
        st = load().gqa_attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), Q, KV, Hq, Hkv, D,
                                     float(scale), _stream_ptr(stream))
    _check(st, "gqa_attn_prefill")
    return out


def prefill_e4m3(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, kscale: torch.Tensor,
                 vscale: torch.Tensor, scale: float = 1.0 / 16, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """Dense causal GQA prefill over an E4M3 K/V cache: q [Q,Hq,D] fp16, k/v
    [KV,Hkv,D] uint8 codes, kscale/vscale one-element fp32 CUDA tensors."""
    dev = _need_cuda(q, k, v, kscale, vscale)
    Q, Hq, D = q.shape
    KV, Hkv, _ = k.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        ensure_workspace(workspace_bytes(KIND_PREFILL, Q, KV, Hq, D), dev)
        st = load().gqa_attn_prefill_e4m3(_ptr(q), _ptr(k), _ptr(v), _ptr(kscale), _ptr(vscale),
                                          _ptr(out), Q, KV, Hq, Hkv, D, float(scale),
                                          _stream_ptr(stream))
    _check(st, "gqa_attn_prefill_e4m3")
    return out


def paged_e4m3(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
               kscale: torch.Tensor, vscale: torch.Tensor, block_table: torch.Tensor,
               ctx_len: int, scale: float = 1.0 / 16, out: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """Paged E4M3 verifier tail: q [R,Hq,D] fp16, caches [pages,page,Hkv,D] uint8,
    kscale/vscale one-element fp32 CUDA tensors, block_table int32."""
    dev = _need_cuda(q, kcache, vcache, kscale, vscale, block_table)
    R, Hq, D = q.shape
    num_pages, page, Hkv, _ = kcache.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        ensure_workspace(workspace_bytes(KIND_PAGED_E4M3, R, ctx_len, Hq, D), dev)
        st = load().gqa_attn_paged_e4m3(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(kscale),
                                        _ptr(vscale), _ptr(block_table), num_pages, page,
                                        int(ctx_len), R, Hq, Hkv, D, float(scale), _ptr(out),
                                        _stream_ptr(stream))
    _check(st, "gqa_attn_paged_e4m3")
    return out


def paged_e4m3_devctx(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                      kscale: torch.Tensor, vscale: torch.Tensor, block_table: torch.Tensor,
                      ctx_len_dev: torch.Tensor, max_ctx_len: int, scale: float = 1.0 / 16,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Paged E4M3 tail with the context length read on the device when the
    kernels run: ctx_len_dev is a one-element int32 CUDA tensor, max_ctx_len
    the host bound that sizes the grid and the workspace."""
    dev = _need_cuda(q, kcache, vcache, kscale, vscale, block_table, ctx_len_dev)
    if ctx_len_dev.dtype != torch.int32 or ctx_len_dev.numel() < 1:
        raise GQAError(GQA_ERR_INVALID_ARG, "ctx_len_dev must be a CUDA int32 tensor")
    R, Hq, D = q.shape
    num_pages, page, Hkv, _ = kcache.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        ensure_workspace(workspace_bytes(KIND_PAGED_E4M3, R, max_ctx_len, Hq, D), dev)
        st = load().gqa_attn_paged_e4m3_devctx(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(kscale),
                                               _ptr(vscale), _ptr(block_table), num_pages, page,
                                               _ptr(ctx_len_dev), int(max_ctx_len), R, Hq, Hkv, D,
                                               float(scale), _ptr(out), _stream_ptr(stream))
    _check(st, "gqa_attn_paged_e4m3_devctx")
    return out


def paged_e4m3_batch(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                     kscale: torch.Tensor, vscale: torch.Tensor, block_tables: torch.Tensor,
                     ctx_lens_dev: torch.Tensor, max_ctx_len: int, scale: float = 1.0 / 16,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Batched variable-length E4M3 tails: q [B,R,Hq,D] fp16, one shared page
    cache, block_tables [B, stride] int32, ctx_lens_dev [B] CUDA int32 read when
    the kernels run, max_ctx_len the host bound."""
    dev = _need_cuda(q, kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev)
    if ctx_lens_dev.dtype != torch.int32 or block_tables.dtype != torch.int32:
        raise GQAError(GQA_ERR_INVALID_ARG, "ctx_lens_dev and block_tables must be int32")
    B, R, Hq, D = q.shape
    if ctx_lens_dev.numel() != B or block_tables.shape[0] != B or not block_tables.is_contiguous():
        raise GQAError(GQA_ERR_INVALID_ARG, "one context length and table row per sequence")
    num_pages, page, Hkv, _ = kcache.shape
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        ensure_workspace(workspace_bytes(KIND_PAGED_E4M3_BATCH, R, B, Hq, D), dev)
        st = load().gqa_attn_paged_e4m3_batch(_ptr(q), _ptr(kcache), _ptr(vcache), _ptr(kscale),
                                              _ptr(vscale), _ptr(block_tables),
                                              block_tables.shape[1], num_pages, page,
                                              _ptr(ctx_lens_dev), int(max_ctx_len), B, R, Hq, Hkv,
                                              D, float(scale), _ptr(out), _stream_ptr(stream))
    _check(st, "gqa_attn_paged_e4m3_batch")
    return out


def sparse_blocks(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                  block_table: torch.Tensor, sel_idx: torch.Tensor, sel_cnt: torch.Tensor,
                  ctx_len: int, scale: float = 1.0 / 16, out: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """Selected-block sparse paged prefill over an fp16 page cache."""
    dev = _need_cuda(q, kcache, vcache, block_table, sel_idx, sel_cnt)
    rows, Hq, D = q.shape
    num_pages, page, Hkv, _ = kcache.shape
    max_sel = sel_idx.shape[1]
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        st = load().gqa_attn_sparse_blocks(_ptr(q), _ptr(kcache), _ptr(vcache),
                                           _ptr(block_table), _ptr(sel_idx), _ptr(sel_cnt),
                                           max_sel, num_pages, page, int(ctx_len), rows, Hq,
                                           Hkv, D, float(scale), _ptr(out), _stream_ptr(stream))
    _check(st, "gqa_attn_sparse_blocks")
    return out


def sparse_blocks_e4m3(q: torch.Tensor, kcache: torch.Tensor, vcache: torch.Tensor,
                       kscale: torch.Tensor, vscale: torch.Tensor, block_table: torch.Tensor,
                       sel_idx: torch.Tensor, sel_cnt: torch.Tensor, ctx_len: int,
                       scale: float = 1.0 / 16, out: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Selected-block sparse paged prefill over an E4M3 page cache: caches
    [pages,page,Hkv,D] uint8 codes, kscale/vscale one-element fp32 CUDA tensors."""
    dev = _need_cuda(q, kcache, vcache, kscale, vscale, block_table, sel_idx, sel_cnt)
    rows, Hq, D = q.shape
    num_pages, page, Hkv, _ = kcache.shape
    max_sel = sel_idx.shape[1]
    if out is None:
        out = _empty(q.shape, q.dtype, q.device, stream)
    _need_cuda(out)
    with torch.cuda.device(dev):
        st = load().gqa_attn_sparse_blocks_e4m3(_ptr(q), _ptr(kcache), _ptr(vcache),
                                                _ptr(kscale), _ptr(vscale), _ptr(block_table),
                                                _ptr(sel_idx), _ptr(sel_cnt), max_sel, num_pages,
                                                page, int(ctx_len), rows, Hq, Hkv, D,
                                                float(scale), _ptr(out), _stream_ptr(stream))
    _check(st, "gqa_attn_sparse_blocks_e4m3")
    return out


# ---- the cache write, cache read, block index and block selection ----------
#
# These run once a layer and step beside a single small kernel, so their
# wrappers keep to what costs little on the host: plain integers instead of
# ctypes objects, no device switch when the tensors' device is current, and one
# look at each property of a tensor that is as it should be.

# gqa_cache_write_args, in the C compiler's layout.
_WRITE_ARGS = struct.Struct("@14P6q3if9i4x")


def _refuse(what: str):
    raise GQAError(GQA_ERR_INVALID_ARG, what)


def _want(name: str, t, dtype, idx, dims: int):
    """Pointer of a contiguous CUDA tensor of the given type, device and dimensions."""
    try:
        if t.dtype is dtype and t.get_device() == idx and t.dim() == dims and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(f"{name} must be a contiguous {dims}-dimensional {dtype} tensor on cuda:{idx}")


def _heads(name: str, t, dtype, idx, tokens, D):
    """Heads and strides of a [tokens, heads, D] tensor with D contiguous."""
    try:
        if t.dtype is dtype and t.get_device() == idx and t.dim() == 3:
            n, heads, d = t.shape
            a, b, c = t.stride()
            if n == tokens and d == D and c == 1:
                return heads, a, b
    except AttributeError:
        pass
    _refuse(f"{name} must be [tokens, heads, D] like k, with D contiguous")


def _call(fn, idx, stream, *args):
    """One library call on the tensors' device and the given (or current) stream."""
    if torch._C._cuda_getDevice() != idx:
        with torch.cuda.device(idx):
            return _call(fn, idx, stream, *args)
    if stream is not None:
        stream = stream.cuda_stream
    else:
        stream = torch._C._cuda_getCurrentRawStream(idx)
    st = fn(*args, stream)
    if st != GQA_OK:
        raise GQAError(st, fn.__name__)


def _call_with_workspace(fn, idx, stream, args, kind, *shape):
    """The call; where the workspace is too small for it, again with one that is not."""
    try:
        _call(fn, idx, stream, *args)
    except ctypes.ArgumentError as e:
        _refuse(str(e))
    except GQAError as e:
        if e.status != GQA_ERR_WORKSPACE:
            raise
        with torch.cuda.device(idx):
            ensure_workspace(workspace_bytes(kind, *shape), idx)
        _call(fn, idx, stream, *args)


def _device_of(t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse("tensors must be CUDA tensors")
    return t.get_device()


def _scale(name, t, idx):
    try:
        if t.dtype is torch.float32 and t.numel() == 1 and t.get_device() == idx:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(f"{name} must be a one-element fp32 tensor on cuda:{idx}")


def _pages(kcache, vcache, dtype, idx):
    """Pointers of the two caches and their [pages, page, Hkv, D]."""
    kp = _want("kcache", kcache, dtype, idx, 4)
    vp = _want("vcache", vcache, dtype, idx, 4)
    shape = kcache.shape
    if vcache.shape != shape:
        _refuse("kcache and vcache must have the same shape")
    return kp, vp, shape


def _rows(block_tables, ctx_lens_dev, row_starts, idx):
    """(tables, stride, row_starts, ctx_lens, batch) of the rows' sequences."""
    bt = _want("block_tables", block_tables, torch.int32, idx, 2)
    cl = _want("ctx_lens_dev", ctx_lens_dev, torch.int32, idx, 1)
    batch, stride = block_tables.shape
    if ctx_lens_dev.numel() != batch:
        _refuse("one context length and table row per sequence")
    rs = 0
    if row_starts is not None:
        rs = _want("row_starts", row_starts, torch.int32, idx, 1)
        if row_starts.numel() != batch + 1:
            _refuse("row_starts must hold batch + 1 starts")
    return bt, stride, rs, cl, batch


def _fp4_pages(kcache, vcache, idx):
    """Pointers of two 4-bit caches [pages, Hkv, page, 9 D / 16] and (pages, page, Hkv, D)."""
    kp, vp, (num_pages, Hkv, page, row) = _pages(kcache, vcache, torch.uint8, idx)
    if row % 9:
        _refuse("a row of a 4-bit cache must have 9 D / 16 bytes")
    return kp, vp, (num_pages, page, Hkv, row // 9 * 16)


def _cache_write(q, k, v, kcache, vcache, kscale, vscale, bits, block_tables, ctx_lens_dev,
                 max_ctx_len, q_weight, k_weight, eps, inv_freq, interleaved, row_starts, q_out,
                 stream):
    lib = load() if _lib is None else _lib
    idx = _device_of(k)
    dtype = k.dtype
    if dtype is torch.float16:
        kind = DTYPE_F16
    elif dtype is torch.bfloat16:
        kind = DTYPE_BF16
    else:
        _refuse("k must be fp16 or bf16")
    if bits == 4:
        kp, vp, (num_pages, page, Hkv, D) = _fp4_pages(kcache, vcache, idx)
    else:
        kp, vp, (num_pages, page, Hkv, D) = _pages(
            kcache, vcache, torch.uint8 if bits == 8 else torch.float16, idx)
    tokens = len(k)
    hk, kt, kh = _heads("k", k, dtype, idx, tokens, D)
    hv, vt, vh = _heads("v", v, dtype, idx, tokens, D)
    if hk != Hkv or hv != Hkv:
        _refuse("k and v must have the cache's KV heads")
    if q is not None:
        Hq, qt, qh = _heads("q", q, dtype, idx, tokens, D)
        if q_out is None:
            q_out = _empty((tokens, Hq, D), torch.float16, k.device, stream)
        qp, op = q.data_ptr(), _want("q_out", q_out, torch.float16, idx, 3)
        if q_out.shape != q.shape:
            _refuse("q_out must have q's shape")
    elif q_out is None:
        Hq, qt, qh, qp, op = Hkv, 0, 0, 0, 0
    else:
        _refuse("q_out without q")
    qw = kw = fp = rot = ks = vs = 0
    if q_weight is not None:
        qw = _want("q_weight", q_weight, dtype, idx, 1)
        if q_weight.numel() != D:
            _refuse("q_weight must hold D weights")
    if k_weight is not None:
        kw = _want("k_weight", k_weight, dtype, idx, 1)
        if k_weight.numel() != D:
            _refuse("k_weight must hold D weights")
    if inv_freq is not None:
        fp = _want("inv_freq", inv_freq, torch.float32, idx, 1)
        rot = 2 * inv_freq.numel()
    if bits < 16:
        ks, vs = _scale("kscale", kscale, idx), _scale("vscale", vscale, idx)
    bt, stride, rs, cl, batch = _rows(block_tables, ctx_lens_dev, row_starts, idx)
    try:
        args = _WRITE_ARGS.pack(qp, k.data_ptr(), v.data_ptr(), qw, kw, fp, ks, vs, bt, rs, cl,
                                op, kp, vp, qt, qh, kt, kh, vt, vh, kind, rot,
                                1 if interleaved else 0, eps, stride, num_pages, page,
                                max_ctx_len, batch, tokens, Hq, Hkv, D)
    except (struct.error, OverflowError, TypeError) as e:
        _refuse(str(e))
    _call(lib.gqa_cache_write if bits == 16 else
          lib.gqa_cache_write_e4m3 if bits == 8 else lib.gqa_cache_write_fp4, idx, stream, args)
    return q_out


def cache_write_e4m3(q, k, v, kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev,
                     max_ctx_len, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                     interleaved=False, row_starts=None, q_out=None, stream=None):
    """Norm, rotation and store of a step's rows into an E4M3 cache
    (gqa_cache_write_e4m3): q [T,Hq,D] (or None), k/v [T,Hkv,D] fp16 or bf16,
    views of a fused projection included; caches [pages,page,Hkv,D] uint8;
    block_tables [B, stride], ctx_lens_dev [B], row_starts [B+1] int32.
    Returns q_out [T,Hq,D] fp16 (None without q); rows that belong to no
    sequence, or to one whose context length is refused, are left as they were
    (in a q_out allocated here: not initialised)."""
    return _cache_write(q, k, v, kcache, vcache, kscale, vscale, 8, block_tables,
                        ctx_lens_dev, max_ctx_len, q_weight, k_weight, eps, inv_freq,
                        interleaved, row_starts, q_out, stream)


def cache_write(q, k, v, kcache, vcache, block_tables, ctx_lens_dev, max_ctx_len, q_weight=None,
                k_weight=None, eps=1e-6, inv_freq=None, interleaved=False, row_starts=None,
                q_out=None, stream=None):
    """cache_write_e4m3 over an fp16 cache (caches [pages,page,Hkv,D] fp16, no scales)."""
    return _cache_write(q, k, v, kcache, vcache, None, None, 16, block_tables, ctx_lens_dev,
                        max_ctx_len, q_weight, k_weight, eps, inv_freq, interleaved, row_starts,
                        q_out, stream)


def cache_write_fp4(q, k, v, kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev,
                    max_ctx_len, q_weight=None, k_weight=None, eps=1e-6, inv_freq=None,
                    interleaved=False, row_starts=None, q_out=None, stream=None):
    """cache_write_e4m3 into a 4-bit cache (gqa_cache_write_fp4): caches
    [pages,Hkv,page,9*D/16] uint8, E2M1 codes with an E4M3 scale for every 16."""
    return _cache_write(q, k, v, kcache, vcache, kscale, vscale, 4, block_tables, ctx_lens_dev,
                        max_ctx_len, q_weight, k_weight, eps, inv_freq, interleaved, row_starts,
                        q_out, stream)


def _out_rows(name, t, tokens, Hkv, D, dtype, idx, stream):
    if t is None:
        return _empty((tokens, Hkv, D), dtype, idx, stream), None
    p = _want(name, t, dtype, idx, 3)
    if t.shape != (tokens, Hkv, D):
        _refuse(f"{name} must be [tokens, Hkv, D]")
    return t, p


def _cache_read(kcache, vcache, kscale, vscale, e4m3, block_tables, ctx_lens_dev, max_ctx_len,
                tokens, row_starts, k_out, v_out, stream):
    lib = load() if _lib is None else _lib
    idx = _device_of(kcache)
    dtype = kcache.dtype
    if dtype is not torch.uint8 and (e4m3 or dtype is not torch.float16):
        _refuse("caches must be uint8 codes" + ("" if e4m3 else " or fp16"))
    kp, vp, (num_pages, page, Hkv, D) = _pages(kcache, vcache, dtype, idx)
    out_type = torch.float16 if e4m3 else dtype
    k_out, ko = _out_rows("k_out", k_out, tokens, Hkv, D, out_type, idx, stream)
    v_out, vo = _out_rows("v_out", v_out, tokens, Hkv, D, out_type, idx, stream)
    bt, stride, rs, cl, batch = _rows(block_tables, ctx_lens_dev, row_starts, idx)
    tail = (bt, stride, num_pages, page, rs, cl, max_ctx_len, batch, tokens, Hkv, D,
            ko or k_out.data_ptr(), vo or v_out.data_ptr())
    if e4m3:
        _call(lib.gqa_cache_read_e4m3, idx, stream, kp, vp, _scale("kscale", kscale, idx),
              _scale("vscale", vscale, idx), *tail)
    else:
        _call(lib.gqa_cache_read, idx, stream, kp, vp, 1 if dtype is torch.uint8 else 2, *tail)
    return k_out, v_out


def cache_read_e4m3(kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev, max_ctx_len,
                    tokens, row_starts=None, k_out=None, v_out=None, stream=None):
    """The cached tokens of a batch's rows as dense fp16 K, V [tokens,Hkv,D]
    (gqa_cache_read_e4m3); the last tokens / B (or row_starts') of each context.
    Rows that belong to no sequence, or to one whose context length is refused,
    are left as they were (in outputs allocated here: not initialised)."""
    return _cache_read(kcache, vcache, kscale, vscale, True, block_tables, ctx_lens_dev,
                       max_ctx_len, tokens, row_starts, k_out, v_out, stream)


def cache_read(kcache, vcache, block_tables, ctx_lens_dev, max_ctx_len, tokens, row_starts=None,
               k_out=None, v_out=None, stream=None):
    """The same rows in the cache's own type: fp16, or E4M3 codes (uint8)."""
    return _cache_read(kcache, vcache, None, None, False, block_tables, ctx_lens_dev,
                       max_ctx_len, tokens, row_starts, k_out, v_out, stream)


def cache_read_fp4(kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev, max_ctx_len,
                   tokens, row_starts=None, k_out=None, v_out=None, stream=None):
    """cache_read_e4m3 of a 4-bit cache (caches [pages,Hkv,page,9*D/16] uint8)."""
    lib = load() if _lib is None else _lib
    idx = _device_of(kcache)
    kp, vp, (num_pages, page, Hkv, D) = _fp4_pages(kcache, vcache, idx)
    k_out, ko = _out_rows("k_out", k_out, tokens, Hkv, D, torch.float16, idx, stream)
    v_out, vo = _out_rows("v_out", v_out, tokens, Hkv, D, torch.float16, idx, stream)
    bt, stride, rs, cl, batch = _rows(block_tables, ctx_lens_dev, row_starts, idx)
    _call(lib.gqa_cache_read_fp4, idx, stream, kp, vp, _scale("kscale", kscale, idx),
          _scale("vscale", vscale, idx), bt, stride, num_pages, page, rs, cl, max_ctx_len, batch,
          tokens, Hkv, D, ko or k_out.data_ptr(), vo or v_out.data_ptr())
    return k_out, v_out


# ---- tails over a 4-bit cache, and attention with a sliding window ---------------


def _tails(fn, kind, q, idx, pages, pointers, kscale, vscale, block_tables, ctx_lens_dev,
           max_ctx_len, scale, window, sinks, out, stream):
    """A batch's tails: one library call, or two where the workspace has to grow first."""
    num_pages, page, Hkv, D = pages
    qp = _want("q", q, torch.float16, idx, 4)
    B, R, Hq, d = q.shape
    if d != D:
        _refuse("q and the caches must have the same head size")
    bt, stride, _, cl, batch = _rows(block_tables, ctx_lens_dev, None, idx)
    if batch != B:
        _refuse("one context length and table row per sequence")
    if out is None:
        out = _empty(q.shape, torch.float16, q.device, stream)
        op = out.data_ptr()
    else:
        op = _want("out", out, torch.float16, idx, 4)
        if out.shape != q.shape:
            _refuse("out must have q's shape")
    args = (qp, *pointers, _scale("kscale", kscale, idx), _scale("vscale", vscale, idx), bt,
            stride, num_pages, page, cl, max_ctx_len, B, R, Hq, Hkv, D, scale,
            0 if window is None else window, sinks, op)
    _call_with_workspace(fn, idx, stream, args, kind, R, B, Hq, D)
    return out


def paged_fp4(q, kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev, max_ctx_len,
              scale=1.0 / 16, window=None, sinks=0, out=None, stream=None):
    """Tails of a batch over a 4-bit cache (gqa_attn_paged_fp4): q [B,R,Hq,D] fp16, caches
    [pages,Hkv,page,9*D/16] uint8, block_tables [B, stride] and ctx_lens_dev [B] int32.
    window: a row sees its last `window` positions (its own among them) and the first
    `sinks` tokens; None: the whole context."""
    lib = load() if _lib is None else _lib
    idx = _device_of(q)
    kp, vp, pages = _fp4_pages(kcache, vcache, idx)
    return _tails(lib.gqa_attn_paged_fp4, KIND_TAILS, q, idx, pages, (kp, vp), kscale, vscale,
                  block_tables, ctx_lens_dev, max_ctx_len, scale, window, sinks, out, stream)


def paged_e4m3_window(q, kcache, vcache, kscale, vscale, block_tables, ctx_lens_dev, max_ctx_len,
                      window, sinks=0, scale=1.0 / 16, out=None, stream=None):
    """paged_e4m3_batch with a sliding window (gqa_attn_paged_e4m3_window): a row sees its
    last `window` positions (its own among them) and the first `sinks` tokens; contexts
    may be shorter than the rows, whose places in front of the first token give zeros."""
    lib = load() if _lib is None else _lib
    idx = _device_of(q)
    kp, vp, pages = _pages(kcache, vcache, torch.uint8, idx)
    return _tails(lib.gqa_attn_paged_e4m3_window, KIND_TAILS, q, idx, pages, (kp, vp),
                  kscale, vscale, block_tables, ctx_lens_dev, max_ctx_len, scale, window, sinks,
                  out, stream)


def _prefill_window(fn, q, k, v, scales, scale, window, sinks, out, stream):
    idx = _device_of(q)
    dtype = torch.uint8 if scales else torch.float16
    qp, kp, vp = _want("q", q, torch.float16, idx, 3), _want("k", k, dtype, idx, 3), \
        _want("v", v, dtype, idx, 3)
    Q, Hq, D = q.shape
    KV, Hkv, d = k.shape
    if v.shape != k.shape or d != D:
        _refuse("k and v must have the same shape, and q's head size")
    if out is None:
        out = _empty(q.shape, torch.float16, q.device, stream)
        op = out.data_ptr()
    else:
        op = _want("out", out, torch.float16, idx, 3)
        if out.shape != q.shape:
            _refuse("out must have q's shape")
    scales = [_scale("kscale" if i == 0 else "vscale", x, idx) for i, x in enumerate(scales)]
    args = (qp, kp, vp, *scales, op, Q, KV, Hq, Hkv, D, scale, window, sinks)
    _call_with_workspace(fn, idx, stream, args, KIND_PREFILL, Q, KV, Hq, D)
    return out


def prefill_window(q, k, v, window, sinks=0, scale=1.0 / 16, out=None, stream=None):
    """Dense causal prefill with a sliding window (gqa_attn_prefill_window): q [Q,Hq,D],
    k/v [KV,Hkv,D] fp16.  A row sees its last `window` positions (its own among them)
    and the first `sinks` tokens."""
    lib = load() if _lib is None else _lib
    return _prefill_window(lib.gqa_attn_prefill_window, q, k, v, (), scale, window, sinks, out,
                           stream)


def prefill_e4m3_window(q, k, v, kscale, vscale, window, sinks=0, scale=1.0 / 16, out=None,
                        stream=None):
    """prefill_window over an E4M3 K/V cache: k/v [KV,Hkv,D] uint8 codes, kscale/vscale
    one-element fp32 CUDA tensors."""
    lib = load() if _lib is None else _lib
    return _prefill_window(lib.gqa_attn_prefill_e4m3_window, q, k, v, (kscale, vscale), scale,
                           window, sinks, out, stream)


def _index_pointers(index, index_scale, idx):
    """Pointers of a block index and its [pages, page / 4, Hkv, D]."""
    ip = _want("index", index, torch.int8, idx, 4)
    sp = _want("index_scale", index_scale, torch.float32, idx, 2)
    shape = index.shape
    if index_scale.shape != shape[:2]:
        _refuse("index must be [pages, page / 4, Hkv, D], index_scale [pages, page / 4]")
    return ip, sp, shape


def _block_index(kcache, kscale, e4m3, block_tables, ctx_lens_dev, max_ctx_len, tokens, index,
                 index_scale, row_starts, stream):
    lib = load() if _lib is None else _lib
    idx = _device_of(kcache)
    kp = _want("kcache", kcache, torch.uint8 if e4m3 else torch.float16, idx, 4)
    num_pages, page, Hkv, D = kcache.shape
    ip, sp, shape = _index_pointers(index, index_scale, idx)
    if shape != (num_pages, page // 4, Hkv, D):
        _refuse("index must be [pages, page / 4, Hkv, D], index_scale [pages, page / 4]")
    bt, stride, rs, cl, batch = _rows(block_tables, ctx_lens_dev, row_starts, idx)
    tail = (bt, stride, num_pages, page, rs, cl, max_ctx_len, batch, tokens, Hkv, D, ip, sp)
    if e4m3:
        _call(lib.gqa_block_index_e4m3, idx, stream, kp, _scale("kscale", kscale, idx), *tail)
    else:
        _call(lib.gqa_block_index, idx, stream, kp, *tail)


def block_index_e4m3(kcache, kscale, block_tables, ctx_lens_dev, max_ctx_len, tokens, index,
                     index_scale, row_starts=None, stream=None):
    """Summaries of the 4-token blocks that a step's rows finish
    (gqa_block_index_e4m3), into index [pages,page/4,Hkv,D] int8 and
    index_scale [pages,page/4] fp32."""
    _block_index(kcache, kscale, True, block_tables, ctx_lens_dev, max_ctx_len, tokens, index,
                 index_scale, row_starts, stream)


def block_index(kcache, block_tables, ctx_lens_dev, max_ctx_len, tokens, index, index_scale,
                row_starts=None, stream=None):
    """block_index_e4m3 over an fp16 cache."""
    _block_index(kcache, None, False, block_tables, ctx_lens_dev, max_ctx_len, tokens, index,
                 index_scale, row_starts, stream)


def select_blocks(q, index, index_scale, block_table, ctx_len, max_sel, n_first=0, n_last=1,
                  sel_idx=None, sel_cnt=None, stream=None):
    """The blocks each of the last rows of one sequence attends
    (gqa_select_blocks): q [rows,Hq,D] fp16, the sequence's block index and
    block_table [pages of ctx_len] int32.  Returns sel_idx [rows,max_sel] and
    sel_cnt [rows], as sparse_blocks takes them."""
    lib = load() if _lib is None else _lib
    idx = _device_of(q)
    qp = _want("q", q, torch.float16, idx, 3)
    ip, sp, (num_pages, ppb, Hkv, d) = _index_pointers(index, index_scale, idx)
    bt = _want("block_table", block_table, torch.int32, idx, 1)
    rows, Hq, D = q.shape
    if d != D:
        _refuse("q and index must have the same head size")
    if block_table.numel() * ppb * 4 < ctx_len:
        _refuse("block_table must cover ctx_len")
    if sel_idx is None:
        sel_idx = _empty((rows, max_sel), torch.int32, idx, stream)
        xp = sel_idx.data_ptr()
    else:
        xp = _want("sel_idx", sel_idx, torch.int32, idx, 2)
        if sel_idx.shape != (rows, max_sel):
            _refuse("sel_idx must be [rows, max_sel]")
    if sel_cnt is None:
        sel_cnt = _empty((rows,), torch.int32, idx, stream)
        cp = sel_cnt.data_ptr()
    else:
        cp = _want("sel_cnt", sel_cnt, torch.int32, idx, 1)
        if sel_cnt.numel() != rows:
            _refuse("sel_cnt must be [rows]")
    args = (qp, ip, sp, bt, num_pages, ppb * 4, ctx_len, rows, Hq, Hkv, D, max_sel, n_first,
            n_last, xp, cp)
    try:
        _call(lib.gqa_select_blocks, idx, stream, *args)
    except GQAError as e:
        if e.status != GQA_ERR_WORKSPACE:
            raise
        with torch.cuda.device(idx):
            # (by the heads its size goes by: those of the index)
            ensure_workspace(workspace_bytes(KIND_SELECT_BLOCKS, rows, ctx_len, Hkv, D), idx)
        _call(lib.gqa_select_blocks, idx, stream, *args)
    return sel_idx, sel_cnt
