"""Python binding of the kvq C ABI (include/kvq.h): argument marshalling only.

Every function here checks tensor devices, dtypes and shapes, takes raw
device pointers and the current CUDA stream, and calls the function of the
same name in libkvq.so.  All computation happens in the library's kernels;
there is no fallback: if the library cannot be built or loaded, every call
raises.

Tensor conventions (torch is used for device memory and streams only):
  pools          uint8 (e4m3 codes) or bfloat16, [num_pages, Hkv, P, D]
  q              bfloat16 [B, Hq, D]; out float32 [B, Hq, D]
  k_new, v_new   bfloat16 [N, Hkv, D]
  block_table    int32 [B, MP]; seq_lens, req_idx, pos int32
  page_tags      int32/uint32 [num_pages]; expected_tags [B, MP]
  abort_mask     uint8 [B]; err_word int32/uint32 [1]
"""
from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional

import torch

from . import _build

KV_E4M3 = 0
KV_BF16 = 1
W_INT4 = 0
W_E4M3 = 1

ROPE_HALF = 0
ROPE_INTERLEAVED = 1
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_RAMP = 3
ROPE_BANDS = 4

ERRBIT_PAGE = 1 << 0
ERRBIT_SEQLEN = 1 << 1
ERRBIT_POS = 1 << 2
ERRBIT_REQ = 1 << 3
ERRBIT_TIMEOUT = 1 << 4
ERRBIT_EXHAUSTED = 1 << 5

STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_WORKSPACE", 3: "KVQ_ERR_CUDA",
          4: "KVQ_ERR_UNSUPPORTED"}

# every symbol include/kvq.h declares
EXPORTS = ("kvq_append", "kvq_append_check", "kvq_handoff_pages", "kvq_check_tags",
           "kvq_pages_update", "kvq_decode_attn_workspace_size", "kvq_decode_attn",
           "kvq_decode_attn_static", "kvq_wq_gemm", "kvq_selftest_wait", "kvq_status_string",
           "kvq_rope_inv_freq", "kvq_rope", "kvq_block_append", "kvq_rope_block_append",
           "kvq_block_read", "kvq_block_attn_workspace_size", "kvq_block_attn",
           "kvq_pages_workspace_size", "kvq_pages_fork", "kvq_pages_release", "kvq_pages_compact",
           "kvq_copy_pages", "kvq_block_copy_pages", "kvq_block_prefix_attn_workspace_size",
           "kvq_block_prefix_attn")
STATIC_SCRATCH_BYTES = 64 << 20


class KvqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")
        self.status = status


class CCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("kv_dtype", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class CBlockCache(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class CRope(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("mscale", ctypes.c_float)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libkvq.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_missing and not _build.up_to_date():
        _build.build()
    if not os.path.exists(_build.LIB):
        raise RuntimeError(f"CUDA library missing: {_build.LIB}")
    L = ctypes.CDLL(_build.LIB)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    cp = ctypes.POINTER(CCache)
    L.kvq_append.argtypes = [cp, vp, vp, vp, vp, i32, vp, i32, i32, vp, vp]
    L.kvq_append.restype = ctypes.c_int
    L.kvq_append_check.argtypes = [cp, vp, vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, vp, vp]
    L.kvq_append_check.restype = ctypes.c_int
    L.kvq_handoff_pages.argtypes = [cp, vp, i32, cp, vp, i32, vp, vp, i32, vp, vp]
    L.kvq_handoff_pages.restype = ctypes.c_int
    L.kvq_check_tags.argtypes = [vp, i32, i32, vp, i32, vp, i32, vp, vp, vp]
    L.kvq_check_tags.restype = ctypes.c_int
    L.kvq_pages_update.argtypes = [vp, vp, vp, i32, vp, vp, i32, i32, vp, vp, i32, vp, vp, vp,
                                   i32, vp, vp, vp]
    L.kvq_pages_update.restype = ctypes.c_int
    L.kvq_wq_gemm.argtypes = [i32, vp, vp, vp, vp, i32, i32, i32, vp, vp]
    L.kvq_wq_gemm.restype = ctypes.c_int
    L.kvq_selftest_wait.argtypes = [i32, vp, vp, vp, vp]
    L.kvq_selftest_wait.restype = ctypes.c_int
    L.kvq_decode_attn_workspace_size.argtypes = [i32, i32, i32, i32]
    L.kvq_decode_attn_workspace_size.restype = sz
    L.kvq_decode_attn.argtypes = [cp, vp, i32, i32, vp, i32, vp, vp, f32, vp, vp, sz, vp, vp]
    L.kvq_decode_attn.restype = ctypes.c_int
    L.kvq_decode_attn_static.argtypes = [cp, vp, i32, i32, vp, i32, vp, vp, f32, vp, vp, vp]
    L.kvq_decode_attn_static.restype = ctypes.c_int
    i64, f64, bp, rp = ctypes.c_int64, ctypes.c_double, ctypes.POINTER(CBlockCache), \
        ctypes.POINTER(CRope)
    L.kvq_rope_inv_freq.argtypes = [i32, f64, i32, f64, f64, f64, f64, vp, vp]
    L.kvq_rope_inv_freq.restype = ctypes.c_int
    L.kvq_rope.argtypes = [rp, vp, i32, i32, vp, i64, vp, i64, i32, vp, i64, vp, i64, i32, vp]
    L.kvq_rope.restype = ctypes.c_int
    L.kvq_block_append.argtypes = [bp, vp, i64, vp, i64, vp, i32, vp, vp, i32, i32, vp, vp]
    L.kvq_block_append.restype = ctypes.c_int
    L.kvq_rope_block_append.argtypes = [bp, rp, vp, i64, vp, i64, i32, vp, i64, vp, i64, vp, i32,
                                        vp, vp, i32, i32, vp, vp]
    L.kvq_rope_block_append.restype = ctypes.c_int
    L.kvq_block_read.argtypes = [bp, vp, i32, vp, vp, i32, i32, vp, i64, vp, i64, vp, vp]
    L.kvq_block_read.restype = ctypes.c_int
    L.kvq_block_attn_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    L.kvq_block_attn_workspace_size.restype = sz
    L.kvq_block_attn.argtypes = [bp, vp, i64, i32, vp, i32, i32, vp, vp, i32, i32, vp, f32, vp,
                                 vp, sz, vp, vp]
    L.kvq_block_attn.restype = ctypes.c_int
    L.kvq_block_prefix_attn_workspace_size.argtypes = [i32, i32, i32, i32]
    L.kvq_block_prefix_attn_workspace_size.restype = sz
    L.kvq_block_prefix_attn.argtypes = [bp, vp, i64, i32, vp, i32, i32, vp, vp, i32, i32, vp, vp,
                                        i32, vp, f32, vp, vp, sz, vp, vp]
    L.kvq_block_prefix_attn.restype = ctypes.c_int
    L.kvq_pages_workspace_size.argtypes = [i32, i32]
    L.kvq_pages_workspace_size.restype = sz
    L.kvq_pages_fork.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, i32, vp, vp, vp, i32, vp,
                                 vp, vp, vp, sz, vp, vp]
    L.kvq_pages_fork.restype = ctypes.c_int
    L.kvq_pages_release.argtypes = [vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, i32, vp, sz, vp, vp]
    L.kvq_pages_release.restype = ctypes.c_int
    L.kvq_pages_compact.argtypes = [vp, vp, vp, vp, i32, vp, vp, i32, i32, vp, vp, vp, i32, vp, vp,
                                    sz, vp, vp]
    L.kvq_pages_compact.restype = ctypes.c_int
    L.kvq_copy_pages.argtypes = [cp, vp, vp, i32, vp, vp]
    L.kvq_copy_pages.restype = ctypes.c_int
    L.kvq_block_copy_pages.argtypes = [bp, vp, vp, i32, vp, vp]
    L.kvq_block_copy_pages.restype = ctypes.c_int
    L.kvq_status_string.argtypes = [ctypes.c_int]
    L.kvq_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


# ----------------------------------------------------------------------------
# helpers
# ----------------------------------------------------------------------------

def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t: Optional[torch.Tensor], name: str, dtypes, ndim=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, has {t.dim()}")
    return ctypes.c_void_p(t.data_ptr())


def _check(fn: str, status: int):
    if status != 0:
        raise KvqError(fn, status)


I32 = (torch.int32,)
U32 = (torch.int32, torch.uint32) if hasattr(torch, "uint32") else (torch.int32,)
U8 = (torch.uint8, torch.bool)
BF16 = (torch.bfloat16,)


@dataclass
class KVCache:
    """Caller-owned paged K/V pools ([num_pages, Hkv, P, D]) and their scales."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    k_scale: float = 1.0
    v_scale: float = 1.0

    @property
    def kv_dtype(self) -> int:
        return KV_E4M3 if self.k_pool.element_size() == 1 else KV_BF16

    @property
    def shape(self):
        return tuple(self.k_pool.shape)

    def c(self) -> CCache:
        dt = (torch.uint8, torch.float8_e4m3fn, torch.bfloat16)
        _dev(self.k_pool, "k_pool", dt, 4)
        _dev(self.v_pool, "v_pool", dt, 4)
        if self.k_pool.shape != self.v_pool.shape or self.k_pool.dtype != self.v_pool.dtype:
            raise ValueError("k_pool and v_pool must match")
        NP, H, P, D = self.k_pool.shape
        return CCache(self.k_pool.data_ptr(), self.v_pool.data_ptr(), self.kv_dtype, NP, P, H, D,
                      float(self.k_scale), float(self.v_scale))

    @staticmethod
    def empty(num_pages, num_kv_heads, page_size, head_dim, kv_dtype=KV_E4M3, k_scale=1.0,
              v_scale=1.0, device="cuda"):
        dt = torch.uint8 if kv_dtype == KV_E4M3 else torch.bfloat16
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        return KVCache(torch.empty(shape, dtype=dt, device=device),
                       torch.empty(shape, dtype=dt, device=device), k_scale, v_scale)


# ----------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ----------------------------------------------------------------------------

def kvq_append(cache: KVCache, k_new, v_new, req_idx, pos, block_table, err_word=None,
               stream=None) -> None:
    L = load()
    c = cache.c()
    N = int(req_idx.shape[0])
    B, MP = block_table.shape
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        if tuple(t.shape) != (N, c.num_kv_heads, c.head_dim):
            raise ValueError(f"{n} must be [{N}, {c.num_kv_heads}, {c.head_dim}]")
    st = L.kvq_append(ctypes.byref(c), _dev(k_new, "k_new", BF16, 3), _dev(v_new, "v_new", BF16, 3),
                      _dev(req_idx, "req_idx", I32, 1), _dev(pos, "pos", I32, 1), N,
                      _dev(block_table, "block_table", I32, 2), B, MP,
                      _dev(err_word, "err_word", U32), _stream(stream))
    _check("kvq_append", st)


def kvq_append_check(cache: KVCache, k_new, v_new, req_idx, pos, block_table, seq_lens,
                     page_tags, expected_tags, abort_mask, err_word=None, stream=None) -> None:
    """kvq_append and kvq_check_tags (the cache's page size and page count)
    in one launch, with the same results as the two calls."""
    L = load()
    c = cache.c()
    N = int(req_idx.shape[0])
    B, MP = block_table.shape
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        if tuple(t.shape) != (N, c.num_kv_heads, c.head_dim):
            raise ValueError(f"{n} must be [{N}, {c.num_kv_heads}, {c.head_dim}]")
    if tuple(expected_tags.shape) != (B, MP) or abort_mask.shape[0] != B or \
            seq_lens.shape[0] != B or page_tags.shape[0] != c.num_pages:
        raise ValueError("expected_tags must be [B, MP], seq_lens and abort_mask [B], "
                         "page_tags [num_pages]")
    st = L.kvq_append_check(ctypes.byref(c), _dev(k_new, "k_new", BF16, 3),
                            _dev(v_new, "v_new", BF16, 3), _dev(req_idx, "req_idx", I32, 1),
                            _dev(pos, "pos", I32, 1), N, _dev(block_table, "block_table", I32, 2),
                            B, MP, _dev(seq_lens, "seq_lens", I32, 1),
                            _dev(page_tags, "page_tags", U32, 1),
                            _dev(expected_tags, "expected_tags", U32, 2),
                            _dev(abort_mask, "abort_mask", U8, 1), _dev(err_word, "err_word", U32),
                            _stream(stream))
    _check("kvq_append_check", st)


def kvq_handoff_pages(src: KVCache, src_block_table, dst: KVCache, dst_block_table, count,
                      first=None, err_word=None, stream=None) -> None:
    """Prefill -> decode handoff: tokens [first[b], first[b] + count[b]) of
    every request b, read from the paged bf16 cache `src` through
    src_block_table [B, src_MP] and stored into `dst` through
    dst_block_table [B, dst_MP] with kvq_append's rounding."""
    L = load()
    cs, cd = src.c(), dst.c()
    B, src_MP = src_block_table.shape
    if dst_block_table.shape[0] != B or count.shape[0] != B or \
            (first is not None and first.shape[0] != B):
        raise ValueError("dst_block_table, count and first must have B rows")
    st = L.kvq_handoff_pages(ctypes.byref(cs), _dev(src_block_table, "src_block_table", I32, 2),
                             src_MP, ctypes.byref(cd),
                             _dev(dst_block_table, "dst_block_table", I32, 2),
                             int(dst_block_table.shape[1]), _dev(first, "first", I32, 1),
                             _dev(count, "count", I32, 1), B, _dev(err_word, "err_word", U32),
                             _stream(stream))
    _check("kvq_handoff_pages", st)


def kvq_check_tags(block_table, seq_lens, page_size: int, page_tags, expected_tags, abort_mask,
                   stream=None) -> None:
    L = load()
    B, MP = block_table.shape
    if tuple(expected_tags.shape) != (B, MP) or abort_mask.shape[0] != B:
        raise ValueError("expected_tags must be [B, MP] and abort_mask [B]")
    st = L.kvq_check_tags(_dev(block_table, "block_table", I32, 2), B, MP,
                          _dev(seq_lens, "seq_lens", I32, 1), int(page_size),
                          _dev(page_tags, "page_tags", U32, 1), int(page_tags.shape[0]),
                          _dev(expected_tags, "expected_tags", U32, 2),
                          _dev(abort_mask, "abort_mask", U8, 1), _stream(stream))
    _check("kvq_check_tags", st)


@dataclass
class PageState:
    """The page allocator's device state (include/kvq.h, kvq_pages_update):
    free_stack int32 [num_pages] with free_count[0] live entries (top = last),
    page_tags int32/uint32 [num_pages], block_table int32 [B, MP] and
    expected_tags int32/uint32 [B, MP] (the tables kvq_check_tags reads)."""
    free_stack: torch.Tensor
    free_count: torch.Tensor
    page_tags: torch.Tensor
    block_table: torch.Tensor
    expected_tags: torch.Tensor


def kvq_pages_update(state: PageState, rel_req=None, rel_npages=None, acq_req=None,
                     acq_first=None, acq_npages=None, acq_ok=None, err_word=None,
                     stream=None) -> None:
    """One batch of page releases then acquisitions (see include/kvq.h)."""
    L = load()
    num_pages = int(state.free_stack.shape[0])
    B, MP = state.block_table.shape
    if tuple(state.page_tags.shape) != (num_pages,) or state.free_count.numel() != 1:
        raise ValueError("page_tags must be [num_pages] and free_count [1]")
    if tuple(state.expected_tags.shape) != (B, MP):
        raise ValueError("expected_tags must match block_table")
    n_rel = 0 if rel_req is None else int(rel_req.shape[0])
    n_acq = 0 if acq_req is None else int(acq_req.shape[0])
    if n_rel and rel_npages.shape != rel_req.shape:
        raise ValueError("rel_npages must match rel_req")
    if n_acq and (acq_first.shape != acq_req.shape or acq_npages.shape != acq_req.shape or
                  acq_ok is None or acq_ok.shape != acq_req.shape):
        raise ValueError("acq_first, acq_npages and acq_ok must match acq_req")
    st = L.kvq_pages_update(_dev(state.free_stack, "free_stack", I32, 1),
                            _dev(state.free_count, "free_count", I32),
                            _dev(state.page_tags, "page_tags", U32, 1), num_pages,
                            _dev(state.block_table, "block_table", I32, 2),
                            _dev(state.expected_tags, "expected_tags", U32, 2), B, MP,
                            _dev(rel_req, "rel_req", I32, 1), _dev(rel_npages, "rel_npages", I32, 1),
                            n_rel, _dev(acq_req, "acq_req", I32, 1),
                            _dev(acq_first, "acq_first", I32, 1),
                            _dev(acq_npages, "acq_npages", I32, 1), n_acq,
                            _dev(acq_ok, "acq_ok", U8, 1), _dev(err_word, "err_word", U32),
                            _stream(stream))
    _check("kvq_pages_update", st)


def kvq_wq_gemm(w_dtype: int, w, scales, x, y, err_word=None, stream=None) -> None:
    """y [M, N] fp32 = x [M, K] bf16 times the quantised weights (include/kvq.h):
    W_INT4: w uint8 [N, K/2], scales bf16 (or int16 bits) [N, K/128];
    W_E4M3: w uint8 [N, K], scales fp32 [N].  err_word: optional int32 [1]
    device tensor that collects KVQ_ERRBIT_TIMEOUT."""
    L = load()
    M, K = x.shape
    N = int(w.shape[0])
    if tuple(y.shape) != (M, N):
        raise ValueError("y must be [M, N]")
    if w_dtype == W_INT4:
        if tuple(w.shape) != (N, K // 2) or tuple(scales.shape) != (N, K // 128):
            raise ValueError("INT4 weights must be [N, K/2] with scales [N, K/128]")
        sc = _dev(scales, "scales", (torch.bfloat16, torch.int16), 2)
    else:
        if tuple(w.shape) != (N, K) or tuple(scales.shape) != (N,):
            raise ValueError("e4m3 weights must be [N, K] with scales [N]")
        sc = _dev(scales, "scales", (torch.float32,), 1)
    st = L.kvq_wq_gemm(int(w_dtype), _dev(w, "w", U8, 2), sc, _dev(x, "x", BF16, 2),
                       _dev(y, "y", (torch.float32,), 2), M, N, K,
                       _dev(err_word, "err_word", U32), _stream(stream))
    _check("kvq_wq_gemm", st)


def kvq_selftest_wait(which: int, src, err_word, landed, stream=None) -> None:
    """Launch the bounded-wait self-test (include/kvq.h): which = 0 the split
    attention kernels' wait, 1 the weight ring's.  src: 16 int32 on the
    device; err_word, landed: int32 [1] device tensors."""
    L = load()
    st = L.kvq_selftest_wait(int(which), _dev(src, "src", U32), _dev(err_word, "err_word", U32),
                             _dev(landed, "landed", U32), _stream(stream))
    _check("kvq_selftest_wait", st)


def kvq_decode_attn_workspace_size(B: int, Hq: int, num_kv_heads: int, head_dim: int) -> int:
    return int(load().kvq_decode_attn_workspace_size(B, Hq, num_kv_heads, head_dim))


def workspace(B: int, Hq: int, num_kv_heads: int, head_dim: int, device="cuda") -> torch.Tensor:
    """Allocate (with torch) a workspace of the size kvq_decode_attn needs."""
    n = kvq_decode_attn_workspace_size(B, Hq, num_kv_heads, head_dim)
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_decode_attn(cache: KVCache, q, block_table, seq_lens, out, workspace, abort_mask=None,
                    sm_scale: Optional[float] = None, err_word=None, stream=None) -> None:
    L = load()
    c = cache.c()
    B, Hq, D = q.shape
    if D != c.head_dim or tuple(out.shape) != (B, Hq, D):
        raise ValueError("q / out shapes do not match the cache")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens must have B rows")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    st = L.kvq_decode_attn(ctypes.byref(c), _dev(q, "q", BF16, 3), B, Hq,
                           _dev(block_table, "block_table", I32, 2), int(block_table.shape[1]),
                           _dev(seq_lens, "seq_lens", I32, 1),
                           _dev(abort_mask, "abort_mask", U8, 1), float(sm_scale),
                           _dev(out, "out", (torch.float32,), 3),
                           _dev(workspace, "workspace", (torch.uint8,), 1),
                           workspace.numel() * workspace.element_size(),
                           _dev(err_word, "err_word", U32), _stream(stream))
    _check("kvq_decode_attn", st)


def kvq_decode_attn_static(cache: KVCache, q, block_table, seq_lens, out, abort_mask=None,
                           sm_scale: Optional[float] = None, err_word=None, stream=None) -> None:
    """kvq_decode_attn with the library's own static scratch instead of a
    caller workspace, for callers that cannot allocate device memory (see
    include/kvq.h).  Calls that can overlap on the GPU must not be issued."""
    L = load()
    c = cache.c()
    B, Hq, D = q.shape
    if D != c.head_dim or tuple(out.shape) != (B, Hq, D):
        raise ValueError("q / out shapes do not match the cache")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table / seq_lens must have B rows")
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(D)
    st = L.kvq_decode_attn_static(ctypes.byref(c), _dev(q, "q", BF16, 3), B, Hq,
                                  _dev(block_table, "block_table", I32, 2),
                                  int(block_table.shape[1]), _dev(seq_lens, "seq_lens", I32, 1),
                                  _dev(abort_mask, "abort_mask", U8, 1), float(sm_scale),
                                  _dev(out, "out", (torch.float32,), 3),
                                  _dev(err_word, "err_word", U32), _stream(stream))
    _check("kvq_decode_attn_static", st)


# ----------------------------------------------------------------------------
# the block-scaled cache (include/kvq.h): rotary positions, append, read-back
# and attention over ragged steps.  Request b's rows are tok_start[b] ..
# tok_start[b + 1] - 1 (int32 [B + 1]; None: one row a request) and seq_lens[b]
# its length after the step.  q, k and v are [rows, heads, D] bf16 whose
# last two dims are contiguous; the rows may be slices of a wider projection.
# Every tensor of a call lies on one device; without `stream` the call runs on
# that device's current stream.
# ----------------------------------------------------------------------------

_F8 = (torch.uint8, torch.float8_e4m3fn)
_F32 = (torch.float32,)
_F64 = (torch.float64,)
_BYTES = (torch.uint8,)


# The checks below run on every call of a decode step, so they are written for
# few attribute look-ups: a decode step's kernels take a few microseconds.

def _arr(t, name, dtypes, shape, dev):
    """Pointer of a contiguous array of the given dtypes and shape on device dev."""
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != dev or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtypes[0]} tensor {list(shape)} on "
                         f"cuda:{dev}; it is {t.dtype} {list(t.shape)} on {t.device}"
                         f"{'' if t.is_contiguous() else ', not contiguous'}")
    return t.data_ptr()


def _rows(t, name, n, heads, D, dev):
    """(pointer, token stride) of a bf16 [n, heads, D] tensor strided by token."""
    if t is None:
        raise ValueError(f"{name} is missing")
    st = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != (n, heads, D) or t.get_device() != dev or \
            st[2] != 1 or (st[1] != D and heads > 1):
        raise ValueError(f"{name} must be a bfloat16 tensor {[n, heads, D]} on cuda:{dev} with "
                         f"contiguous rows of heads; it is {t.dtype} {list(t.shape)}, strides "
                         f"{list(st)}, on {t.device}")
    return t.data_ptr(), (st[0] if n > 1 else heads * D)


def _device(t, name) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _launch(fn, name, dev, stream, args):
    """Calls the library with device `dev` current, on `stream` or that device's
    current stream."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, raw)
    if st != 0:
        raise KvqError(name, st)


@dataclass(frozen=True)
class BlockKVCache:
    """Caller-owned e4m3 pools [num_pages, Hkv, P, D] and the scale of each
    (page, kv head) block of K and of V: scales fp32 [num_pages, Hkv, 2].  A
    handle: the tensors are checked once, here, and held."""
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    scales: torch.Tensor

    def __post_init__(self):
        shape, dev = tuple(self.k_pool.shape), _device(self.k_pool, "k_pool")
        if len(shape) != 4:
            raise ValueError("k_pool must have 4 dims")
        NP, H, P, D = shape
        c = CBlockCache(_arr(self.k_pool, "k_pool", _F8, shape, dev),
                        _arr(self.v_pool, "v_pool", _F8, shape, dev),
                        _arr(self.scales, "scales", _F32, (NP, H, 2), dev), NP, P, H, D)
        object.__setattr__(self, "_c", (ctypes.byref(c), dev, H, D))

    def c(self):
        """(reference to the C descriptor, device, kv heads, head_dim)"""
        return self._c

    @staticmethod
    def empty(num_pages, num_kv_heads, page_size, head_dim, device="cuda"):
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        return BlockKVCache(torch.empty(shape, dtype=torch.uint8, device=device),
                            torch.empty(shape, dtype=torch.uint8, device=device),
                            torch.ones((num_pages, num_kv_heads, 2), device=device))


@dataclass(frozen=True)
class Rope:
    """Rotary positions: inv_freq float64 [rotary_dim / 2] on the device
    (radians per position), the pairs' layout and the factor on the result.  A
    handle, like BlockKVCache."""
    inv_freq: torch.Tensor
    layout: int = ROPE_HALF
    mscale: float = 1.0

    def __post_init__(self):
        dev = _device(self.inv_freq, "inv_freq")
        n = self.inv_freq.numel()
        c = CRope(_arr(self.inv_freq, "inv_freq", _F64, (n,), dev), 2 * n, int(self.layout),
                  float(self.mscale))
        object.__setattr__(self, "_c", (ctypes.byref(c), dev))

    def c(self):
        """(reference to the C descriptor, device)"""
        return self._c


def kvq_rope_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: int = ROPE_PLAIN,
                      factor: float = 1.0, orig_len: float = 0.0, low: float = 1.0,
                      high: float = 32.0):
    """(float64 tensor [rotary_dim / 2] on the host, mscale) of a frequency
    scheme (include/kvq.h): move the tensor to the device once and keep it."""
    out = torch.empty(max(rotary_dim, 0) // 2, dtype=torch.float64)
    m = ctypes.c_float()
    st = load().kvq_rope_inv_freq(int(rotary_dim), float(base), int(scaling), float(factor),
                                  float(orig_len), float(low), float(high),
                                  ctypes.c_void_p(out.data_ptr()), ctypes.byref(m))
    _check("kvq_rope_inv_freq", st)
    return out, m.value


def _rope(rope, dev):
    r, d = rope.c()
    if d != dev:
        raise ValueError(f"inv_freq lies on cuda:{d}, the call's tensors on cuda:{dev}")
    return r


def kvq_rope(rope: Rope, pos, q, q_out, k=None, k_out=None, stream=None) -> None:
    """Rotate rows of q into q_out (and of k into k_out); row t stands at
    position pos[t] (int32).  An output may be its input."""
    L = _lib or load()
    N, Hq, D = q.shape
    dev = _device(q, "q")
    qa, qb = _rows(q, "q", N, Hq, D, dev), _rows(q_out, "q_out", N, Hq, D, dev)
    Hk, ka, kb = 0, (None, 0), (None, 0)
    if k is None and k_out is not None:
        raise ValueError("k is missing")
    if k is not None:
        Hk = k.shape[1]
        ka, kb = _rows(k, "k", N, Hk, D, dev), _rows(k_out, "k_out", N, Hk, D, dev)
    _launch(L.kvq_rope, "kvq_rope", dev, stream,
            (_rope(rope, dev), _arr(pos, "pos", I32, (N,), dev), N, D, *qa, *qb, Hq, *ka, *kb, Hk))


def _step(tok_start, seq_lens, block_table, dev, name="seq_lens"):
    B, MP = block_table.shape
    return (None if tok_start is None else _arr(tok_start, "tok_start", I32, (B + 1,), dev),
            None if seq_lens is None else _arr(seq_lens, name, I32, (B,), dev),
            _arr(block_table, "block_table", I32, (B, MP), dev), B, MP)


def _err(err_word, dev):
    return None if err_word is None else _arr(err_word, "err_word", U32, (1,), dev)


def kvq_block_append(cache: BlockKVCache, k_new, v_new, tok_start, seq_lens, block_table,
                     err_word=None, stream=None) -> None:
    """Quantise rows of k_new / v_new [rows, Hkv, D] into their requests' pages
    and set the blocks' scales (include/kvq.h)."""
    L = _lib or load()
    c, dev, H, D = cache.c()
    N = k_new.shape[0]
    ts, sl, bt, B, MP = _step(tok_start, seq_lens, block_table, dev)
    _launch(L.kvq_block_append, "kvq_block_append", dev, stream,
            (c, *_rows(k_new, "k_new", N, H, D, dev), *_rows(v_new, "v_new", N, H, D, dev), ts, N,
             sl, bt, B, MP, _err(err_word, dev)))


def kvq_rope_block_append(cache: BlockKVCache, rope: Rope, q, q_out, k_new, v_new, tok_start,
                          seq_lens, block_table, err_word=None, stream=None) -> None:
    """kvq_block_append with K rotated on the way in, and q rotated into q_out
    (both may be None), in one launch."""
    L = _lib or load()
    c, dev, H, D = cache.c()
    N = k_new.shape[0]
    Hq, qa, qb = 0, (None, 0), (None, 0)
    if q is None and q_out is not None:
        raise ValueError("q is missing")
    if q is not None:
        Hq = q.shape[1]
        qa, qb = _rows(q, "q", N, Hq, D, dev), _rows(q_out, "q_out", N, Hq, D, dev)
    ts, sl, bt, B, MP = _step(tok_start, seq_lens, block_table, dev)
    _launch(L.kvq_rope_block_append, "kvq_rope_block_append", dev, stream,
            (c, _rope(rope, dev), *qa, *qb, Hq, *_rows(k_new, "k_new", N, H, D, dev),
             *_rows(v_new, "v_new", N, H, D, dev), ts, N, sl, bt, B, MP, _err(err_word, dev)))


def kvq_block_read(cache: BlockKVCache, tok_start, first, block_table, k_out, v_out,
                   err_word=None, stream=None) -> None:
    """Read cached tokens back into k_out / v_out [rows, Hkv, D] bf16: row i of
    request b is its position first[b] + i (first None: from position 0)."""
    L = _lib or load()
    c, dev, H, D = cache.c()
    N = k_out.shape[0]
    ts, fi, bt, B, MP = _step(tok_start, first, block_table, dev, "first")
    _launch(L.kvq_block_read, "kvq_block_read", dev, stream,
            (c, ts, N, fi, bt, B, MP, *_rows(k_out, "k_out", N, H, D, dev),
             *_rows(v_out, "v_out", N, H, D, dev), _err(err_word, dev)))


def kvq_block_attn_workspace_size(B: int, max_q: int, Hq: int, num_kv_heads: int,
                                  head_dim: int) -> int:
    return int(load().kvq_block_attn_workspace_size(B, max_q, Hq, num_kv_heads, head_dim))


def block_workspace(B: int, max_q: int, Hq: int, num_kv_heads: int, head_dim: int,
                    device="cuda") -> torch.Tensor:
    """Allocate (with torch) a workspace of the size kvq_block_attn needs."""
    with torch.cuda.device(device):
        n = kvq_block_attn_workspace_size(B, max_q, Hq, num_kv_heads, head_dim)
    if n == 0:
        raise ValueError("kvq_block_attn does not support these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_block_attn(cache: BlockKVCache, q, tok_start, seq_lens, block_table, out, workspace,
                   max_q: int = 1, abort_mask=None, sm_scale: Optional[float] = None,
                   err_word=None, stream=None) -> None:
    """Causal attention of each request's rows (at most max_q a request) over
    its cached tokens: q [rows, Hq, D] bf16, out [rows, Hq, D] fp32."""
    L = _lib or load()
    c, dev, _, D = cache.c()
    N, Hq = q.shape[0], q.shape[1]
    ts, sl, bt, B, MP = _step(tok_start, seq_lens, block_table, dev)
    _launch(L.kvq_block_attn, "kvq_block_attn", dev, stream,
            (c, *_rows(q, "q", N, Hq, D, dev), Hq, ts, N, max_q, sl, bt, B, MP,
             None if abort_mask is None else _arr(abort_mask, "abort_mask", U8, (B,), dev),
             D ** -0.5 if sm_scale is None else sm_scale,
             _arr(out, "out", _F32, (N, Hq, D), dev),
             _arr(workspace, "workspace", _BYTES, workspace.shape, dev), workspace.numel(),
             _err(err_word, dev)))


def kvq_block_prefix_attn_workspace_size(n_tokens: int, Hq: int, num_kv_heads: int,
                                         head_dim: int) -> int:
    return int(load().kvq_block_prefix_attn_workspace_size(n_tokens, Hq, num_kv_heads, head_dim))


def block_prefix_workspace(n_tokens: int, Hq: int, num_kv_heads: int, head_dim: int,
                           device="cuda") -> torch.Tensor:
    """Allocate (with torch) a workspace of the size kvq_block_prefix_attn needs for at most
    n_tokens rows."""
    with torch.cuda.device(device):
        n = kvq_block_prefix_attn_workspace_size(n_tokens, Hq, num_kv_heads, head_dim)
    if n == 0:
        raise ValueError("kvq_block_prefix_attn does not support these sizes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def kvq_block_prefix_attn(cache: BlockKVCache, q, tok_start, seq_lens, block_table, group_start,
                          prefix_pages, out, workspace, max_q: int = 1, abort_mask=None,
                          sm_scale: Optional[float] = None, err_word=None, stream=None) -> None:
    """Causal attention of each request's rows (at most max_q a request) over its cached tokens,
    for requests in groups that share their first pages: requests group_start[g] ..
    group_start[g + 1] - 1 (int32 [groups + 1]; None: no groups) hold the same prefix_pages[g]
    pages in front (int32 [groups]), which are read once for the group.  q and out [rows, Hq,
    D] bf16."""
    L = _lib or load()
    c, dev, _, D = cache.c()
    N, Hq = q.shape[0], q.shape[1]
    ts, sl, bt, B, MP = _step(tok_start, seq_lens, block_table, dev)
    if group_start is None:
        gs, pp, n_groups = None, None, 0
        if prefix_pages is not None:
            raise ValueError("group_start is missing")
    else:
        n_groups = group_start.shape[0] - 1
        gs = _arr(group_start, "group_start", I32, (n_groups + 1,), dev)
        if prefix_pages is None:
            raise ValueError("prefix_pages is missing")
        pp = _arr(prefix_pages, "prefix_pages", I32, (n_groups,), dev)
    _launch(L.kvq_block_prefix_attn, "kvq_block_prefix_attn", dev, stream,
            (c, *_rows(q, "q", N, Hq, D, dev), Hq, ts, N, max_q, sl, bt, B, MP, gs, pp, n_groups,
             None if abort_mask is None else _arr(abort_mask, "abort_mask", U8, (B,), dev),
             D ** -0.5 if sm_scale is None else sm_scale,
             _arr(out, "out", BF16, (N, Hq, D), dev), *_ws(workspace, dev), _err(err_word, dev)))


# ----------------------------------------------------------------------------
# pages that several requests hold (include/kvq.h).  `state` is the allocator's
# PageState and `shares` int32 [num_pages] its count of holders beyond the first
# (zeros at the start).  Every tensor of a call lies on one device, as above.
# ----------------------------------------------------------------------------

def kvq_pages_workspace_size(num_pages: int, B: int) -> int:
    return int(load().kvq_pages_workspace_size(num_pages, B))


def pages_workspace(num_pages: int, B: int, device="cuda") -> torch.Tensor:
    """Allocate (with torch) a workspace for kvq_pages_fork, _release and _compact."""
    n = kvq_pages_workspace_size(num_pages, B)
    if n == 0:
        raise ValueError("num_pages and B must lie between 1 and 2^30")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _pages(state: PageState, shares, tags=True):
    """(device, num_pages, B, MP, pointers of the state's arrays)"""
    dev = _device(state.block_table, "block_table")
    n = state.free_stack.numel()
    B, MP = state.block_table.shape
    p = [_arr(state.free_stack, "free_stack", I32, (n,), dev),
         _arr(state.free_count, "free_count", I32, (1,), dev)]
    if tags:
        p.append(_arr(state.page_tags, "page_tags", U32, (n,), dev))
    p += [_arr(shares, "shares", I32, (n,), dev), n,
          _arr(state.block_table, "block_table", I32, (B, MP), dev)]
    if tags:
        p.append(_arr(state.expected_tags, "expected_tags", U32, (B, MP), dev))
    return dev, B, [*p, B, MP]


def _ws(workspace, dev):
    return _arr(workspace, "workspace", _BYTES, workspace.shape, dev), workspace.numel()


def kvq_pages_fork(state: PageState, shares, src, dst, tokens, page_size: int, copy_src, copy_dst,
                   fork_ok, workspace, err_word=None, stream=None) -> None:
    """Give request dst[i] the first tokens[i] tokens of request src[i]: whole pages
    shared, a part-filled last one replaced by a fresh page, whose copy is
    (copy_src[i], copy_dst[i]) for kvq_copy_pages or kvq_block_copy_pages."""
    L = _lib or load()
    dev, _, p = _pages(state, shares)
    n = src.shape[0]
    _launch(L.kvq_pages_fork, "kvq_pages_fork", dev, stream,
            (*p, page_size, _arr(src, "src", I32, (n,), dev), _arr(dst, "dst", I32, (n,), dev),
             _arr(tokens, "tokens", I32, (n,), dev), n, _arr(copy_src, "copy_src", I32, (n,), dev),
             _arr(copy_dst, "copy_dst", I32, (n,), dev), _arr(fork_ok, "fork_ok", U8, (n,), dev),
             *_ws(workspace, dev), _err(err_word, dev)))


def kvq_pages_release(state: PageState, shares, req, first, npages, workspace, err_word=None,
                      stream=None) -> None:
    """Request req[j] lets go of logical pages first[j] .. first[j] + npages[j] - 1 (first
    None: from page 0); a page is free when its last holder is gone."""
    L = _lib or load()
    dev, _, p = _pages(state, shares, tags=False)
    n = req.shape[0]
    _launch(L.kvq_pages_release, "kvq_pages_release", dev, stream,
            (*p, _arr(req, "req", I32, (n,), dev),
             None if first is None else _arr(first, "first", I32, (n,), dev),
             _arr(npages, "npages", I32, (n,), dev), n, *_ws(workspace, dev), _err(err_word, dev)))


def kvq_pages_compact(state: PageState, shares, held, copy_src, copy_dst, n_moves, workspace,
                      err_word=None, stream=None) -> None:
    """Rename the pages in use to the lowest ids; copy_src[k] -> copy_dst[k] (the rest -1)
    are the pages that kvq_copy_pages or kvq_block_copy_pages then moves.  held int32
    [B]: block-table entries in use of every request; the lists have num_pages // 2
    entries or more; n_moves int32 [1]."""
    L = _lib or load()
    dev, B, p = _pages(state, shares)
    cap = copy_src.shape[0]
    _launch(L.kvq_pages_compact, "kvq_pages_compact", dev, stream,
            (*p, _arr(held, "held", I32, (B,), dev), _arr(copy_src, "copy_src", I32, (cap,), dev),
             _arr(copy_dst, "copy_dst", I32, (cap,), dev), cap,
             _arr(n_moves, "n_moves", I32, (1,), dev), *_ws(workspace, dev), _err(err_word, dev)))


def _pairs(src, dst, dev):
    n = src.shape[0]
    return _arr(src, "src", I32, (n,), dev), _arr(dst, "dst", I32, (n,), dev), n


def kvq_copy_pages(cache: KVCache, src, dst, err_word=None, stream=None) -> None:
    """Copy whole pages of K and V: src[i] to dst[i]; pairs with a negative page are left
    out."""
    L = _lib or load()
    c = cache.c()
    dev = cache.k_pool.get_device()
    if cache.v_pool.get_device() != dev:
        raise ValueError("k_pool and v_pool lie on different devices")
    _launch(L.kvq_copy_pages, "kvq_copy_pages", dev, stream,
            (ctypes.byref(c), *_pairs(src, dst, dev), _err(err_word, dev)))


def kvq_block_copy_pages(cache: BlockKVCache, src, dst, err_word=None, stream=None) -> None:
    """kvq_copy_pages for the block-scaled cache: codes and scales."""
    L = _lib or load()
    c, dev, _, _ = cache.c()
    _launch(L.kvq_block_copy_pages, "kvq_block_copy_pages", dev, stream,
            (c, *_pairs(src, dst, dev), _err(err_word, dev)))
