"""Python binding of libdescbuild.so: batched GPU-range -> DMA-descriptor translation.

The functions here have the names of the C ABI in ``include/descbuild.h``
(without the ``db_`` prefix) and only marshal arguments: torch CUDA tensors
become device pointers, the stream becomes a ``cudaStream_t``, and a negative
return code becomes a ``DescBuildError``. Every step of the computation runs
in the library's CUDA kernels; there is no fallback. Importing this package
fails loudly when the library has not been built.

Record layouts (all tensors contiguous, on the GPU):
  PRP request  16 B  {u64 off; u32 len; u32 rsvd}     -> int64 [n, 2]
  PRP output   16 B  {u64 prp1; u64 prp2}             -> int64 [n, 2]
  range        16 B  {u64 addr; u64 size}             -> int64 [n, 2]
  put          16 B  {u64 off; u32 bytes; u16 pe; u16 qp} -> int64 [n, 2]
  WQE          64 B                                    -> uint8 [rings, depth, 64]
  counters     32 B  {total, n_invalid, n_overflow, err} -> int64 [4]
Records of the paged cache (include/pagecache.h), u32 fields as int32 bits:
  cut           8 B  {seq, keep}                       -> int32 [n, 2]
  grow          8 B  {seq, tokens}                     -> int32 [n, 2]
  fork         16 B  {parent, child, tokens, rsvd}     -> int32 [n, 4]
  move         16 B  {src, dst, tokens, rsvd}          -> int32 [n, 4]
What the pages hold (include/cachedata.h) are tensors of their own types: the
keys or values of a layer [pages, tokens, heads, width] (token_dim 1) or
[pages, heads, tokens, width] (token_dim 2), bfloat16, float16, float8_e4m3fn
or int8, the 8-bit ones with float32 scales of the same axes but the last.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct

import numpy as np
import torch

from . import build as _build

__all__ = [
    "DescBuildError", "lib_path", "workspace", "prp_workspace_size", "prp_build",
    "prp_build_static", "PRP_STATIC_MAX_REQUESTS",
    "mr_workspace_size", "mr_lookup", "mr_lookup_overlap", "wqe_workspace_size",
    "wqe_vmm_workspace_size", "wqe_bucket", "wqe_bucket_vmm", "wqe_bucket_transport",
    "XPORT_RDMA", "XPORT_P2P", "XPORT_SDMA",
    "strerror", "CQ_SLOT_DTYPE", "CQ_MAX_SLOTS", "CQ_MAX_DEPTH", "CQ_TIMED", "cq_slots",
    "cq_slot_fields",
    "mr_capacity_for", "mr_register_workspace_size", "mr_register",
    "mr_deregister_workspace_size", "mr_deregister", "MR_NEW", "MR_NEW_DUP", "DEREG_OK",
    "DEREG_RELEASED", "DEREG_STALE",
    "cq_mirror", "cq_attach", "cq_detach", "cq_wait_ack", "cq_host_reap", "cq_request_stop",
    "PRP_OK", "PRP_INVALID", "PRP_OVERFLOW", "MR_MISS", "MR_EXACT", "MR_CONTAINED",
    "MR_INVALID", "ERR_TIMEOUT", "ERR_RING_OVERFLOW", "ERR_TABLE_ORDER", "PRP_ZERO_TAIL",
    "PRP_SCHED_SINGLE", "PRP_SCHED_SPLIT",
    "PageTables", "page_workspace_size", "page_extend", "page_fork", "page_free", "page_compact",
    "page_copy", "PAGE_NONE", "PAGE_ALL", "PAGE_OK", "PAGE_INVALID", "PAGE_SHORT",
    "ERR_PAGE_TABLE",
    "cache_write", "cache_read", "cache_attention_workspace_size", "cache_attention",
    "draft_verify", "cache_keep",
]

PRP_OK, PRP_INVALID, PRP_OVERFLOW = 0, 1, 2
MR_MISS, MR_EXACT, MR_CONTAINED, MR_INVALID = 0, 1, 2, 3
ERR_TIMEOUT, ERR_RING_OVERFLOW, ERR_TABLE_ORDER = 1, 2, 4
PRP_ZERO_TAIL = 1
PRP_SCHED_SINGLE, PRP_SCHED_SPLIT = 2, 4
XPORT_RDMA, XPORT_P2P, XPORT_SDMA = 0, 1, 2
PAGE_NONE, PAGE_ALL = -1, -1  # a table entry without a page; "every token" of a move (0xFFFFFFFF)
PAGE_OK, PAGE_INVALID, PAGE_SHORT = 0, 1, 2
ERR_PAGE_TABLE = 8

lib_path = _build.LIB


class DescBuildError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = _lib.db_strerror(code).decode()
        if code == -5:
            msg += f" (cudaError {_lib.db_last_cuda_error()})"
        super().__init__(f"{fn}: {msg} [{code}]")


def _load():
    if not os.path.exists(lib_path):
        raise ImportError(
            f"{lib_path} is missing: build it with `python -c 'import __graft_entry__ as g; "
            f"g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(lib_path)
    vp, u64, u32, i32, sz = (ctypes.c_void_p, ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int,
                             ctypes.c_size_t)
    psz = ctypes.POINTER(ctypes.c_size_t)
    lib.db_prp_workspace_size.argtypes = [u64, psz]
    lib.db_prp_build.argtypes = [vp, u64, vp, u64, u64, u64, vp, vp, vp, vp, vp, u32, vp, sz, vp]
    lib.db_prp_build_static.argtypes = [vp, u64, vp, u64, u64, u64, vp, vp, vp, vp, vp, u32, vp]
    lib.db_mr_workspace_size.argtypes = [u64, psz]
    lib.db_mr_lookup.argtypes = [vp, u64, vp, vp, vp, u64, vp, vp, vp, vp, vp, sz, vp]
    lib.db_mr_lookup_overlap.argtypes = lib.db_mr_lookup.argtypes
    lib.db_wqe_workspace_size.argtypes = [u64, u32, psz]
    lib.db_wqe_vmm_workspace_size.argtypes = [u64, u32, u32, u64, u32, psz]
    lib.db_wqe_vmm_workspace_size.restype = i32
    lib.db_wqe_bucket.argtypes = [vp, u64, vp, vp, u32, u32, u64, u32, u64, vp, u64, vp, vp, vp,
                                  vp, sz, vp]
    lib.db_wqe_bucket_vmm.argtypes = [vp, u64, vp, vp, vp, u32, u32, u32, u64, u64, vp, u64, vp,
                                      vp, u32, vp, vp, vp, sz, vp]
    lib.db_wqe_bucket_transport.argtypes = [vp, u64, vp, vp, vp, u32, u32, u64, u32, u64, vp,
                                            u64, vp, vp, vp, vp, vp, vp, sz, vp]
    for name in ("db_prp_workspace_size", "db_prp_build", "db_prp_build_static",
                 "db_mr_workspace_size",
                 "db_mr_lookup", "db_mr_lookup_overlap", "db_wqe_workspace_size", "db_wqe_bucket",
                 "db_wqe_bucket_vmm", "db_wqe_bucket_transport",
                 "db_last_cuda_error"):
        getattr(lib, name).restype = i32
    lib.db_mr_capacity_for.argtypes = [u64]
    lib.db_mr_capacity_for.restype = u64
    lib.db_mr_register_workspace_size.argtypes = [u64, u64, psz]
    lib.db_mr_register.argtypes = [vp, u64, vp, u32, vp, vp, vp, vp, u64, vp, vp, vp, vp, u64,
                                   vp, vp, vp, vp, vp, sz, vp]
    lib.db_mr_deregister_workspace_size.argtypes = [u64, u64, psz]
    lib.db_mr_deregister.argtypes = [vp, u64, vp, vp, vp, vp, u64, vp, vp, vp, vp, vp, vp, vp,
                                     vp, sz, vp]
    for name in ("db_mr_register_workspace_size", "db_mr_register",
                 "db_mr_deregister_workspace_size", "db_mr_deregister"):
        getattr(lib, name).restype = i32
    lib.db_cq_mirror.argtypes = [vp, u32, vp, u64, vp, vp]
    lib.db_cq_attach.argtypes = [vp, u64, u64, u32, ctypes.POINTER(ctypes.c_uint32)]
    lib.db_cq_detach.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.db_cq_wait_ack.argtypes = [vp, u32, u64]
    lib.db_cq_host_reap.argtypes = [vp, u32, ctypes.POINTER(ctypes.c_uint32),
                                    ctypes.POINTER(ctypes.c_uint32), vp, u32]
    lib.db_cq_request_stop.argtypes = [vp]
    lib.db_cq_request_stop.restype = None
    for name in ("db_cq_mirror", "db_cq_attach", "db_cq_detach", "db_cq_wait_ack",
                 "db_cq_host_reap"):
        getattr(lib, name).restype = i32
    lib.db_page_workspace_size.argtypes = [u32, u32, psz]
    lib.db_page_extend.argtypes = [vp, vp, u32, vp, vp, vp, vp, vp, sz, vp]
    lib.db_page_fork.argtypes = [vp, vp, u32, vp, vp, vp, sz, vp]
    lib.db_page_free.argtypes = lib.db_page_fork.argtypes
    lib.db_page_compact.argtypes = [vp, vp, vp, u32, vp, vp, vp, sz, vp]
    lib.db_page_copy.argtypes = [vp, u32, vp, vp, vp, vp, vp, vp]
    for name in ("db_page_workspace_size", "db_page_extend", "db_page_fork", "db_page_free",
                 "db_page_compact", "db_page_copy"):
        getattr(lib, name).restype = i32
    f32 = ctypes.c_float
    lib.db_cache_write.argtypes = [vp, vp, vp, vp, vp, u32, vp, vp, vp]
    lib.db_cache_read.argtypes = [vp, vp, vp, vp, vp, vp, u32, vp, vp, vp]
    lib.db_cache_attention_workspace_size.argtypes = [u32, u32, u32, u32, u32, psz]
    lib.db_cache_attention.argtypes = [vp, vp, vp, vp, vp, u32, u32, u32, f32, vp, u32, vp, vp, vp,
                                       vp, sz, vp]
    lib.db_draft_verify.argtypes = [vp, u32, u32, vp, vp, vp, u64, vp, u64, u32, u32, vp, vp, vp,
                                    vp, vp, vp, vp]
    lib.db_cache_keep.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    for name in ("db_cache_write", "db_cache_read", "db_cache_attention_workspace_size",
                 "db_cache_attention", "db_draft_verify", "db_cache_keep"):
        getattr(lib, name).restype = i32
    lib.db_strerror.argtypes = [i32]
    lib.db_strerror.restype = ctypes.c_char_p
    lib.db_last_cuda_error.argtypes = []
    return lib


_lib = _load()


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise DescBuildError(fn, rc)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libdescbuild must be contiguous")
    return t.data_ptr()


def _records(t: torch.Tensor, size: int) -> int:
    nbytes = t.numel() * t.element_size()
    if nbytes % size:
        raise ValueError(f"buffer of {nbytes} bytes is not a whole number of {size}-byte records")
    return nbytes // size


# The current device's current stream as a number. torch.cuda.current_stream()
# builds a Stream object for it (2.9 us a call on the GPU's host, these 0.2 us).
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cuda_ready = False


def _stream(stream) -> int:
    global _cuda_ready
    if stream is None:
        if _cuda_ready:
            return _raw_stream(_device())
        now = torch.cuda.current_stream().cuda_stream  # initialises CUDA
        _cuda_ready = _raw_stream is not None and _device is not None
        return now
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _size(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(fn.__name__, fn(*args, ctypes.byref(out)))
    return out.value


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled device workspace of ``nbytes`` (256-byte aligned by torch)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def strerror(code: int) -> str:
    return _lib.db_strerror(code).decode()


# ------------------------------------------------------------------ PRP build
def prp_workspace_size(n: int) -> int:
    return _size(_lib.db_prp_workspace_size, n)


def prp_build(req: torch.Tensor, lut: torch.Tensor, heap_size: int, arena_base: int,
              arena_cap_pages: int, arena: torch.Tensor | None, prp: torch.Tensor,
              ws: torch.Tensor, page_base: torch.Tensor | None = None,
              status: torch.Tensor | None = None, ctr: torch.Tensor | None = None,
              flags: int = 0, stream=None) -> None:
    """db_prp_build: PRP1/PRP2 per request and the chained list pages in ``arena``."""
    n = _records(req, 16)
    _check("db_prp_build", _lib.db_prp_build(
        _ptr(req), n, _ptr(lut), heap_size, arena_base, arena_cap_pages, _ptr(arena), _ptr(prp),
        _ptr(page_base), _ptr(status), _ptr(ctr), flags, _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


PRP_STATIC_MAX_REQUESTS = 1 << 24


def prp_build_static(req: torch.Tensor, lut: torch.Tensor, heap_size: int, arena_base: int,
                     arena_cap_pages: int, arena: torch.Tensor | None, prp: torch.Tensor,
                     page_base: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     ctr: torch.Tensor | None = None, flags: int = 0, stream=None) -> None:
    """db_prp_build_static: prp_build with the library's own static scratch
    array, for callers that must not allocate device memory while submitting
    (cudaMalloc may wait on queued device work and takes driver locks).
    At most PRP_STATIC_MAX_REQUESTS requests per call; calls that may overlap
    on the GPU share the array and must be ordered by the caller. The first
    call on a device looks the array up, so make it before any stream capture."""
    n = _records(req, 16)
    _check("db_prp_build_static", _lib.db_prp_build_static(
        _ptr(req), n, _ptr(lut), heap_size, arena_base, arena_cap_pages, _ptr(arena), _ptr(prp),
        _ptr(page_base), _ptr(status), _ptr(ctr), flags, _stream(stream)))


# ------------------------------------------------------------------ MR lookup
def mr_workspace_size(n_mr: int) -> int:
    return _size(_lib.db_mr_workspace_size, n_mr)


def mr_lookup(q: torch.Tensor, mr_start: torch.Tensor, mr_end: torch.Tensor,
              mr_lkey: torch.Tensor, idx: torch.Tensor, lkey: torch.Tensor, kind: torch.Tensor,
              ws: torch.Tensor, ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_mr_lookup: classify each range against a sorted registration table."""
    n_q = _records(q, 16)
    n_mr = _records(mr_start, 8)
    _check("db_mr_lookup", _lib.db_mr_lookup(
        _ptr(q), n_q, _ptr(mr_start), _ptr(mr_end), _ptr(mr_lkey), n_mr, _ptr(idx), _ptr(lkey),
        _ptr(kind), _ptr(ctr), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def mr_lookup_overlap(q: torch.Tensor, mr_start: torch.Tensor, mr_end: torch.Tensor,
                      mr_lkey: torch.Tensor, idx: torch.Tensor, lkey: torch.Tensor,
                      kind: torch.Tensor, ws: torch.Tensor, ctr: torch.Tensor | None = None,
                      stream=None) -> None:
    """db_mr_lookup_overlap: the same on a start-sorted table whose ranges may overlap."""
    n_q = _records(q, 16)
    n_mr = _records(mr_start, 8)
    _check("db_mr_lookup_overlap", _lib.db_mr_lookup_overlap(
        _ptr(q), n_q, _ptr(mr_start), _ptr(mr_end), _ptr(mr_lkey), n_mr, _ptr(idx), _ptr(lkey),
        _ptr(kind), _ptr(ctr), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


# ------------------------------------------------------- MR cache mutation
MR_NEW, MR_NEW_DUP = 4, 5
DEREG_OK, DEREG_RELEASED, DEREG_STALE = 0, 1, 2


def mr_capacity_for(n: int) -> int:
    """Table capacity after growth to n records: 0, 32, then doubling."""
    return int(_lib.db_mr_capacity_for(n))


def mr_register_workspace_size(n_q: int, n_mr: int) -> int:
    return _size(_lib.db_mr_register_workspace_size, n_q, n_mr)


def mr_register(q: torch.Tensor, new_lkey: torch.Tensor, start: torch.Tensor, end: torch.Tensor,
                lkey: torch.Tensor, refs: torch.Tensor, out_start: torch.Tensor,
                out_end: torch.Tensor, out_lkey: torch.Tensor, out_refs: torch.Tensor,
                handle: torch.Tensor, kind: torch.Tensor, remap: torch.Tensor, ws: torch.Tensor,
                granule_shift: int = 12, ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_mr_register: a batch of registrations; the table after it goes to out_*."""
    n_q = _records(q, 16)
    n_mr = _records(start, 8)
    out_cap = _records(out_start, 8)
    _check("db_mr_register", _lib.db_mr_register(
        _ptr(q), n_q, _ptr(new_lkey), granule_shift, _ptr(start), _ptr(end), _ptr(lkey),
        _ptr(refs), n_mr, _ptr(out_start), _ptr(out_end), _ptr(out_lkey), _ptr(out_refs),
        out_cap, _ptr(handle), _ptr(kind), _ptr(remap), _ptr(ctr), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def mr_deregister_workspace_size(n_h: int, n_mr: int) -> int:
    return _size(_lib.db_mr_deregister_workspace_size, n_h, n_mr)


def mr_deregister(handle: torch.Tensor, start: torch.Tensor, end: torch.Tensor,
                  lkey: torch.Tensor, refs: torch.Tensor, out_start: torch.Tensor,
                  out_end: torch.Tensor, out_lkey: torch.Tensor, out_refs: torch.Tensor,
                  remap: torch.Tensor, status: torch.Tensor, ws: torch.Tensor,
                  ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_mr_deregister: a batch of deregistrations, in batch order."""
    n_h = _records(handle, 8)
    n_mr = _records(start, 8)
    _check("db_mr_deregister", _lib.db_mr_deregister(
        _ptr(handle), n_h, _ptr(start), _ptr(end), _ptr(lkey), _ptr(refs), n_mr,
        _ptr(out_start), _ptr(out_end), _ptr(out_lkey), _ptr(out_refs), _ptr(remap),
        _ptr(status), _ptr(ctr), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


# --------------------------------------------------------------- WQE bucketing
def wqe_workspace_size(n: int, n_rings: int) -> int:
    return _size(_lib.db_wqe_workspace_size, n, n_rings)


def wqe_vmm_workspace_size(n: int, world: int, n_qp: int, heap_size: int,
                           chunk_shift: int) -> int:
    """Workspace bytes of db_wqe_bucket_vmm (columns plus the packed chunk tables)."""
    return _size(_lib.db_wqe_vmm_workspace_size, n, world, n_qp, heap_size, chunk_shift)


def wqe_bucket(req: torch.Tensor, peer_ptrs: torch.Tensor, rkeys: torch.Tensor, world: int,
               n_qp: int, local_base: int, lkey: int, heap_size: int, rings: torch.Tensor,
               depth: int, head: torch.Tensor, count: torch.Tensor, ws: torch.Tensor,
               ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_wqe_bucket: translate puts and stable-partition them into WQE rings."""
    n = _records(req, 16)
    _check("db_wqe_bucket", _lib.db_wqe_bucket(
        _ptr(req), n, _ptr(peer_ptrs), _ptr(rkeys), world, n_qp, local_base, lkey, heap_size,
        _ptr(rings), depth, _ptr(head), _ptr(count), _ptr(ctr), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def wqe_bucket_transport(req: torch.Tensor, peer_ptrs: torch.Tensor, rkeys: torch.Tensor,
                         transport: torch.Tensor, world: int, n_qp: int, local_base: int,
                         lkey: int, heap_size: int, rings: torch.Tensor, depth: int,
                         head: torch.Tensor, count: torch.Tensor, direct: torch.Tensor,
                         n_direct: torch.Tensor, ws: torch.Tensor,
                         ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_wqe_bucket_transport: puts dispatched on their PE's transport (uint8
    [world] of XPORT_*): RDMA puts into WQE rings as wqe_bucket, P2P and SDMA
    puts as 32-byte direct records (uint8 [n, 32]) in batch order; n_direct
    (int64 [1]) gets their number."""
    n = _records(req, 16)
    _check("db_wqe_bucket_transport", _lib.db_wqe_bucket_transport(
        _ptr(req), n, _ptr(peer_ptrs), _ptr(rkeys), _ptr(transport), world, n_qp, local_base,
        lkey, heap_size, _ptr(rings), depth, _ptr(head), _ptr(count), _ptr(direct),
        _ptr(n_direct), _ptr(ctr), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def wqe_bucket_vmm(req: torch.Tensor, chunk_raddr: torch.Tensor, chunk_rkey: torch.Tensor,
                   chunk_lkey: torch.Tensor, chunk_shift: int, world: int, n_qp: int,
                   local_base: int, heap_size: int, rings: torch.Tensor, depth: int,
                   head: torch.Tensor, count: torch.Tensor, ws: torch.Tensor,
                   ctr: torch.Tensor | None = None, stream=None, mtu: int = 0,
                   psn_head: torch.Tensor | None = None) -> None:
    """db_wqe_bucket_vmm: puts on a chunked (VMM) heap, one WQE per chunk
    touched; with an mtu, each WQE also gets its first PSN."""
    n = _records(req, 16)
    _check("db_wqe_bucket_vmm", _lib.db_wqe_bucket_vmm(
        _ptr(req), n, _ptr(chunk_raddr), _ptr(chunk_rkey), _ptr(chunk_lkey), chunk_shift, world,
        n_qp, local_base, heap_size, _ptr(rings), depth, _ptr(head), _ptr(count), mtu,
        _ptr(psn_head), _ptr(ctr), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


# ------------------------------------------------------------------ CQ mirror
CQ_MAX_SLOTS, CQ_MAX_DEPTH = 64, 65536
CQ_TIMED = 1  # slot flag: record each batch's latency in lat_ns / lat_seq
# db_cq_slot, 64 bytes
CQ_SLOT_DTYPE = np.dtype([("dev_cq", "<u8"), ("host_cq", "<u8"), ("depth", "<u4"),
                          ("generation", "<u4"), ("ack", "<u4"), ("seen", "<u4"),
                          ("head", "<u4"), ("phase", "<u4"), ("copied", "<u8"),
                          ("flags", "<u4"), ("lat_ns", "<u4"), ("lat_seq", "<u8")])
assert CQ_SLOT_DTYPE.itemsize == 64


def _host(t: torch.Tensor) -> int:
    if t.device.type != "cpu" or not t.is_contiguous():
        raise ValueError("expected a contiguous host tensor")
    return t.data_ptr()


def cq_slots(n: int) -> torch.Tensor:
    """A zero-filled slot table of n slots in pinned host memory."""
    return torch.zeros((n, 64), dtype=torch.uint8).pin_memory()


def cq_slot_fields(slots: torch.Tensor) -> np.ndarray:
    """A live structured view of a slot table (reads see the kernel's writes)."""
    return slots.numpy().view(CQ_SLOT_DTYPE).reshape(-1)


def cq_mirror(slots: torch.Tensor, stop: torch.Tensor, limit_s: float,
              ctr: torch.Tensor | None = None, stream=None, n_slots: int | None = None) -> None:
    """db_cq_mirror: launch the bounded resident mirror over the slots."""
    n = slots.shape[0] if n_slots is None else n_slots
    _check("db_cq_mirror", _lib.db_cq_mirror(_host(slots), n, _host(stop),
                                             int(limit_s * 1e9), _ptr(ctr), _stream(stream)))


def cq_attach(slots: torch.Tensor, i: int, dev_cq: torch.Tensor, host_cq: torch.Tensor) -> int:
    """db_cq_attach: serve the device CQ dev_cq ([depth, 4] int32, device)
    into host_cq ([depth, 4] int32, pinned); returns the odd generation."""
    depth = _records(dev_cq, 16)
    if _records(host_cq, 16) != depth:
        raise ValueError("device and host CQ differ in depth")
    g = ctypes.c_uint32(0)
    _check("db_cq_attach", _lib.db_cq_attach(_host(slots) + 64 * i, _ptr(dev_cq),
                                             _host(host_cq), depth, ctypes.byref(g)))
    return g.value


def cq_detach(slots: torch.Tensor, i: int) -> int:
    """db_cq_detach: returns the odd generation whose acknowledgement to wait for."""
    g = ctypes.c_uint32(0)
    _check("db_cq_detach", _lib.db_cq_detach(_host(slots) + 64 * i, ctypes.byref(g)))
    return g.value


def cq_wait_ack(slots: torch.Tensor, i: int, generation: int, timeout_s: float) -> bool:
    rc = _lib.db_cq_wait_ack(_host(slots) + 64 * i, generation, int(timeout_s * 1e9))
    if rc not in (0, -110):
        _check("db_cq_wait_ack", rc)
    return rc == 0


def cq_host_reap(host_cq: torch.Tensor, head: int, phase: int, max_entries: int | None = None):
    """db_cq_host_reap: returns (entries [n, 4] uint32, head, phase)."""
    depth = _records(host_cq, 16)
    m = depth if max_entries is None else max_entries
    out = np.zeros((max(m, 1), 4), dtype=np.uint32)
    h, ph = ctypes.c_uint32(head), ctypes.c_uint32(phase)
    n = _lib.db_cq_host_reap(_host(host_cq), depth, ctypes.byref(h), ctypes.byref(ph),
                             out.ctypes.data, m)
    if n < 0:
        _check("db_cq_host_reap", n)
    return out[:n], h.value, ph.value


def cq_request_stop(stop: torch.Tensor) -> None:
    _lib.db_cq_request_stop(_host(stop))


# ---------------------------------------------------------------- paged cache
class _Tables(ctypes.Structure):  # db_page_tables
    _fields_ = [("table", ctypes.c_void_p), ("length", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("free", ctypes.c_void_p), ("n_seqs", ctypes.c_uint32),
                ("columns", ctypes.c_uint32), ("n_pages", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32)]


class _Pool(ctypes.Structure):  # db_page_pool
    _fields_ = [("base", ctypes.c_void_p), ("n_pages", ctypes.c_uint64),
                ("plane_stride", ctypes.c_uint64), ("page_stride", ctypes.c_uint64)]


class _Shape(ctypes.Structure):  # db_page_shape
    _fields_ = [("planes", ctypes.c_uint32), ("segments", ctypes.c_uint32),
                ("page_tokens", ctypes.c_uint32), ("token_bytes", ctypes.c_uint32)]


def _refuse(t: torch.Tensor) -> None:
    if not (t.is_cuda or t.is_pinned()):  # the GPU would fault in it
        raise ValueError("a paged cache's tensors must be on the GPU or in pinned host memory")
    raise ValueError("tensors passed to libdescbuild must be contiguous")


def _at(t: torch.Tensor, nbytes: int) -> int:
    """The address of a tensor of which the GPU reads or writes ``nbytes``."""
    if not (t.is_contiguous() and (t.is_cuda or t.is_pinned())):
        _refuse(t)
    if t.nbytes < nbytes:
        raise ValueError(f"tensor of {t.nbytes} bytes where {nbytes} are read or written")
    return t.data_ptr()


def _whole(t: torch.Tensor) -> tuple[int, int]:
    """A tensor's address and size."""
    if not (t.is_contiguous() and (t.is_cuda or t.is_pinned())):
        _refuse(t)
    return t.data_ptr(), t.nbytes


_I32, _U32 = torch.int32, torch.uint32


def _batch(t: torch.Tensor, width: int) -> tuple[int, int]:
    """The address and the number of a batch's records of ``width`` 32-bit
    fields. (Another type's bytes would be read as other records.)"""
    shape = t.shape
    if len(shape) == 2 and shape[1] == width:
        n = shape[0]
    elif shape[-1:] == (width,) or (len(shape) == 1 and shape[0] % width == 0):
        n = t.numel() // width
    else:
        n = -1
    if not (0 <= n <= 0xFFFFFFFF and (t.dtype is _I32 or t.dtype is _U32)):
        raise ValueError(f"a batch is an int32 tensor [n, {width}], n below 2^32, not "
                         f"{t.dtype} {list(shape)}")
    if not (t.is_contiguous() and (t.is_cuda or t.is_pinned())):
        _refuse(t)
    return t.data_ptr(), n


class PageTables:
    """The state of a paged cache: int32 CUDA tensors table [n_seqs, columns],
    length [n_seqs], refs [n_pages] and free [ceil(n_pages / 32)], which the
    calls below update in place (their bits are the header's u32). n_seqs and
    n_pages are below 2^31, and free starts on a multiple of 16 bytes."""

    def __init__(self, table: torch.Tensor, length: torch.Tensor, refs: torch.Tensor,
                 free: torch.Tensor, page_tokens: int):
        if table.dim() != 2:
            raise ValueError("table must be [n_seqs, columns]")
        n_seqs, columns = table.shape
        n_pages, page_tokens = refs.numel(), int(page_tokens)
        if not (0 < n_seqs < 1 << 31 and 0 < n_pages < 1 << 31):
            raise ValueError("a cache has at least one sequence and one page, and below 2^31 of them")
        if not (0 < columns < 1 << 32 and 0 < page_tokens < 1 << 32):
            raise ValueError("columns and page_tokens are from 1 to 2^32 - 1")
        for name, t, n in (("table", table, n_seqs * columns), ("length", length, n_seqs),
                           ("refs", refs, n_pages), ("free", free, (n_pages + 31) // 32)):
            if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"{name} must be a contiguous int32 tensor of {n} elements")
        self.table, self.length, self.refs, self.free = table, length, refs, free
        self.page_tokens = page_tokens
        self._c = _Tables(*(_at(t, 0) for t in (table, length, refs, free)), n_seqs, columns,
                          n_pages, self.page_tokens)
        if self._c.free % 16:
            raise ValueError("free must start on a multiple of 16 bytes")
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_seqs: int, columns: int, n_pages: int, page_tokens: int,
              device=None) -> "PageTables":
        """An empty cache: no sequence holds a token and every page is free."""
        device = device or "cuda"
        free = torch.full(((n_pages + 31) // 32,), -1, dtype=torch.int32, device=device)
        if n_pages % 32:
            free[-1] = (1 << (n_pages % 32)) - 1
        return cls(torch.full((n_seqs, columns), PAGE_NONE, dtype=torch.int32, device=device),
                   torch.zeros(n_seqs, dtype=torch.int32, device=device),
                   torch.zeros(n_pages, dtype=torch.int32, device=device), free, page_tokens)


def page_workspace_size(n_seqs: int, n_pages: int) -> int:
    """Bytes of the workspace of a cache of these sizes. Calls on a cache of
    other sizes need another workspace."""
    return _size(_lib.db_page_workspace_size, n_seqs, n_pages)


def page_extend(tables: PageTables, req: torch.Tensor, moves: torch.Tensor,
                n_moves: torch.Tensor, ws: torch.Tensor, status: torch.Tensor | None = None,
                ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_page_extend: sequences grow by tokens (req [n, 2] {seq, tokens});
    moves [>= n, 4] and n_moves [1] get the copies page_copy has to make."""
    at, n = _batch(req, 2)
    to, room = _batch(moves, 4)
    if room < n:
        raise ValueError(f"moves holds fewer than {n} records")
    space, nbytes = _whole(ws)
    _check("db_page_extend", _lib.db_page_extend(
        tables._ref, at, n, to, _at(n_moves, 4), None if status is None else _at(status, n),
        None if ctr is None else _at(ctr, 32), space, nbytes, _stream(stream)))


def page_fork(tables: PageTables, req: torch.Tensor, ws: torch.Tensor,
              status: torch.Tensor | None = None, ctr: torch.Tensor | None = None,
              stream=None) -> None:
    """db_page_fork: children share their parents' first tokens (req [n, 4]
    {parent, child, tokens, ignored})."""
    at, n = _batch(req, 4)
    space, nbytes = _whole(ws)
    _check("db_page_fork", _lib.db_page_fork(
        tables._ref, at, n, None if status is None else _at(status, n),
        None if ctr is None else _at(ctr, 32), space, nbytes, _stream(stream)))


def page_free(tables: PageTables, req: torch.Tensor, ws: torch.Tensor,
              status: torch.Tensor | None = None, ctr: torch.Tensor | None = None,
              stream=None) -> None:
    """db_page_free: sequences cut back to their first tokens (req [n, 2]
    {seq, keep}) give their other pages back."""
    at, n = _batch(req, 2)
    space, nbytes = _whole(ws)
    _check("db_page_free", _lib.db_page_free(
        tables._ref, at, n, None if status is None else _at(status, n),
        None if ctr is None else _at(ctr, 32), space, nbytes, _stream(stream)))


def page_compact(tables: PageTables, out: PageTables, moves: torch.Tensor, n_moves: torch.Tensor,
                 ws: torch.Tensor, ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_page_compact: live pages move down to the lowest indices. The cache
    after the moves goes to ``out`` (``tables`` itself, or other tensors of the
    same sizes); moves [cap, 4] and n_moves [1] get what page_copy has to
    move."""
    at, cap = _batch(moves, 4)
    space, nbytes = _whole(ws)
    _check("db_page_compact", _lib.db_page_compact(
        tables._ref, out._ref, at, cap, _at(n_moves, 4), None if ctr is None else _at(ctr, 32),
        space, nbytes, _stream(stream)))


def _strides(shape, stride, item: int) -> tuple[int, int]:
    """Bytes between the planes and the pages of a pool [planes, pages, ...]."""
    if len(shape) < 3:
        raise ValueError("a pool is [planes, pages, ...]")
    want = 1
    for size, step in zip(reversed(shape[2:]), reversed(stride[2:])):
        if size != 1 and step != want:
            raise ValueError("a pool's pages must be contiguous")
        want *= size
    return stride[0] * item, stride[1] * item


@functools.lru_cache(maxsize=1024)
def _copy_plan(shape, stride, item: int, token_dim, dst_shape=None, dst_stride=None):
    """What a copy's pools have in common and their strides, from their shapes
    alone (without dst_shape they are one pool)."""
    a = b = _strides(shape, stride, item)
    if dst_shape is not None:
        if shape[0] != dst_shape[0] or shape[2:] != dst_shape[2:]:
            raise ValueError("source and destination pools differ in planes or page shape")
        b = _strides(dst_shape, dst_stride, item)
    page = shape[2:]
    if token_dim is None:
        segments, page_tokens, k = 1, 1, 0
    else:
        if not 2 <= token_dim < len(shape):
            raise ValueError("token_dim must be one of a page's axes (2 and up)")
        k = token_dim - 1
        segments, page_tokens = math.prod(page[:k - 1]), page[k - 1]
    if math.prod(page) * item * shape[0] > 1 << 31:
        raise ValueError("a page has at most 2^31 bytes in all planes")
    form = _Shape(shape[0], segments, page_tokens, math.prod(page[k:]) * item)
    return form, ctypes.byref(form), a, b


def page_copy(moves: torch.Tensor, n_moves: torch.Tensor, src: torch.Tensor, dst: torch.Tensor,
              token_dim: int | None = None, ctr: torch.Tensor | None = None,
              stream=None) -> None:
    """db_page_copy: the bytes of ``moves`` ({src, dst, tokens, ignored}, of
    which n_moves [1] counts), from pages of ``src`` to pages of ``dst`` (the
    same tensor, or another of the same page shape). Pools are [planes, pages,
    ...], on the GPU or in pinned host memory, strided in the first two axes;
    ``token_dim`` is the axis of a page's tokens, None when it has none (then
    every move takes whole pages)."""
    shape = src.shape
    if not (src.is_cuda or src.is_pinned()):
        _refuse(src)
    if dst is src:
        _, form, a, _ = _copy_plan(shape, src.stride(), src.element_size(), token_dim)
        here = there = ctypes.byref(_Pool(src.data_ptr(), shape[1], *a))
    else:
        if not (dst.is_cuda or dst.is_pinned()):
            _refuse(dst)
        if src.dtype != dst.dtype:
            raise ValueError("source and destination pools differ in type")
        _, form, a, b = _copy_plan(shape, src.stride(), src.element_size(), token_dim, dst.shape,
                                   dst.stride())
        here = ctypes.byref(_Pool(src.data_ptr(), shape[1], *a))
        there = ctypes.byref(_Pool(dst.data_ptr(), dst.shape[1], *b))
    at, most = _batch(moves, 4)
    _check("db_page_copy", _lib.db_page_copy(
        at, most, _at(n_moves, 4), here, there, form, None if ctr is None else _at(ctr, 32),
        _stream(stream)))


# ------------------------------------------------------- a paged cache's contents
# The C structs as bytes, which a call reads before it returns (making a
# ctypes.Structure takes four times as long).
_pack_batch = struct.Struct("=2Q2I").pack  # db_cache_batch: seq, start, n, rows
_pack_layer = struct.Struct("=4Q").pack  # db_cache_layer: k, v, k_scale, v_scale, and after them
_pack_layer_plan = struct.Struct("=4Q4I").pack  # their strides, heads, width, type, heads_first
_pack_rows = struct.Struct("=3Q").pack  # db_cache_rows: base, row_stride, head_stride

_ROW_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_CACHE_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 3, torch.int8: 4}


def _i32(t: torch.Tensor, n: int, what: str) -> int:
    """The address of an int32 tensor of at least ``n`` elements."""
    if t.dtype is not _I32 and t.dtype is not _U32:
        raise ValueError(f"{what} must be an int32 tensor, not {t.dtype}")
    return _at(t, 4 * n)


def _cache_batch(seq: torch.Tensor, start: torch.Tensor, rows: int) -> tuple[bytes, int]:
    n = seq.numel()
    if start.numel() != n + 1:
        raise ValueError(f"start must have {n + 1} elements for {n} sequences")
    return _pack_batch(_i32(seq, n, "seq"), _i32(start, n + 1, "start"), n, rows), n


def _cache_rows(t: torch.Tensor, heads: int, width: int) -> bytes:
    """Rows [rows, heads, width] outside the cache, of any strides but the last."""
    if t.shape[1:] != (heads, width):
        raise ValueError(f"rows must be [rows, {heads}, {width}]")
    row, head, one = t.stride()
    if one != 1:
        raise ValueError("the values of a row must be neighbours")
    if not (t.is_cuda or t.is_pinned()):
        _refuse(t)
    size = t.element_size()
    return _pack_rows(t.data_ptr(), row * size, head * size)


def _pool_plan(shape, stride, dtype, token_dim, page_tokens, scale_shape, scale_stride):
    """What a pool of keys or values says: (page stride and scales' page stride
    in bytes, heads, width, type)."""
    if len(shape) != 4 or token_dim not in (1, 2):
        raise ValueError("a layer's pool is [pages, tokens, heads, width] (token_dim 1) or "
                         "[pages, heads, tokens, width] (token_dim 2)")
    if dtype not in _CACHE_TYPES:
        raise ValueError(f"a cache holds bfloat16, float16, float8_e4m3fn or int8, not {dtype}")
    if shape[token_dim] != page_tokens:
        raise ValueError(f"the pool's pages hold {shape[token_dim]} tokens, the tables' {page_tokens}")

    def contiguous(inner, steps):
        want = 1
        for size, step in zip(reversed(inner), reversed(steps)):
            if size != 1 and step != want:
                raise ValueError("a pool's pages must be contiguous")
            want *= size

    contiguous(shape[1:], stride[1:])
    size = dtype.itemsize
    scale = 0
    if size == 1:
        if scale_shape is None or scale_shape != shape[:3]:
            raise ValueError(f"a cache of {dtype} needs scales {list(shape[:3])}")
        contiguous(scale_shape[1:], scale_stride[1:])
        scale = scale_stride[0] * 4
    elif scale_shape is not None:
        raise ValueError("only 8-bit caches have scales")
    return stride[0] * size, scale, shape[3 - token_dim], shape[3], _CACHE_TYPES[dtype]


@functools.lru_cache(maxsize=1024)
def _layer_plan(token_dim, page_tokens, k, k_scale, v, v_scale) -> tuple[bytes, int, int]:
    """The rest of a layer's struct, its heads and width, from what the tensors
    look like (shape, stride and a pool's type)."""
    k_step, ks_step, *of_k = _pool_plan(*k, token_dim, page_tokens, *k_scale)
    v_step, vs_step, *of_v = _pool_plan(*v, token_dim, page_tokens, *v_scale)
    if of_k != of_v:
        raise ValueError("the pools of keys and values differ in heads, width or type")
    heads, width, kind = of_k
    return (_pack_layer_plan(k_step, v_step, ks_step, vs_step, heads, width, kind, token_dim == 2),
            heads, width)


_NO_SCALE = (None, None)


def _cache_layer(tables: PageTables, k_pool, v_pool, k_scale, v_scale, token_dim):
    """The layer's struct, its heads and width."""
    k_shape, v_shape, pages = k_pool.shape, v_pool.shape, tables._c.n_pages
    if not (k_pool.is_cuda or k_pool.is_pinned()):
        _refuse(k_pool)
    if not (v_pool.is_cuda or v_pool.is_pinned()):
        _refuse(v_pool)
    like_k = like_v = _NO_SCALE
    at_k = at_v = 0
    for scale in (k_scale, v_scale):
        if scale is not None:
            if not (scale.is_cuda or scale.is_pinned()):
                _refuse(scale)
            if scale.dtype is not torch.float32:
                raise ValueError("scales are float32")
    if k_scale is not None:
        like_k, at_k = (k_scale.shape, k_scale.stride()), k_scale.data_ptr()
    if v_scale is not None:
        like_v, at_v = (v_scale.shape, v_scale.stride()), v_scale.data_ptr()
    rest, heads, width = _layer_plan(token_dim, tables.page_tokens, (k_shape, k_pool.stride(), k_pool.dtype), like_k,
                                     (v_shape, v_pool.stride(), v_pool.dtype), like_v)
    if k_shape[0] < pages or v_shape[0] < pages:
        raise ValueError(f"a pool of {min(k_shape[0], v_shape[0])} pages where the tables have {pages}")
    return _pack_layer(k_pool.data_ptr(), v_pool.data_ptr(), at_k, at_v) + rest, heads, width


def _row_type(*tensors: torch.Tensor) -> int:
    dtype = tensors[0].dtype
    kind = _ROW_TYPES.get(dtype)
    if kind is None or tensors[-1].dtype is not dtype:
        raise ValueError("rows are bfloat16, float16 or float32, all of one type")
    return kind


def _maybe(t: torch.Tensor | None, nbytes: int) -> int | None:
    return None if t is None else _at(t, nbytes)


def cache_write(tables: PageTables, seq: torch.Tensor, start: torch.Tensor, k: torch.Tensor,
                v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
                k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                token_dim: int = 1, status: torch.Tensor | None = None,
                ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_cache_write: rows start[i] to start[i + 1] of k and v [rows, heads,
    width] go to the slots of the last tokens of sequence seq[i], rounded to
    the pools' type or quantised with a scale for each row."""
    layer, heads, width = _cache_layer(tables, k_pool, v_pool, k_scale, v_scale, token_dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v differ in rows")
    batch, n = _cache_batch(seq, start, k.shape[0])
    _check("db_cache_write", _lib.db_cache_write(
        tables._ref, batch, layer, _cache_rows(k, heads, width), _cache_rows(v, heads, width),
        _row_type(k, v), _maybe(status, n), _maybe(ctr, 32), _stream(stream)))


def cache_read(tables: PageTables, seq: torch.Tensor, start: torch.Tensor, k: torch.Tensor,
               v: torch.Tensor, k_pool: torch.Tensor, v_pool: torch.Tensor,
               k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
               first: torch.Tensor | None = None, token_dim: int = 1,
               status: torch.Tensor | None = None, ctr: torch.Tensor | None = None,
               stream=None) -> None:
    """db_cache_read: rows start[i] to start[i + 1] of k and v [rows, heads,
    width] get the tokens of sequence seq[i] from position first[i] (0) on;
    rows past its last token become zeros."""
    layer, heads, width = _cache_layer(tables, k_pool, v_pool, k_scale, v_scale, token_dim)
    if k.shape[0] != v.shape[0]:
        raise ValueError("k and v differ in rows")
    batch, n = _cache_batch(seq, start, k.shape[0])
    _check("db_cache_read", _lib.db_cache_read(
        tables._ref, batch, None if first is None else _i32(first, n, "first"), layer,
        _cache_rows(k, heads, width), _cache_rows(v, heads, width), _row_type(k, v),
        _maybe(status, n), _maybe(ctr, 32), _stream(stream)))


def cache_attention_workspace_size(n: int, q_heads: int, heads: int, width: int,
                                   max_tokens: int) -> int:
    """Bytes of cache_attention's workspace on the current device."""
    return _size(_lib.db_cache_attention_workspace_size, n, q_heads, heads, width, max_tokens)


def cache_attention(tables: PageTables, seq: torch.Tensor, start: torch.Tensor, q: torch.Tensor,
                    k_pool: torch.Tensor, v_pool: torch.Tensor, out: torch.Tensor,
                    ws: torch.Tensor, max_tokens: int, scale: float | None = None,
                    mask: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                    token_dim: int = 1, status: torch.Tensor | None = None,
                    ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_cache_attention: the last tokens of sequences (rows of q and out
    [rows, q_heads, width], at most max_tokens of a sequence) attend to all
    tokens before them and to those of their own that mask [rows, words] of
    bits names (None: themselves and the ones before). scale None: 1 /
    sqrt(width). lse: float32 [rows, q_heads]. max_tokens chooses the kernel
    for the whole call, so single tokens go faster in one of their own."""
    layer, heads, width = _cache_layer(tables, k_pool, v_pool, k_scale, v_scale, token_dim)
    rows, q_heads, _ = q.shape
    if out.shape[0] != rows:
        raise ValueError("q and out differ in rows")
    batch, n = _cache_batch(seq, start, rows)
    words = 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[0] != rows:
            raise ValueError(f"mask must be [{rows}, words]")
        words = mask.shape[1]
    if lse is not None and lse.dtype is not torch.float32:
        raise ValueError("lse is float32")
    space, nbytes = _whole(ws)
    _check("db_cache_attention", _lib.db_cache_attention(
        tables._ref, batch, layer, _cache_rows(q, q_heads, width), _cache_rows(out, q_heads, width),
        _row_type(q, out), q_heads, max_tokens, width ** -0.5 if scale is None else scale,
        None if mask is None else _i32(mask, rows * words, "mask"), words,
        _maybe(lse, 4 * rows * q_heads), _maybe(status, n), _maybe(ctr, 32), space, nbytes,
        _stream(stream)))


def draft_verify(start: torch.Tensor, parent: torch.Tensor, token: torch.Tensor, p: torch.Tensor,
                 u: torch.Tensor, path: torch.Tensor, accepted: torch.Tensor, next: torch.Tensor,
                 q: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_draft_verify: trees of drafted tokens (rows start[i] to start[i + 1]
    of parent, token, u, and of the probabilities p and q [rows, vocab])
    accepted or not; path [rows], accepted [n] and next [n] get the result. Of
    a tree that is refused none is accepted, not the root either: cache_keep
    and page_free then take its sequence's step back."""
    n, rows = start.numel() - 1, p.shape[0]
    if n < 0 or p.dim() != 2 or p.stride(1) != 1:
        raise ValueError("start must be [n + 1], p [rows, vocab] with neighbouring values")
    if q is not None and (q.shape != p.shape or q.stride(1) != 1):
        raise ValueError("q must be of p's shape, with neighbouring values")
    for t in (p, q):
        if t is not None and not (t.is_cuda or t.is_pinned()):
            _refuse(t)
    if u.dtype is not torch.float32:
        raise ValueError("u is float32")
    kind = _row_type(p) if q is None else _row_type(p, q)
    _check("db_draft_verify", _lib.db_draft_verify(
        _i32(start, n + 1, "start"), n, rows, _i32(parent, rows, "parent"), _i32(token, rows, "token"),
        p.data_ptr(), p.stride(0), None if q is None else q.data_ptr(), 0 if q is None else q.stride(0),
        kind, p.shape[1], _at(u, 4 * rows), _i32(path, rows, "path"), _i32(accepted, n, "accepted"),
        _i32(next, n, "next"), _maybe(status, n), _maybe(ctr, 32), _stream(stream)))


def cache_keep(tables: PageTables, seq: torch.Tensor, start: torch.Tensor, path: torch.Tensor,
               accepted: torch.Tensor, pool: torch.Tensor, token_dim: int = 2,
               cut: torch.Tensor | None = None, status: torch.Tensor | None = None,
               ctr: torch.Tensor | None = None, stream=None) -> None:
    """db_cache_keep: in every plane of ``pool`` [planes, pages, ...] (as in
    page_copy; token_dim is the axis of a page's tokens) the tokens on the
    accepted paths move together. cut [n, 2] gets the requests of page_free
    that give the others' slots back."""
    shape = pool.shape
    if not (pool.is_cuda or pool.is_pinned()):
        _refuse(pool)
    if token_dim is None:
        raise ValueError("token_dim must be one of a page's axes (2 and up)")
    _, form, a, _ = _copy_plan(shape, pool.stride(), pool.element_size(), token_dim)
    if shape[token_dim] != tables.page_tokens:
        raise ValueError(f"the pool's pages hold {shape[token_dim]} tokens, the tables' {tables.page_tokens}")
    if shape[1] < tables._c.n_pages:
        raise ValueError(f"a pool of {shape[1]} pages where the tables have {tables._c.n_pages}")
    rows = path.numel()
    batch, n = _cache_batch(seq, start, rows)
    if cut is not None and _batch(cut, 2)[1] < n:
        raise ValueError(f"cut holds fewer than {n} records")
    _check("db_cache_keep", _lib.db_cache_keep(
        tables._ref, batch, _i32(path, rows, "path"), _i32(accepted, n, "accepted"),
        ctypes.byref(_Pool(pool.data_ptr(), shape[1], *a)), form, _maybe(cut, 8 * n),
        _maybe(status, n), _maybe(ctr, 32), _stream(stream)))
