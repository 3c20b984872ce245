"""ctypes binding of libdsv4sa.so (include/dsv4sa.h): same names, torch tensors in.

Argument marshalling only: every function here checks that its tensors live on
a CUDA device with the expected dtype and shape, passes their data pointers and
the current torch stream to the C entry point of the same name, and raises
``DSV4SAError`` on a non-zero status.  There is no fallback: if the shared
library is missing or a tensor is on the CPU, the call fails loudly.

``pack_kv_pool`` / ``pack_key_pool`` lay logical cache arrays out in the
library's paged byte layout (offsets taken from ``dsv4sa_pool_desc_init``),
and ``DeviceWorkload`` + ``run_path`` drive the whole hot path through the C
ABI for tests and the benchmark.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsv4sa.so")

POOL_KV = 0
POOL_IDXK = 1
POOL_IDXK_FP4 = 2
POOL_KV_FP4 = 3
MAX_POOLS = 4
ATTN_DECODE = 0
ATTN_PREFILL = 1
ROPE_PAIRS = 0     # pairs (2i, 2i + 1)
ROPE_HALVES = 1    # pairs (i, i + half)
PAGE = 64
HEAD_DIM = 512

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported size", 3: "workspace missing or too small",
          4: "CUDA runtime error", 5: "index or page id out of range (device)", 6: "device wait timed out",
          7: "no free page left (device)"}


class DSV4SAError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed: {status} ({STATUS.get(status, 'unknown')})")
        self.status = status


class PoolDesc(ctypes.Structure):
    device = None   # of the tensor it was made from
    _fields_ = [("kind", ctypes.c_int32), ("page_size", ctypes.c_int32), ("nope_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("scale_group", ctypes.c_int32), ("n_scales", ctypes.c_int32),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("nope_off", ctypes.c_int64),
                ("rope_off", ctypes.c_int64), ("scale_off", ctypes.c_int64), ("nope_row", ctypes.c_int32),
                ("rope_row", ctypes.c_int32), ("scale_row", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("base", ctypes.c_void_p)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("flags", ctypes.c_int32),
                ("attn_sink", ctypes.c_void_p), ("q_seq", ctypes.c_void_p),
                ("comp", ctypes.POINTER(PoolDesc)), ("comp_pt", ctypes.c_void_p),
                ("comp_pt_stride", ctypes.c_int32), ("kc", ctypes.c_int32), ("idx_c", ctypes.c_void_p),
                ("idx_c_stride", ctypes.c_int32), ("kw", ctypes.c_int32),
                ("win", ctypes.POINTER(PoolDesc)), ("win_pt", ctypes.c_void_p),
                ("win_pt_stride", ctypes.c_int32), ("idx_w_stride", ctypes.c_int32),
                ("idx_w", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("ws", ctypes.c_void_p), ("ws_bytes", ctypes.c_size_t),
                ("win_pos", ctypes.c_void_p), ("win_ring", ctypes.c_int32), ("reserved1", ctypes.c_int32),
                ("rope_cs", ctypes.c_void_p), ("rope_pos", ctypes.c_void_p), ("rope_rows", ctypes.c_int32),
                ("reserved2", ctypes.c_int32)]


class CacheDesc(ctypes.Structure):
    device = None   # of its tensors
    _fields_ = [("pools", ctypes.POINTER(PoolDesc)), ("n_pools", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("pt_stride", ctypes.c_int32), ("reserved", ctypes.c_int32), ("page_table", ctypes.c_void_p),
                ("use", ctypes.c_void_p)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_tok_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_tok_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64),
                ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("dim", ctypes.c_int32), ("rope_off", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("rope_rows", ctypes.c_int32), ("rope_cs", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("norm_w", ctypes.c_void_p)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("pool", ctypes.POINTER(PoolDesc)), ("page_table", ctypes.c_void_p), ("pt_stride", ctypes.c_int32),
                ("ring", ctypes.c_int32), ("row_seq", ctypes.c_void_p), ("row_pos", ctypes.c_void_p),
                ("row_entry", ctypes.c_void_p), ("src_row", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("row_stride", ctypes.c_int64), ("n_src", ctypes.c_int32), ("n", ctypes.c_int32),
                ("rope_cs", ctypes.c_void_p), ("rope_rows", ctypes.c_int32), ("norm", ctypes.c_int32),
                ("norm_w", ctypes.c_void_p), ("eps", ctypes.c_float), ("pt_rows", ctypes.c_int32)]


class TreeArgs(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("n_seqs", ctypes.c_int32), ("attn_sink", ctypes.c_void_p), ("node_start", ctypes.c_void_p),
                ("seq_row", ctypes.c_void_p), ("ctx", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("anc", ctypes.c_void_p),
                ("n_vis", ctypes.c_void_p), ("n_max", ctypes.c_int32), ("max_nodes", ctypes.c_int32),
                ("comp", ctypes.POINTER(PoolDesc)), ("comp_pt", ctypes.c_void_p), ("win", ctypes.POINTER(PoolDesc)),
                ("win_pt", ctypes.c_void_p), ("comp_pt_stride", ctypes.c_int32), ("win_pt_stride", ctypes.c_int32),
                ("window", ctypes.c_int32), ("win_ring", ctypes.c_int32), ("draft_entry", ctypes.c_int32),
                ("rope_rows", ctypes.c_int32), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("rope_cs", ctypes.c_void_p), ("rope_pos", ctypes.c_void_p), ("ws", ctypes.c_void_p),
                ("ws_bytes", ctypes.c_size_t), ("comp_pt_rows", ctypes.c_int32), ("win_pt_rows", ctypes.c_int32)]


class StepDesc(ctypes.Structure):
    _fields_ = [("host_in", ctypes.c_void_p), ("dev_in", ctypes.c_void_p), ("in_bytes", ctypes.c_size_t),
                ("in_split", ctypes.c_size_t), ("kpool", ctypes.POINTER(PoolDesc)), ("page_table", ctypes.c_void_p),
                ("pt_stride", ctypes.c_int32), ("T", ctypes.c_int32), ("q_seq", ctypes.c_void_p),
                ("n_vis", ctypes.c_void_p), ("q_fp8", ctypes.c_void_p), ("q_scale", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("Hi", ctypes.c_int32), ("n_max", ctypes.c_int32), ("logits", ctypes.c_void_p),
                ("logits_stride", ctypes.c_int64), ("k", ctypes.c_int32), ("idx_stride", ctypes.c_int32),
                ("idx", ctypes.c_void_p), ("topk_ws", ctypes.c_void_p), ("topk_ws_bytes", ctypes.c_size_t),
                ("attn", ctypes.POINTER(AttnArgs))]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_SIGS = {
    "dsv4sa_version": ([], ctypes.c_int),
    "dsv4sa_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "dsv4sa_pool_bytes": ([_I32, _I64], _SZ),
    "dsv4sa_pool_desc_init": ([ctypes.POINTER(PoolDesc), _I32, _P, _I64], ctypes.c_int),
    "dsv4sa_indexer_logits": ([ctypes.POINTER(PoolDesc), _P, _I32, _P, _P, _P, _P, _P, _I32, _I32, _I32, _P,
                               _I64, _P], ctypes.c_int),
    "dsv4sa_indexer_logits_fp4": ([ctypes.POINTER(PoolDesc), _P, _I32, _P, _P, _P, _P, _P, _I32, _I32, _I32,
                                   _P, _I64, _P], ctypes.c_int),
    "dsv4sa_topk_workspace_size": ([_I32, _I32, _I32], _SZ),
    "dsv4sa_attn_plan": ([_I32, _I32, _I32, _I32, _I32, ctypes.POINTER(_I32), ctypes.POINTER(_I32),
                          ctypes.POINTER(_I32)], ctypes.c_int),
    "dsv4sa_topk": ([_P, _I64, _P, _I32, _I32, _I32, _P, _I32, _P, _SZ, _P], ctypes.c_int),
    "dsv4sa_topk_noalloc": ([_P, _I64, _P, _I32, _I32, _I32, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_topk_prefetch": ([_P, _I64, _P, _I32, _I32, _I32, _P, _I32, _P, _SZ, ctypes.POINTER(PoolDesc), _P, _I32,
                              _P, _P], ctypes.c_int),
    "dsv4sa_window_indices": ([_P, _I32, _I32, _I32, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_cache_write": ([ctypes.POINTER(PoolDesc), _P, _I32, _P, _P, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_cache_write_rotated": ([ctypes.POINTER(PoolDesc), _P, _I32, _P, _P, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_cache_read": ([ctypes.POINTER(PoolDesc), _P, _I32, _P, _P, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_pages_copy": ([ctypes.POINTER(PoolDesc), _I32, _P, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_cache_release": ([ctypes.POINTER(CacheDesc), _P, _I32, _P], ctypes.c_int),
    "dsv4sa_cache_fork": ([ctypes.POINTER(CacheDesc), _P, _P, _P, _I32, _P, _P], ctypes.c_int),
    "dsv4sa_cache_compact": ([ctypes.POINTER(CacheDesc), ctypes.POINTER(CacheDesc), _P, _P, _P], ctypes.c_int),
    "dsv4sa_rmsnorm_quant": ([_P, _I64, _P, _I64, _P, ctypes.c_float, _I32, _I32, _I32, _P, _P, _P, _P, _P],
                             ctypes.c_int),
    "dsv4sa_rope_table": ([_P, _I64, _I32, _I64, ctypes.c_double, ctypes.c_double, _I64, ctypes.c_double, ctypes.c_double,
                           _P], ctypes.c_int),
    "dsv4sa_rope": ([ctypes.POINTER(RopeArgs), _P], ctypes.c_int),
    "dsv4sa_cache_append": ([ctypes.POINTER(AppendArgs), _P], ctypes.c_int),
    "dsv4sa_tree_attn_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "dsv4sa_tree_attn": ([ctypes.POINTER(TreeArgs), _P], ctypes.c_int),
    "dsv4sa_tree_window_indices": ([_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _I64, _P], ctypes.c_int),
    "dsv4sa_compress_indices": ([_P, _I32, _I32, _P, _I32, _P], ctypes.c_int),
    "dsv4sa_selftest_wait_timeout": ([_P, _P], ctypes.c_int),
    "dsv4sa_copy_async": ([_P, _P, _SZ, _P], ctypes.c_int),
    "dsv4sa_copy_async_background": ([_P, _P, _SZ, _P], ctypes.c_int),
    "dsv4sa_compress_windows": ([_P, _P, _I64, _I64, _P, _P, _P, _I32, _I32, _I32, _P, _P, ctypes.c_float, _P, _I32,
                                 _P, _P], ctypes.c_int),
    "dsv4sa_compress_online_c128": ([_P, _P, _I64, _I32, _P, _P, _P, _I32, _P, _P, _P, ctypes.c_float, _P, _I32,
                                     _P, _P, _P], ctypes.c_int),
    "dsv4sa_attn_workspace_size": ([_I32, _I32, _I32, _I32, _I32], _SZ),
    "dsv4sa_sparse_attn_decode": ([ctypes.POINTER(AttnArgs), _P], ctypes.c_int),
    "dsv4sa_topk_sparse_attn_decode": ([ctypes.POINTER(AttnArgs), _P, _I64, _P, _I32, _I32, _P, _SZ, _P], ctypes.c_int),
    "dsv4sa_sparse_attn_prefill": ([ctypes.POINTER(AttnArgs), _P], ctypes.c_int),
    "dsv4sa_check_errors": ([_P, ctypes.POINTER(ctypes.c_uint32)], ctypes.c_int),
    "dsv4sa_step_create": ([ctypes.POINTER(_P), ctypes.POINTER(StepDesc), _P], ctypes.c_int),
    "dsv4sa_step_launch": ([_P, _P], ctypes.c_int),
    "dsv4sa_step_destroy": ([_P], ctypes.c_int),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded shared library (loaded on first use; raises if it is not built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built: run `python -m compressed_sparse_attention_c4_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _LIB = L
    return _LIB


def exported_symbols():
    return list(_SIGS)


def _check(fn, status):
    if status != 0:
        raise DSV4SAError(fn, status)


# a small call is bound by the host: names of this module instead of attributes of torch
_Tensor, _int32, _bf16, _f32, _u8 = torch.Tensor, torch.int32, torch.bfloat16, torch.float32, torch.uint8
_int64 = torch.int64


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here() -> int:
    """The current device; -2 (no tensor's) on a host without one."""
    try:
        return _current_device()
    except RuntimeError:
        return -2


def _refuse_device(name: str, device: int):
    """The library launches on the current device: memory of another one is refused."""
    raise ValueError(f"{name} is on cuda:{device}, the current device is cuda:{_current_device()}")


def _dev(t: torch.Tensor, name: str, dtype=None, here=None):
    """The address of a contiguous tensor (of that dtype) on the current CUDA device, or an
    error.  A call of many tensors looks the device up once and gives it as `here`."""
    if here is None:
        here = _here()
    if type(t) is _Tensor and t.get_device() == here and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.get_device() != here:
        _refuse_device(name, t.get_device())
    return t.data_ptr()


def _dev_or_pinned(t: torch.Tensor, name: str, dtype=None, here=None):
    """A CUDA tensor, or a pinned host tensor: with unified addressing its
    pointer is valid on the device and the kernel's stores cross the host link."""
    if isinstance(t, _Tensor) and not t.is_cuda and t.is_pinned():
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()
    return _dev(t, name, dtype, here)


# The current stream's handle without a Stream object around it (3 us a call less).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, here=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device() if here is None else here)
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@contextlib.contextmanager
def _running_on(stream):
    """Torch's work and the library's inside the block run on `stream` (a torch stream or a
    handle; None: the current one), after what the current stream holds already; the
    current stream then waits for it.  Tensors made inside belong to `stream`, so their
    memory is not used again before its kernels have read them."""
    if stream is None:
        yield
        return
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream))
    caller = torch.cuda.current_stream()
    s.wait_stream(caller)
    try:
        with torch.cuda.stream(s):
            yield
    finally:
        caller.wait_stream(s)


# ---------------------------------------------------------------- pools

def dsv4sa_pool_bytes(kind: int, num_pages: int) -> int:
    return int(lib().dsv4sa_pool_bytes(kind, num_pages))


def dsv4sa_pool_desc_init(kind: int, base: int | torch.Tensor, num_pages: int) -> PoolDesc:
    """The descriptor of a pool at `base`, a device tensor or an address.  It does not keep
    the memory alive; calls refuse a pool made from a CUDA tensor that is not on the current
    device (of an address, or of pinned host memory, there is nothing to compare)."""
    d = PoolDesc()
    ptr = base.data_ptr() if isinstance(base, torch.Tensor) else int(base)
    _check("dsv4sa_pool_desc_init", lib().dsv4sa_pool_desc_init(ctypes.byref(d), kind, ctypes.c_void_p(ptr), num_pages))
    if isinstance(base, torch.Tensor) and base.is_cuda:
        d.device = base.get_device()
    return d


def _pool(d: PoolDesc, name: str, here=None) -> PoolDesc:
    if d.device is not None and d.device != (_here() if here is None else here):
        _refuse_device(name, d.device)
    return d


def _cache(c: "CacheDesc", name: str, here: int):
    """A reference to a cache on the current device."""
    if c.device is not None and c.device != here:
        _refuse_device(name, c.device)
    return ctypes.byref(c)


def _layout(kind: int, num_pages: int) -> PoolDesc:
    return dsv4sa_pool_desc_init(kind, 1 << 20, num_pages)   # any aligned base: offsets only


def _alloc_pool(kind: int, num_pages: int, device) -> torch.Tensor:
    nbytes = dsv4sa_pool_bytes(kind, num_pages)
    buf = torch.empty(nbytes + 1024, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 1024
    return buf[off:off + nbytes]


def pack_kv_pool(nope_codes: np.ndarray, nope_scale: np.ndarray, rope_bits: np.ndarray, device="cuda"):
    """Logical KV pool arrays -> (device byte tensor, PoolDesc) in the library layout."""
    P = nope_codes.shape[0]
    L = _layout(POOL_KV, P)
    host = np.zeros((P, L.page_stride), dtype=np.uint8)
    host[:, L.nope_off:L.nope_off + PAGE * L.nope_row] = nope_codes.reshape(P, -1)
    host[:, L.rope_off:L.rope_off + PAGE * L.rope_row] = np.ascontiguousarray(rope_bits).view(np.uint8).reshape(P, -1)
    sc = np.zeros((P, PAGE, L.scale_row // 4), dtype=np.float32)
    sc[:, :, :nope_scale.shape[-1]] = nope_scale
    host[:, L.scale_off:L.scale_off + PAGE * L.scale_row] = sc.view(np.uint8).reshape(P, -1)
    dev = _alloc_pool(POOL_KV, P, device)
    dev.copy_(torch.from_numpy(host.reshape(-1)))
    return dev, dsv4sa_pool_desc_init(POOL_KV, dev, P)


def pack_key_pool(codes: np.ndarray, scale: np.ndarray, device="cuda"):
    """Logical indexer-key pool arrays -> (device byte tensor, PoolDesc)."""
    P = codes.shape[0]
    L = _layout(POOL_IDXK, P)
    host = np.zeros((P, L.page_stride), dtype=np.uint8)
    host[:, L.nope_off:L.nope_off + PAGE * L.nope_row] = codes.reshape(P, -1)
    host[:, L.scale_off:L.scale_off + PAGE * L.scale_row] = \
        np.ascontiguousarray(scale, dtype=np.float32).view(np.uint8).reshape(P, -1)
    dev = _alloc_pool(POOL_IDXK, P, device)
    dev.copy_(torch.from_numpy(host.reshape(-1)))
    return dev, dsv4sa_pool_desc_init(POOL_IDXK, dev, P)


def pack_key_pool_fp4(codes: np.ndarray, e8m0: np.ndarray, device="cuda"):
    """Logical FP4 indexer-key pool arrays (E2M1 codes uint8 [P, 64, 128], one
    per byte; E8M0 bytes [P, 64, 4]) -> (device byte tensor, PoolDesc): codes two
    per byte, value 2j in the low nibble of byte j."""
    P = codes.shape[0]
    L = _layout(POOL_IDXK_FP4, P)
    c = np.asarray(codes, np.uint8) & 0xF
    packed = (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)
    host = np.zeros((P, L.page_stride), dtype=np.uint8)
    host[:, L.nope_off:L.nope_off + PAGE * L.nope_row] = packed.reshape(P, -1)
    host[:, L.scale_off:L.scale_off + PAGE * L.scale_row] = np.asarray(e8m0, np.uint8).reshape(P, -1)
    dev = _alloc_pool(POOL_IDXK_FP4, P, device)
    dev.copy_(torch.from_numpy(host.reshape(-1)))
    return dev, dsv4sa_pool_desc_init(POOL_IDXK_FP4, dev, P)


def pack_kv_pool_fp4(nope_codes: np.ndarray, nope_e8m0: np.ndarray, rope_bits: np.ndarray, device="cuda"):
    """Logical FP4 KV pool arrays (E2M1 codes uint8 [P, 64, 448], one per byte; E8M0
    bytes [P, 64, 14]; BF16 bits [P, 64, 64]) -> (device byte tensor, PoolDesc)."""
    P = nope_codes.shape[0]
    L = _layout(POOL_KV_FP4, P)
    host = np.zeros((P, L.page_stride), dtype=np.uint8)
    host[:, L.nope_off:L.nope_off + PAGE * L.nope_row] = pack_fp4_codes(nope_codes).reshape(P, -1)
    host[:, L.rope_off:L.rope_off + PAGE * L.rope_row] = np.ascontiguousarray(rope_bits).view(np.uint8).reshape(P, -1)
    sc = np.zeros((P, PAGE, L.scale_row), dtype=np.uint8)
    sc[:, :, :L.n_scales] = nope_e8m0
    host[:, L.scale_off:L.scale_off + PAGE * L.scale_row] = sc.reshape(P, -1)
    dev = _alloc_pool(POOL_KV_FP4, P, device)
    dev.copy_(torch.from_numpy(host.reshape(-1)))
    return dev, dsv4sa_pool_desc_init(POOL_KV_FP4, dev, P)


# ---------------------------------------------------------------- stage 1: indexer

def dsv4sa_indexer_logits(kpool: PoolDesc, page_table, q_seq, n_vis, q_fp8, q_scale, w, n_max: int, logits,
                          stream=None):
    T, Hi = q_fp8.shape[0], q_fp8.shape[1]
    st = lib().dsv4sa_indexer_logits(
        ctypes.byref(_pool(kpool, "kpool")), _dev(page_table, "page_table", torch.int32), page_table.shape[-1],
        _dev(q_seq, "q_seq", torch.int32), _dev(n_vis, "n_vis", torch.int32), _dev(q_fp8, "q_fp8", torch.uint8),
        _dev(q_scale, "q_scale", torch.float32), _dev(w, "w", torch.float32), T, Hi, n_max,
        _dev(logits, "logits", torch.float32), logits.shape[-1], _stream(stream))
    _check("dsv4sa_indexer_logits", st)


def pack_fp4_codes(codes: np.ndarray) -> np.ndarray:
    """E2M1 codes one per byte [..., 2 m] -> packed bytes [..., m], value 2j in
    the low nibble of byte j (the layout of FP4 q and FP4 pool codes)."""
    c = np.asarray(codes, np.uint8) & 0xF
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def dsv4sa_indexer_logits_fp4(kpool: PoolDesc, page_table, q_seq, n_vis, q_fp4, q_e8m0, w, n_max: int, logits,
                              stream=None):
    """q_fp4: device uint8 [T, Hi, 64] packed E2M1 codes; q_e8m0: uint8 [T, Hi, 4]."""
    T, Hi = q_fp4.shape[0], q_fp4.shape[1]
    st = lib().dsv4sa_indexer_logits_fp4(
        ctypes.byref(_pool(kpool, "kpool")), _dev(page_table, "page_table", torch.int32), page_table.shape[-1],
        _dev(q_seq, "q_seq", torch.int32), _dev(n_vis, "n_vis", torch.int32), _dev(q_fp4, "q_fp4", torch.uint8),
        _dev(q_e8m0, "q_e8m0", torch.uint8), _dev(w, "w", torch.float32), T, Hi, n_max,
        _dev(logits, "logits", torch.float32), logits.shape[-1], _stream(stream))
    _check("dsv4sa_indexer_logits_fp4", st)


# ---------------------------------------------------------------- stage 2: top-k

def dsv4sa_topk_workspace_size(T: int, n_max: int, k: int) -> int:
    return int(lib().dsv4sa_topk_workspace_size(T, n_max, k))


def dsv4sa_topk(logits, n_vis, n_max: int, k: int, idx, ws=None, stream=None):
    T = n_vis.shape[0]
    wsp = _dev(ws, "ws", torch.uint8) if ws is not None else None
    st = lib().dsv4sa_topk(_dev(logits, "logits", torch.float32), logits.shape[-1], _dev(n_vis, "n_vis", torch.int32),
                           T, n_max, k, _dev(idx, "idx", torch.int32), idx.shape[-1], wsp,
                           0 if ws is None else ws.numel(), _stream(stream))
    _check("dsv4sa_topk", st)


def dsv4sa_topk_prefetch(logits, n_vis, n_max: int, k: int, idx, kv_pool: PoolDesc, kv_pt, q_seq, ws=None,
                         stream=None):
    """dsv4sa_topk, with each selected entry's row of the compressed KV pool
    prefetched into L2 for the attention that gathers it next."""
    T = n_vis.shape[0]
    wsp = _dev(ws, "ws", torch.uint8) if ws is not None else None
    st = lib().dsv4sa_topk_prefetch(_dev(logits, "logits", torch.float32), logits.shape[-1],
                                    _dev(n_vis, "n_vis", torch.int32), T, n_max, k, _dev(idx, "idx", torch.int32),
                                    idx.shape[-1], wsp, 0 if ws is None else ws.numel(), ctypes.byref(_pool(kv_pool, "kv_pool")),
                                    _dev(kv_pt, "kv_pt", torch.int32), kv_pt.shape[-1],
                                    _dev(q_seq, "q_seq", torch.int32), _stream(stream))
    _check("dsv4sa_topk_prefetch", st)


def dsv4sa_topk_noalloc(logits, n_vis, n_max: int, k: int, idx, stream=None):
    """dsv4sa_topk without a workspace: for callers that cannot allocate device
    memory when they call; uses the library's fixed 8 MiB device scratch (see
    include/dsv4sa.h for the size limit and the sharing rules)."""
    T = n_vis.shape[0]
    st = lib().dsv4sa_topk_noalloc(_dev(logits, "logits", torch.float32), logits.shape[-1],
                                   _dev(n_vis, "n_vis", torch.int32), T, n_max, k, _dev(idx, "idx", torch.int32),
                                   idx.shape[-1], _stream(stream))
    _check("dsv4sa_topk_noalloc", st)


# ---------------------------------------------------------------- index assembly

def dsv4sa_window_indices(pos, window: int, ring: int, idx_w, stream=None):
    st = lib().dsv4sa_window_indices(_dev(pos, "pos", torch.int32), pos.shape[0], window, ring,
                                     _dev(idx_w, "idx_w", torch.int32), idx_w.shape[-1], _stream(stream))
    _check("dsv4sa_window_indices", st)


def _one_for_each_row(row_seq, row_entry, n: int):
    if row_seq.numel() < n or row_entry.numel() < n:
        raise ValueError(f"row_seq and row_entry must have one entry for each of the {n} rows")


def dsv4sa_cache_write(pool: PoolDesc, page_table, row_seq, row_entry, rows, stream=None):
    """Quantise BF16 rows [n, 512] (KV and KV_FP4 pools) or [n, 128] (indexer-key pools) into the pool
    (of longer lists the first n entries count)."""
    want = HEAD_DIM if pool.kind in (POOL_KV, POOL_KV_FP4) else 128
    shape = rows.shape
    if len(shape) != 2 or shape[1] != want:
        raise ValueError(f"rows must be [n, {want}]")
    _one_for_each_row(row_seq, row_entry, shape[0])
    here = _here()
    st = lib().dsv4sa_cache_write(
        ctypes.byref(_pool(pool, "pool", here)), _dev(page_table, "page_table", _int32, here), page_table.shape[-1],
        _dev(row_seq, "row_seq", _int32, here), _dev(row_entry, "row_entry", _int32, here), _dev(rows, "rows", _bf16, here),
        shape[0], _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_cache_write", st)


def dsv4sa_cache_write_rotated(pool: PoolDesc, page_table, row_seq, row_entry, rows, stream=None):
    """Rotate BF16 keys [n, 128] by the order-128 Hadamard transform, then quantise
    them into an FP4 indexer-key pool."""
    if rows.dim() != 2 or rows.shape[1] != 128:
        raise ValueError("rows must be [n, 128]")
    _one_for_each_row(row_seq, row_entry, rows.shape[0])
    _check("dsv4sa_cache_write_rotated", lib().dsv4sa_cache_write_rotated(
        ctypes.byref(_pool(pool, "pool")), _dev(page_table, "page_table", torch.int32), page_table.shape[-1],
        _dev(row_seq, "row_seq", torch.int32), _dev(row_entry, "row_entry", torch.int32),
        _dev(rows, "rows", torch.bfloat16), rows.shape[0], _stream(stream)))


def dsv4sa_cache_read(pool: PoolDesc, page_table, row_seq, row_entry, rows, stream=None):
    """Rows of a KV or KV_FP4 pool into BF16 rows [n, 512]: the values the attention reads."""
    n = row_entry.shape[0]
    if rows.shape != (n, HEAD_DIM) or row_seq.shape[0] != n:
        raise ValueError("rows must be [n, 512] for n entries")
    here = _here()
    st = lib().dsv4sa_cache_read(
        ctypes.byref(_pool(pool, "pool", here)), _dev(page_table, "page_table", _int32, here), page_table.shape[-1],
        _dev(row_seq, "row_seq", _int32, here), _dev(row_entry, "row_entry", _int32, here), _dev(rows, "rows", _bf16, here),
        n, _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_cache_read", st)


# ---------------------------------------------------------------- pages of a cache

def _pool_array(pools):
    if not 1 <= len(pools) <= MAX_POOLS:
        raise ValueError(f"a cache has 1 to {MAX_POOLS} pools")
    return (PoolDesc * len(pools))(*[_pool(d, "pool") for d in pools])


def page_cache(pools, page_table, use) -> CacheDesc:
    """The descriptor of a cache: pools that share page ids, the page table int32
    [rows, pt_stride] and the use counts int32 [num_pages] (table entries that
    hold each page).  The descriptor keeps these two tensors alive, not the pools' memory."""
    if page_table.dim() != 2:
        raise ValueError("page_table must be [rows, pt_stride]")
    if use.shape != (pools[0].num_pages,):
        raise ValueError("use must have one count per page")
    c = CacheDesc()
    c._keep = (_pool_array(pools), page_table, use)
    c.pools = ctypes.cast(c._keep[0], ctypes.POINTER(PoolDesc))
    c.n_pools = len(pools)
    c.rows, c.pt_stride = page_table.shape
    c.page_table = _dev(page_table, "page_table", torch.int32)
    c.use = _dev(use, "use", torch.int32)
    c.device = page_table.get_device()
    return c


def dsv4sa_pages_copy(pools, src_page, dst_page, stream=None):
    """Copy pages src_page[i] -> dst_page[i] of every pool in the list (int32 [n]; -1: skip)."""
    if src_page.shape != dst_page.shape:
        raise ValueError("src_page and dst_page differ in length")
    arr = _pool_array(pools)
    _check("dsv4sa_pages_copy", lib().dsv4sa_pages_copy(
        arr, len(pools), _dev(src_page, "src_page", torch.int32), _dev(dst_page, "dst_page", torch.int32),
        src_page.numel(), _stream(stream)))


def dsv4sa_cache_release(cache: CacheDesc, row, stream=None):
    """Release rows (int32 [n]) of the page table: entries -1, their pages' counts down by one."""
    here = _here()
    st = lib().dsv4sa_cache_release(_cache(cache, "cache", here), _dev(row, "row", _int32, here), row.numel(),
                                    _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_cache_release", st)


def dsv4sa_cache_fork(cache: CacheDesc, src_row, dst_row, length, new_page, stream=None):
    """Fork the first length[i] entries of row src_row[i] into the empty row dst_row[i]:
    full pages shared, a partial last page copied into new_page[i] (all int32 [n])."""
    n = src_row.numel()
    if dst_row.numel() != n or length.numel() != n or new_page.numel() != n:
        raise ValueError("src_row, dst_row, length and new_page differ in length")
    here = _here()
    st = lib().dsv4sa_cache_fork(
        _cache(cache, "cache", here), _dev(src_row, "src_row", _int32, here), _dev(dst_row, "dst_row", _int32, here),
        _dev(length, "length", _int32, here), n, _dev(new_page, "new_page", _int32, here), _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_cache_fork", st)


def dsv4sa_cache_compact(src: CacheDesc, dst: CacheDesc, new_id, n_used, stream=None):
    """Move the pages in use to the front of dst's pools (dst may be src: in place),
    with dst's table and counts by the new ids.  new_id int32 [src pages], n_used int32 [1]."""
    if new_id.numel() != src.pools[0].num_pages or n_used.numel() != 1:
        raise ValueError("new_id must have one entry per page, n_used one")
    here = _here()
    _check("dsv4sa_cache_compact", lib().dsv4sa_cache_compact(
        _cache(src, "src", here), _cache(dst, "dst", here), _dev(new_id, "new_id", _int32, here),
        _dev(n_used, "n_used", _int32, here), _stream(stream, here)))


# ---------------------------------------------------------------- norm

def _bf16_rows(t: torch.Tensor, name: str, shape, here):
    """A BF16 tensor [n, dim] on the current CUDA device whose rows may be strided -> (pointer, row stride)."""
    if t.get_device() != here:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        _refuse_device(name, t.get_device())
    if t.dtype is not _bf16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    n, dim = shape
    row, col = t.stride() if t.shape == shape else (0, 0)
    if col != 1 and dim > 1:
        raise ValueError(f"{name} must be [{n}, {dim}] with consecutive values in a row")
    return t.data_ptr(), (row if n > 1 else dim)


def dsv4sa_rmsnorm_quant(x, norm_w, codes=None, scale=None, group: int = 128, residual=None, residual_out=None, y=None,
                         eps: float = 1e-6, stream=None):
    """RMSNorm of BF16 rows x [n, dim] (+ residual) with fp32 weights [dim]: E4M3 codes
    uint8 [n, dim] with fp32 scales [n, dim / group], the sum x + residual and
    the norm's output as BF16 [n, dim], each where a tensor is given (see dsv4sa.h)."""
    shape = x.shape
    n, dim = shape
    if norm_w.shape != (dim,):
        raise ValueError("norm_w must be [dim]")
    here = _here()
    xp, xs = _bf16_rows(x, "x", shape, here)
    rp, rs = _bf16_rows(residual, "residual", shape, here) if residual is not None else (None, 0)
    op = yp = cp = sp = None
    if residual_out is not None:
        if residual_out.shape != shape:
            raise ValueError("residual_out must be [n, dim]")
        op = _dev(residual_out, "residual_out", _bf16, here)
    if y is not None:
        if y.shape != shape:
            raise ValueError("y must be [n, dim]")
        yp = _dev(y, "y", _bf16, here)
    if codes is not None:
        if codes.shape != shape:
            raise ValueError("codes must be [n, dim]")
        cp = _dev(codes, "codes", _u8, here)
    if scale is not None:
        if group < 1 or scale.shape != (n, dim // group):
            raise ValueError("scale must be [n, dim / group]")
        sp = _dev(scale, "scale", _f32, here)
    st = lib().dsv4sa_rmsnorm_quant(xp, xs, rp, rs, _dev(norm_w, "norm_w", _f32, here), eps, n, dim, group, op, yp, cp, sp,
                                    _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_rmsnorm_quant", st)


# ---------------------------------------------------------------- rotary positions

def dsv4sa_rope_table(cs, base: float = 10000.0, first: int = 0, factor: float = 1.0, original_len: int = 0,
                      beta_fast: float = 32.0, beta_slow: float = 1.0, stream=None):
    """The rotation table cs fp32 [rows, pairs, 2]: (cos, sin) of positions first, first + 1, ...
    (first plus a table of 32 pairs is what the attention, the compressor and cache_append
    take as rope_cs); factor > 1 scales the context, by YaRN with original_len > 0."""
    if cs.dim() != 3 or cs.shape[2] != 2:
        raise ValueError("cs must be [rows, pairs, 2]")
    here = _here()
    _check("dsv4sa_rope_table", lib().dsv4sa_rope_table(
        _dev(cs, "cs", _f32, here), cs.shape[0], cs.shape[1], first, base, factor, original_len, beta_fast, beta_slow,
        _stream(stream, here)))


def _heads(t: torch.Tensor, name: str, shape, here):
    """A BF16 tensor [T, H, dim] on the current CUDA device, tokens and heads strided -> (pointer, strides)."""
    if t.get_device() != here:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        _refuse_device(name, t.get_device())
    if t.dtype is not _bf16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    tok, head, col = t.stride()
    if col != 1 and shape[2] > 1:
        raise ValueError(f"{name} must have consecutive values in a head")
    return t.data_ptr(), tok, head


def _table_of(rope_cs, pairs, here):
    if rope_cs.dim() != 3 or rope_cs.shape[2] != 2 or (pairs and rope_cs.shape[1] != pairs):
        raise ValueError(f"rope_cs must be [rows, {pairs or 'pairs'}, 2]")
    return _dev(rope_cs, "rope_cs", _f32, here)


def dsv4sa_rope(x, rope_cs, pos, out=None, rope_off=None, layout: int = ROPE_PAIRS, inverse: bool = False, eps=None,
                norm_w=None, stream=None):
    """Heads x bf16 [T, H, dim] (tokens and heads may be strided) with dims rope_off .. rope_off +
    2 pairs (the last ones by default) rotated by rows pos int32 [T] of rope_cs [rows, pairs, 2],
    into out, or in place.  With eps each head is divided by its root mean square first, and
    multiplied by norm_w fp32 [dim] if given (see dsv4sa.h)."""
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [T, H, dim]")
    T, H, dim = shape
    here = _here()
    xp, xt, xh = _heads(x, "x", shape, here)
    op, ot, oh = (xp, xt, xh) if out is None else _heads(out, "out", shape, here)
    cs = _table_of(rope_cs, None, here)
    rope_dim = 2 * rope_cs.shape[1]
    if pos.numel() < T:
        raise ValueError(f"pos must have an entry for each of the {T} tokens")
    wp = None
    if norm_w is not None:
        if eps is None or norm_w.shape != (dim,):
            raise ValueError("norm_w must be [dim], with eps")
        wp = _dev(norm_w, "norm_w", _f32, here)
    a = RopeArgs(xp, xt, xh, op, ot, oh, T, H, dim, dim - rope_dim if rope_off is None else rope_off, rope_dim, layout,
                 1 if inverse else 0, rope_cs.shape[0], cs, _dev(pos, "pos", _int32, here), 0 if eps is None else 1, eps or 0.0, wp)
    st = lib().dsv4sa_rope(ctypes.byref(a), _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_rope", st)


def _page_table(pt, name, least, here):
    """Address, entries a row and rows of a page table, which has to have at least so many."""
    p, shape = _dev(pt, name, _int32, here), pt.shape
    rows, stride = shape if len(shape) == 2 else (pt.numel() // max(shape[-1], 1), shape[-1])
    if rows < least:
        raise ValueError(f"{name} must have a row for each sequence ({least} at least)")
    return p, stride, rows


def dsv4sa_cache_append(pool: PoolDesc, page_table, row_seq, row_pos, rows, rope_cs=None, row_entry=None, ring: int = 0,
                        src_row=None, norm_w=None, eps=None, stream=None):
    """New rows bf16 [n_src, 512] (rows may be strided) of the KV projection into a KV or KV_FP4 pool:
    normed where eps is given (times norm_w fp32 [512] if given), the last 64 dims rotated by row
    row_pos[r] of rope_cs [rows, 32, 2] where it is given, quantised.  Row r is rows[src_row[r]] or
    rows[r]; it goes to entry row_entry[r], or by its position (modulo ring > 0), of page-table row
    row_seq[r] (-1: skipped).  row_seq's length is the number of rows (all lists int32)."""
    n = row_seq.shape[0]
    shape = rows.shape
    if len(shape) != 2 or shape[1] != HEAD_DIM:
        raise ValueError("rows must be [n, 512]")
    if src_row is None and shape[0] < n:
        raise ValueError(f"rows must have one row for each of the {n} entries of row_seq")
    here = _here()
    rp, rs = _bf16_rows(rows, "rows", shape, here)
    lists = []
    for t, name in ((row_pos, "row_pos"), (row_entry, "row_entry"), (src_row, "src_row")):
        if t is not None and t.numel() < n:
            raise ValueError(f"{name} must have an entry for each of the {n} rows")
        lists.append(None if t is None else _dev(t, name, _int32, here))
    cs = None if rope_cs is None else _table_of(rope_cs, 32, here)
    wp = None
    if norm_w is not None:
        if eps is None or norm_w.shape != (HEAD_DIM,):
            raise ValueError("norm_w must be [512], with eps")
        wp = _dev(norm_w, "norm_w", _f32, here)
    pt, pt_stride, pt_rows = _page_table(page_table, "page_table", 1 if n else 0, here)
    a = AppendArgs(ctypes.pointer(_pool(pool, "pool", here)), pt, pt_stride, ring, _dev(row_seq, "row_seq", _int32, here), lists[0],
                   lists[1], lists[2], rp, rs, shape[0], n, cs, 0 if rope_cs is None else rope_cs.shape[0], 0 if eps is None else 1, wp,
                   eps or 0.0, pt_rows)
    st = lib().dsv4sa_cache_append(ctypes.byref(a), _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_cache_append", st)


def dsv4sa_compress_windows(kv, score, first_tok, prev_tok, position, ratio: int, overlap: bool, ape, norm_w,
                            rope_cs, out, eps: float = 1e-6, stream=None):
    """Pool windows of projected tokens into compressed entries (see dsv4sa.h).
    kv, score: bf16 [n_tok, coff * 512] (rows may be strided); first_tok,
    prev_tok (overlap only), position: int32 [n]; ape fp32 [ratio, coff * 512];
    norm_w fp32 [512]; rope_cs fp32 [rows, 32, 2]; out bf16 [n, 512]."""
    n = first_tok.shape[0]
    if kv.stride(1) != 1 or score.stride(0) != kv.stride(0) or score.shape != kv.shape:
        raise ValueError("kv and score must be row-major with the same row stride")
    _check("dsv4sa_compress_windows", lib().dsv4sa_compress_windows(
        _dev(kv, "kv", torch.bfloat16), _dev(score, "score", torch.bfloat16), kv.stride(0), kv.shape[0],
        _dev(first_tok, "first_tok", torch.int32), _dev(prev_tok, "prev_tok", torch.int32) if overlap else None,
        _dev(position, "position", torch.int32), n, int(ratio), 1 if overlap else 0,
        _dev(ape, "ape", torch.float32), _dev(norm_w, "norm_w", torch.float32), float(eps),
        _dev(rope_cs, "rope_cs", torch.float32), rope_cs.shape[0], _dev(out, "out", torch.bfloat16), _stream(stream)))


def dsv4sa_compress_online_c128(kv, score, state_idx, state, state_count, position, ape, norm_w, rope_cs, out,
                                done, eps: float = 1e-6, stream=None):
    """Fold one new token per sequence into its online C128 state (see dsv4sa.h).
    kv, score: bf16 [T, 512]; state fp32 [slots, 3, 512]; state_count int32
    [slots]; out bf16 [T, 512]; done int32 [T]."""
    T = kv.shape[0]
    if kv.stride(1) != 1 or score.stride(0) != kv.stride(0) or score.shape != kv.shape:
        raise ValueError("kv and score must be row-major with the same row stride")
    _check("dsv4sa_compress_online_c128", lib().dsv4sa_compress_online_c128(
        _dev(kv, "kv", torch.bfloat16), _dev(score, "score", torch.bfloat16), kv.stride(0), T,
        _dev(state_idx, "state_idx", torch.int32), _dev(state, "state", torch.float32),
        _dev(state_count, "state_count", torch.int32), state.shape[0], _dev(position, "position", torch.int32),
        _dev(ape, "ape", torch.float32), _dev(norm_w, "norm_w", torch.float32), float(eps),
        _dev(rope_cs, "rope_cs", torch.float32), rope_cs.shape[0], _dev(out, "out", torch.bfloat16),
        _dev(done, "done", torch.int32), _stream(stream)))


def dsv4sa_selftest_wait_timeout(result, stream=None):
    """Launch the failure-path self-test (a bounded wait that runs out; see dsv4sa.h)."""
    _check("dsv4sa_selftest_wait_timeout", lib().dsv4sa_selftest_wait_timeout(_dev(result, "result", torch.int32),
                                                                              _stream(stream)))


def dsv4sa_copy_async(dst, src, stream=None):
    """Copy src into dst (same byte size, a multiple of 16) with the library's copy
    kernel; either may be a CUDA tensor or a pinned host tensor."""
    if dst.numel() * dst.element_size() != src.numel() * src.element_size():
        raise ValueError("dst and src differ in size")
    _check("dsv4sa_copy_async", lib().dsv4sa_copy_async(_dev_or_pinned(dst, "dst"), _dev_or_pinned(src, "src"),
                                                        dst.numel() * dst.element_size(), _stream(stream)))


def dsv4sa_copy_async_background(dst, src, stream=None):
    """dsv4sa_copy_async by one warp per SM: for a copy on a side stream that runs
    beside the indexer (see dsv4sa.h)."""
    if dst.numel() * dst.element_size() != src.numel() * src.element_size():
        raise ValueError("dst and src differ in size")
    _check("dsv4sa_copy_async_background",
           lib().dsv4sa_copy_async_background(_dev_or_pinned(dst, "dst"), _dev_or_pinned(src, "src"),
                                              dst.numel() * dst.element_size(), _stream(stream)))


def online_c128_state(slots: int, device="cuda"):
    """Fresh online C128 states: (state fp32 [slots, 3, 512] = (-inf, 0, 0), count int32 [slots] = 0)."""
    state = torch.zeros((slots, 3, 512), dtype=torch.float32, device=device)
    state[:, 0] = float("-inf")
    return state, torch.zeros(slots, dtype=torch.int32, device=device)


def dsv4sa_compress_indices(n_vis, kc: int, idx, stream=None):
    st = lib().dsv4sa_compress_indices(_dev(n_vis, "n_vis", torch.int32), n_vis.shape[0], kc,
                                       _dev(idx, "idx", torch.int32), idx.shape[-1], _stream(stream))
    _check("dsv4sa_compress_indices", st)


# ---------------------------------------------------------------- stage 3: attention

def dsv4sa_attn_workspace_size(mode: int, T: int, H: int, kc: int, kw: int) -> int:
    return int(lib().dsv4sa_attn_workspace_size(mode, T, H, kc, kw))


def dsv4sa_attn_plan(mode: int, T: int, H: int, kc: int, kw: int) -> dict:
    """Splits, rows per split and kernel launches of an attention call on the current device."""
    ns, rps, nl = _I32(), _I32(), _I32()
    _check("dsv4sa_attn_plan", lib().dsv4sa_attn_plan(mode, T, H, kc, kw, ctypes.byref(ns), ctypes.byref(rps),
                                                      ctypes.byref(nl)))
    return {"nsplit": ns.value, "rows_per_split": rps.value, "launches": nl.value}


ATTN_EARLY_WINDOW = 1


def _attn_args(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale, lse, ws,
               win_pos=None, kw=None, win_ring=0, flags=0, rope_cs=None, rope_pos=None):
    T, H, dim = q.shape
    if dim != HEAD_DIM:
        raise ValueError("q must be [T, H, 512]")
    # what the kernel reads and writes for T queries of H heads is there
    if out.numel() < q.numel() or sink.numel() < H or q_seq.numel() < T or (lse is not None and lse.numel() < T * H):
        raise ValueError(f"out, attn_sink, q_seq or lse is too small for {T} queries of {H} heads")
    here = _here()
    qp = _dev(q, "q", _bf16, here)
    cd = cpt = ic = wd = wpt = iw = wpos = rcs = rpos = None
    cpt_stride = kc = wpt_stride = n_w = iw_stride = ring = rope_rows = 0
    if idx_c is not None:
        cd = ctypes.pointer(_pool(comp, "comp", here))
        cpt = _dev(comp_pt, "comp_pt", _int32, here)
        cpt_stride = comp_pt.shape[-1]
        ic = _dev(idx_c, "idx_c", _int32, here)
        kc = idx_c.shape[-1]
        if idx_c.numel() < T * kc:
            raise ValueError(f"idx_c must have a row for each of the {T} queries")
    if idx_w is not None:
        iw = _dev(idx_w, "idx_w", _int32, here)
        n_w = iw_stride = idx_w.shape[-1]
        if idx_w.numel() < T * n_w:
            raise ValueError(f"idx_w must have a row for each of the {T} queries")
    elif win_pos is not None and kw:
        # window indices computed in the kernel from the positions
        wpos = _dev(win_pos, "win_pos", _int32, here)
        n_w, ring = int(kw), int(win_ring)
        if win_pos.numel() < T:
            raise ValueError(f"win_pos must have an entry for each of the {T} queries")
    if idx_w is not None or wpos is not None:
        wd = ctypes.pointer(_pool(win, "win", here))
        wpt = _dev(win_pt, "win_pt", _int32, here)
        wpt_stride = win_pt.shape[-1]
    if rope_cs is not None:
        # (cos, sin) table [rows, 32, 2] fp32: the inverse rotary embedding of the output
        if rope_cs.dim() != 3 or rope_cs.shape[1:] != (32, 2):
            raise ValueError("rope_cs must be [rows, 32, 2]")
        rcs = _dev(rope_cs, "rope_cs", _f32, here)
        rpos = _dev(rope_pos, "rope_pos", _int32, here)
        if rope_pos.numel() < T:
            raise ValueError(f"rope_pos must have an entry for each of the {T} queries")
        rope_rows = rope_cs.shape[0]
    # in the order of the fields: one construction costs a third of as many assignments
    return AttnArgs(qp, T, H, float(softmax_scale), int(flags), _dev(sink, "attn_sink", _f32, here),
                    _dev(q_seq, "q_seq", _int32, here), cd, cpt, cpt_stride, kc, ic, kc, n_w, wd, wpt, wpt_stride, iw_stride,
                    iw, _dev_or_pinned(out, "out", _bf16, here),
                    _dev_or_pinned(lse, "lse", _f32, here) if lse is not None else None,
                    _dev(ws, "ws", _u8, here) if ws is not None else None, ws.numel() if ws is not None else 0,
                    wpos, ring, 0, rcs, rpos, rope_rows, 0)


def dsv4sa_sparse_attn_decode(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale,
                              lse=None, ws=None, stream=None, win_pos=None, kw=None, win_ring=0, flags=0,
                              rope_cs=None, rope_pos=None):
    """idx_w=None with win_pos, kw (and win_ring) given: the window indices are
    computed in the kernel from the positions.  flags: ATTN_EARLY_WINDOW (see
    dsv4sa.h).  rope_cs [rows, 32, 2] with rope_pos [T]: the output's last 64
    dims are rotated back by the table row of each query."""
    a = _attn_args(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale, lse, ws,
                   win_pos, kw, win_ring, flags, rope_cs, rope_pos)
    _check("dsv4sa_sparse_attn_decode", lib().dsv4sa_sparse_attn_decode(ctypes.byref(a), _stream(stream)))


def dsv4sa_topk_sparse_attn_decode(logits, n_vis, n_max: int, k: int, q, sink, q_seq, comp, comp_pt, idx_c, win,
                                   win_pt, idx_w, out, softmax_scale, lse=None, ws=None, topk_ws=None, stream=None,
                                   win_pos=None, kw=None, win_ring=0, flags=0, rope_cs=None, rope_pos=None):
    """dsv4sa_topk into idx_c, then dsv4sa_sparse_attn_decode over it, as one call
    (one kernel when the decode runs as clusters over rows of <= 16384 entries)."""
    a = _attn_args(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale, lse, ws,
                   win_pos, kw, win_ring, flags, rope_cs, rope_pos)
    twp = _dev(topk_ws, "topk_ws", torch.uint8) if topk_ws is not None else None
    _check("dsv4sa_topk_sparse_attn_decode", lib().dsv4sa_topk_sparse_attn_decode(
        ctypes.byref(a), _dev(logits, "logits", torch.float32), logits.shape[-1], _dev(n_vis, "n_vis", torch.int32),
        n_max, k, twp, 0 if topk_ws is None else topk_ws.numel(), _stream(stream)))


def dsv4sa_sparse_attn_prefill(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale,
                               lse=None, ws=None, stream=None, win_pos=None, kw=None, win_ring=0, flags=0,
                               rope_cs=None, rope_pos=None):
    a = _attn_args(q, sink, q_seq, comp, comp_pt, idx_c, win, win_pt, idx_w, out, softmax_scale, lse, ws,
                   win_pos, kw, win_ring, flags, rope_cs, rope_pos)
    _check("dsv4sa_sparse_attn_prefill", lib().dsv4sa_sparse_attn_prefill(ctypes.byref(a), _stream(stream)))


# ---------------------------------------------------------------- drafted tokens

def _nodes(node_start, ctx, pos, anc, T, here):
    """Addresses of a batch of trees' lists: first nodes [B + 1], committed tokens [B], positions and ancestors [T]."""
    if ctx.numel() < node_start.numel() - 1:
        raise ValueError("ctx must have an entry for each sequence")
    if pos.numel() < T or (anc is not None and anc.numel() < T):
        raise ValueError(f"pos and anc must have an entry for each of the {T} nodes")
    return (_dev(node_start, "node_start", _int32, here), _dev(ctx, "ctx", _int32, here), _dev(pos, "pos", _int32, here),
            None if anc is None else _dev(anc, "anc", _int64, here))


def dsv4sa_tree_attn_workspace_size(n_seqs: int, max_nodes: int, H: int, n_max: int, window: int) -> int:
    return int(lib().dsv4sa_tree_attn_workspace_size(n_seqs, max_nodes, H, n_max, window))


def dsv4sa_tree_attn(q, sink, node_start, ctx, pos, comp, comp_pt, n_vis, n_max: int, win, win_pt, window: int, out,
                     softmax_scale, max_nodes: int, seq_row=None, anc=None, win_ring: int = 0, draft_entry: int = -1, lse=None,
                     ws=None, stream=None, rope_cs=None, rope_pos=None):
    """Attention of drafted tokens: q bf16 [T, H, 512], sequence b's being rows node_start[b] ..
    node_start[b + 1] - 1 (int32 [B + 1]), over compressed entries below n_vis [T], the window of
    committed tokens (positions below ctx [B]) and the drafted rows that the bits of anc (int64 [T];
    None: a chain) name, at draft_entry + j of the window pool (see dsv4sa.h).  Sequence b's pages are
    row seq_row[b] (None: b) of comp_pt and win_pt.  comp with n_max 0,
    and win with window 0 and no draft_entry, may be None.  rope_cs, rope_pos: as in the sparse attention."""
    T, H, dim = q.shape
    if dim != HEAD_DIM:
        raise ValueError("q must be [T, H, 512]")
    if out.shape != q.shape or sink.numel() < H or n_vis.numel() < T or (lse is not None and lse.numel() < T * H):
        raise ValueError(f"out, attn_sink, n_vis or lse does not fit {T} queries of {H} heads")
    here = _here()
    B = node_start.numel() - 1
    ns, cx, ps, an = _nodes(node_start, ctx, pos, anc, T, here)
    rows = None
    if seq_row is not None:
        if seq_row.numel() < B:
            raise ValueError("seq_row must have an entry for each sequence")
        rows = _dev(seq_row, "seq_row", _int32, here)
    cd = cpt = wd = wpt = rcs = rpos = None
    cpt_stride = wpt_stride = cpt_rows = wpt_rows = rope_rows = 0
    least = B if seq_row is None else min(B, 1)
    if comp is not None:
        cd = ctypes.pointer(_pool(comp, "comp", here))
        cpt, cpt_stride, cpt_rows = _page_table(comp_pt, "comp_pt", least if n_max > 0 else 0, here)
    if win is not None:
        wd = ctypes.pointer(_pool(win, "win", here))
        wpt, wpt_stride, wpt_rows = _page_table(win_pt, "win_pt", least if window > 0 or draft_entry >= 0 else 0, here)
    if rope_cs is not None:
        rcs = _table_of(rope_cs, 32, here)
        rpos = _dev(rope_pos, "rope_pos", _int32, here)
        if rope_pos.numel() < T:
            raise ValueError(f"rope_pos must have an entry for each of the {T} queries")
        rope_rows = rope_cs.shape[0]
    a = TreeArgs(_dev(q, "q", _bf16, here), T, H, float(softmax_scale), B, _dev(sink, "attn_sink", _f32, here), ns, rows, cx, ps, an,
                 _dev(n_vis, "n_vis", _int32, here), n_max, max_nodes, cd, cpt, wd, wpt, cpt_stride, wpt_stride, window, win_ring,
                 draft_entry, rope_rows, _dev(out, "out", _bf16, here), _dev(lse, "lse", _f32, here) if lse is not None else None,
                 rcs, rpos, _dev(ws, "ws", _u8, here) if ws is not None else None, ws.numel() if ws is not None else 0,
                 cpt_rows, wpt_rows)
    st = lib().dsv4sa_tree_attn(ctypes.byref(a), _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_tree_attn", st)


def dsv4sa_tree_window_indices(node_start, ctx, pos, window: int, ring: int, draft_entry: int, max_nodes: int, idx_w, anc=None,
                               stream=None):
    """The window list of each drafted token for the sparse attention: idx_w int32 [T, window +
    max_nodes] (committed positions, then drafted rows; -1: none), as dsv4sa_tree_attn sees them."""
    if idx_w.dim() != 2:
        raise ValueError("idx_w must be [T, window + max_nodes]")
    T = idx_w.shape[0]
    here = _here()
    ns, cx, ps, an = _nodes(node_start, ctx, pos, anc, T, here)
    st = lib().dsv4sa_tree_window_indices(ns, cx, ps, an, node_start.numel() - 1, T, max_nodes, window, ring, draft_entry,
                                          _dev(idx_w, "idx_w", _int32, here), idx_w.shape[1], _stream(stream, here))
    if st:
        raise DSV4SAError("dsv4sa_tree_window_indices", st)


def dsv4sa_check_errors(stream=None) -> tuple[int, int]:
    bits = ctypes.c_uint32(0)
    st = lib().dsv4sa_check_errors(_stream(stream), ctypes.byref(bits))
    return int(st), int(bits.value)


# ---------------------------------------------------------------- whole path (tests / bench)

@dataclass
class DeviceWorkload:
    """A workload resident on the GPU: pools, page tables, queries, outputs, workspaces."""
    w: object
    mode: int
    comp_buf: torch.Tensor
    comp: PoolDesc
    key_buf: torch.Tensor
    keys: PoolDesc
    win_buf: torch.Tensor
    win: PoolDesc
    comp_pt: torch.Tensor
    win_pt: torch.Tensor
    q: torch.Tensor
    q_idx: torch.Tensor
    q_idx_scale: torch.Tensor
    wts: torch.Tensor
    sink: torch.Tensor
    q_seq: torch.Tensor
    pos: torch.Tensor
    n_vis_idx: torch.Tensor      # indexer / top-k rows (-1: not routed through top-k)
    n_vis_c128: torch.Tensor     # rows taking every visible entry (0 otherwise)
    has_c128: bool
    logits: torch.Tensor
    idx_c: torch.Tensor
    idx_w: torch.Tensor
    out: torch.Tensor
    lse: torch.Tensor
    topk_ws: torch.Tensor | None
    attn_ws: torch.Tensor | None
    in_arena: torch.Tensor       # the STEP_INPUTS tensors are views of this buffer
    in_layout: list
    out_arena: torch.Tensor      # out and lse are views of this buffer
    out_layout: list


# indexer / top-k inputs first, then those only the attention reads (the graph
# step copies the second group while the indexer runs)
STEP_INPUTS = ("q_idx", "q_idx_scale", "wts", "q_seq", "n_vis_idx", "comp_pt", "q", "sink", "pos", "win_pt")
ATTN_ONLY_INPUTS = ("q", "sink", "pos", "win_pt")
STEP_OUTPUTS = ("out", "lse")


def _arena_layout(specs):
    """Byte offsets of tensors packed into one buffer, each 256-byte aligned; the
    buffer size is a multiple of 256 bytes (whole 16-byte units for the copy
    kernel)."""
    off, layout = 0, []
    for name, shape, dtype in specs:
        off = (off + 255) // 256 * 256
        nbytes = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        layout.append((name, off, nbytes, tuple(shape), dtype))
        off += nbytes
    return layout, max((off + 255) // 256 * 256, 256)


def _arena_views(buf, layout):
    return {name: buf[o:o + nb].view(dtype).view(shape) for name, o, nb, shape, dtype in layout}


def requantize_kv_pool_fp4(pool: PoolDesc, device="cuda", stream=None):
    """A KV pool's rows, all of them, as a KV_FP4 pool of as many pages -> (device byte
    tensor, PoolDesc): read back as BF16 and written again, 1024 pages at a time.  With a
    stream the work runs there, after the current stream's and before what follows on it."""
    pages = int(pool.num_pages)
    buf = _alloc_pool(POOL_KV_FP4, pages, device)
    desc = dsv4sa_pool_desc_init(POOL_KV_FP4, buf, pages)
    with _running_on(stream):
        table = torch.arange(pages, dtype=torch.int32, device=device).view(1, pages)
        for p0 in range(0, pages, 1024):
            entry = torch.arange(p0 * PAGE, min(pages, p0 + 1024) * PAGE, dtype=torch.int32, device=device)
            seq = torch.zeros_like(entry)
            rows = torch.empty(entry.shape[0], HEAD_DIM, dtype=torch.bfloat16, device=device)
            dsv4sa_cache_read(pool, table, seq, entry, rows)
            dsv4sa_cache_write(desc, table, seq, entry, rows)
    return buf, desc


def upload(w, device="cuda", mode=None, kv_fp4=False) -> DeviceWorkload:
    """Copy a workloads.Workload to the GPU in the library's formats; with kv_fp4 the
    KV pools are requantised into KV_FP4 pools."""
    dev = torch.device(device)
    if mode is None:
        mode = ATTN_PREFILL if w.T > 4 * w.B else ATTN_DECODE
    comp_buf, comp = pack_kv_pool(w.comp_pool["nope_codes"], w.comp_pool["nope_scale"], w.comp_pool["rope_bits"], dev)
    key_buf, keys = pack_key_pool(w.key_pool["codes"], w.key_pool["scale"], dev)
    win_buf, win = pack_kv_pool(w.win_pool["nope_codes"], w.win_pool["nope_scale"], w.win_pool["rope_bits"], dev)
    if kv_fp4:
        comp_buf, comp = requantize_kv_pool_fp4(comp, dev)
        win_buf, win = requantize_kv_pool_fp4(win, dev)

    def t(x, dt):
        return torch.from_numpy(np.ascontiguousarray(x)).to(dt).to(dev)

    c128 = np.asarray(w.c128, bool)
    n_max = max(1, int(w.n_max))
    logits_stride = (n_max + 3) // 4 * 4
    topk_ws_bytes = dsv4sa_topk_workspace_size(w.T, n_max, w.k)
    attn_ws_bytes = 0 if kv_fp4 else dsv4sa_attn_workspace_size(mode, w.T, w.H, w.kc, w.kw)
    # the per-step inputs and outputs each live in one buffer, so a step moves
    # them with one host-to-device and one device-to-host copy
    host = {
        "q": torch.from_numpy(np.ascontiguousarray(w.q).view(np.int16)).view(torch.bfloat16),
        "q_idx": torch.from_numpy(np.ascontiguousarray(w.q_idx, np.uint8)),
        "q_idx_scale": torch.from_numpy(np.ascontiguousarray(w.q_idx_scale, np.float32)),
        "wts": torch.from_numpy(np.ascontiguousarray(w.w, np.float32)),
        "sink": torch.from_numpy(np.ascontiguousarray(w.sink, np.float32)),
        "q_seq": torch.from_numpy(np.ascontiguousarray(w.q_seq, np.int32)),
        "pos": torch.from_numpy(np.ascontiguousarray(w.pos, np.int32)),
        "n_vis_idx": torch.from_numpy(np.where(c128, -1, w.n_vis).astype(np.int32)),
        "comp_pt": torch.from_numpy(np.ascontiguousarray(w.comp_pt, np.int32)),
        "win_pt": torch.from_numpy(np.ascontiguousarray(w.win_pt, np.int32)),
    }
    in_layout, in_bytes = _arena_layout([(n, host[n].shape, host[n].dtype) for n in STEP_INPUTS])
    in_arena = torch.empty(in_bytes, dtype=torch.uint8, device=dev)
    ins = _arena_views(in_arena, in_layout)
    for n in STEP_INPUTS:
        ins[n].copy_(host[n])
    out_layout, out_bytes = _arena_layout([("out", (w.T, w.H, HEAD_DIM), torch.bfloat16),
                                           ("lse", (w.T, w.H), torch.float32)])
    out_arena = torch.empty(out_bytes, dtype=torch.uint8, device=dev)
    outs = _arena_views(out_arena, out_layout)
    return DeviceWorkload(
        w=w, mode=mode, comp_buf=comp_buf, comp=comp, key_buf=key_buf, keys=keys, win_buf=win_buf, win=win,
        in_arena=in_arena, in_layout=in_layout, out_arena=out_arena, out_layout=out_layout,
        n_vis_c128=t(np.where(c128, w.n_vis, 0), torch.int32), has_c128=bool(c128.any()),
        logits=torch.empty((w.T, logits_stride), dtype=torch.float32, device=dev),
        idx_c=torch.empty((w.T, w.kc), dtype=torch.int32, device=dev),
        idx_w=torch.empty((w.T, w.kw), dtype=torch.int32, device=dev),
        topk_ws=torch.empty(topk_ws_bytes, dtype=torch.uint8, device=dev) if topk_ws_bytes else None,
        attn_ws=torch.empty(attn_ws_bytes, dtype=torch.uint8, device=dev) if attn_ws_bytes else None,
        **ins, **outs)


def run_path(d: DeviceWorkload, stream=None, fused_window=False, before_attention=None, out=None, lse=None,
             after_indexer=None, fused_topk=False):
    """One pass of the hot path on the GPU, every step in the library's kernels:
    index assembly -> indexer logits -> top-k -> sparse attention.  With
    fused_window the attention kernel computes the window indices from the
    positions itself (one launch fewer; d.idx_w is then not written)."""
    w = d.w
    n_max = max(1, int(w.n_max))
    if d.has_c128 or w.kc > w.k:
        dsv4sa_compress_indices(d.n_vis_c128, w.kc, d.idx_c, stream)
    if not fused_window:
        dsv4sa_window_indices(d.pos, w.kw, w.win_ring, d.idx_w, stream)
    dsv4sa_indexer_logits(d.keys, d.comp_pt, d.q_seq, d.n_vis_idx, d.q_idx, d.q_idx_scale, d.wts, n_max, d.logits,
                          stream)
    if after_indexer is not None:
        after_indexer()
    if fused_topk and d.mode != ATTN_PREFILL and w.kc == w.k:
        # the top-k and the decode attention as one call (fused_window: window indices from positions)
        if before_attention is not None:
            before_attention()
        dsv4sa_topk_sparse_attn_decode(
            d.logits, d.n_vis_idx, n_max, w.k, d.q, d.sink, d.q_seq, d.comp, d.comp_pt, d.idx_c, d.win, d.win_pt,
            None if fused_window else d.idx_w, d.out if out is None else out, w.softmax_scale,
            lse=d.lse if lse is None else lse, ws=d.attn_ws, topk_ws=d.topk_ws, stream=stream,
            win_pos=d.pos if fused_window else None, kw=w.kw if fused_window else None,
            win_ring=w.win_ring if fused_window else 0, flags=ATTN_EARLY_WINDOW if fused_window else 0)
        return
    if d.comp.kind == POOL_KV:
        # the top-k also prefetches the selected compressed rows into L2 for the attention
        dsv4sa_topk_prefetch(d.logits, d.n_vis_idx, n_max, w.k, d.idx_c, d.comp, d.comp_pt, d.q_seq, d.topk_ws, stream)
    else:
        dsv4sa_topk(d.logits, d.n_vis_idx, n_max, w.k, d.idx_c, d.topk_ws, stream)
    if before_attention is not None:
        before_attention()
    fn = dsv4sa_sparse_attn_prefill if d.mode == ATTN_PREFILL else dsv4sa_sparse_attn_decode
    if fused_window:
        # the kernels before it on the stream (indexer, top-k) write only logits and idx_c
        fn(d.q, d.sink, d.q_seq, d.comp, d.comp_pt, d.idx_c, d.win, d.win_pt, None,
           d.out if out is None else out, w.softmax_scale, lse=d.lse if lse is None else lse, ws=d.attn_ws,
           stream=stream, win_pos=d.pos, kw=w.kw, win_ring=w.win_ring, flags=ATTN_EARLY_WINDOW)
    else:
        fn(d.q, d.sink, d.q_seq, d.comp, d.comp_pt, d.idx_c, d.win, d.win_pt, d.idx_w, d.out, w.softmax_scale,
           lse=d.lse, ws=d.attn_ws, stream=stream)


class StepGraph:
    """One step of a serving loop as a single CUDA graph launch.

    The graph holds: two host-to-device copies of the step's packed inputs
    (`d.in_arena`) from a pinned host buffer of the same layout, made by the
    library's copy kernels (a copy-engine transfer node costs about 20 us of
    latency in the graph) -- the indexer's part first, the attention-only part
    (mostly q) on a side stream beside the indexer (dsv4sa_copy_async_background,
    one warp per SM) -- and the whole path (run_path, window indices
    derived in the attention kernel), whose attention kernel writes out and lse
    straight into a pinned host buffer over the host link.  `host_in[name]` / `host_out[name]` are views of
    those host buffers: the caller fills host_in, calls replay(), and
    synchronises `stream` before reading host_out.  The cache pools stay
    resident on the device; programmatic-dependent launches keep their overlap
    inside the graph."""

    def __init__(self, d: DeviceWorkload):
        self.d = d
        # byte offset where the attention-only inputs start in the packed layout
        self.split = min(o for n, o, _, _, _ in d.in_layout if n in ATTN_ONLY_INPUTS)
        self.side = torch.cuda.Stream(device=d.in_arena.device)
        self.host_in_arena = torch.empty_like(d.in_arena, device="cpu").pin_memory()
        self.host_out_arena = torch.empty_like(d.out_arena, device="cpu").pin_memory()
        self.host_in = _arena_views(self.host_in_arena, d.in_layout)
        self.host_out = _arena_views(self.host_out_arena, d.out_layout)
        self.host_in_arena.copy_(d.in_arena)
        self.stream = torch.cuda.Stream(device=d.in_arena.device)
        self.h2d_bytes = self.host_in_arena.numel()
        self.d2h_bytes = self.host_out_arena.numel()
        # one eager pass first: per-device set-up (kernel attributes, driver
        # entry points) happens outside the capture
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            self._body()
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self._body()
        self.stream.synchronize()

    def _body(self):
        # the indexer's inputs first; the attention-only inputs (mostly q) then
        # travel on a side stream, by one warp per SM beside the indexer (it
        # leaves a warp's worth of registers free on every SM), joined before
        # the attention
        dsv4sa_copy_async(self.d.in_arena[:self.split], self.host_in_arena[:self.split], self.stream)
        joined = torch.cuda.Event()
        ev = torch.cuda.Event()
        ev.record(self.stream)
        self.side.wait_event(ev)
        with torch.cuda.stream(self.side):
            dsv4sa_copy_async_background(self.d.in_arena[self.split:], self.host_in_arena[self.split:], self.side)
        joined.record(self.side)
        # the attention writes out and lse straight into the pinned host buffer
        run_path(self.d, self.stream, fused_window=True,
                 before_attention=lambda: self.stream.wait_event(joined),
                 out=self.host_out["out"], lse=self.host_out["lse"])

    def replay(self):
        """Launch the step on `stream` (the graph is launched on the current stream)."""
        with torch.cuda.stream(self.stream):
            self.graph.replay()


class NativeStep:
    """The same serving step as StepGraph, built and owned by the library
    (dsv4sa_step_create: a CUDA graph of the copy kernels and the three calls,
    captured in C++), launched by one C-ABI call with no torch graph in
    between.  host_in / host_out are views of pinned host buffers with the
    packed layouts of `d`; the caller fills host_in, calls launch() and
    synchronises `stream` before reading host_out."""

    def __init__(self, d: DeviceWorkload):
        w = d.w
        self.d = d
        self.split = min(o for n, o, _, _, _ in d.in_layout if n in ATTN_ONLY_INPUTS)
        self.host_in_arena = torch.empty_like(d.in_arena, device="cpu").pin_memory()
        self.host_out_arena = torch.empty_like(d.out_arena, device="cpu").pin_memory()
        self.host_in = _arena_views(self.host_in_arena, d.in_layout)
        self.host_out = _arena_views(self.host_out_arena, d.out_layout)
        self.host_in_arena.copy_(d.in_arena)
        self.stream = torch.cuda.Stream(device=d.in_arena.device)
        self.h2d_bytes = self.host_in_arena.numel()
        self.d2h_bytes = self.host_out_arena.numel()
        self.attn = _attn_args(d.q, d.sink, d.q_seq, d.comp, d.comp_pt, d.idx_c, d.win, d.win_pt, None,
                               self.host_out["out"], w.softmax_scale, self.host_out["lse"], d.attn_ws,
                               win_pos=d.pos, kw=w.kw, win_ring=w.win_ring, flags=ATTN_EARLY_WINDOW)
        n_max = max(1, int(w.n_max))
        sd = StepDesc()
        sd.host_in = self.host_in_arena.data_ptr()
        sd.dev_in = d.in_arena.data_ptr()
        sd.in_bytes = d.in_arena.numel()
        sd.in_split = self.split
        sd.kpool = ctypes.pointer(_pool(d.keys, "keys"))
        sd.page_table = _dev(d.comp_pt, "page_table", torch.int32)
        sd.pt_stride = d.comp_pt.shape[-1]
        sd.T = w.T
        sd.q_seq = _dev(d.q_seq, "q_seq", torch.int32)
        sd.n_vis = _dev(d.n_vis_idx, "n_vis", torch.int32)
        sd.q_fp8 = _dev(d.q_idx, "q_fp8", torch.uint8)
        sd.q_scale = _dev(d.q_idx_scale, "q_scale", torch.float32)
        sd.w = _dev(d.wts, "w", torch.float32)
        sd.Hi = d.q_idx.shape[1]
        sd.n_max = n_max
        sd.logits = _dev(d.logits, "logits", torch.float32)
        sd.logits_stride = d.logits.shape[-1]
        sd.k = w.k
        sd.idx_stride = d.idx_c.shape[-1]
        sd.idx = _dev(d.idx_c, "idx", torch.int32)
        sd.topk_ws = d.topk_ws.data_ptr() if d.topk_ws is not None else None
        sd.topk_ws_bytes = d.topk_ws.numel() if d.topk_ws is not None else 0
        sd.attn = ctypes.pointer(self.attn)
        self.desc = sd
        self.handle = ctypes.c_void_p()
        _check("dsv4sa_step_create", lib().dsv4sa_step_create(ctypes.byref(self.handle), ctypes.byref(sd),
                                                              ctypes.c_void_p(self.stream.cuda_stream)))

    def launch(self):
        _check("dsv4sa_step_launch", lib().dsv4sa_step_launch(self.handle, ctypes.c_void_p(self.stream.cuda_stream)))

    def close(self):
        if self.handle:
            self.stream.synchronize()
            lib().dsv4sa_step_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
