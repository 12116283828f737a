"""Python binding of libpagedattn (paged GQA attention for GB300).

Argument marshalling only: torch tensors become device pointers and sizes for the
C ABI in include/pagedattn.h; every step of the computation runs in the CUDA
kernels of libpagedattn.so.  There is no CPU or PyTorch fallback -- if the
library is not built, loading it raises.

Names follow the C ABI: pa_kv_append, pa_decode, pa_decode_splitkv,
pa_combine, pa_prefill_chunked, pa_device_status; on an 8-bit pool (PaPool8) pa_kv_append8,
pa_decode8, pa_prefill_chunked8; pa_decode_weights / pa_decode8_weights and pa_kv_evict for
eviction by accumulated attention weight.  Tensors must be CUDA,
contiguous, and of the dtypes the header states (bf16 data, int32 tables,
int64 slot mapping, fp32 split-KV workspace).  Calls are asynchronous on the
given stream (default: torch's current stream).  For a step of full and linear attention: pa_prefill_packed
(cold prompts, rows strided as a fused projection leaves them), pa_kv_grow and pa_kv_free (tables,
lengths and slots built on the GPU from a free list) and pa_linear_decode / pa_linear_prefill
(linear attention with a fixed decay for each head).
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path
from typing import Optional, Tuple

import torch

__all__ = ["PaPool", "PaPool8", "pa_kv_append8", "pa_decode8", "pa_prefill_chunked8", "pa_decode_weights",
           "pa_decode8_weights", "pa_weights_workspace_bytes", "pa_kv_evict", "pa_kv_append", "pa_kv_copy", "pa_decode", "pa_append_decode", "pa_decode_splitkv",
           "pa_combine", "pa_prefill_chunked",
           "pa_device_status", "pa_selftest_wait_timeout", "pa_selftest_packed_pairs", "pa_splitkv_workspace_bytes", "pa_decode_num_splits", "pa_splitkv_num_partitions",
           "pa_decode_splitkv_noalloc", "pa_noalloc_scratch_bytes", "PagedAttnError",
           "pa_prefill_packed", "pa_kv_grow", "pa_kv_free", "pa_linear_decode", "pa_linear_prefill",
           "pa_linear_workspace_bytes", "BlockManager", "pa_kv_block_bytes", "pa_kv_budget_blocks",
           "library", "library_path", "BLOCK_SIZE", "EXPORTED_SYMBOLS"]

BLOCK_SIZE = 16
PKG = Path(__file__).resolve().parent
_LIB_PATH = PKG / "libpagedattn.so"
EXPORTED_SYMBOLS = ("pa_kv_append8", "pa_decode8", "pa_prefill_chunked8", "pa_decode_weights", "pa_decode8_weights",
                    "pa_weights_workspace_bytes", "pa_kv_evict", "pa_bm_evict", "pa_kv_append", "pa_kv_copy", "pa_decode", "pa_append_decode", "pa_splitkv_workspace_bytes",
                    "pa_decode_splitkv", "pa_combine",
                    "pa_prefill_chunked", "pa_device_status", "pa_decode_num_splits", "pa_splitkv_num_partitions",
                    "pa_status_str", "pa_version", "pa_decode_splitkv_noalloc", "pa_noalloc_scratch_bytes",
                    "pa_selftest_wait_timeout", "pa_selftest_packed_pairs", "pa_prefill_packed", "pa_kv_grow", "pa_kv_free", "pa_linear_decode",
                    "pa_linear_prefill", "pa_linear_workspace_bytes",
                    "pa_kv_block_bytes", "pa_kv_budget_blocks", "pa_bm_create", "pa_bm_destroy", "pa_bm_admit", "pa_bm_admit_cow",
                    "pa_bm_commit", "pa_bm_release", "pa_bm_slots", "pa_bm_stats")

PA_OK = 0
PA_ERR_INVALID_ARG = -1
PA_ERR_REJECTED = -7
PA_ERR_UNSUPPORTED = -2
PA_ERR_CUDA = -3
PA_ERR_OUT_OF_RANGE = -4
PA_ERR_TIMEOUT = -5
PA_ERR_TOO_LARGE = -6
PA_ERR_NO_MEMORY = -8
PA_DEV_OUT_OF_RANGE = 1
PA_DEV_TIMEOUT = 2


class PagedAttnError(RuntimeError):
    def __init__(self, what: str, code: int):
        super().__init__(f"{what} failed: {_status_str(code)} ({code})")
        self.code = code


class _PaPoolC(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class _PaPool8C(ctypes.Structure):
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("exps", ctypes.c_void_p),
                ("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


_lib: Optional[ctypes.CDLL] = None


def library_path() -> Path:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """Load libpagedattn.so (built by paged_kv_gqa_slot_gb300.build); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not _LIB_PATH.exists():
        raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m paged_kv_gqa_slot_gb300.build` "
                           "(or __graft_entry__.build()) first -- there is no fallback path")
    lib = ctypes.CDLL(str(_LIB_PATH))
    P, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    I64 = ctypes.c_int64
    pool = ctypes.POINTER(_PaPoolC)
    pool8 = ctypes.POINTER(_PaPool8C)
    weights_args = [P, P, I32, P, I32, I32, F32, F32, P, P, P, P]
    sig = {
        "pa_kv_append8": (ctypes.c_int, [pool8, P, P, P, I32, P]),
        "pa_decode8": (ctypes.c_int, [pool8, P, P, I32, P, I32, I32, F32, P, P]),
        "pa_prefill_chunked8": (ctypes.c_int, [pool8, P, P, P, I32, P, I32, I32, I32, F32, P, P]),
        "pa_decode_weights": (ctypes.c_int, [pool, *weights_args]),
        "pa_decode8_weights": (ctypes.c_int, [pool8, *weights_args]),
        "pa_weights_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "pa_kv_evict": (ctypes.c_int, [P, P, P, I32, I32, I32, I32, I32, I32, P, P, P, P, P, P]),
        "pa_bm_evict": (ctypes.c_int, [P, ctypes.c_int64, P, I32]),
        "pa_prefill_packed": (ctypes.c_int, [P, P, P, P, I32, I32, I32, I32, I32, I64, I64, I64, I32, F32, P, P]),
        "pa_selftest_packed_pairs": (ctypes.c_int, [P, I32, I32, I32, I32, P, I32, P, P]),
        "pa_kv_grow": (ctypes.c_int, [P, I32, P, P, I32, P, I32, P, I32, P, P, P, P, P, P, P]),
        "pa_kv_free": (ctypes.c_int, [P, P, I32, I32, P, I32, P, P, P]),
        "pa_linear_decode": (ctypes.c_int, [P, I32, P, P, P, P, P, P, I32, I32, I32, I32, I64, I64, I64, F32, P, P]),
        "pa_linear_prefill": (ctypes.c_int, [P, I32, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, I64, I64, I64, I32,
                                             F32, P, P, P]),
        "pa_linear_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "pa_kv_append": (ctypes.c_int, [pool, P, P, P, I32, P]),
        "pa_kv_copy": (ctypes.c_int, [pool, P, P, I32, P]),
        "pa_decode": (ctypes.c_int, [pool, P, P, I32, P, I32, I32, F32, P, P]),
        "pa_append_decode": (ctypes.c_int, [pool, P, P, P, P, P, I32, P, I32, I32, F32, P, P]),
        "pa_splitkv_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "pa_decode_splitkv": (ctypes.c_int, [pool, P, P, I32, P, I32, I32, F32, I32, P, P, P]),
        "pa_combine": (ctypes.c_int, [P, P, I32, I32, I32, I32, P, P]),
        "pa_prefill_chunked": (ctypes.c_int, [pool, P, P, P, I32, P, I32, I32, I32, F32, P, P]),
        "pa_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), I32, P]),
        "pa_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint64, P]),
        "pa_decode_num_splits": (ctypes.c_int, [I32, I32, I32]),
        "pa_splitkv_num_partitions": (ctypes.c_int, [I32, I32, I32]),
        "pa_decode_splitkv_noalloc": (ctypes.c_int, [pool, P, P, I32, P, I32, I32, F32, I32, P, P]),
        "pa_noalloc_scratch_bytes": (SZ, []),
        "pa_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "pa_kv_block_bytes": (ctypes.c_int64, [I32, I32, I32, I32, I32]),
        "pa_kv_budget_blocks": (I32, [ctypes.c_int64, I32, I32, I32, I32, I32]),
        "pa_bm_create": (P, [I32, I32, I32]),
        "pa_bm_destroy": (None, [P]),
        "pa_bm_admit": (ctypes.c_int, [P, ctypes.c_int64, P, I32, I32, P, I32, P, P]),
        "pa_bm_admit_cow": (ctypes.c_int, [P, ctypes.c_int64, P, I32, I32, P, I32, P, P, P, P, P]),
        "pa_bm_commit": (ctypes.c_int, [P, ctypes.c_int64, P, I32, I32]),
        "pa_bm_release": (ctypes.c_int, [P, ctypes.c_int64]),
        "pa_bm_slots": (ctypes.c_int, [P, ctypes.c_int64, I32, I32, P]),
        "pa_bm_stats": (ctypes.c_int, [P, P, P, P]),
        "pa_version": (ctypes.c_int, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _status_str(code: int) -> str:
    try:
        return library().pa_status_str(code).decode()
    except Exception:  # pragma: no cover - used while raising
        return str(code)


def _check(code: int, what: str) -> None:
    if code != PA_OK:
        raise PagedAttnError(what, code)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    return t.data_ptr()


def _tables(block_tables: torch.Tensor, seq_lens: torch.Tensor, batch: int) -> None:
    """The kernels read block_tables[b] and seq_lens[b] for every b < batch."""
    if block_tables.dim() != 2 or block_tables.shape[0] != batch or seq_lens.numel() != batch:
        raise ValueError(f"block_tables [batch, max_blocks] and seq_lens [batch] must match batch {batch}, got "
                         f"{tuple(block_tables.shape)} and {tuple(seq_lens.shape)}")


def _rows(k_new: torch.Tensor, v_new: torch.Tensor, pool: "PaPool", n: int) -> None:
    """The append kernels read n rows of [num_kv_heads, head_dim] from k_new and v_new."""
    shape = (n, pool.num_kv_heads, pool.head_dim)
    if tuple(k_new.shape) != shape or tuple(v_new.shape) != shape:
        raise ValueError(f"k_new / v_new: need shape {shape}, got {tuple(k_new.shape)} / {tuple(v_new.shape)}")


def _out(out: Optional[torch.Tensor], shape, like: torch.Tensor) -> torch.Tensor:
    """The caller's output tensor, checked to be exactly `shape` (the kernels write all of it),
    or a new one."""
    if out is None:
        return torch.empty(tuple(shape), dtype=torch.bfloat16, device=like.device)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out: need shape {tuple(shape)}, got {tuple(out.shape)}")
    return out


class PaPool:
    """The paged KV pool: k_cache, v_cache = [num_blocks, num_kv_heads, 16, head_dim] bf16 on the GPU."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor):
        if k_cache.shape != v_cache.shape or k_cache.dim() != 4:
            raise ValueError("k_cache and v_cache must both be [num_blocks, num_kv_heads, block_size, head_dim]")
        self.k_cache, self.v_cache = k_cache, v_cache
        nb, hkv, bs, d = k_cache.shape
        self.c = _PaPoolC(_dev(k_cache, torch.bfloat16, "k_cache"), _dev(v_cache, torch.bfloat16, "v_cache"),
                          nb, bs, hkv, d)
        self.ref = ctypes.byref(self.c)

    @property
    def num_kv_heads(self) -> int:
        return self.c.num_kv_heads

    @property
    def head_dim(self) -> int:
        return self.c.head_dim


def pa_kv_append(pool: PaPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                 stream=None) -> None:
    T = int(slot_mapping.numel())
    _rows(k_new, v_new, pool, T)
    rc = library().pa_kv_append(pool.ref, _dev(k_new, torch.bfloat16, "k_new") if T else None,
                                _dev(v_new, torch.bfloat16, "v_new") if T else None,
                                _dev(slot_mapping, torch.int64, "slot_mapping") if T else None, T, _stream(stream))
    _check(rc, "pa_kv_append")


def pa_kv_copy(pool: PaPool, src_slots: torch.Tensor, dst_slots: torch.Tensor, stream=None) -> None:
    """Copy pool rows src_slots[t] -> dst_slots[t] (K and V, every kv head)."""
    n = int(src_slots.numel())
    if dst_slots.numel() != n:
        raise ValueError(f"src_slots / dst_slots: need equal lengths, got {n} / {dst_slots.numel()}")
    rc = library().pa_kv_copy(pool.ref, _dev(src_slots, torch.int64, "src_slots") if n else None,
                              _dev(dst_slots, torch.int64, "dst_slots") if n else None, n, _stream(stream))
    _check(rc, "pa_kv_copy")


def pa_decode(pool: PaPool, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    B, Hq, _ = q.shape
    _tables(block_tables, seq_lens, B)
    out = _out(out, q.shape, q)
    rc = library().pa_decode(pool.ref, _dev(q, torch.bfloat16, "q"), _dev(block_tables, torch.int32, "block_tables"),
                             block_tables.shape[1], _dev(seq_lens, torch.int32, "seq_lens"), B, Hq, float(scale),
                             _dev(out, torch.bfloat16, "out"), _stream(stream))
    _check(rc, "pa_decode")
    return out


def pa_append_decode(pool: PaPool, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                     q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_kv_append of one new row per sequence followed by pa_decode, in one launch."""
    B, Hq, _ = q.shape
    _tables(block_tables, seq_lens, B)
    _rows(k_new, v_new, pool, B)
    if slot_mapping.numel() != B:
        raise ValueError(f"slot_mapping: need {B} entries, got {slot_mapping.numel()}")
    out = _out(out, q.shape, q)
    rc = library().pa_append_decode(pool.ref, _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"),
                                    _dev(slot_mapping, torch.int64, "slot_mapping"), _dev(q, torch.bfloat16, "q"),
                                    _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                    _dev(seq_lens, torch.int32, "seq_lens"), B, Hq, float(scale),
                                    _dev(out, torch.bfloat16, "out"), _stream(stream))
    _check(rc, "pa_append_decode")
    return out


def pa_splitkv_workspace_bytes(batch: int, num_heads: int, head_dim: int, num_partitions: int) -> int:
    return int(library().pa_splitkv_workspace_bytes(batch, num_heads, head_dim, num_partitions))


def pa_decode_splitkv(pool: PaPool, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float, num_partitions: int, ws_o: Optional[torch.Tensor] = None,
                      ws_lse: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    B, Hq, D = q.shape
    _tables(block_tables, seq_lens, B)
    P = int(num_partitions)
    if ws_o is None:
        ws_o = torch.empty((B, Hq, P, D), dtype=torch.float32, device=q.device)
    if ws_lse is None:
        ws_lse = torch.empty((B, Hq, P), dtype=torch.float32, device=q.device)
    if tuple(ws_o.shape) != (B, Hq, P, D) or tuple(ws_lse.shape) != (B, Hq, P):
        raise ValueError(f"ws_o / ws_lse: need shapes {(B, Hq, P, D)} / {(B, Hq, P)}, "
                         f"got {tuple(ws_o.shape)} / {tuple(ws_lse.shape)}")
    rc = library().pa_decode_splitkv(pool.ref, _dev(q, torch.bfloat16, "q"),
                                     _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                     _dev(seq_lens, torch.int32, "seq_lens"), B, Hq, float(scale), P,
                                     _dev(ws_o, torch.float32, "ws_o"), _dev(ws_lse, torch.float32, "ws_lse"),
                                     _stream(stream))
    _check(rc, "pa_decode_splitkv")
    return ws_o, ws_lse


def pa_decode_splitkv_noalloc(pool: PaPool, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                              scale: float, num_partitions: int, out: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """Split-KV decode + merge with no workspace argument: for callers that cannot allocate
    device memory (see include/pagedattn.h).  Pass a preallocated `out` to allocate nothing
    at all; its partition results live in a static array inside the library."""
    B, Hq, _ = q.shape
    _tables(block_tables, seq_lens, B)
    out = _out(out, q.shape, q)
    rc = library().pa_decode_splitkv_noalloc(pool.ref, _dev(q, torch.bfloat16, "q"),
                                             _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                             _dev(seq_lens, torch.int32, "seq_lens"), B, Hq, float(scale),
                                             int(num_partitions), _dev(out, torch.bfloat16, "out"), _stream(stream))
    _check(rc, "pa_decode_splitkv_noalloc")
    return out


def pa_noalloc_scratch_bytes() -> int:
    return int(library().pa_noalloc_scratch_bytes())


def pa_combine(ws_o: torch.Tensor, ws_lse: torch.Tensor, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    B, Hq, P, D = ws_o.shape
    if tuple(ws_lse.shape) != (B, Hq, P):
        raise ValueError(f"ws_lse: need shape {(B, Hq, P)}, got {tuple(ws_lse.shape)}")
    out = _out(out, (B, Hq, D), ws_o)
    rc = library().pa_combine(_dev(ws_o, torch.float32, "ws_o"), _dev(ws_lse, torch.float32, "ws_lse"), B, Hq, D, P,
                              _dev(out, torch.bfloat16, "out"), _stream(stream))
    _check(rc, "pa_combine")
    return out


def pa_prefill_chunked(pool: PaPool, q: torch.Tensor, cu_q_lens: torch.Tensor, block_tables: torch.Tensor,
                       seq_lens: torch.Tensor, scale: float, max_chunk: int, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    _, Hq, _ = q.shape
    B = int(seq_lens.numel())
    _tables(block_tables, seq_lens, B)
    if cu_q_lens.numel() != B + 1:
        raise ValueError(f"cu_q_lens: need {B + 1} entries, got {cu_q_lens.numel()}")
    out = _out(out, q.shape, q)
    rc = library().pa_prefill_chunked(pool.ref, _dev(q, torch.bfloat16, "q"), _dev(cu_q_lens, torch.int32, "cu_q_lens"),
                                      _dev(block_tables, torch.int32, "block_tables"), block_tables.shape[1],
                                      _dev(seq_lens, torch.int32, "seq_lens"), B, Hq, int(max_chunk), float(scale),
                                      _dev(out, torch.bfloat16, "out"), _stream(stream))
    _check(rc, "pa_prefill_chunked")
    return out


# ----------------------------------------------------------------------------- 8-bit pool, weights, eviction
# (looked up once: a call's own arithmetic is a few microseconds, and so is what Python adds to it)
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_empty_like = torch.empty_like
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _arg(t: torch.Tensor, dtype, name: str, device: int) -> int:
    """Address of a contiguous CUDA tensor of `dtype` on the call's device."""
    if t.dtype is dtype and t.get_device() == device and t.is_contiguous() and device >= 0:
        return t.data_ptr()
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    raise ValueError(f"{name}: on cuda:{t.get_device()}, the call's other tensors are on cuda:{device}")


def _like(t: torch.Tensor, stream) -> torch.Tensor:
    """A result tensor of t's shape, type and device, allocated for the stream that writes it."""
    if stream is None:
        return torch.empty_like(t)
    with _on(stream, t.device):
        return torch.empty_like(t)


def _on(stream, device):
    """The given stream (an object or a raw handle) as the current one, for allocations."""
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def _width(block_tables: torch.Tensor, seq_lens: torch.Tensor, batch: int) -> int:
    """The tables' width, once they and the lengths are known to match the batch."""
    shape = block_tables.shape
    if len(shape) != 2 or shape[0] != batch or seq_lens.numel() != batch:
        _tables(block_tables, seq_lens, batch)
    return shape[1]


def _call(what: str, device: int, stream, *args) -> None:
    """The library's call on `device` (its current stream unless one is given)."""
    fn = getattr(_lib or library(), what)
    if stream is None:
        raw = _raw_stream(device)
    else:
        raw = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if _current_device() == device:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc != PA_OK:
        raise PagedAttnError(what, rc)


class PaPool8:
    """The 8-bit paged KV pool: k_cache, v_cache = [num_blocks, num_kv_heads, 16, head_dim] e4m3 codes
    (torch.uint8 or torch.float8_e4m3fn), exps = [num_blocks, num_kv_heads, 2] uint8, all on one GPU:
    K = code * 2^(exps[..., 0] - 127), V = code * 2^(exps[..., 1] - 127)."""

    def __init__(self, k_cache: torch.Tensor, v_cache: torch.Tensor, exps: torch.Tensor):
        if k_cache.shape != v_cache.shape or k_cache.dim() != 4 or k_cache.dtype != v_cache.dtype:
            raise ValueError("k_cache and v_cache must both be [num_blocks, num_kv_heads, block_size, head_dim]")
        if k_cache.dtype not in (torch.uint8, torch.float8_e4m3fn):
            raise ValueError(f"k_cache and v_cache: need uint8 or float8_e4m3fn codes, got {k_cache.dtype}")
        nb, hkv, bs, d = k_cache.shape
        if tuple(exps.shape) != (nb, hkv, 2):
            raise ValueError(f"exps: need shape {(nb, hkv, 2)}, got {tuple(exps.shape)}")
        self.k_cache, self.v_cache, self.exps = k_cache, v_cache, exps
        self.device = k_cache.get_device()
        self.c = _PaPool8C(_arg(k_cache, k_cache.dtype, "k_cache", self.device),
                           _arg(v_cache, k_cache.dtype, "v_cache", self.device),
                           _arg(exps, torch.uint8, "exps", self.device), nb, bs, hkv, d)
        self.ref = ctypes.byref(self.c)
        self.num_kv_heads, self.head_dim = hkv, d

    @classmethod
    def zeros(cls, num_blocks: int, num_kv_heads: int, head_dim: int, device="cuda") -> "PaPool8":
        shape = (num_blocks, num_kv_heads, BLOCK_SIZE, head_dim)
        return cls(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros((num_blocks, num_kv_heads, 2), dtype=torch.uint8, device=device))


def pa_kv_append8(pool: PaPool8, k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                  stream=None) -> None:
    """Quantise new bf16 rows into the pool; the rows of one block are consecutive entries."""
    T = slot_mapping.numel()
    _rows(k_new, v_new, pool, T)
    if T == 0:
        return
    d = pool.device
    _call("pa_kv_append8", d, stream, pool.ref, _arg(k_new, _BF16, "k_new", d),
          _arg(v_new, _BF16, "v_new", d), _arg(slot_mapping, _I64, "slot_mapping", d), T)


def _query(pool, q: torch.Tensor, out: Optional[torch.Tensor], stream) -> torch.Tensor:
    """Check q against the pool; the output tensor (the caller's, checked, or a new one)."""
    shape = q.shape
    if len(shape) != 3 or shape[2] != pool.head_dim:
        raise ValueError(f"q: need [rows, num_heads, {pool.head_dim}], got {tuple(shape)}")
    if out is None:
        return _empty_like(q) if stream is None else _like(q, stream)
    if out.shape != shape:
        raise ValueError(f"out: need shape {tuple(shape)}, got {tuple(out.shape)}")
    return out


def pa_decode8(pool: PaPool8, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
               out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    d = pool.device
    out = _query(pool, q, out, stream)
    B, heads, _ = q.shape
    width = _width(block_tables, seq_lens, B)
    _call("pa_decode8", d, stream, pool.ref, _arg(q, _BF16, "q", d), _arg(block_tables, _I32, "block_tables", d), width,
          _arg(seq_lens, _I32, "seq_lens", d), B, heads, float(scale),
          _arg(out, _BF16, "out", d))
    return out


def pa_prefill_chunked8(pool: PaPool8, q: torch.Tensor, cu_q_lens: torch.Tensor, block_tables: torch.Tensor,
                        seq_lens: torch.Tensor, scale: float, max_chunk: int, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    d = pool.device
    out = _query(pool, q, out, stream)
    B = seq_lens.numel()
    width = _width(block_tables, seq_lens, B)
    if cu_q_lens.numel() != B + 1:
        raise ValueError(f"cu_q_lens: need {B + 1} entries, got {cu_q_lens.numel()}")
    _call("pa_prefill_chunked8", d, stream, pool.ref, _arg(q, _BF16, "q", d),
          _arg(cu_q_lens, _I32, "cu_q_lens", d), _arg(block_tables, _I32, "block_tables", d),
          width, _arg(seq_lens, _I32, "seq_lens", d), B, q.shape[1], int(max_chunk),
          float(scale), _arg(out, _BF16, "out", d))
    return out


def pa_weights_workspace_bytes(batch: int, num_heads: int, num_kv_heads: int, max_blocks: int) -> int:
    return int(library().pa_weights_workspace_bytes(batch, num_heads, num_kv_heads, max_blocks))


def _decode_weights(what, pool, device, q, block_tables, seq_lens, scale, weights, decay, workspace, out, stream):
    out = _query(pool, q, out, stream)
    B, Hq, _ = q.shape
    width = _width(block_tables, seq_lens, B)
    if weights.shape != (B, pool.num_kv_heads, width):
        raise ValueError(f"weights: need shape {(B, pool.num_kv_heads, width)}, got {tuple(weights.shape)}")
    if B == 0:
        return out
    need = B * pool.num_kv_heads * width * (16 if Hq // pool.num_kv_heads > 8 else 8)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.float32, device=weights.device) if stream is None else \
            _like(weights.expand(need // max(weights.numel(), 1), *weights.shape), stream)
    elif workspace.numel() < need:
        raise ValueError(f"workspace: need {need} floats, got {workspace.numel()}")
    _call(what, device, stream, pool.ref, _arg(q, _BF16, "q", device),
          _arg(block_tables, _I32, "block_tables", device), width,
          _arg(seq_lens, _I32, "seq_lens", device), B, Hq, float(scale), float(decay),
          _arg(weights, _F32, "weights", device), _arg(workspace, _F32, "workspace", device),
          _arg(out, _BF16, "out", device))
    return out


def pa_decode_weights(pool: PaPool, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float, weights: torch.Tensor, decay: float = 1.0,
                      workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """pa_decode that also does weights[b, kvh, j] = decay * weights[b, kvh, j] + the attention weight
    that logical block j got from the query heads of kv head kvh (fp32, in place)."""
    return _decode_weights("pa_decode_weights", pool, pool.k_cache.get_device(), q, block_tables, seq_lens, scale,
                           weights, decay, workspace, out, stream)


def pa_decode8_weights(pool: PaPool8, q: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor,
                       scale: float, weights: torch.Tensor, decay: float = 1.0,
                       workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """pa_decode8 with the accumulated block weights of pa_decode_weights."""
    return _decode_weights("pa_decode8_weights", pool, pool.device, q, block_tables, seq_lens, scale, weights, decay,
                           workspace, out, stream)


def pa_kv_evict(block_tables: torch.Tensor, seq_lens: torch.Tensor, weights: torch.Tensor, keep_blocks: int,
                sink_blocks: int = 1, recent_blocks: int = 1, in_place: bool = False, stream=None):
    """Evict each sequence's blocks past `keep_blocks` with the lowest accumulated weight, but none of
    the first sink_blocks and last recent_blocks.  Returns (block_tables, seq_lens, weights, evicted,
    num_evicted): new tensors, or with in_place the given ones updated; evicted [batch, max_blocks]
    lists the ids that left (-1 behind them) for BlockManager.evict."""
    if weights.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("need block_tables [batch, max_blocks] and weights [batch, num_kv_heads, max_blocks]")
    B, hkv, width = weights.shape
    if block_tables.shape != (B, width) or seq_lens.shape != (B,):
        raise ValueError(f"block_tables / seq_lens: need shapes {(B, width)} / {(B,)}, got "
                         f"{tuple(block_tables.shape)} / {tuple(seq_lens.shape)}")
    d = weights.get_device()
    like = _empty_like if stream is None else lambda t: _like(t, stream)
    if in_place:
        new_tables, new_lens, new_weights = block_tables, seq_lens, weights
    else:
        new_tables, new_lens, new_weights = like(block_tables), like(seq_lens), like(weights)
    evicted, num = like(block_tables), like(seq_lens)
    _call("pa_kv_evict", d, stream, _arg(block_tables, _I32, "block_tables", d),
          _arg(seq_lens, _I32, "seq_lens", d), _arg(weights, _F32, "weights", d), B, width, hkv,
          int(keep_blocks), int(sink_blocks), int(recent_blocks), new_tables.data_ptr(), new_lens.data_ptr(),
          new_weights.data_ptr(), evicted.data_ptr(), num.data_ptr())
    return new_tables, new_lens, new_weights, evicted, num


# ----------------------------------------------------------------------------- a step of full and linear attention
def _strided(t: torch.Tensor, heads: int, dim: int, name: str, device: int) -> Tuple[int, int]:
    """Address and row stride of bf16 rows [heads, dim] on the call's device: each row contiguous, the
    rows any multiple of 8 elements apart (a view of a fused projection)."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: need [rows, {heads}, {dim}], got {tuple(shape)}")
    if t.dtype is not _BF16 or t.get_device() != device or device < 0:
        if t.dtype is not _BF16 or not t.is_cuda:
            raise ValueError(f"{name}: need a CUDA {_BF16} tensor, got {t.dtype} on {t.device}")
        raise ValueError(f"{name}: on cuda:{t.get_device()}, the call's other tensors are on cuda:{device}")
    row, head, one = t.stride()
    if shape[0] <= 1:
        row = heads * dim
    if one != 1 or (head != dim and heads > 1) or row < heads * dim or row % 8:
        raise ValueError(f"{name}: need rows of {heads} x {dim} contiguous elements, a multiple of 8 apart, got strides "
                         f"{t.stride()}")
    return t.data_ptr(), row


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A result tensor on `like`'s device, allocated for the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _on(stream, like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _most(n) -> int:
    """An upper bound as int32: larger ones mean the same as the largest (and negative ones are refused as such)."""
    return max(-1, min(int(n), 0x7fffffff))


def _packed(q, k, v, out, stream):
    """Check the rows of a packed call; (device, rows, heads, kv heads, dim, addresses, strides, out)."""
    shape, kshape = q.shape, k.shape
    if len(shape) != 3 or len(kshape) != 3:
        raise ValueError(f"q / k: need [rows, heads, head_dim], got {tuple(shape)} / {tuple(kshape)}")
    rows, heads, dim = shape
    kvh, d = kshape[1], q.get_device()
    if kshape[0] != rows or v.shape[0] != rows:
        raise ValueError(f"q, k, v: need equal row counts, got {rows}, {kshape[0]}, {v.shape[0]}")
    qp, qs = _strided(q, heads, dim, "q", d)
    kp, ks = _strided(k, kvh, dim, "k", d)
    vp, vs = _strided(v, kvh, dim, "v", d)
    if out is None:
        out = _new(q, shape, _BF16, stream)
    elif out.shape != shape:
        raise ValueError(f"out: need shape {tuple(shape)}, got {tuple(out.shape)}")
    return d, rows, heads, kvh, dim, (qp, kp, vp), (qs, ks, vs), out


def pa_prefill_packed(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_lens: torch.Tensor, scale: float,
                      max_len: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention over packed prompts: rows cu_lens[b] .. cu_lens[b+1] of q [rows, num_heads, head_dim],
    k and v [rows, num_kv_heads, head_dim] are sequence b.  Rows may be strided views."""
    d, rows, heads, kvh, dim, p, s, out = _packed(q, k, v, out, stream)
    _call("pa_prefill_packed", d, stream, *p, _arg(cu_lens, _I32, "cu_lens", d), cu_lens.numel() - 1, rows, heads, kvh,
          dim, *s, _most(max_len), float(scale), _arg(out, _BF16, "out", d))
    return out


def pa_kv_grow(block_tables: torch.Tensor, seq_lens: torch.Tensor, new_lens: torch.Tensor, free_blocks: torch.Tensor,
               num_free: torch.Tensor, max_tokens: int, in_place: bool = False, stream=None):
    """Give every sequence its new_lens tokens while the free list and max_tokens last.  block_tables is
    updated in place, and seq_lens and num_free [1] with in_place.  Returns (block_tables, seq_lens, num_free,
    cu_lens, slot_mapping, positions, token_seqs)."""
    if block_tables.dim() != 2:
        raise ValueError(f"block_tables: need [batch, max_blocks], got {tuple(block_tables.shape)}")
    B, width = block_tables.shape
    if seq_lens.shape != (B,) or new_lens.shape != (B,) or num_free.numel() != 1:
        raise ValueError(f"seq_lens / new_lens / num_free: need shapes {(B,)} / {(B,)} / (1,), got "
                         f"{tuple(seq_lens.shape)} / {tuple(new_lens.shape)} / {tuple(num_free.shape)}")
    d, rows = block_tables.get_device(), int(max_tokens)
    if rows < 0:
        raise ValueError(f"max_tokens: need 0 or more, got {rows}")
    lens = seq_lens if in_place else _like(seq_lens, stream)
    left = num_free if in_place else _like(num_free, stream)
    cu = _new(block_tables, (B + 1,), _I32, stream)
    slots = _new(block_tables, (rows,), _I64, stream)
    positions = _new(block_tables, (rows,), _I32, stream)
    token_seqs = _new(block_tables, (rows,), _I32, stream)
    _call("pa_kv_grow", d, stream, _arg(block_tables, _I32, "block_tables", d), width, _arg(seq_lens, _I32, "seq_lens", d),
          _arg(new_lens, _I32, "new_lens", d), B, _arg(free_blocks, _I32, "free_blocks", d), free_blocks.numel(),
          _arg(num_free, _I32, "num_free", d), rows, lens.data_ptr(), left.data_ptr(), cu.data_ptr(),
          slots.data_ptr(), positions.data_ptr(), token_seqs.data_ptr())
    return block_tables, lens, left, cu, slots, positions, token_seqs


def pa_kv_free(ids: torch.Tensor, counts: torch.Tensor, free_blocks: torch.Tensor, num_free: torch.Tensor,
               in_place: bool = False, stream=None) -> torch.Tensor:
    """Push the blocks ids[r, :counts[r]] (negative entries do not count) onto the free list, which is updated
    in place; returns num_free [1] after that (num_free itself with in_place)."""
    if ids.dim() != 2 or counts.shape != (ids.shape[0],) or num_free.numel() != 1:
        raise ValueError(f"ids / counts / num_free: need [rows, width] / [rows] / [1], got {tuple(ids.shape)} / "
                         f"{tuple(counts.shape)} / {tuple(num_free.shape)}")
    d = free_blocks.get_device()
    left = num_free if in_place else _like(num_free, stream)
    _call("pa_kv_free", d, stream, _arg(ids, _I32, "ids", d), _arg(counts, _I32, "counts", d), ids.shape[0],
          ids.shape[1], _arg(free_blocks, _I32, "free_blocks", d), free_blocks.numel(),
          _arg(num_free, _I32, "num_free", d), left.data_ptr())
    return left


def _linear_state(state, kvh, dim, state_slots, log_decay, seq_lens, batch, device):
    """Check the state pool and the arrays beside it; their addresses."""
    shape = state.shape
    if len(shape) != 4 or shape[1] != kvh or shape[2] != dim or shape[3] != dim:
        raise ValueError(f"state: need [num_slots, {kvh}, {dim}, {dim}], got {tuple(state.shape)}")
    if state_slots.shape != (batch,) or seq_lens.shape != (batch,) or log_decay.shape != (kvh,):
        raise ValueError(f"state_slots / seq_lens / log_decay: need shapes {(batch,)} / {(batch,)} / {(kvh,)}, got "
                         f"{tuple(state_slots.shape)} / {tuple(seq_lens.shape)} / {tuple(log_decay.shape)}")
    return (_arg(state, _F32, "state", device), _arg(state_slots, _I32, "state_slots", device),
            _arg(log_decay, _F32, "log_decay", device), _arg(seq_lens, _I32, "seq_lens", device))


def pa_linear_decode(state: torch.Tensor, state_slots: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                     v: torch.Tensor, log_decay: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One token a sequence of linear attention: state [num_slots, num_kv_heads, d, d] fp32, updated in place at
    state_slots [batch]; q [batch, num_heads, d], k and v [batch, num_kv_heads, d], which may be strided views."""
    d, rows, heads, kvh, dim, p, s, out = _packed(q, k, v, out, stream)
    st, slots, decay, lens = _linear_state(state, kvh, dim, state_slots, log_decay, seq_lens, rows, d)
    _call("pa_linear_decode", d, stream, st, state.shape[0], slots, *p, decay, lens, rows, heads, kvh, dim, *s,
          float(scale), _arg(out, _BF16, "out", d))
    return out


def pa_linear_workspace_bytes(batch: int, num_kv_heads: int, head_dim: int, max_chunk: int) -> int:
    return int(library().pa_linear_workspace_bytes(batch, num_kv_heads, head_dim, _most(max_chunk)))


def pa_linear_prefill(state: torch.Tensor, state_slots: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                      v: torch.Tensor, log_decay: torch.Tensor, cu_q_lens: torch.Tensor, seq_lens: torch.Tensor,
                      scale: float, max_chunk: int, workspace: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A chunk of tokens a sequence of linear attention: rows cu_q_lens[b] .. cu_q_lens[b+1] are sequence b's newest
    tokens, and its state goes on from slot state_slots[b] (from zero when seq_lens[b] counts no others)."""
    d, rows, heads, kvh, dim, p, s, out = _packed(q, k, v, out, stream)
    B = cu_q_lens.numel() - 1
    st, slots, decay, lens = _linear_state(state, kvh, dim, state_slots, log_decay, seq_lens, B, d)
    if _current_device() == d:
        need = pa_linear_workspace_bytes(B, kvh, dim, int(max_chunk))
    else:  # (a device of more SMs cuts sequences into more segments)
        with torch.cuda.device(d):
            need = pa_linear_workspace_bytes(B, kvh, dim, int(max_chunk))
    if workspace is None:
        workspace = _new(q, ((need + 3) // 4,), _F32, stream)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace: need {need} bytes, got {workspace.numel() * workspace.element_size()}")
    _call("pa_linear_prefill", d, stream, st, state.shape[0], slots, *p, decay, _arg(cu_q_lens, _I32, "cu_q_lens", d),
          lens, B, rows, heads, kvh, dim, *s, _most(max_chunk), float(scale),
          _arg(workspace, workspace.dtype, "workspace", d) or None, _arg(out, _BF16, "out", d))
    return out


def pa_device_status(clear: bool = True, stream=None) -> int:
    """Synchronise the stream and return the device status bits (0 = clean)."""
    flags = ctypes.c_uint32(0)
    rc = library().pa_device_status(ctypes.byref(flags), 1 if clear else 0, _stream(stream))
    if rc == PA_ERR_CUDA:
        raise PagedAttnError("pa_device_status", rc)
    return int(flags.value)


def pa_selftest_wait_timeout(limit_cycles: int = 2_000_000, stream=None) -> None:
    """Make one bounded device wait run out (an mbarrier nothing arrives on); afterwards the
    device status has PA_DEV_TIMEOUT set.  Asynchronous on `stream`."""
    _check(library().pa_selftest_wait_timeout(int(limit_cycles), _stream(stream)), "pa_selftest_wait_timeout")


def pa_selftest_packed_pairs(cu_lens: torch.Tensor, num_tokens: int, max_len: int, pair_tokens: int, pairs: torch.Tensor,
                             stream=None) -> torch.Tensor:
    """[n, 3] int32: for each of `pairs`, in turn, the first row and the length of its sequence and its first token, as a
    block of pa_prefill_packed finds them; -1 past the last pair."""
    d = cu_lens.get_device()
    out = _new(cu_lens, (pairs.numel(), 3), _I32, stream)
    _call("pa_selftest_packed_pairs", d, stream, _arg(cu_lens, _I32, "cu_lens", d), cu_lens.numel() - 1, int(num_tokens),
          int(max_len), int(pair_tokens), _arg(pairs, _I32, "pairs", d), pairs.numel(), out.data_ptr())
    return out


def pa_decode_num_splits(batch: int, num_kv_heads: int, max_blocks: int) -> int:
    return int(library().pa_decode_num_splits(batch, num_kv_heads, max_blocks))


def pa_splitkv_num_partitions(batch: int, num_kv_heads: int, max_blocks: int) -> int:
    return int(library().pa_splitkv_num_partitions(batch, num_kv_heads, max_blocks))


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)


# ----------------------------------------------------------------------------- host block manager
def pa_kv_block_bytes(num_layers: int, num_kv_heads: int, head_dim: int, block_size: int = BLOCK_SIZE,
                      dtype_bytes: int = 2) -> int:
    return int(library().pa_kv_block_bytes(num_layers, num_kv_heads, head_dim, block_size, dtype_bytes))


def pa_kv_budget_blocks(budget_bytes: int, num_layers: int, num_kv_heads: int, head_dim: int,
                        block_size: int = BLOCK_SIZE, dtype_bytes: int = 2) -> int:
    return int(library().pa_kv_budget_blocks(int(budget_bytes), num_layers, num_kv_heads, head_dim, block_size,
                                             dtype_bytes))


class BlockManager:
    """The library's host-side KV block manager (pa_bm_*): refcounted blocks, a prefix cache
    of full blocks, full-lifetime admission.  Block tables and slot mappings come back as
    int32 / int64 numpy arrays, ready for the attention calls."""

    def __init__(self, num_blocks: int, block_size: int = BLOCK_SIZE, prefix_cache: bool = True):
        import numpy as np
        self._np = np
        self.block_size = block_size
        self._h = library().pa_bm_create(num_blocks, block_size, 1 if prefix_cache else 0)
        if not self._h:
            raise PagedAttnError("pa_bm_create", PA_ERR_INVALID_ARG if num_blocks <= 0 or block_size <= 0 else PA_ERR_NO_MEMORY)

    def close(self):
        if self._h:
            library().pa_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def admit(self, request_id: int, tokens, max_new_tokens: int):
        """(block_table, n_cached_tokens), or None when the request is rejected."""
        np = self._np
        toks = np.ascontiguousarray(tokens, dtype=np.int32)
        cap = (len(toks) + max_new_tokens + self.block_size - 1) // self.block_size
        table = np.empty(max(cap, 1), dtype=np.int32)
        nb, nc = ctypes.c_int32(0), ctypes.c_int32(0)
        rc = library().pa_bm_admit(self._h, request_id, toks.ctypes.data, len(toks), max_new_tokens,
                                   table.ctypes.data, len(table), ctypes.byref(nb), ctypes.byref(nc))
        if rc == PA_ERR_REJECTED:
            return None
        _check(rc, "pa_bm_admit")
        return table[:nb.value].copy(), nc.value

    def admit_cow(self, request_id: int, tokens, max_new_tokens: int):
        """(block_table, n_cached_tokens, copy_src, copy_dst), or None when rejected: a prefix
        hit may end inside a block, whose leading rows copy_src -> copy_dst (slot arrays for
        pa_kv_copy) must be copied before the request's own tokens are appended."""
        np = self._np
        toks = np.ascontiguousarray(tokens, dtype=np.int32)
        cap = (len(toks) + max_new_tokens + self.block_size - 1) // self.block_size
        table = np.empty(max(cap, 1), dtype=np.int32)
        src = np.empty(self.block_size, dtype=np.int64)
        dst = np.empty(self.block_size, dtype=np.int64)
        nb, nc, ncp = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
        rc = library().pa_bm_admit_cow(self._h, request_id, toks.ctypes.data, len(toks), max_new_tokens,
                                       table.ctypes.data, len(table), ctypes.byref(nb), ctypes.byref(nc),
                                       src.ctypes.data, dst.ctypes.data, ctypes.byref(ncp))
        if rc == PA_ERR_REJECTED:
            return None
        _check(rc, "pa_bm_admit_cow")
        return table[:nb.value].copy(), nc.value, src[:ncp.value].copy(), dst[:ncp.value].copy()

    def commit(self, request_id: int, new_tokens, computed: int):
        np = self._np
        toks = np.ascontiguousarray(new_tokens if new_tokens is not None else [], dtype=np.int32)
        _check(library().pa_bm_commit(self._h, request_id, toks.ctypes.data if len(toks) else None, len(toks),
                                      computed), "pa_bm_commit")

    def release(self, request_id: int):
        _check(library().pa_bm_release(self._h, request_id), "pa_bm_release")

    def evict(self, request_id: int, block_ids):
        """The given blocks (one row of pa_kv_evict's `evicted`; negative entries do not count) leave the
        request; its table, positions and reserved lifetime shrink by them."""
        np = self._np
        ids = np.ascontiguousarray(block_ids, dtype=np.int32)
        ids = np.ascontiguousarray(ids[ids >= 0])
        _check(library().pa_bm_evict(self._h, request_id, ids.ctypes.data if len(ids) else None, len(ids)),
               "pa_bm_evict")

    def slots(self, request_id: int, start: int, n: int):
        np = self._np
        out = np.empty(max(n, 1), dtype=np.int64)
        _check(library().pa_bm_slots(self._h, request_id, start, n, out.ctypes.data), "pa_bm_slots")
        return out[:n].copy()

    def stats(self):
        """(free, cached_idle, used) block counts."""
        f, c, u = ctypes.c_int32(0), ctypes.c_int32(0), ctypes.c_int32(0)
        _check(library().pa_bm_stats(self._h, ctypes.byref(f), ctypes.byref(c), ctypes.byref(u)), "pa_bm_stats")
        return f.value, c.value, u.value

