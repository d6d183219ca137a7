"""Python binding of libpkv (paged KV-cache attention on GB300 / sm_103a).

Argument marshalling only: every step of the path runs in libpkv's CUDA kernels
(see ``include/pkv.h`` for the contracts).  PyTorch provides device memory and
the current stream.  There is no fallback: if ``libpkv.so`` is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpkv.so")

PKV_F32 = 0
PKV_BF16 = 1
BLOCK_SIZE = 16

_STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration", 3: "CUDA error",
           4: "device pipeline wait timed out", 5: "slot or block id outside the pool",
           6: "out of blocks or workspace too small", 7: "unknown or duplicate sequence id"}


class PkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {_STATUS.get(status, 'unknown status')} ({status})")
        self.status = status


class PoolDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class PrefillLayout(ctypes.Structure):
    """Byte offsets of one prefill step's inputs in a packed host buffer: the part copied
    to the device (q and the control arrays, `copied_bytes`), then the new rows."""
    _fields_ = [("q", ctypes.c_uint64), ("block_tables", ctypes.c_uint64),
                ("cached_lens", ctypes.c_uint64), ("new_lens", ctypes.c_uint64),
                ("q_offsets", ctypes.c_uint64), ("copied_bytes", ctypes.c_uint64),
                ("k_new", ctypes.c_uint64), ("v_new", ctypes.c_uint64),
                ("slot_mapping", ctypes.c_uint64), ("bytes", ctypes.c_uint64)]


class StepLayout(ctypes.Structure):
    """Byte offsets of one decode step's inputs in a packed host buffer (and its size)."""
    _fields_ = [("q", ctypes.c_uint64), ("k_new", ctypes.c_uint64), ("v_new", ctypes.c_uint64),
                ("block_tables", ctypes.c_uint64), ("context_lens", ctypes.c_uint64),
                ("bytes", ctypes.c_uint64)]


class RopeScaling(ctypes.Structure):
    """How rotary frequencies are scaled (pkv_rope_scaling)."""
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("original_context", ctypes.c_double)]


class QuantCacheDesc(ctypes.Structure):
    """A quantised cache: sizes, format and the four arrays (pkv_quant_cache)."""
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("format", ctypes.c_int32), ("k_codes", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p)]


_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libpkv.so is not built ({LIB_PATH}); run "
                          "paged_kv_cache_58_gb300.build.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, \
        ctypes.c_size_t
    P = ctypes.POINTER
    lib.pkv_status_string.restype = ctypes.c_char_p
    lib.pkv_status_string.argtypes = [ctypes.c_int]
    lib.pkv_version.restype = ctypes.c_int
    lib.pkv_pool_bytes.restype = ctypes.c_uint64
    lib.pkv_pool_bytes.argtypes = [P(PoolDesc)]
    lib.pkv_kv_append.restype = ctypes.c_int
    lib.pkv_kv_append.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, i64, vp]
    lib.pkv_paged_decode_workspace_bytes.restype = sz
    lib.pkv_paged_decode_workspace_bytes.argtypes = [ctypes.c_int] * 6
    lib.pkv_paged_decode_auto_partition.restype = ctypes.c_int
    lib.pkv_paged_decode_auto_partition.argtypes = [ctypes.c_int] * 4
    lib.pkv_paged_decode.restype = ctypes.c_int
    lib.pkv_paged_decode.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_int, f32, ctypes.c_int,
                                     vp, sz, vp]
    lib.pkv_paged_decode_append.restype = ctypes.c_int
    lib.pkv_paged_decode_append.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, vp, vp,
                                            ctypes.c_int, vp, ctypes.c_int, ctypes.c_int,
                                            ctypes.c_int, f32, ctypes.c_int, vp, sz, vp]
    lib.pkv_paged_decode_cascade_append.restype = ctypes.c_int
    lib.pkv_paged_decode_cascade_append.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, vp, vp,
                                                    ctypes.c_int, vp, ctypes.c_int, vp,
                                                    ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                    f32, ctypes.c_int, vp, sz, vp]
    lib.pkv_decode_step_layout.restype = ctypes.c_int
    lib.pkv_decode_step_layout.argtypes = [P(PoolDesc), ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           P(StepLayout)]
    lib.pkv_paged_decode_append_host_staging_bytes.restype = sz
    lib.pkv_paged_decode_append_host_staging_bytes.argtypes = [P(PoolDesc)] + [ctypes.c_int] * 5
    lib.pkv_prefill_step_layout.restype = ctypes.c_int
    lib.pkv_prefill_step_layout.argtypes = [P(PoolDesc)] + [ctypes.c_int] * 4 + [P(PrefillLayout)]
    lib.pkv_paged_prefill_append_host_staging_bytes.restype = sz
    lib.pkv_paged_prefill_append_host_staging_bytes.argtypes = [P(PoolDesc)] + [ctypes.c_int] * 4
    lib.pkv_paged_prefill_append_host.restype = ctypes.c_int
    lib.pkv_paged_prefill_append_host.argtypes = [P(PoolDesc), vp, vp, vp, vp] + \
        [ctypes.c_int] * 5 + [f32, vp, sz, vp]
    lib.pkv_paged_decode_append_host.restype = ctypes.c_int
    lib.pkv_paged_decode_append_host.argtypes = [P(PoolDesc), vp, vp, vp, vp, ctypes.c_int,
                                                 ctypes.c_int, ctypes.c_int, ctypes.c_int, f32,
                                                 ctypes.c_int, vp, sz, vp]
    lib.pkv_paged_prefill.restype = ctypes.c_int
    lib.pkv_paged_prefill.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, ctypes.c_int, vp, vp, vp,
                                      ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, f32,
                                      vp]
    lib.pkv_copy_blocks.restype = ctypes.c_int
    lib.pkv_copy_blocks.argtypes = [P(PoolDesc), vp, vp, vp, ctypes.c_int, vp]
    lib.pkv_read_device_status.restype = ctypes.c_int
    lib.pkv_read_device_status.argtypes = [P(ctypes.c_int), vp]
    lib.pkv_alloc_create.restype = vp
    lib.pkv_alloc_create.argtypes = [i64, ctypes.c_int, ctypes.c_uint64]
    lib.pkv_alloc_destroy.restype = None
    lib.pkv_alloc_destroy.argtypes = [vp]
    lib.pkv_alloc_add_seq.restype = ctypes.c_int
    lib.pkv_alloc_add_seq.argtypes = [vp, i64, i64]
    lib.pkv_alloc_fork.restype = ctypes.c_int
    lib.pkv_alloc_fork.argtypes = [vp, i64, i64]
    lib.pkv_alloc_append.restype = ctypes.c_int
    lib.pkv_alloc_append.argtypes = [vp, i64, i64, P(i64), P(i32), P(ctypes.c_int)]
    lib.pkv_alloc_free_seq.restype = ctypes.c_int
    lib.pkv_alloc_free_seq.argtypes = [vp, i64]
    lib.pkv_alloc_block_table.restype = ctypes.c_int
    lib.pkv_alloc_block_table.argtypes = [vp, P(i64), ctypes.c_int, P(i32), ctypes.c_int]
    lib.pkv_alloc_num_free.restype = i64
    lib.pkv_alloc_num_free.argtypes = [vp]
    lib.pkv_alloc_refcount.restype = ctypes.c_int
    lib.pkv_alloc_refcount.argtypes = [vp, i64]
    lib.pkv_alloc_seq_len.restype = i64
    lib.pkv_alloc_seq_len.argtypes = [vp, i64]
    lib.pkv_alloc_seq_num_blocks.restype = i64
    lib.pkv_alloc_seq_num_blocks.argtypes = [vp, i64]
    lib.pkv_alloc_add_seq_shared.restype = ctypes.c_int
    lib.pkv_alloc_add_seq_shared.argtypes = [vp, i64, P(i32), ctypes.c_int, i64]
    lib.pkv_paged_decode_cascade_workspace_bytes.restype = sz
    lib.pkv_paged_decode_cascade_workspace_bytes.argtypes = [ctypes.c_int] * 7
    lib.pkv_paged_decode_cascade.restype = ctypes.c_int
    lib.pkv_paged_decode_cascade.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, ctypes.c_int, vp,
                                             ctypes.c_int, vp, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, f32, ctypes.c_int, vp, sz, vp]
    ci = ctypes.c_int
    lib.pkv_rope_frequencies.restype = ci
    lib.pkv_rope_frequencies.argtypes = [P(ctypes.c_double), P(f32), ci, ctypes.c_double,
                                         P(RopeScaling)]
    lib.pkv_rope.restype = ci
    lib.pkv_rope.argtypes = [ci, vp, i64, vp, i64, vp, vp, ci, ci, ci, f32, i64, ci, ci, vp]
    lib.pkv_rope_append.restype = ci
    lib.pkv_rope_append.argtypes = [P(PoolDesc), vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, i64,
                                    vp, vp, ci, ci, f32, i64, ci, vp]
    lib.pkv_paged_decode_weights_workspace_bytes.restype = sz
    lib.pkv_paged_decode_weights_workspace_bytes.argtypes = [P(PoolDesc)] + [ci] * 4
    lib.pkv_paged_decode_weights.restype = ci
    lib.pkv_paged_decode_weights.argtypes = [P(PoolDesc), vp, vp, vp, vp, vp, vp, vp, ci, vp, ci,
                                             ci, ci, f32, ci, vp, i64, vp, ci, f32, vp, sz, vp]
    lib.pkv_paged_prefill_weights_workspace_bytes.restype = sz
    lib.pkv_paged_prefill_weights_workspace_bytes.argtypes = [P(PoolDesc)] + [ci] * 5
    lib.pkv_paged_prefill_weights.restype = ci
    lib.pkv_paged_prefill_weights.argtypes = [P(PoolDesc), vp, vp, vp, ci, vp, vp, vp, ci, ci, ci,
                                              ci, ci, f32, ci, vp, i64, vp, ci, f32, vp, sz, vp]
    lib.pkv_evict_workspace_bytes.restype = sz
    lib.pkv_evict_workspace_bytes.argtypes = [P(PoolDesc), ci, ci]
    lib.pkv_evict.restype = ci
    lib.pkv_evict.argtypes = [P(PoolDesc), vp, vp, vp, ci, vp, ci, ci, vp, ci, ci, vp, vp, vp, vp,
                              vp, vp, i64, vp, ci, vp, vp, sz, vp]
    QC = P(QuantCacheDesc)
    lib.pkv_quant_codes_bytes.restype = ctypes.c_uint64
    lib.pkv_quant_codes_bytes.argtypes = [QC]
    lib.pkv_quant_scales_bytes.restype = ctypes.c_uint64
    lib.pkv_quant_scales_bytes.argtypes = [QC]
    lib.pkv_kv_append_quant.restype = ci
    lib.pkv_kv_append_quant.argtypes = [QC, vp, ci, vp, i64, vp, i64, i64, vp]
    lib.pkv_kv_read_quant.restype = ci
    lib.pkv_kv_read_quant.argtypes = [QC, vp, ci, vp, i64, vp, i64, i64, vp]
    lib.pkv_quantize_blocks.restype = ci
    lib.pkv_quantize_blocks.argtypes = [QC, P(PoolDesc), vp, vp, vp, ci, vp]
    lib.pkv_dequantize_blocks.restype = ci
    lib.pkv_dequantize_blocks.argtypes = [QC, P(PoolDesc), vp, vp, vp, ci, vp]
    lib.pkv_copy_blocks_quant.restype = ci
    lib.pkv_copy_blocks_quant.argtypes = [QC, vp, ci, vp]
    lib.pkv_paged_decode_quant_workspace_bytes.restype = sz
    lib.pkv_paged_decode_quant_workspace_bytes.argtypes = [QC] + [ci] * 4
    lib.pkv_paged_decode_quant.restype = ci
    lib.pkv_paged_decode_quant.argtypes = [QC, ci, vp, vp, vp, vp, vp, ci, vp, ci, ci, ci, f32, ci,
                                           vp, sz, vp]
    lib.pkv_alloc_privatize.restype = ci
    lib.pkv_alloc_privatize.argtypes = [vp, i64, i64, P(i32), ci, P(ci)]
    lib.pkv_alloc_truncate.restype = ci
    lib.pkv_alloc_truncate.argtypes = [vp, i64, i64]
    u64 = ctypes.c_uint64
    lib.pkv_block_hash.restype = u64
    lib.pkv_block_hash.argtypes = [u64, u64, P(i32), ctypes.c_int, u64]
    lib.pkv_pcache_create.restype = vp
    lib.pkv_pcache_create.argtypes = [vp]
    lib.pkv_pcache_destroy.restype = None
    lib.pkv_pcache_destroy.argtypes = [vp]
    lib.pkv_pcache_match.restype = ctypes.c_int
    lib.pkv_pcache_match.argtypes = [vp, P(i32), i64, u64, P(i32), ctypes.c_int]
    lib.pkv_pcache_insert.restype = ctypes.c_int
    lib.pkv_pcache_insert.argtypes = [vp, i64, P(i32), i64, u64]
    lib.pkv_pcache_evict.restype = i64
    lib.pkv_pcache_evict.argtypes = [vp, i64]
    lib.pkv_pcache_size.restype = i64
    lib.pkv_pcache_size.argtypes = [vp]
    lib.pkv_radix_create.restype = vp
    lib.pkv_radix_create.argtypes = [vp]
    lib.pkv_radix_destroy.restype = None
    lib.pkv_radix_destroy.argtypes = [vp]
    lib.pkv_radix_match.restype = i64
    lib.pkv_radix_match.argtypes = [vp, P(i32), i64, P(i32), ctypes.c_int]
    lib.pkv_radix_insert.restype = ctypes.c_int
    lib.pkv_radix_insert.argtypes = [vp, i64, P(i32), i64]
    lib.pkv_radix_lock.restype = ctypes.c_int
    lib.pkv_radix_lock.argtypes = [vp, P(i32), i64, ctypes.c_int]
    lib.pkv_radix_evict.restype = i64
    lib.pkv_radix_evict.argtypes = [vp, i64]
    lib.pkv_radix_num_nodes.restype = i64
    lib.pkv_radix_num_nodes.argtypes = [vp]
    lib.pkv_radix_cached_tokens.restype = i64
    lib.pkv_radix_cached_tokens.argtypes = [vp]
    _lib = lib
    return lib


def lib():
    """The loaded libpkv handle (ctypes.CDLL)."""
    return _load()


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise PkvError(fn, st)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PKV_BF16
    if t.dtype == torch.float32:
        return PKV_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


_POOL_DESCS: dict = {}


def pool_desc(k_pool: torch.Tensor) -> PoolDesc:
    """The pool descriptor of a [num_blocks, Hkv, B, D] pool (cached per shape and dtype:
    it holds sizes only)."""
    key = (k_pool.shape, k_pool.dtype)
    d = _POOL_DESCS.get(key)
    if d is None:
        nb, hkv, bs, dim = key[0]
        d = PoolDesc(nb, bs, hkv, dim, _dtype_code(k_pool))
        if len(_POOL_DESCS) > 64:
            _POOL_DESCS.clear()
        _POOL_DESCS[key] = d
    return d


def _dev(t: torch.Tensor, name: str, dtype=None) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def pool_bytes(num_blocks: int, num_kv_heads: int, head_dim: int, dtype=torch.bfloat16,
               block_size: int = BLOCK_SIZE) -> int:
    """Bytes of one (K or V) pool of this shape, as computed by libpkv."""
    d = PoolDesc(num_blocks, block_size, num_kv_heads, head_dim, _dtype_code(torch.empty(0,
                                                                                       dtype=dtype)))
    return int(_load().pkv_pool_bytes(ctypes.byref(d)))


def kv_append(k_pool, v_pool, slot_mapping, k, v, stream=None) -> None:
    """Scatter k/v [T, Hkv, D] into their pool slots (slot < 0 = skip)."""
    d = pool_desc(k_pool)
    T = k.shape[0]
    st = _load().pkv_kv_append(ctypes.byref(d), _dev(k_pool, "k_pool"),
                               _dev(v_pool, "v_pool", k_pool.dtype),
                               _dev(slot_mapping, "slot_mapping", torch.int64),
                               _dev(k, "k", k_pool.dtype), _dev(v, "v", k_pool.dtype), T,
                               _stream(stream))
    _check("pkv_kv_append", st)


def decode_workspace_bytes(num_seqs, num_q_heads, head_dim, max_context, partition_blocks=0,
                           block_size=BLOCK_SIZE):
    return int(_load().pkv_paged_decode_workspace_bytes(num_seqs, num_q_heads, head_dim,
                                                        max_context, block_size,
                                                        partition_blocks))


def auto_partition(num_seqs, num_q_heads, max_context, block_size=BLOCK_SIZE) -> int:
    """Partition size (in pool blocks) paged_decode picks when partition_blocks == 0."""
    return int(_load().pkv_paged_decode_auto_partition(num_seqs, num_q_heads, max_context,
                                                       block_size))


def paged_decode(q, k_pool, v_pool, block_tables, context_lens, scale, *, max_context,
                 out=None, partition_blocks=0, workspace=None, stream=None):
    """Decode attention: q [S, Hq, D] over the paged pools; returns out [S, Hq, D].

    `max_context` is the host-side upper bound of context_lens (no device sync).
    `workspace` (uint8 CUDA tensor) is allocated here when not given.
    """
    d = pool_desc(k_pool)
    S, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:   # the library checks a given workspace's size itself
        need = decode_workspace_bytes(S, Hq, D, max_context, partition_blocks, d.block_size)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = _load().pkv_paged_decode(ctypes.byref(d), _dev(out, "out", q.dtype),
                                  _dev(q, "q", k_pool.dtype), _dev(k_pool, "k_pool"),
                                  _dev(v_pool, "v_pool", k_pool.dtype),
                                  _dev(block_tables, "block_tables", torch.int32),
                                  block_tables.shape[1],
                                  _dev(context_lens, "context_lens", torch.int32),
                                  int(max_context), S, Hq, float(scale), int(partition_blocks),
                                  wptr, wbytes, _stream(stream))
    _check("pkv_paged_decode", st)
    return out


def paged_decode_append(q, k_pool, v_pool, k_new, v_new, block_tables, context_lens, scale, *,
                        max_context, out=None, partition_blocks=0, workspace=None, stream=None):
    """kv_append + paged_decode in one pass: k_new / v_new [S, Hkv, D] are the K / V of
    each sequence's token context_lens[s] - 1, stored into the slot the block table gives
    for that position and attended; returns out [S, Hq, D]."""
    d = pool_desc(k_pool)
    S, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:   # the library checks a given workspace's size itself
        need = decode_workspace_bytes(S, Hq, D, max_context, partition_blocks, d.block_size)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    wptr = workspace.data_ptr() if workspace is not None else None
    wbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if tuple(k_new.shape) != (S, d.num_kv_heads, D) or tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError("k_new / v_new must be [num_seqs, num_kv_heads, head_dim]")
    st = _load().pkv_paged_decode_append(
        ctypes.byref(d), _dev(out, "out", q.dtype), _dev(q, "q", k_pool.dtype),
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool", k_pool.dtype),
        _dev(k_new, "k_new", k_pool.dtype), _dev(v_new, "v_new", k_pool.dtype),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), int(max_context), S, Hq, float(scale),
        int(partition_blocks), wptr, wbytes, _stream(stream))
    _check("pkv_paged_decode_append", st)
    return out


def decode_step_layout(k_pool, num_seqs, num_q_heads, max_blocks_per_seq) -> StepLayout:
    """Packed host-buffer layout of one decode step's inputs (pkv_decode_step_layout)."""
    lay = StepLayout()
    _check("pkv_decode_step_layout",
           _load().pkv_decode_step_layout(ctypes.byref(pool_desc(k_pool)), num_seqs, num_q_heads,
                                          max_blocks_per_seq, ctypes.byref(lay)))
    return lay


def pack_decode_step(host_in, layout, q, k_new, v_new, block_tables, context_lens):
    """Write one step's inputs (CPU tensors) into the packed host buffer `host_in` (uint8)."""
    for off, t in ((layout.q, q), (layout.k_new, k_new), (layout.v_new, v_new),
                   (layout.block_tables, block_tables), (layout.context_lens, context_lens)):
        b = t.contiguous().view(torch.uint8).reshape(-1)
        host_in[off:off + b.numel()].copy_(b)


def decode_host_staging_bytes(k_pool, num_seqs, num_q_heads, max_blocks_per_seq, max_context,
                              partition_blocks=0):
    return int(_load().pkv_paged_decode_append_host_staging_bytes(
        ctypes.byref(pool_desc(k_pool)), num_seqs, num_q_heads, max_blocks_per_seq, max_context,
        partition_blocks))


def paged_decode_append_host(k_pool, v_pool, host_in, host_out, scale, *, num_seqs, num_q_heads,
                             max_blocks_per_seq, max_context, staging, partition_blocks=0,
                             stream=None):
    """One decode step from host memory: host_in (uint8, packed as decode_step_layout)
    -> fused append + decode -> host_out ([S, Hq, D]).  Pinned buffers are read and
    written by the kernels in place; pageable ones go through `staging` with one copy
    each way.  Queued on the stream; host_out is complete after a synchronise."""
    if host_in.is_cuda or host_out.is_cuda:
        raise ValueError("host_in and host_out must be host tensors")
    st = _load().pkv_paged_decode_append_host(
        ctypes.byref(pool_desc(k_pool)), _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool",
                                                                       k_pool.dtype),
        host_in.data_ptr(), host_out.data_ptr(), int(max_blocks_per_seq), int(max_context),
        int(num_seqs), int(num_q_heads), float(scale), int(partition_blocks),
        _dev(staging, "staging"), staging.numel() * staging.element_size(), _stream(stream))
    _check("pkv_paged_decode_append_host", st)
    return host_out


class HostDecodeStep:
    """paged_decode_append_host with every argument bound once, for a loop that runs
    the same step shape over the same buffers (refilling host_in between calls): each
    call is then one ctypes call on pre-converted arguments, about 3 us less host time
    than the keyword form.  The stream is bound too (stream=None: the current stream
    at construction).  The tensors are held for the object's lifetime."""

    def __init__(self, k_pool, v_pool, host_in, host_out, scale, *, num_seqs, num_q_heads,
                 max_blocks_per_seq, max_context, staging, partition_blocks=0, stream=None):
        if host_in.is_cuda or host_out.is_cuda:
            raise ValueError("host_in and host_out must be host tensors")
        self._keep = (k_pool, v_pool, host_in, host_out, staging)
        self._desc = pool_desc(k_pool)
        vp = ctypes.c_void_p
        self._fn = _load().pkv_paged_decode_append_host
        self._args = (ctypes.byref(self._desc), vp(_dev(k_pool, "k_pool")),
                      vp(_dev(v_pool, "v_pool", k_pool.dtype)), vp(host_in.data_ptr()),
                      vp(host_out.data_ptr()), ctypes.c_int(int(max_blocks_per_seq)),
                      ctypes.c_int(int(max_context)), ctypes.c_int(int(num_seqs)),
                      ctypes.c_int(int(num_q_heads)), ctypes.c_float(float(scale)),
                      ctypes.c_int(int(partition_blocks)), vp(_dev(staging, "staging")),
                      ctypes.c_size_t(staging.numel() * staging.element_size()),
                      vp(_stream(stream)))
        self.host_out = host_out

    def __call__(self):
        st = self._fn(*self._args)
        if st != 0:
            raise PkvError("pkv_paged_decode_append_host", st)
        return self.host_out


def prefill_step_layout(k_pool, num_reqs, total_new, num_q_heads,
                        max_blocks_per_seq) -> PrefillLayout:
    """Packed host-buffer layout of one prefill step's inputs (pkv_prefill_step_layout)."""
    lay = PrefillLayout()
    _check("pkv_prefill_step_layout",
           _load().pkv_prefill_step_layout(ctypes.byref(pool_desc(k_pool)), num_reqs, total_new,
                                           num_q_heads, max_blocks_per_seq, ctypes.byref(lay)))
    return lay


def pack_prefill_step(host_in, layout, q, block_tables, cached_lens, new_lens, q_offsets,
                      k_new, v_new, slot_mapping):
    """Write one prefill step's inputs (CPU tensors) into the packed host buffer
    `host_in` (uint8)."""
    for off, t in ((layout.q, q), (layout.block_tables, block_tables),
                   (layout.cached_lens, cached_lens), (layout.new_lens, new_lens),
                   (layout.q_offsets, q_offsets), (layout.k_new, k_new),
                   (layout.v_new, v_new), (layout.slot_mapping, slot_mapping)):
        b = t.contiguous().view(torch.uint8).reshape(-1)
        host_in[off:off + b.numel()].copy_(b)


def prefill_host_staging_bytes(k_pool, num_reqs, total_new, num_q_heads, max_blocks_per_seq):
    return int(_load().pkv_paged_prefill_append_host_staging_bytes(
        ctypes.byref(pool_desc(k_pool)), num_reqs, total_new, num_q_heads, max_blocks_per_seq))


def paged_prefill_append_host(k_pool, v_pool, host_in, host_out, scale, *, num_reqs, total_new,
                              max_new, num_q_heads, max_blocks_per_seq, staging, stream=None):
    """One prefill step from host memory: host_in (uint8, packed as prefill_step_layout)
    -> kv_append of the new rows + paged_prefill -> host_out ([total_new, Hq, D]),
    through `staging`, with the copies pipelined against the kernels over request chunks.
    Queued on the stream; host_out is complete after a synchronise."""
    if host_in.is_cuda or host_out.is_cuda:
        raise ValueError("host_in and host_out must be host tensors")
    st = _load().pkv_paged_prefill_append_host(
        ctypes.byref(pool_desc(k_pool)), _dev(k_pool, "k_pool"),
        _dev(v_pool, "v_pool", k_pool.dtype), host_in.data_ptr(), host_out.data_ptr(),
        int(num_reqs), int(total_new), int(max_new), int(num_q_heads), int(max_blocks_per_seq),
        float(scale), _dev(staging, "staging"), staging.numel() * staging.element_size(),
        _stream(stream))
    _check("pkv_paged_prefill_append_host", st)
    return host_out


def cascade_workspace_bytes(num_seqs, num_q_heads, head_dim, prefix_len, max_context,
                            partition_blocks=0, block_size=BLOCK_SIZE):
    return int(_load().pkv_paged_decode_cascade_workspace_bytes(
        num_seqs, num_q_heads, head_dim, prefix_len, max_context, block_size, partition_blocks))


def paged_decode_cascade(q, k_pool, v_pool, prefix_blocks, prefix_len, block_tables,
                         context_lens, scale, *, max_context, out=None, partition_blocks=0,
                         workspace=None, stream=None):
    """Decode of sequences sharing their first `prefix_len` tokens in `prefix_blocks`
    (int32 [prefix_len / block_size] CUDA tensor); same result as paged_decode."""
    d = pool_desc(k_pool)
    S, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    need = cascade_workspace_bytes(S, Hq, D, prefix_len, max_context, partition_blocks,
                                   d.block_size)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = _load().pkv_paged_decode_cascade(
        ctypes.byref(d), _dev(out, "out", q.dtype), _dev(q, "q", k_pool.dtype),
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool", k_pool.dtype),
        _dev(prefix_blocks, "prefix_blocks", torch.int32), int(prefix_len),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), int(max_context), S, Hq, float(scale),
        int(partition_blocks), workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check("pkv_paged_decode_cascade", st)
    return out


def paged_decode_cascade_append(q, k_pool, v_pool, k_new, v_new, prefix_blocks, prefix_len,
                                block_tables, context_lens, scale, *, max_context, out=None,
                                partition_blocks=0, workspace=None, stream=None):
    """Cascade decode with the append fused in: k_new / v_new [S, Hkv, D] are the K / V
    of each sequence's token context_lens[s] - 1 (in its private suffix)."""
    d = pool_desc(k_pool)
    S, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = cascade_workspace_bytes(S, Hq, D, prefix_len, max_context, partition_blocks,
                                       d.block_size)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if tuple(k_new.shape) != (S, d.num_kv_heads, D) or tuple(v_new.shape) != tuple(k_new.shape):
        raise ValueError("k_new / v_new must be [num_seqs, num_kv_heads, head_dim]")
    st = _load().pkv_paged_decode_cascade_append(
        ctypes.byref(d), _dev(out, "out", q.dtype), _dev(q, "q", k_pool.dtype),
        _dev(k_pool, "k_pool"), _dev(v_pool, "v_pool", k_pool.dtype),
        _dev(k_new, "k_new", k_pool.dtype), _dev(v_new, "v_new", k_pool.dtype),
        _dev(prefix_blocks, "prefix_blocks", torch.int32), int(prefix_len),
        _dev(block_tables, "block_tables", torch.int32), block_tables.shape[1],
        _dev(context_lens, "context_lens", torch.int32), int(max_context), S, Hq, float(scale),
        int(partition_blocks), workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check("pkv_paged_decode_cascade_append", st)
    return out


def paged_prefill(q, k_pool, v_pool, block_tables, cached_lens, new_lens, q_offsets, scale, *,
                  max_new, out=None, stream=None):
    """Causal prefill of q [N, Hq, D] over cached prefix + new tokens; returns out."""
    d = pool_desc(k_pool)
    N, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    R = cached_lens.shape[0]
    st = _load().pkv_paged_prefill(ctypes.byref(d), _dev(out, "out", q.dtype),
                                   _dev(q, "q", k_pool.dtype), _dev(k_pool, "k_pool"),
                                   _dev(v_pool, "v_pool", k_pool.dtype),
                                   _dev(block_tables, "block_tables", torch.int32),
                                   block_tables.shape[1],
                                   _dev(cached_lens, "cached_lens", torch.int32),
                                   _dev(new_lens, "new_lens", torch.int32),
                                   _dev(q_offsets, "q_offsets", torch.int32), R, N, int(max_new),
                                   Hq, float(scale), _stream(stream))
    _check("pkv_paged_prefill", st)
    return out


# The raw handle of the current stream of a device, and the current device, without the
# Python objects around them: a decode step's calls are a few microseconds each.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_on(stream, dev: int) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _wrong(t, name, dev, dtype, shape):
    """The error for a tensor that `_arg` refuses."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev}, the current device")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t: torch.Tensor, name: str, dev: int, dtype, shape) -> int:
    """Address of a contiguous tensor that must be of this device, dtype and shape."""
    if t.get_device() == dev and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _wrong(t, name, dev, dtype, shape)


def _opt(t, name: str, dev: int, dtype, shape):
    return None if t is None else _arg(t, name, dev, dtype, shape)


def _rows_arg(t: torch.Tensor, name: str, dev: int, dtype, shape):
    """(address, token stride) of [tokens, heads, head_dim] rows whose tokens may be apart
    (a slice of a fused projection)."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape:
        _wrong(t, name, dev, dtype, shape)
    tokens, heads, dim = shape
    if tokens == 0 or heads == 0:
        return t.data_ptr(), heads * dim
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return t.data_ptr(), (s0 if tokens > 1 else heads * dim)


def _device(t: torch.Tensor, name: str) -> int:
    """The CUDA device of the call: `t`'s, which must be the current one (the library's
    streams and status word are the current device's)."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != _cur_device():
        raise ValueError(f"{name} is on cuda:{dev}, not on the current device")
    return dev


def _fresh(shape, dtype, dev, stream):
    """A tensor the call writes, allocated on the stream that will use it, so that its memory
    is not handed on while that stream still works in it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace_arg(ws, need, dev, stream):
    """(tensor, address, bytes) of the given workspace, or of one made here."""
    if ws is None:
        ws = _fresh((max(need(), 16),), torch.uint8, dev, stream)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _pools(k_pool, v_pool):
    """(descriptor, device, K address, V address) of a pair of pools."""
    dev, dt, shape = k_pool.get_device(), k_pool.dtype, k_pool.shape
    if dev < 0 or dev != _cur_device():
        _device(k_pool, "k_pool")
    d = _POOL_DESCS.get((shape, dt))
    if d is None:
        if len(shape) != 4:
            raise ValueError("k_pool must be [num_blocks, num_kv_heads, block_size, head_dim]")
        d = pool_desc(k_pool)
    if not k_pool.is_contiguous():
        raise ValueError("k_pool must be contiguous")
    return d, dev, k_pool.data_ptr(), _arg(v_pool, "v_pool", dev, dt, shape)


def _weights_arg(weights, dev, dtype, hkv, name="weights"):
    """(address, rows, stride) of a [rows, Hkv, stride] array."""
    if weights.dim() != 3 or weights.shape[1] != hkv:
        raise ValueError(f"{name} must be [num_rows, num_kv_heads, stride]")
    return _arg(weights, name, dev, dtype, weights.shape), weights.shape[0], weights.shape[2]


ROPE_KINDS = {None: 0, "linear": 1, "ntk": 2, "llama3": 3, "yarn": 4, "yarn_pairs": 5}


def rope_frequencies(rotary_dim, theta=10000.0, *, scaling=None, factor=1.0, low=None, high=None,
                     original_context=0, device="cuda"):
    """Rotary frequencies (float64 [rotary_dim / 2] on `device`) and the attention scale that
    goes with them.  `scaling`: None, "linear", "ntk", "llama3" (low 1, high 4 unless given),
    "yarn" or "yarn_pairs" (low 1, high 32), the last three over a trained context of
    `original_context`.  "yarn_pairs" is what released YaRN models were trained with: the blend
    between kept and stretched frequencies goes by pair index; "yarn" blends by turns, as the
    method's paper has it."""
    if scaling not in ROPE_KINDS:
        raise ValueError(f"scaling must be one of {list(ROPE_KINDS)}")
    sc = RopeScaling(ROPE_KINDS[scaling], float(factor), float(1 if low is None else low),
                     float((4 if scaling == "llama3" else 32) if high is None else high),
                     float(original_context))
    out = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.float64, device="cpu")
    scale = ctypes.c_float(1.0)
    _check("pkv_rope_frequencies", _load().pkv_rope_frequencies(
        ctypes.cast(out.data_ptr(), ctypes.POINTER(ctypes.c_double)), ctypes.byref(scale),
        int(rotary_dim), float(theta), ctypes.byref(sc)))
    return out.to(device), scale.value


def rope(x, positions, inv_freq, *, interleaved=False, inverse=False, attn_scale=1.0, out=None,
         stream=None):
    """Rows x [T, H, D] turned by their token's position (int32 [T]); returns out (a new
    contiguous tensor, or the one given, which may be x itself but not overlap it otherwise).

    The first 2 * len(inv_freq) elements of a row turn (inv_freq float64, radians per
    position: rope_frequencies).  x may be a slice of a fused projection: its tokens any
    multiple of 16 bytes apart.  `inverse` turns the other way: it undoes the turn, and takes
    a gradient with respect to the output to one with respect to x.  Gradients flow to x through
    the new tensor; where one is asked for, `out` is refused.
    """
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("rope: no gradient flows through out=; leave it out, or call under "
                             "torch.no_grad()")
        return _Rope.apply(x, positions, inv_freq, interleaved, inverse, attn_scale, stream)
    return _rope(x, positions, inv_freq, interleaved, inverse, attn_scale, out, stream)


class _Rope(torch.autograd.Function):
    """The turn with its gradient: the opposite turn, same scale, of the output's gradient."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, interleaved, inverse, attn_scale, stream):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = interleaved, inverse, attn_scale
        return _rope(x, positions, inv_freq, interleaved, inverse, attn_scale, None, stream)

    @staticmethod
    def backward(ctx, grad):
        positions, inv_freq = ctx.saved_tensors
        interleaved, inverse, attn_scale = ctx.how
        grad = grad.contiguous()
        if grad.data_ptr() % 16:
            grad = grad.clone()
        return (rope(grad, positions, inv_freq, interleaved=interleaved, inverse=not inverse,
                     attn_scale=attn_scale),) + (None,) * 6


def _rope(x, positions, inv_freq, interleaved, inverse, attn_scale, out, stream):
    dev = _device(x, "x")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError("x must be [tokens, heads, head_dim]")
    T, H, D = shape
    xp, xs = _rows_arg(x, "x", dev, x.dtype, shape)
    if out is None:
        out = _fresh(shape, x.dtype, dev, stream)
    op, os_ = _rows_arg(out, "out", dev, x.dtype, shape)
    half = inv_freq.numel()
    st = _load().pkv_rope(_dtype_code(x), op, os_, xp, xs,
                          _arg(positions, "positions", dev, torch.int32, (T,)),
                          _arg(inv_freq, "inv_freq", dev, torch.float64, (half,)), 2 * half,
                          bool(interleaved), bool(inverse), attn_scale, T, H, D,
                          _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_rope", st)
    return out


def rope_append(q, k, v, k_pool, v_pool, slot_mapping, positions, inv_freq, *, interleaved=False,
                attn_scale=1.0, q_out=None, stream=None):
    """One launch for a step's new tokens: q [T, Hq, D] turned into q_out (returned), k [T, Hkv,
    D] turned and v [T, Hkv, D] as it is stored into their pool slots (slot < 0 = skip).
    Arguments as rope and kv_append; q, k and v may be slices of one fused projection.  As with
    every call that writes the cache, no gradient flows."""
    d, dev, kp, vp_ = _pools(k_pool, v_pool)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    T, Hq, _ = q.shape
    dt, D = k_pool.dtype, d.head_dim
    qp, qs = _rows_arg(q, "q", dev, dt, (T, Hq, D))
    kr, ks = _rows_arg(k, "k", dev, dt, (T, d.num_kv_heads, D))
    vr, vs = _rows_arg(v, "v", dev, dt, (T, d.num_kv_heads, D))
    if q_out is None:
        q_out = _fresh((T, Hq, D), dt, dev, stream)
    op, os_ = _rows_arg(q_out, "q_out", dev, dt, (T, Hq, D))
    half = inv_freq.numel()
    st = _load().pkv_rope_append(ctypes.byref(d), kp, vp_,
                                 _arg(slot_mapping, "slot_mapping", dev, torch.int64, (T,)), op,
                                 os_, qp, qs, kr, ks, vr, vs,
                                 _arg(positions, "positions", dev, torch.int32, (T,)),
                                 _arg(inv_freq, "inv_freq", dev, torch.float64, (half,)),
                                 2 * half, bool(interleaved), attn_scale, T, Hq,
                                 _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_rope_append", st)
    return q_out


def decode_weights_workspace_bytes(k_pool, num_seqs, num_q_heads, max_context,
                                   partition_blocks=0) -> int:
    """Workspace of paged_decode_weights (partials, and every score: 4 bytes per query head
    and token)."""
    return int(_load().pkv_paged_decode_weights_workspace_bytes(
        ctypes.byref(pool_desc(k_pool)), num_seqs, num_q_heads, max_context, partition_blocks))


def paged_decode_weights(q, k_pool, v_pool, block_tables, context_lens, scale, weights, *,
                         max_context, k_new=None, v_new=None, row_ids=None, decay=1.0, out=None,
                         partition_blocks=0, workspace=None, stream=None):
    """paged_decode (or, with k_new / v_new [S, Hkv, D], paged_decode_append) that also adds up
    the attention each cached token receives: weights [rows, Hkv, stride] (fp32, in place)
    becomes decay * weights + the probabilities summed over the kv head's query heads, in row
    row_ids[s] (default s; negative: not counted).  Returns out [S, Hq, D]."""
    d, dev, kp, vp_ = _pools(k_pool, v_pool)
    if q.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q must be [num_seqs, heads, head_dim], block_tables [num_seqs, blocks]")
    S, Hq, _ = q.shape
    dt, D, Hkv = k_pool.dtype, d.head_dim, d.num_kv_heads
    if out is None:
        out = _fresh((S, Hq, D), dt, dev, stream)
    wp, rows, stride = _weights_arg(weights, dev, torch.float32, Hkv)
    _, ws, wsb = _keep = _workspace_arg(
        workspace, lambda: decode_weights_workspace_bytes(k_pool, S, Hq, max_context,
                                                          partition_blocks), dev, stream)
    st = _load().pkv_paged_decode_weights(
        ctypes.byref(d), _arg(out, "out", dev, dt, (S, Hq, D)), _arg(q, "q", dev, dt, (S, Hq, D)),
        kp, vp_, _opt(k_new, "k_new", dev, dt, (S, Hkv, D)),
        _opt(v_new, "v_new", dev, dt, (S, Hkv, D)),
        _arg(block_tables, "block_tables", dev, torch.int32, (S, block_tables.shape[1])),
        block_tables.shape[1], _arg(context_lens, "context_lens", dev, torch.int32, (S,)),
        max_context, S, Hq, scale, partition_blocks, wp, stride,
        _opt(row_ids, "row_ids", dev, torch.int32, (S,)), rows, decay, ws, wsb,
        _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_paged_decode_weights", st)
    return out


def prefill_weights_workspace_bytes(k_pool, num_reqs, num_q_heads, max_new, max_context,
                                    window=0) -> int:
    """Workspace of paged_prefill_weights (the query rows' softmax statistics; for fp32 pools
    also scores, up to 256 MB, or 1 GB where one kv head of a request alone has that many)."""
    return int(_load().pkv_paged_prefill_weights_workspace_bytes(
        ctypes.byref(pool_desc(k_pool)), num_reqs, num_q_heads, max_new, max_context, window))


def paged_prefill_weights(q, k_pool, block_tables, cached_lens, new_lens, q_offsets, scale,
                          weights, *, max_new, max_context, window=0, row_ids=None, decay=1.0,
                          workspace=None, stream=None):
    """The attention that each cached token receives from the last `window` new tokens of its
    request (0: all of them), added to weights [rows, Hkv, stride] (fp32, in place) as
    paged_decode_weights does; q and the lengths as paged_prefill.  Returns weights."""
    if k_pool.dim() != 4 or q.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q must be [tokens, heads, head_dim], block_tables [num_reqs, blocks], "
                         "k_pool [num_blocks, num_kv_heads, block_size, head_dim]")
    dev = _device(k_pool, "k_pool")
    d = pool_desc(k_pool)
    N, Hq, _ = q.shape
    R = block_tables.shape[0]
    dt = k_pool.dtype
    wp, rows, stride = _weights_arg(weights, dev, torch.float32, d.num_kv_heads)
    _, ws, wsb = _keep = _workspace_arg(
        workspace, lambda: prefill_weights_workspace_bytes(k_pool, R, Hq, max_new, max_context,
                                                           window), dev, stream)
    st = _load().pkv_paged_prefill_weights(
        ctypes.byref(d), _arg(q, "q", dev, dt, (N, Hq, d.head_dim)),
        _arg(k_pool, "k_pool", dev, dt, k_pool.shape),
        _arg(block_tables, "block_tables", dev, torch.int32, block_tables.shape),
        block_tables.shape[1], _arg(cached_lens, "cached_lens", dev, torch.int32, (R,)),
        _arg(new_lens, "new_lens", dev, torch.int32, (R,)),
        _arg(q_offsets, "q_offsets", dev, torch.int32, (R + 1,)), R, N, max_new, max_context, Hq,
        scale, window, wp, stride, _opt(row_ids, "row_ids", dev, torch.int32, (R,)), rows, decay,
        ws, wsb, _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_paged_prefill_weights", st)
    return weights


def evict_workspace_bytes(k_pool, num_seqs, max_context) -> int:
    return int(_load().pkv_evict_workspace_bytes(ctypes.byref(pool_desc(k_pool)), num_seqs,
                                                 max_context))


def evict(k_pool, v_pool, block_tables, context_lens, budgets, weights, positions, *, max_context,
          sinks=0, recent=0, seen_lens=None, tracked_lens=None, row_ids=None, weights_out=None,
          positions_out=None, new_lens=None, workspace=None, stream=None):
    """Shrink sequences with more than budgets[s] cached tokens to that many per kv head:
    the first `sinks` and last `recent` positions are kept, then the largest weights (ties:
    lowest index); kept rows past the budget move into the freed places below it.

    weights (fp32) and positions (int32), [rows, Hkv, stride], shrink along: in place, or into
    weights_out / positions_out.  seen_lens: tokens each sequence has had in all (default
    context_lens); tracked_lens: the new_lens of its last eviction (default zeros).  Returns
    new_lens (int32 [S]).  The blocks below a budget must be the sequence's own
    (BlockAllocator.privatize); those past it can go back (BlockAllocator.truncate)."""
    d, dev, kp, vp_ = _pools(k_pool, v_pool)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, blocks]")
    S = block_tables.shape[0]
    i32, one = torch.int32, (S,)
    wp, rows, stride = _weights_arg(weights, dev, torch.float32, d.num_kv_heads)
    pp = _arg(positions, "positions", dev, i32, weights.shape)
    wo = wp if weights_out is None else _arg(weights_out, "weights_out", dev, torch.float32,
                                             weights.shape)
    po = pp if positions_out is None else _arg(positions_out, "positions_out", dev, i32,
                                               weights.shape)
    if new_lens is None:
        new_lens = _fresh(one, i32, dev, stream)
    _, ws, wsb = _keep = _workspace_arg(
        workspace, lambda: evict_workspace_bytes(k_pool, S, max_context), dev, stream)
    st = _load().pkv_evict(
        ctypes.byref(d), kp, vp_, _arg(block_tables, "block_tables", dev, i32, block_tables.shape),
        block_tables.shape[1], _arg(context_lens, "context_lens", dev, i32, one), max_context, S,
        _arg(budgets, "budgets", dev, i32, one), sinks, recent,
        _opt(seen_lens, "seen_lens", dev, i32, one),
        _opt(tracked_lens, "tracked_lens", dev, i32, one), wp, wo, pp, po, stride,
        _opt(row_ids, "row_ids", dev, i32, one), rows, _arg(new_lens, "new_lens", dev, i32, one),
        ws, wsb, _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_evict", st)
    return new_lens


QUANT_FORMATS = {"fp8": 0, "fp4": 1}


class QuantCache:
    """A paged cache whose rows are held in 8 or 4 bits (pkv_quant_cache): the blocks, slots and
    tables of a pool, codes and scales in place of its rows.

    `format` "fp8": e4m3 codes and a power of two per row; "fp4": e2m1 codes with an e4m3 scale
    per 16 elements, and a power of two per row.  k, v: uint8 [num_blocks, Hkv, B, D] (fp4:
    [..., D / 2]); k_scales, v_scales: uint8 [num_blocks, Hkv, B], fp4 [num_blocks, Hkv,
    B / 16 * (D + 16)].  QuantCache.empty makes them; given ones are held, not copied.  Its memory
    need not be cleared: a decode does not look at slots that were never written.  kv_read_quant and
    the moves of whole blocks do, and carry on what is there, NaN and infinities included."""

    def __init__(self, k, v, k_scales, v_scales, *, format="fp8"):
        if format not in QUANT_FORMATS:
            raise ValueError(f"format must be one of {list(QUANT_FORMATS)}")
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be [num_blocks, num_kv_heads, block_size, bytes of a row]")
        dev = k.get_device()
        if dev < 0:
            raise ValueError("k must be a CUDA tensor")
        nb, hkv, block, row = k.shape
        dim = row if format == "fp8" else 2 * row
        beside = (nb, hkv, block // 16 * (16 if format == "fp8" else dim + 16))
        u8 = torch.uint8
        self.desc = QuantCacheDesc(nb, block, hkv, dim, QUANT_FORMATS[format],
                                   _arg(k, "k", dev, u8, k.shape), _arg(v, "v", dev, u8, k.shape),
                                   _arg(k_scales, "k_scales", dev, u8, beside),
                                   _arg(v_scales, "v_scales", dev, u8, beside))
        if not _load().pkv_quant_codes_bytes(ctypes.byref(self.desc)):
            raise ValueError("a quantised cache has blocks of 16 or 32 tokens and heads of 64 or "
                             "128, fewer than 2^31 rows in all")
        runs = sorted((t.data_ptr(), t.numel()) for t in (k, v, k_scales, v_scales))
        if any(at + n > after for (at, n), (after, _) in zip(runs, runs[1:])):
            raise ValueError("the four arrays of a quantised cache may not share memory")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.format, self.device = format, dev
        self.num_blocks, self.num_kv_heads, self.block_size, self.head_dim = nb, hkv, block, dim
        self._ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, num_blocks, num_kv_heads, head_dim, *, block_size=BLOCK_SIZE, format="fp8",
              device="cuda"):
        """A cache of `num_blocks` blocks, not initialised."""
        if format not in QUANT_FORMATS:
            raise ValueError(f"format must be one of {list(QUANT_FORMATS)}")
        row = head_dim if format == "fp8" else head_dim // 2
        beside = block_size // 16 * (16 if format == "fp8" else head_dim + 16)
        k, v = (torch.empty((num_blocks, num_kv_heads, block_size, row), dtype=torch.uint8,
                            device=device) for _ in range(2))
        ks, vs = (torch.empty((num_blocks, num_kv_heads, beside), dtype=torch.uint8,
                              device=device) for _ in range(2))
        return cls(k, v, ks, vs, format=format)

    @property
    def nbytes(self) -> int:
        """Bytes of the four arrays."""
        return 2 * (self.k.numel() + self.k_scales.numel())


def _quant(cache):
    """(pointer to the description, device) of a quantised cache on the current device."""
    dev = cache.device
    if dev != _cur_device():
        raise ValueError(f"the cache is on cuda:{dev}, not on the current device")
    return cache._ref, dev


def kv_append_quant(cache, slot_mapping, k, v, stream=None) -> None:
    """Quantise k / v [T, Hkv, D] (bf16 or fp32) into their slots of a QuantCache (slot < 0 =
    skip).  k and v may be slices of a fused projection: tokens any multiple of 16 bytes apart.
    As with every call that writes the cache, no gradient flows."""
    c, dev = _quant(cache)
    T, dt = k.shape[0], k.dtype
    shape = (T, cache.num_kv_heads, cache.head_dim)
    kp, ks = _rows_arg(k, "k", dev, dt, shape)
    vp_, vs = _rows_arg(v, "v", dev, dt, shape)
    st = _load().pkv_kv_append_quant(c, _arg(slot_mapping, "slot_mapping", dev, torch.int64, (T,)),
                                     _dtype_code(k), kp, ks, vp_, vs, T, _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_kv_append_quant", st)


def kv_read_quant(cache, slot_mapping, *, dtype=torch.bfloat16, k_out=None, v_out=None,
                  stream=None):
    """Rows of the slots [T] of a QuantCache, (k, v) [T, Hkv, D] of `dtype` (or into k_out and
    v_out, of their type; tokens may be apart as in kv_append_quant).  A negative slot reads
    zeros."""
    c, dev = _quant(cache)
    T = slot_mapping.shape[0]
    shape = (T, cache.num_kv_heads, cache.head_dim)
    if k_out is None:
        k_out = _fresh(shape, dtype if v_out is None else v_out.dtype, dev, stream)
    if v_out is None:
        v_out = _fresh(shape, k_out.dtype, dev, stream)
    kp, ks = _rows_arg(k_out, "k_out", dev, k_out.dtype, shape)
    vp_, vs = _rows_arg(v_out, "v_out", dev, k_out.dtype, shape)
    st = _load().pkv_kv_read_quant(c, _arg(slot_mapping, "slot_mapping", dev, torch.int64, (T,)),
                                   _dtype_code(k_out), kp, ks, vp_, vs, T, _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_kv_read_quant", st)
    return k_out, v_out


def quantize_blocks(cache, k_pool, v_pool, pairs, stream=None) -> None:
    """Quantise whole blocks of a pool into a QuantCache: cache[dst] = pool[src] for each (src,
    dst) of pairs (int32 [n, 2])."""
    _move_blocks("pkv_quantize_blocks", cache, k_pool, v_pool, pairs, stream)


def dequantize_blocks(cache, k_pool, v_pool, pairs, stream=None) -> None:
    """Read whole blocks of a QuantCache into a pool: pool[dst] = cache[src] for each (src, dst)
    of pairs (int32 [n, 2]), every row of them, also ones never written.  k_pool and v_pool may not
    overlap.  A prefix read back so is what paged_prefill attends to."""
    _move_blocks("pkv_dequantize_blocks", cache, k_pool, v_pool, pairs, stream)


def _move_blocks(fn, cache, k_pool, v_pool, pairs, stream):
    c, dev = _quant(cache)
    d, _, kp, vp_ = _pools(k_pool, v_pool)
    st = getattr(_load(), fn)(c, ctypes.byref(d), kp, vp_,
                              _arg(pairs, "pairs", dev, torch.int32, (pairs.shape[0], 2)),
                              pairs.shape[0], _stream_on(stream, dev))
    if st != 0:
        raise PkvError(fn, st)


def copy_blocks_quant(cache, pairs, stream=None) -> None:
    """copy_blocks within a QuantCache: block dst = block src for each (src, dst) of pairs (int32
    [n, 2]; the allocator's copy-on-write pairs)."""
    c, dev = _quant(cache)
    st = _load().pkv_copy_blocks_quant(c, _arg(pairs, "pairs", dev, torch.int32,
                                               (pairs.shape[0], 2)), pairs.shape[0],
                                       _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_copy_blocks_quant", st)


def decode_quant_workspace_bytes(cache, num_seqs, num_q_heads, max_context,
                                 partition_blocks=0) -> int:
    """Workspace of paged_decode_quant."""
    return int(_load().pkv_paged_decode_quant_workspace_bytes(
        cache._ref, num_seqs, num_q_heads, max_context, partition_blocks))


def paged_decode_quant(q, cache, block_tables, context_lens, scale, *, max_context, k_new=None,
                       v_new=None, out=None, partition_blocks=0, workspace=None, stream=None):
    """paged_decode over a QuantCache: q [S, Hq, D] (bf16 or fp32) -> out [S, Hq, D].  With k_new
    / v_new [S, Hkv, D], the rows of each sequence's token context_lens[s] - 1, they are quantised
    into the slots the block tables give for them first, in the same launch, and attended as
    they come back from there."""
    c, dev = _quant(cache)
    if q.dim() != 3 or block_tables.dim() != 2:
        raise ValueError("q must be [num_seqs, heads, head_dim], block_tables [num_seqs, blocks]")
    S, Hq, _ = q.shape
    dt, D = q.dtype, cache.head_dim
    new = (S, cache.num_kv_heads, D)
    if out is None:
        out = _fresh((S, Hq, D), dt, dev, stream)
    _, ws, wsb = _keep = _workspace_arg(
        workspace, lambda: decode_quant_workspace_bytes(cache, S, Hq, max_context,
                                                        partition_blocks), dev, stream)
    st = _load().pkv_paged_decode_quant(
        c, _dtype_code(q), _arg(out, "out", dev, dt, (S, Hq, D)), _arg(q, "q", dev, dt, (S, Hq, D)),
        _opt(k_new, "k_new", dev, dt, new), _opt(v_new, "v_new", dev, dt, new),
        _arg(block_tables, "block_tables", dev, torch.int32, (S, block_tables.shape[1])),
        block_tables.shape[1], _arg(context_lens, "context_lens", dev, torch.int32, (S,)),
        max_context, S, Hq, scale, partition_blocks, ws, wsb, _stream_on(stream, dev))
    if st != 0:
        raise PkvError("pkv_paged_decode_quant", st)
    return out


def copy_blocks(k_pool, v_pool, pairs, stream=None) -> None:
    """pool[dst] = pool[src] for each row (src, dst) of int32 pairs [P, 2]."""
    d = pool_desc(k_pool)
    st = _load().pkv_copy_blocks(ctypes.byref(d), _dev(k_pool, "k_pool"),
                                 _dev(v_pool, "v_pool", k_pool.dtype),
                                 _dev(pairs, "pairs", torch.int32), pairs.shape[0],
                                 _stream(stream))
    _check("pkv_copy_blocks", st)


def read_device_status(stream=None) -> int:
    """Synchronise and return (and clear) the library's device status word."""
    v = ctypes.c_int(0)
    _check("pkv_read_device_status", _load().pkv_read_device_status(ctypes.byref(v),
                                                                    _stream(stream)))
    return v.value


class BlockAllocator:
    """Host block allocator (libpkv's C++ pkv_alloc): slots, tables, refcounts, CoW."""

    def __init__(self, num_blocks: int, block_size: int = BLOCK_SIZE, seed: int = 0):
        self._lib = _load()
        self._h = self._lib.pkv_alloc_create(num_blocks, block_size, seed)
        if not self._h:
            raise ValueError("pkv_alloc_create: invalid arguments")
        self.num_blocks = num_blocks
        self.block_size = block_size

    def close(self):
        if self._h:
            self._lib.pkv_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def add_seq(self, seq_id: int, num_tokens: int) -> None:
        _check("pkv_alloc_add_seq", self._lib.pkv_alloc_add_seq(self._h, seq_id, num_tokens))

    def add_seq_shared(self, seq_id: int, shared_blocks, num_tokens: int) -> None:
        """New sequence whose first blocks are existing (shared) blocks."""
        arr = (ctypes.c_int32 * max(len(shared_blocks), 1))(*shared_blocks)
        _check("pkv_alloc_add_seq_shared", self._lib.pkv_alloc_add_seq_shared(
            self._h, seq_id, arr, len(shared_blocks), num_tokens))

    def fork(self, parent: int, child: int) -> None:
        _check("pkv_alloc_fork", self._lib.pkv_alloc_fork(self._h, parent, child))

    def append(self, seq_id: int, n: int = 1):
        """Reserve n slots; returns (slots list, cow pair (old, new) or None)."""
        slots = (ctypes.c_int64 * max(n, 1))()
        pairs = (ctypes.c_int32 * 2)()
        ncow = ctypes.c_int(0)
        _check("pkv_alloc_append", self._lib.pkv_alloc_append(self._h, seq_id, n, slots, pairs,
                                                              ctypes.byref(ncow)))
        return list(slots[:n]), ((pairs[0], pairs[1]) if ncow.value else None)

    def privatize(self, seq_id: int, num_tokens: int):
        """Private copies of the blocks of the first num_tokens tokens that others reference;
        returns the (old, new) pairs for copy_blocks."""
        most = min(max(-(-num_tokens // self.block_size), 0), self.num_blocks)
        pairs = (ctypes.c_int32 * max(2 * most, 1))()
        n = ctypes.c_int(0)
        _check("pkv_alloc_privatize", self._lib.pkv_alloc_privatize(self._h, seq_id, num_tokens,
                                                                    pairs, most, ctypes.byref(n)))
        return [(pairs[2 * i], pairs[2 * i + 1]) for i in range(n.value)]

    def truncate(self, seq_id: int, num_tokens: int) -> None:
        """Keep the sequence's first num_tokens tokens; blocks past them lose its reference."""
        _check("pkv_alloc_truncate", self._lib.pkv_alloc_truncate(self._h, seq_id, num_tokens))

    def free_seq(self, seq_id: int) -> None:
        _check("pkv_alloc_free_seq", self._lib.pkv_alloc_free_seq(self._h, seq_id))

    def block_table(self, seq_ids, max_blocks: int) -> torch.Tensor:
        ids = (ctypes.c_int64 * len(seq_ids))(*seq_ids)
        out = torch.empty((len(seq_ids), max_blocks), dtype=torch.int32, device="cpu")
        _check("pkv_alloc_block_table", self._lib.pkv_alloc_block_table(
            self._h, ids, len(seq_ids),
            ctypes.cast(out.data_ptr(), ctypes.POINTER(ctypes.c_int32)), max_blocks))
        return out

    @property
    def num_free(self) -> int:
        return int(self._lib.pkv_alloc_num_free(self._h))

    def refcount(self, block: int) -> int:
        return int(self._lib.pkv_alloc_refcount(self._h, block))

    def seq_len(self, seq_id: int) -> int:
        return int(self._lib.pkv_alloc_seq_len(self._h, seq_id))

    def seq_num_blocks(self, seq_id: int) -> int:
        return int(self._lib.pkv_alloc_seq_num_blocks(self._h, seq_id))


def _i32(values):
    """Token ids as a contiguous int32 buffer for the C ABI: (pointer, count).  A numpy
    conversion, not an element-by-element ctypes array (the pointer keeps its buffer
    alive for the call)."""
    a = np.ascontiguousarray(values, dtype=np.int32).reshape(-1)
    n = int(a.size)
    if n == 0:
        a = np.zeros(1, dtype=np.int32)
    return a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n


def block_hash(parent_hash: int, salt: int, tokens, extra: int = 0) -> int:
    arr, n = _i32(tokens)
    return int(_load().pkv_block_hash(parent_hash, salt, arr, n, extra))


class PrefixCache:
    """Chained block-hash prefix cache (libpkv pkv_pcache) over a BlockAllocator."""

    def __init__(self, alloc: BlockAllocator):
        self._lib = _load()
        self.alloc = alloc
        self._h = self._lib.pkv_pcache_create(alloc._h)

    def close(self):
        if self._h:
            self._lib.pkv_pcache_destroy(self._h)
            self._h = None

    def match(self, tokens, salt: int = 0) -> list:
        arr, n = _i32(tokens)
        out = (ctypes.c_int32 * max(n // self.alloc.block_size, 1))()
        k = self._lib.pkv_pcache_match(self._h, arr, n, salt, out, n // self.alloc.block_size)
        if k < 0:
            raise ValueError("pkv_pcache_match: bad arguments")
        return list(out[:k])

    def insert(self, seq_id: int, tokens, salt: int = 0) -> int:
        arr, n = _i32(tokens)
        k = self._lib.pkv_pcache_insert(self._h, seq_id, arr, n, salt)
        if k < 0:
            raise ValueError("pkv_pcache_insert: unknown sequence or too few tokens")
        return k

    def evict(self, min_free: int) -> int:
        return int(self._lib.pkv_pcache_evict(self._h, min_free))

    def __len__(self):
        return int(self._lib.pkv_pcache_size(self._h))


class RadixTree:
    """Radix tree of token sequences (libpkv pkv_radix) over a BlockAllocator."""

    def __init__(self, alloc: BlockAllocator):
        self._lib = _load()
        self.alloc = alloc
        self._h = self._lib.pkv_radix_create(alloc._h)

    def close(self):
        if self._h:
            self._lib.pkv_radix_destroy(self._h)
            self._h = None

    def match(self, tokens):
        """(matched token count, blocks of the matched positions)."""
        arr, n = _i32(tokens)
        nb = -(-n // self.alloc.block_size)
        out = (ctypes.c_int32 * max(nb, 1))()
        m = int(self._lib.pkv_radix_match(self._h, arr, n, out, nb))
        if m < 0:
            raise ValueError("pkv_radix_match: bad arguments")
        return m, list(out[:-(-m // self.alloc.block_size)])

    def insert(self, seq_id: int, tokens) -> None:
        arr, n = _i32(tokens)
        _check("pkv_radix_insert", self._lib.pkv_radix_insert(self._h, seq_id, arr, n))

    def lock(self, tokens, delta: int = 1) -> None:
        arr, n = _i32(tokens)
        _check("pkv_radix_lock", self._lib.pkv_radix_lock(self._h, arr, n, delta))

    def evict(self, min_free: int) -> int:
        return int(self._lib.pkv_radix_evict(self._h, min_free))

    @property
    def num_nodes(self) -> int:
        return int(self._lib.pkv_radix_num_nodes(self._h))

    @property
    def cached_tokens(self) -> int:
        return int(self._lib.pkv_radix_cached_tokens(self._h))
