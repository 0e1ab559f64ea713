"""paged_kv_cache_93_gb300 -- paged KV-cache decode attention on GB300.

A thin binding over libpkv.so (include/pkv.h).  Every function here only
marshals torch tensors (device pointers, shapes, the current CUDA stream)
into one C call; all arithmetic runs in the library's CUDA kernels.  Outputs
that the caller does not pass are allocated with torch.

Layouts (one layer): k_pool [num_blocks, Hkv, block_size, Dk] bf16,
v_pool [num_blocks, Hkv, block_size, Dv] bf16, block_tables [B, max_blocks]
int32, seq_lens [B] int32, q [B, Hq, Dk] fp32, out [B, Hq, Dv] fp32,
lse [B, Hq] fp32 (natural log).  An FP8 cache holds E4M3 codes in uint8
pools of the same shapes, with fp32 dequantisation scales per KV head
(the *_e4m3 functions).
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _lib
from ._lib import (DECODE_GENERIC, DECODE_NO_TCGEN05, DECODE_TEST_WITHHOLD, DEV_BLOCK_ID,
                   DEV_COPY_CONFLICT, DEV_PREFIX, DEV_SEQ_LEN, DEV_SLOT, DEV_TABLE_RANGE,
                   DEV_QUERY_RANGE, DEV_TIMEOUT, ROPE_INTERLEAVED, ROPE_Q_FP32, CacheDesc,
                   PkvError)

__all__ = [
    "CacheDesc", "PkvError", "ValuesInKeys", "cache_desc", "kv_append", "slot_mapping", "copy_blocks",
    "interleave_slot_mapping", "interleave_partition_len", "decode_workspace_size",
    "decode_auto_splits", "paged_decode_attn", "paged_decode_attn_partial",
    "paged_decode_attn_multi", "lse_merge", "kv_append_e4m3", "copy_blocks_e4m3",
    "paged_decode_attn_e4m3", "paged_decode_attn_partial_e4m3", "paged_decode_attn_multi_e4m3",
    "paged_decode_attn_cascade",
    "decode_cascade_splits", "DEV_PREFIX", "rope_frequencies", "rope_append", "rope_append_e4m3",
    "chunk_workspace_size", "paged_chunk_attn", "paged_chunk_attn_e4m3", "DEV_QUERY_RANGE",
    "ROPE_INTERLEAVED", "ROPE_Q_FP32",
    "device_status", "BlockManager", "library_path", "DECODE_GENERIC", "DECODE_NO_TCGEN05",
    "DECODE_TEST_WITHHOLD", "DEV_BLOCK_ID",
    "DEV_SLOT", "DEV_SEQ_LEN", "DEV_COPY_CONFLICT", "DEV_TIMEOUT", "DEV_TABLE_RANGE",
]

lib = _lib.load()
library_path = _lib.LIB_PATH


def _check(where: str, status: int) -> None:
    if status != _lib.PKV_OK:
        raise PkvError(where, status, lib.pkv_status_string(status).decode())


def _ptr(t: torch.Tensor | None):
    # (a plain address: ctypes converts it for a c_void_p argument at a third of
    # the cost of building the object here)
    return None if t is None else t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    # the current stream's handle, without the Stream object around it
    return _raw_stream(torch.cuda.current_device())


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, dim: int | None = None):
    if t.dtype is dtype and t.is_cuda and t.is_contiguous() and (dim is None or t.dim() == dim):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {t.dim()}")


def _int32(x) -> int:
    """x as a 32-bit argument: past 2^31 - 1 it is that, negative -1 (ctypes would wrap
    it around)."""
    return max(-1, min(int(x), 2 ** 31 - 1))


class ValuesInKeys:
    """Pass as `v_pool` when the cache keeps no separate value pool: the value
    of a token is the first `head_dim_v` dims of its key row (the latent
    layout of multi-head latent attention).  Marshalled as a NULL v_pool."""

    def __init__(self, head_dim_v: int):
        self.head_dim_v = int(head_dim_v)


def _v_ptr(v_pool):
    return None if isinstance(v_pool, ValuesInKeys) else _ptr(v_pool)


def cache_desc(k_pool: torch.Tensor, v_pool) -> CacheDesc:
    """Shape of a bf16 cache, or of an E4M3 one (uint8 code pools)."""
    dtype = torch.uint8 if k_pool.dtype == torch.uint8 else torch.bfloat16
    _need(k_pool, "k_pool", dtype, 4)
    nb, hkv, bs, dk = k_pool.shape
    if isinstance(v_pool, ValuesInKeys):
        if dtype != torch.bfloat16:
            raise ValueError("values inside the keys need a bf16 cache")
        if not 0 < v_pool.head_dim_v <= dk:
            raise ValueError("values inside the keys need 0 < head_dim_v <= head_dim_k")
        return CacheDesc(nb, bs, hkv, dk, v_pool.head_dim_v)
    _need(v_pool, "v_pool", dtype, 4)
    if tuple(v_pool.shape[:3]) != (nb, hkv, bs):
        raise ValueError("k_pool and v_pool disagree on [num_blocks, Hkv, block_size]")
    return CacheDesc(nb, bs, hkv, dk, v_pool.shape[3])


def _bf16_desc(k_pool: torch.Tensor, v_pool) -> CacheDesc:
    """cache_desc for the calls that take bf16 pools only (the C calls size
    every row from the element count at two bytes an element, so a code pool
    given to them would be read and written past its end)."""
    _need(k_pool, "k_pool", torch.bfloat16, 4)
    return cache_desc(k_pool, v_pool)


def device_status(reset: bool = True, stream=None) -> int:
    """Synchronize `stream` and return the device status word (PKV_DEV_* bits)."""
    flags = ctypes.c_uint32(0)
    _check("pkv_device_status", lib.pkv_device_status(ctypes.byref(flags), int(reset),
                                                      _stream(stream)))
    return int(flags.value)


def slot_mapping(k_pool, v_pool, block_tables, seq_ids, positions, out=None, stream=None):
    """Slots of (sequence, position) pairs through the block tables (int64 [T])."""
    desc = cache_desc(k_pool, v_pool)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_ids, "seq_ids", torch.int32, 1)
    _need(positions, "positions", torch.int64, 1)
    T = positions.numel()
    if out is None:
        out = torch.empty(T, dtype=torch.int64, device=positions.device)
    _check("pkv_slot_mapping", lib.pkv_slot_mapping(
        ctypes.byref(desc), _ptr(block_tables), block_tables.shape[0], block_tables.shape[1],
        _ptr(seq_ids), _ptr(positions), T, _ptr(out), _stream(stream)))
    return out


def kv_append(k_pool, v_pool, k_new, v_new, slots, stream=None) -> None:
    """Write k_new [T, Hkv, Dk] / v_new [T, Hkv, Dv] (bf16) at slots [T] (int64).
    With v_pool = ValuesInKeys(Dv), v_new must be None (only K is written)."""
    desc = _bf16_desc(k_pool, v_pool)
    _need(k_new, "k_new", torch.bfloat16, 3)
    if isinstance(v_pool, ValuesInKeys):
        if v_new is not None:
            raise ValueError("v_new must be None when the values are inside the keys")
    else:
        _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slots, "slot_mapping", torch.int64, 1)
    _check("pkv_kv_append", lib.pkv_kv_append(
        ctypes.byref(desc), _ptr(k_pool), _v_ptr(v_pool), _ptr(k_new), _ptr(v_new),
        _ptr(slots), slots.numel(), _stream(stream)))


def copy_blocks(k_pool, v_pool, src, dst, stream=None) -> None:
    """Copy-on-write duplication: block src[i] -> block dst[i] (int32 device
    arrays), bf16 pools (copy_blocks_e4m3 for code pools)."""
    desc = _bf16_desc(k_pool, v_pool)
    _need(src, "src", torch.int32, 1)
    _need(dst, "dst", torch.int32, 1)
    if src.numel() != dst.numel():
        raise ValueError("src and dst lengths differ")
    _check("pkv_copy_blocks", lib.pkv_copy_blocks(
        ctypes.byref(desc), _ptr(k_pool), _v_ptr(v_pool), _ptr(src), _ptr(dst), src.numel(),
        _stream(stream)))


def _e4m3_desc(k_pool, v_pool, k_scale, v_scale) -> CacheDesc:
    _need(k_pool, "k_pool", torch.uint8, 4)
    desc = cache_desc(k_pool, v_pool)
    _need(k_scale, "k_scale", torch.float32, 1)
    _need(v_scale, "v_scale", torch.float32, 1)
    if k_scale.numel() != desc.num_kv_heads or v_scale.numel() != desc.num_kv_heads:
        raise ValueError("k_scale and v_scale hold one scale per KV head")
    return desc


def kv_append_e4m3(k_pool, v_pool, k_new, v_new, slots, k_scale, v_scale, stream=None) -> None:
    """Quantise k_new / v_new (bf16 [T, Hkv, D]) into the E4M3 pools at slots
    [T]: element x of KV head g becomes the code nearest to x / scale[g]."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slots, "slot_mapping", torch.int64, 1)
    _check("pkv_kv_append_e4m3", lib.pkv_kv_append_e4m3(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(k_new), _ptr(v_new),
        _ptr(k_scale), _ptr(v_scale), _ptr(slots), slots.numel(), _stream(stream)))


def copy_blocks_e4m3(k_pool, v_pool, src, dst, stream=None) -> None:
    """copy_blocks for E4M3 pools."""
    _need(k_pool, "k_pool", torch.uint8, 4)
    desc = cache_desc(k_pool, v_pool)
    _need(src, "src", torch.int32, 1)
    _need(dst, "dst", torch.int32, 1)
    if src.numel() != dst.numel():
        raise ValueError("src and dst lengths differ")
    _check("pkv_copy_blocks_e4m3", lib.pkv_copy_blocks_e4m3(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(src), _ptr(dst), src.numel(),
        _stream(stream)))


def rope_frequencies(rotary_dim: int, theta: float = 10000.0, factor: float = 1.0,
                     original_len: float = 0, low_turns: float = 1.0, high_turns: float = 4.0,
                     device=None) -> torch.Tensor:
    """Radians per token of each rotary pair, [rotary_dim / 2] float64:
    theta^(-2i / rotary_dim), divided by `factor` (positions interpolated), or
    with original_len > 0 scaled by parts (pairs of at least high_turns turns
    within original_len keep their frequency, those of low_turns or fewer are
    divided by `factor`, linear between)."""
    host = torch.empty(max(0, int(rotary_dim) // 2), dtype=torch.float64)
    _check("pkv_rope_frequencies", lib.pkv_rope_frequencies(
        int(rotary_dim), float(theta), float(factor), float(original_len), float(low_turns),
        float(high_turns), _ptr(host)))
    return host.to("cuda" if device is None else device)


def _rope_args(desc, v_pool, q, k_new, v_new, positions, slots, inv_freq, interleaved, q_dtype,
               q_out, stream):
    """Checks of the rope_append calls -> (q_out, flags)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(positions, "positions", torch.int64, 1)
    _need(slots, "slot_mapping", torch.int64, 1)
    _need(inv_freq, "inv_freq", torch.float64, 1)
    T = positions.numel()
    Tq, Hq, Dk = q.shape
    if slots.numel() != T or Tq != T:
        raise ValueError("q, positions and slots disagree on the number of tokens")
    if Dk != desc.head_dim_k:
        raise ValueError(f"q must have head dim {desc.head_dim_k}, got {Dk}")
    if k_new.shape != (T, desc.num_kv_heads, Dk):
        raise ValueError("k_new must be [tokens, Hkv, Dk] of the cache")
    if isinstance(v_pool, ValuesInKeys):
        if v_new is not None:
            raise ValueError("v_new must be None when the values are inside the keys")
    else:
        _need(v_new, "v_new", torch.bfloat16, 3)
        if v_new.shape != (T, desc.num_kv_heads, desc.head_dim_v):
            raise ValueError("v_new must be [tokens, Hkv, Dv] of the cache")
    if q_out is None:
        if q_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"q_dtype must be torch.bfloat16 or torch.float32, got {q_dtype}")
        if stream is None:
            q_out = torch.empty_like(q, dtype=q_dtype)
        else:                    # it is written on that stream: let it belong to it
            with torch.cuda.stream(stream):
                q_out = torch.empty_like(q, dtype=q_dtype)
    else:
        if q_out.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"q_out must be torch.bfloat16 or torch.float32, got {q_out.dtype}")
        _need(q_out, "q_out", q_out.dtype, 3)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
    flags = (ROPE_INTERLEAVED if interleaved else 0) | \
        (ROPE_Q_FP32 if q_out.dtype == torch.float32 else 0)
    return q_out, flags


def rope_append(k_pool, v_pool, q, k_new, v_new, positions, slots, inv_freq,
                interleaved: bool = False, rotary_offset: int = 0, amplitude: float = 1.0,
                q_dtype: torch.dtype = torch.bfloat16, q_out=None, stream=None):
    """Rotate q [T, Hq, Dk] and k_new [T, Hkv, Dk] (bf16) by their tokens'
    positions [T] (int64; negative: padding, skipped) and write k_new and
    v_new [T, Hkv, Dv] at slots [T] -> the rotated q (bf16, or fp32 as the
    decode calls take it; q_out may be q itself).  inv_freq: [rotary_dim / 2]
    float64 radians per token (see rope_frequencies); pairs are the halves of
    the rotary part, or neighbours with `interleaved`; amplitude multiplies the
    rotary part."""
    desc = _bf16_desc(k_pool, v_pool)
    q_out, flags = _rope_args(desc, v_pool, q, k_new, v_new, positions, slots, inv_freq,
                              interleaved, q_dtype, q_out, stream)
    _check("pkv_rope_append", lib.pkv_rope_append(
        ctypes.byref(desc), _ptr(k_pool), _v_ptr(v_pool), _ptr(q), q.shape[1], _ptr(k_new),
        _ptr(v_new), _ptr(positions), _ptr(slots), positions.numel(), _ptr(inv_freq),
        2 * inv_freq.numel(), _int32(rotary_offset), float(amplitude), flags, _ptr(q_out),
        _stream(stream)))
    return q_out


def rope_append_e4m3(k_pool, v_pool, q, k_new, v_new, positions, slots, inv_freq, k_scale,
                     v_scale, interleaved: bool = False, rotary_offset: int = 0,
                     amplitude: float = 1.0, q_dtype: torch.dtype = torch.bfloat16, q_out=None,
                     stream=None):
    """rope_append into E4M3 pools (uint8 codes, fp32 scales per KV head)."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    q_out, flags = _rope_args(desc, v_pool, q, k_new, v_new, positions, slots, inv_freq,
                              interleaved, q_dtype, q_out, stream)
    _check("pkv_rope_append_e4m3", lib.pkv_rope_append_e4m3(
        ctypes.byref(desc), _ptr(k_pool), _ptr(v_pool), _ptr(q), q.shape[1], _ptr(k_new),
        _ptr(v_new), _ptr(k_scale), _ptr(v_scale), _ptr(positions), _ptr(slots),
        positions.numel(), _ptr(inv_freq), 2 * inv_freq.numel(), _int32(rotary_offset),
        float(amplitude), flags, _ptr(q_out), _stream(stream)))
    return q_out


def interleave_slot_mapping(k_pool, v_pool, first_token: int, num_tokens: int, num_parts: int,
                            interleave: int, part_block_tables, out=None, part_out=None,
                            stream=None):
    """Slots of tokens first_token.. in their DCP partition's table (int64 [T])."""
    desc = cache_desc(k_pool, v_pool)
    _need(part_block_tables, "part_block_tables", torch.int32, 2)
    if out is None:
        out = torch.empty(num_tokens, dtype=torch.int64, device=part_block_tables.device)
    _check("pkv_interleave_slot_mapping", lib.pkv_interleave_slot_mapping(
        ctypes.byref(desc), int(first_token), int(num_tokens), int(num_parts), int(interleave),
        _ptr(part_block_tables), part_block_tables.shape[1], _ptr(out), _ptr(part_out),
        _stream(stream)))
    return out


def interleave_partition_len(num_tokens: int, num_parts: int, interleave: int, part: int) -> int:
    n = lib.pkv_interleave_partition_len(int(num_tokens), int(num_parts), int(interleave),
                                         int(part))
    if n < 0:
        raise ValueError("invalid interleave arguments")
    return int(n)


def decode_workspace_size(batch: int, num_q_heads: int, head_dim_v: int, num_splits: int) -> int:
    return int(lib.pkv_decode_workspace_size(batch, num_q_heads, head_dim_v, num_splits))


def decode_auto_splits(k_pool, v_pool, batch: int, num_q_heads: int, max_seq_len: int) -> int:
    desc = _bf16_desc(k_pool, v_pool)
    return int(lib.pkv_decode_auto_splits(ctypes.byref(desc), batch, num_q_heads, max_seq_len))


def _decode_common(q, k_pool, v_pool, block_tables, seq_lens):
    desc = _bf16_desc(k_pool, v_pool)
    _need(q, "q", torch.float32, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    return desc


def paged_decode_attn(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                      num_splits: int = 0, workspace=None, out=None, lse=None, flags: int = 0,
                      stream=None):
    """Decode attention of q [B, Hq, Dk] over the paged cache -> (out, lse)."""
    desc = _decode_common(q, k_pool, v_pool, block_tables, seq_lens)
    B, Hq, _ = q.shape
    if out is None:
        out = torch.empty(B, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    S = num_splits
    if S == 0:
        S = int(lib.pkv_decode_auto_splits(ctypes.byref(desc), B, Hq,
                                           block_tables.shape[1] * desc.block_size))
    need = decode_workspace_size(B, Hq, desc.head_dim_v, S)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pkv_paged_decode_attn", lib.pkv_paged_decode_attn(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_pool), _v_ptr(v_pool), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), float(scale), S, _ptr(workspace), ws_bytes,
        _ptr(out), _ptr(lse), int(flags), _stream(stream)))
    return out, lse


def decode_cascade_splits(k_pool, v_pool, batch: int, num_q_heads: int, max_blocks: int,
                          prefix_blocks: int, prefix_splits: int = 0,
                          suffix_splits: int = 0) -> tuple[int, int]:
    """The (prefix, suffix) split counts a cascade call uses (0 = chosen)."""
    desc = _bf16_desc(k_pool, v_pool)
    s1, s2 = ctypes.c_int32(prefix_splits), ctypes.c_int32(suffix_splits)
    _check("pkv_decode_cascade_splits", lib.pkv_decode_cascade_splits(
        ctypes.byref(desc), batch, num_q_heads, max_blocks, prefix_blocks, ctypes.byref(s1),
        ctypes.byref(s2)))
    return int(s1.value), int(s2.value)


def paged_decode_attn_cascade(q, k_pool, v_pool, prefix_table, block_tables, seq_lens,
                              scale: float, prefix_splits: int = 0, suffix_splits: int = 0,
                              workspace=None, out=None, lse=None, flags: int = 0, stream=None):
    """Decode attention of q [B, Hq, Dk] for sequences whose tables begin with
    the shared blocks `prefix_table` [prefix_blocks] int32 -> (out, lse), as a
    cascade: all rows over the shared prefix, each sequence over its rest,
    merged.  Same result as paged_decode_attn on those tables."""
    desc = _decode_common(q, k_pool, v_pool, block_tables, seq_lens)
    _need(prefix_table, "prefix_table", torch.int32, 1)
    B, Hq, _ = q.shape
    if out is None:
        out = torch.empty(B, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    P, mb = prefix_table.shape[0], block_tables.shape[1]
    need = int(lib.pkv_decode_cascade_workspace_size(ctypes.byref(desc), B, Hq, mb, P,
                                                     int(prefix_splits), int(suffix_splits)))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("pkv_paged_decode_attn_cascade", lib.pkv_paged_decode_attn_cascade(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_pool), _v_ptr(v_pool), _ptr(prefix_table), P,
        _ptr(block_tables), mb, _ptr(seq_lens), float(scale), int(prefix_splits),
        int(suffix_splits), _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse), int(flags),
        _stream(stream)))
    return out, lse


def paged_decode_attn_e4m3(q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                           scale: float, num_splits: int = 0, workspace=None, out=None,
                           lse=None, flags: int = 0, stream=None):
    """Decode attention over an E4M3 cache (uint8 code pools, fp32 scales per
    KV head) -> (out, lse); num_splits 0 lets the library choose."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    _need(q, "q", torch.float32, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, _ = q.shape
    if out is None:
        out = torch.empty(B, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, Hq, dtype=torch.float32, device=q.device)
    S = num_splits or int(lib.pkv_decode_auto_splits_e4m3(
        ctypes.byref(desc), B, Hq, block_tables.shape[1] * desc.block_size))
    need = decode_workspace_size(B, Hq, desc.head_dim_v, S)
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("pkv_paged_decode_attn_e4m3", lib.pkv_paged_decode_attn_e4m3(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), float(scale),
        S, _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse), int(flags), _stream(stream)))
    return out, lse


def paged_decode_attn_partial_e4m3(q, k_pool, v_pool, k_scale, v_scale, block_tables,
                                   seq_lens, scale: float, num_splits: int, out_part=None,
                                   lse_part=None, flags: int = 0, stream=None):
    """Per-split partials over an E4M3 cache -> (out_part [S, B, Hq, Dv],
    lse_part [S, B, Hq])."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    _need(q, "q", torch.float32, 3)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, _ = q.shape
    S = int(num_splits)
    if out_part is None:
        out_part = torch.empty(S, B, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty(S, B, Hq, dtype=torch.float32, device=q.device)
    _check("pkv_paged_decode_attn_partial_e4m3", lib.pkv_paged_decode_attn_partial_e4m3(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), float(scale),
        S, _ptr(out_part), _ptr(lse_part), int(flags), _stream(stream)))
    return out_part, lse_part


def paged_decode_attn_multi_e4m3(q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                                 scale: float, num_splits: int = 0, workspace=None, out=None,
                                 lse=None, flags: int = 0, stream=None):
    """The multi-token step (q [B, T, Hq, Dk], causal over the last T tokens) over
    an E4M3 cache -> (out [B, T, Hq, Dv], lse [B, T, Hq])."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    _need(q, "q", torch.float32, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, T, Hq, _ = q.shape
    if out is None:
        out = torch.empty(B, T, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, Hq, dtype=torch.float32, device=q.device)
    S = num_splits or int(lib.pkv_decode_multi_auto_splits_e4m3(
        ctypes.byref(desc), B, T, Hq, block_tables.shape[1] * desc.block_size))
    need = int(lib.pkv_decode_multi_workspace_size(B, T, Hq, desc.head_dim_v,
                                                   block_tables.shape[1], S))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check("pkv_paged_decode_attn_multi_e4m3", lib.pkv_paged_decode_attn_multi_e4m3(
        ctypes.byref(desc), _ptr(q), B, T, Hq, _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), float(scale),
        S, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        int(flags), _stream(stream)))
    return out, lse


def paged_decode_attn_partial(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                              num_splits: int, out_part=None, lse_part=None, flags: int = 0,
                              stream=None):
    """Per-split partials -> (out_part [S, B, Hq, Dv], lse_part [S, B, Hq])."""
    desc = _decode_common(q, k_pool, v_pool, block_tables, seq_lens)
    B, Hq, _ = q.shape
    S = int(num_splits)
    if out_part is None:
        out_part = torch.empty(S, B, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse_part is None:
        lse_part = torch.empty(S, B, Hq, dtype=torch.float32, device=q.device)
    _check("pkv_paged_decode_attn_partial", lib.pkv_paged_decode_attn_partial(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_pool), _v_ptr(v_pool), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), float(scale), S, _ptr(out_part), _ptr(lse_part),
        int(flags), _stream(stream)))
    return out_part, lse_part


def paged_decode_attn_multi(q, k_pool, v_pool, block_tables, seq_lens, scale: float,
                            num_splits: int = 0, workspace=None, out=None, lse=None,
                            flags: int = 0, stream=None):
    """Several new tokens per sequence (q [B, T, Hq, Dk]); query t attends to
    the first seq_lens[b] - T + 1 + t tokens -> (out [B, T, Hq, Dv], lse [B, T, Hq])."""
    desc = _bf16_desc(k_pool, v_pool)
    _need(q, "q", torch.float32, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, T, Hq, _ = q.shape
    if out is None:
        out = torch.empty(B, T, Hq, desc.head_dim_v, dtype=torch.float32, device=q.device)
    if lse is None:
        lse = torch.empty(B, T, Hq, dtype=torch.float32, device=q.device)
    S = num_splits
    if S == 0:
        S = int(lib.pkv_decode_multi_auto_splits(ctypes.byref(desc), B, T, Hq,
                                                 block_tables.shape[1] * desc.block_size,
                                                 int(flags)))
    need = int(lib.pkv_decode_multi_workspace_size(B, T, Hq, desc.head_dim_v,
                                                   block_tables.shape[1], S))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check("pkv_paged_decode_attn_multi", lib.pkv_paged_decode_attn_multi(
        ctypes.byref(desc), _ptr(q), B, T, Hq, _ptr(k_pool), _v_ptr(v_pool),
        _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), float(scale), S,
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
        int(flags), _stream(stream)))
    return out, lse


def chunk_workspace_size(k_pool, v_pool, num_tokens: int, batch: int, num_q_heads: int,
                         max_blocks: int, flags: int = 0) -> int:
    """Workspace bytes of paged_chunk_attn (bf16 pools) or paged_chunk_attn_e4m3."""
    desc = cache_desc(k_pool, v_pool)
    size = (lib.pkv_chunk_workspace_size_e4m3 if k_pool.dtype == torch.uint8
            else lib.pkv_chunk_workspace_size)
    return int(size(ctypes.byref(desc), num_tokens, batch, num_q_heads, max_blocks, int(flags)))


# Workspaces of the chunk attention calls that bring none, or one that is too
# small: one for each thread, device and stream that the kernels run on, kept, as
# a thread's calls on a stream follow one another (two threads' kernels may
# interleave).  A capture gets one of its own (graphs may run beside anything).
_chunk_scratch = threading.local()


def _chunk_args(desc, size, q, cu_q_lens, block_tables, seq_lens, workspace, out, lse, flags,
                stream):
    """Checks of the chunk attention calls -> (workspace, its bytes, out, lse)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(cu_q_lens, "cu_q_lens", torch.int32, 1)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    T, Hq, Dk = q.shape
    B = seq_lens.numel()
    Dv = desc.head_dim_v
    if Dk != desc.head_dim_k:
        raise ValueError(f"q must have head dim {desc.head_dim_k}, got {Dk}")
    if cu_q_lens.numel() != B + 1 or block_tables.shape[0] != B:
        raise ValueError("cu_q_lens must have one entry more, block_tables one row per seq_len")
    if workspace is not None:
        _need(workspace, "workspace", workspace.dtype)
    need = size(ctypes.byref(desc), T, B, Hq, block_tables.shape[1], flags)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if stream is not None and (out is None or lse is None or ws_bytes < need):
        # what is allocated or looked up here is used on that stream: let it belong to it
        with torch.cuda.stream(stream):
            return _chunk_args(desc, size, q, cu_q_lens, block_tables, seq_lens, workspace, out,
                               lse, flags, None)
    if out is None:
        out = torch.empty((T, Hq, Dv), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, "out", torch.bfloat16, 3)
        if out.shape != (T, Hq, Dv):
            raise ValueError("out must be [tokens, Hq, Dv]")
    if lse is None:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", torch.float32, 2)
        if lse.shape != (T, Hq):
            raise ValueError("lse must be [tokens, Hq]")
    if ws_bytes < need:
        if torch.cuda.is_current_stream_capturing():
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            kept = _chunk_scratch.__dict__
            key = (q.device.index, _stream())
            workspace = kept.get(key)
            if workspace is None or workspace.numel() < need:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
                kept[key] = workspace
        ws_bytes = workspace.numel()
    return workspace, ws_bytes, out, lse


def paged_chunk_attn(q, cu_q_lens, k_pool, v_pool, block_tables, seq_lens, scale: float,
                     window: int = 0, sink_tokens: int = 0, workspace=None, out=None, lse=None,
                     flags: int = 0, stream=None):
    """Attention of ragged chunks of new tokens over the paged cache.

    q [T, Hq, Dk] bf16 holds the chunks one after another: sequence b's are
    rows cu_q_lens[b] .. cu_q_lens[b + 1] (int32 [B + 1]), the last tokens of
    its seq_lens[b] stored ones.  Causal; with window > 0 a token sees the last
    `window` positions (its own among them) and the first `sink_tokens`.
    -> (out [T, Hq, Dv] bf16, lse [T, Hq] fp32); rows past the last sequence
    are left as they were."""
    desc = _bf16_desc(k_pool, v_pool)
    workspace, ws_bytes, out, lse = _chunk_args(
        desc, lib.pkv_chunk_workspace_size, q, cu_q_lens, block_tables, seq_lens, workspace, out,
        lse, int(flags), stream)
    _check("pkv_paged_chunk_attn", lib.pkv_paged_chunk_attn(
        ctypes.byref(desc), _ptr(q), q.shape[0], q.shape[1], _ptr(cu_q_lens), seq_lens.numel(),
        _ptr(k_pool), _v_ptr(v_pool), _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens),
        float(scale), _int32(window), _int32(sink_tokens), _ptr(workspace), ws_bytes, _ptr(out),
        _ptr(lse), int(flags), _stream(stream)))
    return out, lse


def paged_chunk_attn_e4m3(q, cu_q_lens, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens,
                          scale: float, window: int = 0, sink_tokens: int = 0, workspace=None,
                          out=None, lse=None, flags: int = 0, stream=None):
    """paged_chunk_attn over an E4M3 cache (uint8 code pools, fp32 scales per
    KV head) -> (out, lse)."""
    desc = _e4m3_desc(k_pool, v_pool, k_scale, v_scale)
    workspace, ws_bytes, out, lse = _chunk_args(
        desc, lib.pkv_chunk_workspace_size_e4m3, q, cu_q_lens, block_tables, seq_lens, workspace,
        out, lse, int(flags), stream)
    _check("pkv_paged_chunk_attn_e4m3", lib.pkv_paged_chunk_attn_e4m3(
        ctypes.byref(desc), _ptr(q), q.shape[0], q.shape[1], _ptr(cu_q_lens), seq_lens.numel(),
        _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
        block_tables.shape[1], _ptr(seq_lens), float(scale), _int32(window), _int32(sink_tokens),
        _ptr(workspace), ws_bytes, _ptr(out), _ptr(lse), int(flags), _stream(stream)))
    return out, lse


def lse_merge(out_part, lse_part, out=None, lse=None, stream=None):
    """Merge P partials: out_part [P, ..., Dv], lse_part [P, ...] -> (out, lse)."""
    _need(out_part, "out_part", torch.float32)
    _need(lse_part, "lse_part", torch.float32)
    P, dv = out_part.shape[0], out_part.shape[-1]
    rows = out_part[0].numel() // dv
    if lse_part.numel() != P * rows:
        raise ValueError("lse_part does not match out_part")
    if out is None:
        out = torch.empty(out_part.shape[1:], dtype=torch.float32, device=out_part.device)
    if lse is None:
        lse = torch.empty(lse_part.shape[1:], dtype=torch.float32, device=lse_part.device)
    _check("pkv_lse_merge", lib.pkv_lse_merge(P, _ptr(out_part), _ptr(lse_part), rows, dv,
                                              _ptr(out), _ptr(lse), _stream(stream)))
    return out, lse


class BlockManager:
    """Host block manager (C++): allocation, reuse, ref-counted sharing, copy-on-write."""

    def __init__(self, num_blocks: int, block_size: int, initial_order=None):
        self.block_size = int(block_size)
        arr = None
        if initial_order is not None:
            order = [int(x) for x in initial_order]
            arr = (ctypes.c_int32 * len(order))(*order)
        self._h = lib.pkv_bm_create(int(num_blocks), int(block_size), arr)
        if not self._h:
            raise ValueError("pkv_bm_create: invalid arguments")

    def __del__(self):
        h = getattr(self, "_h", None)
        if h:
            lib.pkv_bm_destroy(h)
            self._h = None

    def add_sequence(self) -> int:
        sid = ctypes.c_int64(0)
        _check("pkv_bm_add_sequence", lib.pkv_bm_add_sequence(self._h, ctypes.byref(sid)))
        return int(sid.value)

    def fork(self, parent: int) -> int:
        sid = ctypes.c_int64(0)
        _check("pkv_bm_fork", lib.pkv_bm_fork(self._h, int(parent), ctypes.byref(sid)))
        return int(sid.value)

    def append(self, seq: int, num_tokens: int):
        """-> (slots list, copy-on-write pairs [(src, dst)])."""
        slots = (ctypes.c_int64 * max(1, num_tokens))()
        src = (ctypes.c_int32 * 1)()
        dst = (ctypes.c_int32 * 1)()
        n = ctypes.c_int32(0)
        _check("pkv_bm_append", lib.pkv_bm_append(self._h, int(seq), int(num_tokens), slots, src,
                                                  dst, 1, ctypes.byref(n)))
        return list(slots[:num_tokens]), [(src[i], dst[i]) for i in range(n.value)]

    def free(self, seq: int) -> None:
        _check("pkv_bm_free", lib.pkv_bm_free(self._h, int(seq)))

    def block_table(self, seq: int):
        nb = ctypes.c_int32(0)
        ln = ctypes.c_int64(0)
        rc = lib.pkv_bm_block_table(self._h, int(seq), None, 0, ctypes.byref(nb), ctypes.byref(ln))
        if rc not in (0, -2):          # -2: capacity 0 too small, sizes still reported
            _check("pkv_bm_block_table", rc)
        buf = (ctypes.c_int32 * max(1, nb.value))()
        _check("pkv_bm_block_table", lib.pkv_bm_block_table(self._h, int(seq), buf, nb.value,
                                                            ctypes.byref(nb), ctypes.byref(ln)))
        return list(buf[:nb.value])

    def seq_len(self, seq: int) -> int:
        nb = ctypes.c_int32(0)
        ln = ctypes.c_int64(0)
        rc = lib.pkv_bm_block_table(self._h, int(seq), None, 0, ctypes.byref(nb), ctypes.byref(ln))
        if rc not in (0, -2):
            _check("pkv_bm_block_table", rc)
        return int(ln.value)

    @property
    def num_free(self) -> int:
        return int(lib.pkv_bm_num_free(self._h))

    def ref_count(self, block: int) -> int:
        return int(lib.pkv_bm_ref_count(self._h, int(block)))
