"""Python entry points with the C ABI's names (include/pagedattn.h).

Each function checks that tensors are on the GPU, contiguous and of the right
integer type, then calls the library on torch's current stream. Shapes and
sizes are validated by the library itself.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from ._lib import DTYPE_CODE, check, lib, ptr, stream_handle


def _dev(t: torch.Tensor, name: str, dtype=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def pa_compute_slot_mapping(query_start_loc: torch.Tensor, positions: torch.Tensor,
                            block_table: torch.Tensor, block_size: int,
                            slot_mapping: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """slot[t] = block_table[r, pos // B] * B + pos % B for the tokens of each
    request r; -1 for tokens of no request. Returns int64 [num_tokens]."""
    _dev(query_start_loc, "query_start_loc", torch.int32)
    _dev(positions, "positions", torch.int64)
    _dev(block_table, "block_table", torch.int32)
    T = positions.numel()
    if slot_mapping is None:
        slot_mapping = torch.empty(T, dtype=torch.int64, device=positions.device)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    stride = block_table.shape[1] if block_table.dim() == 2 else 0
    check("pa_compute_slot_mapping", lib().pa_compute_slot_mapping(
        ptr(query_start_loc), query_start_loc.numel() - 1, ptr(positions), T,
        ptr(block_table), stride, block_size, ptr(slot_mapping), stream_handle(stream)))
    return slot_mapping


def pa_reshape_and_cache(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                         key_cache: torch.Tensor, value_cache: torch.Tensor,
                         stream=None) -> None:
    """Write k[t], v[t] ([T, Hkv, D]) into pool slot slot_mapping[t]; pools are
    [num_blocks, Hkv, B, D]."""
    for n, t in (("k", k), ("v", v), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    NB, Hkv, B, D = key_cache.shape
    if value_cache.shape != key_cache.shape or k.shape != v.shape:
        raise ValueError("shape mismatch")
    if k.shape[1:] != (Hkv, D) or k.dtype != key_cache.dtype:
        raise ValueError("k/v must be [T, Hkv, D] in the cache dtype")
    check("pa_reshape_and_cache", lib().pa_reshape_and_cache(
        ptr(k), ptr(v), k.shape[0], Hkv, D, DTYPE_CODE[k.dtype], ptr(slot_mapping),
        ptr(key_cache), ptr(value_cache), NB, B, stream_handle(stream)))


def pa_decode_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                              head_size: int, block_size: int, max_seq_len: int,
                              partition_size: int = 0) -> int:
    n = lib().pa_decode_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_size,
                                        block_size, max_seq_len, partition_size)
    if n < 0:
        check("pa_decode_workspace_bytes", int(n))
    return int(n)


def pa_decode_partitioning(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                           block_size: int, max_seq_len: int, partition_size: int = 0):
    """(num_splits, partition_tokens) the attention call will use."""
    s, p = ctypes.c_int(0), ctypes.c_int(0)
    check("pa_decode_partitioning", lib().pa_decode_partitioning(
        num_seqs, num_q_heads, num_kv_heads, block_size, max_seq_len, partition_size,
        ctypes.byref(s), ctypes.byref(p)))
    return s.value, p.value


def pa_decode_window_partitioning(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                  block_size: int, max_seq_len: int, window: int,
                                  partition_size: int = 0):
    """(num_splits, partition_tokens) the windowed attention calls will use."""
    s, p = ctypes.c_int(0), ctypes.c_int(0)
    check("pa_decode_window_partitioning", lib().pa_decode_window_partitioning(
        num_seqs, num_q_heads, num_kv_heads, block_size, max_seq_len, window, partition_size,
        ctypes.byref(s), ctypes.byref(p)))
    return s.value, p.value


def pa_decode_fp8_partitioning(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                               head_size: int, block_size: int, dtype: torch.dtype,
                               max_seq_len: int, window: int = 0, partition_size: int = 0):
    """(num_splits, partition_tokens) the fp8-pool attention calls will use;
    dtype is the query type."""
    s, p = ctypes.c_int(0), ctypes.c_int(0)
    check("pa_decode_fp8_partitioning", lib().pa_decode_fp8_partitioning(
        num_seqs, num_q_heads, num_kv_heads, head_size, block_size, DTYPE_CODE[dtype],
        max_seq_len, window, partition_size, ctypes.byref(s), ctypes.byref(p)))
    return s.value, p.value


KV_FORMAT = {"16bit": 0, "fp8": 1, "fp8_block_scales": 2}


def pa_decode_even_ctas(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_size: int,
                        block_size: int, dtype: torch.dtype, kv_format: str, max_seq_len: int,
                        window: int = 0, partition_size: int = 0) -> int:
    """CTAs of the even schedule a decode call with these sizes runs (0: it
    uses fixed partitions); kv_format is "16bit", "fp8" or
    "fp8_block_scales", dtype the query type."""
    n = lib().pa_decode_even_ctas(num_seqs, num_q_heads, num_kv_heads, head_size, block_size,
                                  DTYPE_CODE[dtype], KV_FORMAT[kv_format], max_seq_len, window,
                                  partition_size)
    if n < 0:
        check("pa_decode_even_ctas", int(n))
    return int(n)


def pa_decode_fp8_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                  head_size: int, block_size: int, dtype: torch.dtype,
                                  max_seq_len: int, window: int = 0,
                                  partition_size: int = 0) -> int:
    """Scratch bytes of the fp8-pool decode calls; dtype is the query type."""
    n = lib().pa_decode_fp8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_size,
                                            block_size, DTYPE_CODE[dtype], max_seq_len, window,
                                            partition_size)
    if n < 0:
        check("pa_decode_fp8_workspace_bytes", int(n))
    return int(n)


def pa_decode_attention(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                        block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                        num_kv_heads: int, out: Optional[torch.Tensor] = None, *,
                        max_seq_len: int, partition_size: int = 0,
                        workspace: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """Paged decode attention. q/out [S, Hq, D]; pools [NB, Hkv, B, D];
    block_tables int32 [S, max_blocks]; seq_lens int32 [S]; max_seq_len is a
    host upper bound of seq_lens."""
    for n, t in (("q", q), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = key_cache.shape
    if Hkv != num_kv_heads or Dk != D or value_cache.shape != key_cache.shape:
        raise ValueError("pool shape does not match q / num_kv_heads")
    if key_cache.dtype != q.dtype or value_cache.dtype != q.dtype:
        raise ValueError("q and pools must share a dtype")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out")
    need = pa_decode_workspace_bytes(S, Hq, Hkv, D, B, max_seq_len, partition_size)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention", lib().pa_decode_attention(
        ptr(q), ptr(key_cache), ptr(value_cache), ptr(block_tables), block_tables.shape[1],
        ptr(seq_lens), S, Hq, Hkv, D, B, NB, DTYPE_CODE[q.dtype], float(scale),
        int(max_seq_len), int(partition_size), ptr(out), ptr(workspace), ws_bytes,
        stream_handle(stream)))
    return out


def pa_copy_blocks(key_caches: Sequence[torch.Tensor], value_caches: Sequence[torch.Tensor],
                   src_dst_pairs: torch.Tensor,
                   src_dst_pairs_host: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy whole blocks src -> dst in every layer's K and V pool.
    src_dst_pairs: int64 [P, 2] on the GPU; src_dst_pairs_host: optional CPU
    copy, which enables the aliasing check before launch."""
    if len(key_caches) != len(value_caches) or not key_caches:
        raise ValueError("need one K and one V pool per layer")
    _dev(src_dst_pairs, "src_dst_pairs", torch.int64)
    kc0 = key_caches[0]
    for t in list(key_caches) + list(value_caches):
        _dev(t, "cache")
        if t.shape != kc0.shape or t.dtype != kc0.dtype:
            raise ValueError("all pools must share shape and dtype")
    nl = len(key_caches)
    kp = (ctypes.c_void_p * nl)(*[t.data_ptr() for t in key_caches])
    vp = (ctypes.c_void_p * nl)(*[t.data_ptr() for t in value_caches])
    host = None
    if src_dst_pairs_host is not None:
        host = src_dst_pairs_host.to(torch.int64).contiguous()
        if host.is_cuda or host.numel() != src_dst_pairs.numel():
            raise ValueError("src_dst_pairs_host must be a CPU copy of the pairs")
    NB = kc0.shape[0]
    block_bytes = kc0[0].numel() * kc0.element_size()
    check("pa_copy_blocks", lib().pa_copy_blocks(
        kp, vp, nl, ptr(src_dst_pairs), None if host is None else host.data_ptr(),
        src_dst_pairs.numel() // 2, NB, block_bytes, stream_handle(stream)))


def pa_get_device_error(stream=None) -> int:
    """Synchronise the stream, then read and clear the latched device error
    (0 = none)."""
    code = ctypes.c_int(0)
    check("pa_get_device_error", lib().pa_get_device_error(ctypes.byref(code),
                                                           stream_handle(stream)))
    return code.value


def pa_map_to_kernel_blocks(manager_table: torch.Tensor, blocks_per_kv_block: int,
                            kernel_table: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Expand an int32 [rows, cols] table of allocator block ids (each owning
    r = blocks_per_kv_block kernel blocks) into an int32 [rows, cols * r]
    table of kernel block ids."""
    _dev(manager_table, "manager_table", torch.int32)
    rows, cols = manager_table.shape
    r = int(blocks_per_kv_block)
    if kernel_table is None:
        kernel_table = torch.empty((rows, cols * r), dtype=torch.int32,
                                   device=manager_table.device)
    _dev(kernel_table, "kernel_table", torch.int32)
    check("pa_map_to_kernel_blocks", lib().pa_map_to_kernel_blocks(
        ptr(manager_table), rows, cols, cols, r, ptr(kernel_table), kernel_table.shape[1],
        stream_handle(stream)))
    return kernel_table


def pa_multi_query_workspace_bytes(num_tokens: int, num_seqs: int, num_q_heads: int,
                                   num_kv_heads: int, head_size: int, block_size: int,
                                   max_query_len: int, max_seq_len: int,
                                   partition_size: int = 0) -> int:
    n = lib().pa_multi_query_workspace_bytes(num_tokens, num_seqs, num_q_heads, num_kv_heads,
                                             head_size, block_size, max_query_len,
                                             max_seq_len, partition_size)
    if n < 0:
        check("pa_multi_query_workspace_bytes", int(n))
    return int(n)


def pa_multi_query_attention(q: torch.Tensor, query_start_loc: torch.Tensor,
                             key_cache: torch.Tensor, value_cache: torch.Tensor,
                             block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                             num_kv_heads: int, out: Optional[torch.Tensor] = None, *,
                             max_query_len: int, max_seq_len: int, partition_size: int = 0,
                             workspace: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """Causal paged attention of several new tokens per sequence.
    q/out [T, Hq, D] with T = query_start_loc[-1]; pools [NB, Hkv, B, D]."""
    for n, t in (("q", q), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(query_start_loc, "query_start_loc", torch.int32)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    T, Hq, D = q.shape
    NB, Hkv, B, Dk = key_cache.shape
    if Hkv != num_kv_heads or Dk != D or value_cache.shape != key_cache.shape:
        raise ValueError("pool shape does not match q / num_kv_heads")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out")
    S = query_start_loc.numel() - 1
    need = pa_multi_query_workspace_bytes(T, S, Hq, Hkv, D, B, max_query_len, max_seq_len,
                                          partition_size)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_multi_query_attention", lib().pa_multi_query_attention(
        ptr(q), ptr(query_start_loc), S, T, ptr(key_cache), ptr(value_cache), ptr(block_tables),
        block_tables.shape[1], ptr(seq_lens), Hq, Hkv, D, B, NB, DTYPE_CODE[q.dtype],
        float(scale), int(max_query_len), int(max_seq_len), int(partition_size), ptr(out),
        ptr(workspace), ws_bytes, stream_handle(stream)))
    return out


def pa_reshape_and_cache_fp8(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                             key_cache: torch.Tensor, value_cache: torch.Tensor,
                             k_scale: float, v_scale: float, stream=None) -> None:
    """KV write into E4M3 pools (uint8 [NB, Hkv, B, D]): code = e4m3(x / scale)."""
    for n, t in (("k", k), ("v", v), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    if key_cache.dtype != torch.uint8 or value_cache.dtype != torch.uint8:
        raise ValueError("fp8 pools are uint8 tensors of E4M3 codes")
    NB, Hkv, B, D = key_cache.shape
    check("pa_reshape_and_cache_fp8", lib().pa_reshape_and_cache_fp8(
        ptr(k), ptr(v), k.shape[0], Hkv, D, DTYPE_CODE[k.dtype], ptr(slot_mapping),
        ptr(key_cache), ptr(value_cache), NB, B, float(k_scale), float(v_scale),
        stream_handle(stream)))


def pa_decode_attention_fp8(q: torch.Tensor, key_cache: torch.Tensor, value_cache: torch.Tensor,
                            block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                            num_kv_heads: int, k_scale: float, v_scale: float,
                            out: Optional[torch.Tensor] = None, *, max_seq_len: int,
                            partition_size: int = 0, workspace: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Decode attention over E4M3 pools; q/out in fp32/fp16/bf16."""
    for n, t in (("q", q), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = key_cache.shape
    if Hkv != num_kv_heads or Dk != D or key_cache.dtype != torch.uint8:
        raise ValueError("pools must be uint8 [NB, Hkv, B, D] matching q")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out")
    need = pa_decode_fp8_workspace_bytes(S, Hq, Hkv, D, B, q.dtype, max_seq_len, 0,
                                         partition_size)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention_fp8", lib().pa_decode_attention_fp8(
        ptr(q), ptr(key_cache), ptr(value_cache), ptr(block_tables), block_tables.shape[1],
        ptr(seq_lens), S, Hq, Hkv, D, B, NB, DTYPE_CODE[q.dtype], float(scale), float(k_scale),
        float(v_scale), int(max_seq_len), int(partition_size), ptr(out), ptr(workspace),
        ws_bytes, stream_handle(stream)))
    return out


def pa_reshape_and_cache_fp8_scaled(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
                                    key_cache: torch.Tensor, value_cache: torch.Tensor,
                                    k_scales: torch.Tensor, v_scales: torch.Tensor,
                                    stream=None) -> None:
    """KV write into E4M3 pools whose blocks carry their own scales
    (k_scales / v_scales: float32 [NB, Hkv], updated where this write stores
    a block's first row)."""
    for n, t in (("k", k), ("v", v), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(slot_mapping, "slot_mapping", torch.int64)
    _dev(k_scales, "k_scales", torch.float32)
    _dev(v_scales, "v_scales", torch.float32)
    if key_cache.dtype != torch.uint8 or value_cache.dtype != torch.uint8:
        raise ValueError("fp8 pools are uint8 tensors of E4M3 codes")
    NB, Hkv, B, D = key_cache.shape
    if tuple(k_scales.shape) != (NB, Hkv) or tuple(v_scales.shape) != (NB, Hkv):
        raise ValueError("scales must be float32 [num_blocks, num_kv_heads]")
    check("pa_reshape_and_cache_fp8_scaled", lib().pa_reshape_and_cache_fp8_scaled(
        ptr(k), ptr(v), k.shape[0], Hkv, D, DTYPE_CODE[k.dtype], ptr(slot_mapping),
        ptr(key_cache), ptr(value_cache), ptr(k_scales), ptr(v_scales), NB, B,
        stream_handle(stream)))


def pa_decode_attention_fp8_scaled(q: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, k_scales: torch.Tensor,
                                   v_scales: torch.Tensor, block_tables: torch.Tensor,
                                   seq_lens: torch.Tensor, scale: float, num_kv_heads: int,
                                   out: Optional[torch.Tensor] = None, *, max_seq_len: int,
                                   window: int = 0, partition_size: int = 0,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream=None) -> torch.Tensor:
    """Decode attention over E4M3 pools with per-(block, KV head) scales;
    window 0 attends the whole sequence."""
    for n, t in (("q", q), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    _dev(k_scales, "k_scales", torch.float32)
    _dev(v_scales, "v_scales", torch.float32)
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = key_cache.shape
    if Hkv != num_kv_heads or Dk != D or key_cache.dtype != torch.uint8:
        raise ValueError("pools must be uint8 [NB, Hkv, B, D] matching q")
    if tuple(k_scales.shape) != (NB, Hkv) or tuple(v_scales.shape) != (NB, Hkv):
        raise ValueError("scales must be float32 [num_blocks, num_kv_heads]")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out")
    need = pa_decode_fp8_workspace_bytes(S, Hq, Hkv, D, B, q.dtype, max_seq_len, window,
                                         partition_size)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check("pa_decode_attention_fp8_scaled", lib().pa_decode_attention_fp8_scaled(
        ptr(q), ptr(key_cache), ptr(value_cache), ptr(k_scales), ptr(v_scales),
        ptr(block_tables), block_tables.shape[1], ptr(seq_lens), S, Hq, Hkv, D, B, NB,
        DTYPE_CODE[q.dtype], float(scale), int(window), int(max_seq_len), int(partition_size),
        ptr(out), ptr(workspace), ws_bytes, stream_handle(stream)))
    return out


def pa_decode_window_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int,
                                     head_size: int, block_size: int, max_seq_len: int,
                                     window: int, partition_size: int = 0) -> int:
    n = lib().pa_decode_window_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_size,
                                               block_size, max_seq_len, window, partition_size)
    if n < 0:
        check("pa_decode_window_workspace_bytes", int(n))
    return int(n)


def _window_call(name, q, key_cache, value_cache, block_tables, seq_lens, scale, num_kv_heads,
                 scales, window, out, max_seq_len, partition_size, workspace, stream):
    for n, t in (("q", q), ("key_cache", key_cache), ("value_cache", value_cache)):
        _dev(t, n)
    _dev(block_tables, "block_tables", torch.int32)
    _dev(seq_lens, "seq_lens", torch.int32)
    S, Hq, D = q.shape
    NB, Hkv, B, Dk = key_cache.shape
    pool_dtype = torch.uint8 if scales else q.dtype
    if Hkv != num_kv_heads or Dk != D or value_cache.shape != key_cache.shape:
        raise ValueError("pool shape does not match q / num_kv_heads")
    if key_cache.dtype != pool_dtype or value_cache.dtype != pool_dtype:
        raise ValueError(f"pools must be {pool_dtype}")
    if out is None:
        out = torch.empty_like(q)
    _dev(out, "out")
    if scales:       # fp8 pools: their own partitioning and scratch
        need = pa_decode_fp8_workspace_bytes(S, Hq, Hkv, D, B, q.dtype, max_seq_len, window,
                                             partition_size)
    else:
        need = pa_decode_window_workspace_bytes(S, Hq, Hkv, D, B, max_seq_len, window,
                                                partition_size)
    if need > 0 and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    check(name, getattr(lib(), name)(
        ptr(q), ptr(key_cache), ptr(value_cache), ptr(block_tables), block_tables.shape[1],
        ptr(seq_lens), S, Hq, Hkv, D, B, NB, DTYPE_CODE[q.dtype], float(scale),
        *[float(x) for x in scales], int(window), int(max_seq_len), int(partition_size),
        ptr(out), ptr(workspace), ws_bytes, stream_handle(stream)))
    return out


def pa_decode_attention_window(q: torch.Tensor, key_cache: torch.Tensor,
                               value_cache: torch.Tensor, block_tables: torch.Tensor,
                               seq_lens: torch.Tensor, scale: float, num_kv_heads: int,
                               window: int, out: Optional[torch.Tensor] = None, *,
                               max_seq_len: int, partition_size: int = 0,
                               workspace: Optional[torch.Tensor] = None,
                               stream=None) -> torch.Tensor:
    """Sliding-window decode: each query attends its sequence's last
    `window` tokens (0 = all); table entries of blocks wholly before the
    window are never read."""
    return _window_call("pa_decode_attention_window", q, key_cache, value_cache, block_tables,
                        seq_lens, scale, num_kv_heads, (), window, out, max_seq_len,
                        partition_size, workspace, stream)


def pa_decode_attention_fp8_window(q: torch.Tensor, key_cache: torch.Tensor,
                                   value_cache: torch.Tensor, block_tables: torch.Tensor,
                                   seq_lens: torch.Tensor, scale: float, num_kv_heads: int,
                                   k_scale: float, v_scale: float, window: int,
                                   out: Optional[torch.Tensor] = None, *, max_seq_len: int,
                                   partition_size: int = 0,
                                   workspace: Optional[torch.Tensor] = None,
                                   stream=None) -> torch.Tensor:
    """pa_decode_attention_window over E4M3 pools."""
    return _window_call("pa_decode_attention_fp8_window", q, key_cache, value_cache,
                        block_tables, seq_lens, scale, num_kv_heads, (k_scale, v_scale),
                        window, out, max_seq_len, partition_size, workspace, stream)


def _current() -> tuple:
    """(current device index, its current stream as an integer)."""
    dev = torch._C._cuda_getDevice()
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _refuse(t: torch.Tensor, name: str, dtype, shape, dense: bool):
    """Say what is wrong with t; None if nothing is."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, not on the current device")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _want(dev: int, t: torch.Tensor, name: str, dtype, *shape) -> int:
    """Address of t, which must be a dense tensor of this dtype and shape on
    the current device. A step makes a dozen of these checks, and small steps
    are bound by them: the passing path asks for as little as it can."""
    if (t.get_device() != dev or t.dtype != dtype or t.shape != shape
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, True)
    return t.data_ptr()


def _buffer(t, name, dtype, device, dev, *shape):
    """The caller's output buffer, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _want(dev, t, name, dtype, *shape)
    return t


_I32, _I64, _U8, _F32, _F64 = torch.int32, torch.int64, torch.uint8, torch.float32, torch.float64


def pa_extend_block_tables(context_lens: torch.Tensor, new_tokens: torch.Tensor,
                           block_tables: torch.Tensor, block_size: int, free_ring: torch.Tensor,
                           ring_state: torch.Tensor, num_blocks: int, num_tokens: int, *,
                           ring_state_out: Optional[torch.Tensor] = None,
                           query_start_loc: Optional[torch.Tensor] = None,
                           block_start_loc: Optional[torch.Tensor] = None,
                           seq_lens: Optional[torch.Tensor] = None,
                           positions: Optional[torch.Tensor] = None,
                           slot_mapping: Optional[torch.Tensor] = None, stream=None):
    """Plan a step on the GPU: request r holds context_lens[r] tokens and gets
    new_tokens[r] more (int32 [S]); the blocks it lacks come from the head of
    the free ring (free_ring int32 [R], ring_state int64 {head, tail}) and are
    entered in block_tables (int32 [S, max_blocks]). num_tokens rows (an upper
    bound of the new tokens) of positions and slots are written, padding rows
    with slot -1. ring_state_out defaults to ring_state (in place); seq_lens
    may be context_lens. Returns (query_start_loc, block_start_loc, seq_lens,
    positions, slot_mapping). A step that lacks blocks changes nothing and
    latches PA_ERR_NO_BLOCKS."""
    if not context_lens.is_cuda:
        raise ValueError("context_lens must be a CUDA tensor")
    dev, st = _current()
    S, T, where = context_lens.numel(), int(num_tokens), context_lens.device
    if T < 0:
        raise ValueError("num_tokens must not be negative")
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks]")
    cols, R = block_tables.shape[1], free_ring.numel()
    if ring_state_out is None:
        ring_state_out = ring_state
    if query_start_loc is None:
        query_start_loc = torch.empty(S + 1, dtype=_I32, device=where)
    if block_start_loc is None:
        block_start_loc = torch.empty(S + 1, dtype=_I32, device=where)
    if seq_lens is None:
        seq_lens = torch.empty(S, dtype=_I32, device=where)
    if positions is None:
        positions = torch.empty(T, dtype=_I64, device=where)
    if slot_mapping is None:
        slot_mapping = torch.empty(T, dtype=_I64, device=where)
    check("pa_extend_block_tables", lib().pa_extend_block_tables(
        _want(dev, context_lens, "context_lens", _I32, S),
        _want(dev, new_tokens, "new_tokens", _I32, S), S,
        _want(dev, block_tables, "block_tables", _I32, S, cols), cols, int(block_size),
        int(num_blocks), _want(dev, free_ring, "free_ring", _I32, R), R,
        _want(dev, ring_state, "ring_state", _I64, 2),
        _want(dev, ring_state_out, "ring_state_out", _I64, 2), T,
        _want(dev, query_start_loc, "query_start_loc", _I32, S + 1),
        _want(dev, block_start_loc, "block_start_loc", _I32, S + 1),
        _want(dev, seq_lens, "seq_lens", _I32, S), _want(dev, positions, "positions", _I64, T),
        _want(dev, slot_mapping, "slot_mapping", _I64, T),
        st if stream is None else stream.cuda_stream))
    return query_start_loc, block_start_loc, seq_lens, positions, slot_mapping


def pa_release_block_tables(finished: torch.Tensor, seq_lens: torch.Tensor,
                            block_tables: torch.Tensor, block_size: int,
                            free_ring: torch.Tensor, ring_state: torch.Tensor, num_blocks: int, *,
                            ring_state_out: Optional[torch.Tensor] = None,
                            release_start_loc: Optional[torch.Tensor] = None,
                            seq_lens_out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Return the blocks of finished requests (uint8 or bool [S]) to the tail
    of the free ring and set their lengths to 0. ring_state_out and
    seq_lens_out default to in place. Returns release_start_loc int32 [S + 1]:
    where each request's blocks begin among those returned."""
    if not seq_lens.is_cuda:
        raise ValueError("seq_lens must be a CUDA tensor")
    dev, st = _current()
    S = seq_lens.numel()
    if finished.dtype == torch.bool:
        finished = finished.view(_U8)
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks]")
    cols, R = block_tables.shape[1], free_ring.numel()
    if ring_state_out is None:
        ring_state_out = ring_state
    if seq_lens_out is None:
        seq_lens_out = seq_lens
    if release_start_loc is None:
        release_start_loc = torch.empty(S + 1, dtype=_I32, device=seq_lens.device)
    check("pa_release_block_tables", lib().pa_release_block_tables(
        _want(dev, finished, "finished", _U8, S), _want(dev, seq_lens, "seq_lens", _I32, S), S,
        _want(dev, block_tables, "block_tables", _I32, S, cols), cols, int(block_size),
        int(num_blocks), _want(dev, free_ring, "free_ring", _I32, R), R,
        _want(dev, ring_state, "ring_state", _I64, 2),
        _want(dev, ring_state_out, "ring_state_out", _I64, 2),
        _want(dev, release_start_loc, "release_start_loc", _I32, S + 1),
        _want(dev, seq_lens_out, "seq_lens_out", _I32, S),
        st if stream is None else stream.cuda_stream))
    return release_start_loc


def _rows(dev: int, t: torch.Tensor, name: str, dtype, shape) -> tuple:
    """(address, elements between tokens) of t [T, H, D] with dense heads;
    tokens may be apart (a slice of a fused projection)."""
    T, H, D = shape
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape:
        _refuse(t, name, dtype, shape, False)
    row, head, one = t.stride()
    if (one != 1 and D > 1) or (head != D and H > 1):
        raise ValueError(f"{name} must have dense rows [heads, head_size]")
    return t.data_ptr(), row if T > 1 else H * D


def _rotary_call(name, q, k, v, positions, inv_freq, slot_mapping, key_cache, value_cache,
                 pool_dtype, scales, axis_of_pair, interleaved, q_out, stream):
    if q.dim() != 3 or k.dim() != 3 or key_cache.dim() != 4:
        raise ValueError("q and k must be [T, heads, head_size], pools [NB, Hkv, B, D]")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev, st = _current()
    T, Hq, D = shape = q.shape
    NB, Hkv, B, Dk = pool = key_cache.shape
    dtype = q.dtype
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"q must be float32, float16 or bfloat16, got {dtype}")
    if Dk != D:
        raise ValueError("pool shape does not match q")
    if positions.dim() == 1:
        axes, pos = 1, _want(dev, positions, "positions", _I64, T)
    elif positions.dim() == 2:
        axes = positions.shape[0]
        pos = _want(dev, positions, "positions", _I64, axes, T)
    else:
        raise ValueError("positions must be [T] or [axes, T]")
    half = inv_freq.numel()
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=q.device)
    kv = (T, Hkv, D)
    check(name, getattr(lib(), name)(
        *_rows(dev, q, "q", dtype, shape), *_rows(dev, k, "k", dtype, kv),
        *_rows(dev, v, "v", dtype, kv), T, Hq, Hkv, D, code, pos, T, axes,
        _want(dev, inv_freq, "inv_freq", _F64, half),
        None if axis_of_pair is None else _want(dev, axis_of_pair, "axis_of_pair", _I32, half),
        2 * half, 1 if interleaved else 0, _want(dev, slot_mapping, "slot_mapping", _I64, T),
        *_rows(dev, q_out, "q_out", dtype, shape),
        _want(dev, key_cache, "key_cache", pool_dtype, *pool),
        _want(dev, value_cache, "value_cache", pool_dtype, *pool), NB, B, *scales,
        st if stream is None else stream.cuda_stream))
    return q_out


def pa_rotary_reshape_and_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                positions: torch.Tensor, inv_freq: torch.Tensor,
                                slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                                value_cache: torch.Tensor, *,
                                axis_of_pair: Optional[torch.Tensor] = None,
                                interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                                stream=None) -> torch.Tensor:
    """Rotary positions of q [T, Hq, D] and k [T, Hkv, D] and the KV write in
    one pass: pair i turns by positions[axis_of_pair[i], t] * inv_freq[i]
    (positions int64 [T] or [axes, T]; inv_freq float64 [rot / 2];
    axis_of_pair int32 [rot / 2], None: axis 0). q, k, v may be slices of one
    projection (dense heads, any token stride). Writes rotated k and v into
    the pools ([NB, Hkv, B, D], q's dtype) at slot_mapping and returns the
    rotated q; q_out may be q."""
    return _rotary_call("pa_rotary_reshape_and_cache", q, k, v, positions, inv_freq, slot_mapping,
                        key_cache, value_cache, q.dtype, (), axis_of_pair, interleaved, q_out,
                        stream)


def pa_rotary_reshape_and_cache_fp8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                    positions: torch.Tensor, inv_freq: torch.Tensor,
                                    slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                                    value_cache: torch.Tensor, k_scale: float, v_scale: float, *,
                                    axis_of_pair: Optional[torch.Tensor] = None,
                                    interleaved: bool = False,
                                    q_out: Optional[torch.Tensor] = None,
                                    stream=None) -> torch.Tensor:
    """pa_rotary_reshape_and_cache into E4M3 pools (uint8) with one scale per
    pool; the fp32 rotated value is quantised."""
    return _rotary_call("pa_rotary_reshape_and_cache_fp8", q, k, v, positions, inv_freq,
                        slot_mapping, key_cache, value_cache, torch.uint8,
                        (float(k_scale), float(v_scale)), axis_of_pair, interleaved, q_out,
                        stream)


def pa_rotary_reshape_and_cache_fp8_scaled(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                           positions: torch.Tensor, inv_freq: torch.Tensor,
                                           slot_mapping: torch.Tensor, key_cache: torch.Tensor,
                                           value_cache: torch.Tensor, k_scales: torch.Tensor,
                                           v_scales: torch.Tensor, *,
                                           axis_of_pair: Optional[torch.Tensor] = None,
                                           interleaved: bool = False,
                                           q_out: Optional[torch.Tensor] = None,
                                           stream=None) -> torch.Tensor:
    """pa_rotary_reshape_and_cache into E4M3 pools whose blocks carry their
    own scales (float32 [NB, Hkv]), updated where this write stores a block's
    first row."""
    NB, Hkv = key_cache.shape[:2]
    dev = key_cache.get_device()
    scales = (_want(dev, k_scales, "k_scales", _F32, NB, Hkv),
              _want(dev, v_scales, "v_scales", _F32, NB, Hkv))
    return _rotary_call("pa_rotary_reshape_and_cache_fp8_scaled", q, k, v, positions, inv_freq,
                        slot_mapping, key_cache, value_cache, torch.uint8,
                        scales, axis_of_pair, interleaved, q_out, stream)


def pa_multi_query_fp8_workspace_bytes(num_tokens: int, num_seqs: int, num_q_heads: int,
                                       num_kv_heads: int, head_size: int, block_size: int,
                                       max_query_len: int, max_seq_len: int, window: int = 0,
                                       partition_size: int = 0) -> int:
    """Scratch bytes of the fp8-pool multi-query calls with these sizes."""
    n = lib().pa_multi_query_fp8_workspace_bytes(num_tokens, num_seqs, num_q_heads, num_kv_heads,
                                                 head_size, block_size, max_query_len,
                                                 max_seq_len, window, partition_size)
    if n < 0:
        check("pa_multi_query_fp8_workspace_bytes", int(n))
    return int(n)


def _chunk_call(name, q, query_start_loc, key_cache, value_cache, scale_tensors, scale_values,
                block_tables, seq_lens, scale, num_kv_heads, out, max_query_len, max_seq_len,
                window, partition_size, workspace, stream):
    if q.dim() != 3 or key_cache.dim() != 4 or block_tables.dim() != 2:
        raise ValueError("q must be [T, Hq, D], pools [NB, Hkv, B, D], block_tables [S, blocks]")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    dev, st = _current()
    T, Hq, D = shape = q.shape
    NB, Hkv, B, Dk = pool = key_cache.shape
    S, cols = seq_lens.numel(), block_tables.shape[1]
    dtype = q.dtype
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"q must be float16 or bfloat16, got {dtype}")
    if Hkv != num_kv_heads or Dk != D:
        raise ValueError("pool shape does not match q / num_kv_heads")
    out = _buffer(out, "out", dtype, q.device, dev, *shape)
    if workspace is None:
        need = pa_multi_query_fp8_workspace_bytes(T, S, Hq, Hkv, D, B, max_query_len, max_seq_len,
                                                  window, partition_size)
        if need > 0:
            workspace = torch.empty(need, dtype=_U8, device=q.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(workspace, "workspace", None, None, True)
    check(name, getattr(lib(), name)(
        _want(dev, q, "q", dtype, *shape),
        _want(dev, query_start_loc, "query_start_loc", _I32, S + 1), S, T,
        _want(dev, key_cache, "key_cache", _U8, *pool),
        _want(dev, value_cache, "value_cache", _U8, *pool),
        *[_want(dev, t, "scales", _F32, NB, Hkv) for t in scale_tensors],
        _want(dev, block_tables, "block_tables", _I32, S, cols), cols,
        _want(dev, seq_lens, "seq_lens", _I32, S), Hq, Hkv, D, B, NB, code, float(scale),
        *scale_values, int(window), int(max_query_len), int(max_seq_len), int(partition_size),
        out.data_ptr(),
        None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.nbytes,
        st if stream is None else stream.cuda_stream))
    return out


def pa_multi_query_attention_fp8(q: torch.Tensor, query_start_loc: torch.Tensor,
                                 key_cache: torch.Tensor, value_cache: torch.Tensor,
                                 block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                 scale: float, num_kv_heads: int, k_scale: float, v_scale: float,
                                 out: Optional[torch.Tensor] = None, *, max_query_len: int,
                                 max_seq_len: int, window: int = 0, partition_size: int = 0,
                                 workspace: Optional[torch.Tensor] = None,
                                 stream=None) -> torch.Tensor:
    """pa_multi_query_attention over E4M3 pools (uint8 [NB, Hkv, B, D]) with
    one scale per pool; window W > 0: the token at position p attends to
    positions max(0, p - W + 1) .. p, and blocks before every window are
    never looked up."""
    return _chunk_call("pa_multi_query_attention_fp8", q, query_start_loc, key_cache, value_cache,
                       (), (float(k_scale), float(v_scale)), block_tables, seq_lens, scale,
                       num_kv_heads, out, max_query_len, max_seq_len, window, partition_size,
                       workspace, stream)


def pa_multi_query_attention_fp8_scaled(q: torch.Tensor, query_start_loc: torch.Tensor,
                                        key_cache: torch.Tensor, value_cache: torch.Tensor,
                                        k_scales: torch.Tensor, v_scales: torch.Tensor,
                                        block_tables: torch.Tensor, seq_lens: torch.Tensor,
                                        scale: float, num_kv_heads: int,
                                        out: Optional[torch.Tensor] = None, *,
                                        max_query_len: int, max_seq_len: int, window: int = 0,
                                        partition_size: int = 0,
                                        workspace: Optional[torch.Tensor] = None,
                                        stream=None) -> torch.Tensor:
    """pa_multi_query_attention_fp8 over blocks that carry their own scales
    (float32 [NB, Hkv] each)."""
    return _chunk_call("pa_multi_query_attention_fp8_scaled", q, query_start_loc, key_cache,
                       value_cache, (k_scales, v_scales), (), block_tables, seq_lens, scale,
                       num_kv_heads, out, max_query_len, max_seq_len, window, partition_size,
                       workspace, stream)


def pa_selftest_bounded_wait(timeout_cycles: int = 2_000_000, stream=None) -> list:
    """Run the bounded-wait self-test; returns [status of warp 0, status of
    warp 1, abort flag] (expected: [PA_ERR_TIMEOUT, PA_ERR_TIMEOUT, 1])."""
    status = torch.full((3,), 12345, dtype=torch.int32, device="cuda")
    check("pa_selftest_bounded_wait", lib().pa_selftest_bounded_wait(
        ptr(status), int(timeout_cycles), stream_handle(stream)))
    torch.cuda.synchronize()
    return status.cpu().tolist()
