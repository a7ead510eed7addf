"""PyTorch-facing wrappers of the libpsk C ABI (same names as include/psk.h).

Argument marshalling only: every step runs in the CUDA kernels of libpsk.
Tensors must live on a CUDA device; each call launches on the current torch
stream of that device and returns without synchronising.  Errors from the
library raise :class:`PskError`.

Cache tensors are uint8 with pages along dim 0: ``num_pages = cache.shape[0]``
and ``page_stride = cache.stride(0)`` bytes (a 2-D ``[pages, bytes]`` tensor or
a 3-D ``[pages, block_size, record_bytes]`` view both work).
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _abi
from ._abi import PSK_REC_FP8_DS_MLA, PSK_REC_FP8_INDEXER, PSK_REC_MXFP4, PskError  # noqa: F401


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# The handle of a device's current stream and the current device as plain numbers:
# the torch.cuda objects for them cost 2 us a call, half of what a launch does.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") \
    else lambda index: torch.cuda.current_stream(index).cuda_stream
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device


def _stream(dev: torch.device) -> int:
    return _raw_stream(dev.index)


def _call(dev: torch.device, name: str, *args) -> None:
    """Call a libpsk entry point on ``dev``'s current stream with ``dev`` as
    the current CUDA device (the library launches, sizes grids and sets kernel
    attributes on the current device)."""
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            _abi.call(name, *args, _stream(dev))
    else:
        _abi.call(name, *args, _stream(dev))


def _need_cuda(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libpsk operates on CUDA tensors only (no CPU fallback)")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"all tensors of one call must be on one device ({dev} and "
                             f"{t.device})")


def _need(t: torch.Tensor, dtype: torch.dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def _page_size(shape, stride) -> int:
    """Bytes of a page, -1 where a page is not contiguous (from the strides: a view of a page
    would cost 2 us)."""
    n, gap = 1, False
    for size, step in zip(shape[:0:-1], stride[:0:-1]):
        gap |= size != 1 and step != n
        n *= size
    return -1 if gap and n > 0 else n


def _pages(cache: torch.Tensor):
    _need(cache, torch.uint8, "cache")
    shape, stride = cache.shape, cache.stride()
    if len(shape) == 2 and stride[1] == 1:
        size = shape[1]
    else:
        size = _page_size(shape, stride) if len(shape) > 1 else -1
    if size < 0 or shape[0] == 0:
        raise ValueError("cache must be [num_pages >= 1, ...] uint8 with contiguous pages")
    if shape[0] == 1:  # a size-1 dim may carry any stride (0 from broadcasting)
        return 1, max(stride[0], size)
    return shape[0], stride[0]


def _rows(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.numel() == 0:
        return t.shape[1]
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have unit inner stride")
    if t.shape[0] == 1:  # a size-1 dim may carry any stride (0 from broadcasting)
        return max(t.stride(0), t.shape[1])
    return t.stride(0)


def quantize_and_insert_k_cache(k: torch.Tensor, k_cache: torch.Tensor,
                                slot_mapping: torch.Tensor, block_size: int = 64, *,
                                rope_dim: int = 64, is_ue8m0: bool = True,
                                head_dim: Optional[int] = None,
                                err_count: Optional[torch.Tensor] = None) -> None:
    """FP8 (fp8_ds_mla) quantize + paged insert of ``k`` [N', D] bf16 at
    ``slot_mapping`` [N] int64 (N <= N'; -1 skips)."""
    _need_cuda(k, k_cache, slot_mapping, err_count)
    _need(k, torch.bfloat16, "k")
    _need(slot_mapping, torch.int64, "slot_mapping")
    if err_count is not None:
        _need(err_count, torch.int32, "err_count")
    if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be 1-D contiguous")
    D = k.shape[1] if head_dim is None else head_dim
    num_pages, page_stride = _pages(k_cache)
    _call(k.device, "quantize_and_insert_k_cache", _ptr(k), _rows(k, "k"), _ptr(slot_mapping),
          slot_mapping.shape[0], _ptr(k_cache), num_pages, page_stride, block_size, D,
          rope_dim, int(bool(is_ue8m0)), _ptr(err_count))


def write_indexer_mxfp4_cache(index_k: torch.Tensor, cache: torch.Tensor,
                              slot_mapping: torch.Tensor, block_size: int = 64, *,
                              err_count: Optional[torch.Tensor] = None) -> None:
    """MXFP4 quantize + paged insert of indexer keys ``index_k`` [N', D] bf16."""
    _need_cuda(index_k, cache, slot_mapping, err_count)
    _need(index_k, torch.bfloat16, "index_k")
    _need(slot_mapping, torch.int64, "slot_mapping")
    if slot_mapping.dim() != 1 or not slot_mapping.is_contiguous():
        raise ValueError("slot_mapping must be 1-D contiguous")
    num_pages, page_stride = _pages(cache)
    _call(index_k.device, "write_indexer_mxfp4_cache", _ptr(index_k), _rows(index_k, "index_k"),
          _ptr(slot_mapping), slot_mapping.shape[0], _ptr(cache), num_pages, page_stride,
          block_size, index_k.shape[1], _ptr(err_count))


def compute_global_topk_indices_and_lens(topk_indices: torch.Tensor,
                                         token_to_req_indices: torch.Tensor,
                                         block_table: torch.Tensor, block_size: int,
                                         is_valid_token: Optional[torch.Tensor] = None, *,
                                         base_offsets: Optional[torch.Tensor] = None,
                                         out: Optional[torch.Tensor] = None,
                                         lens: Optional[torch.Tensor] = None):
    """Map local top-k [T, K] to global slots; returns (indices [T, K], lens [T])."""
    _need_cuda(topk_indices, token_to_req_indices, block_table, is_valid_token, base_offsets)
    for t, n in ((topk_indices, "topk_indices"), (token_to_req_indices, "token_to_req"),
                 (block_table, "block_table")):
        _need(t, torch.int32, n)
    T, K = topk_indices.shape
    if out is None:
        out = torch.empty((T, K), dtype=torch.int32, device=topk_indices.device)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=topk_indices.device)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    _call(topk_indices.device, "compute_global_topk_indices_and_lens", _ptr(topk_indices),
          _rows(topk_indices, "topk_indices"), T, K, _ptr(token_to_req_indices),
          _ptr(block_table), _rows(block_table, "block_table"), block_table.shape[1],
          block_table.shape[0], block_size, _ptr(base_offsets), _ptr(valid), _ptr(out),
          _rows(out, "out"), _ptr(lens))
    return out, lens


def combine_topk_swa_indices(query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                             token_to_req_indices: torch.Tensor,
                             replay_start: Optional[torch.Tensor],
                             swa_block_table: torch.Tensor, swa_block_size: int,
                             compressed_block_table: Optional[torch.Tensor],
                             compressed_block_size: int, window_size: int,
                             compress_ratio: int, topk_indices: torch.Tensor, *,
                             swa_base_offsets: Optional[torch.Tensor] = None,
                             compressed_base_offsets: Optional[torch.Tensor] = None,
                             is_valid_token: Optional[torch.Tensor] = None,
                             num_tokens: Optional[int] = None,
                             out: Optional[torch.Tensor] = None,
                             lens: Optional[torch.Tensor] = None):
    """Fused sparse-index build; returns (sparse_indices [T, W + roundup4(K)], lens [T])."""
    _need_cuda(query_start_loc, seq_lens, token_to_req_indices, replay_start, swa_block_table,
               compressed_block_table, topk_indices, is_valid_token)
    dev = topk_indices.device
    T = topk_indices.shape[0] if num_tokens is None else num_tokens
    K = topk_indices.shape[1]
    width = window_size + (K + 3) // 4 * 4
    if out is None:
        out = torch.empty((T, width), dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=dev)
    cbt = compressed_block_table
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    _call(dev, "combine_topk_swa_indices", _ptr(query_start_loc), _ptr(seq_lens),
          _ptr(token_to_req_indices), _ptr(replay_start), seq_lens.shape[0], T,
          _ptr(swa_block_table), _rows(swa_block_table, "swa_block_table"),
          swa_block_table.shape[1], _ptr(swa_base_offsets), swa_block_size,
          _ptr(cbt), _rows(cbt, "compressed_block_table") if cbt is not None else 0,
          cbt.shape[1] if cbt is not None else 0, _ptr(compressed_base_offsets),
          compressed_block_size, window_size, compress_ratio, _ptr(topk_indices),
          _rows(topk_indices, "topk_indices"), K, _ptr(valid), _ptr(out), _rows(out, "out"),
          _ptr(lens))
    return out, lens


def dequantize_and_gather_k_cache(out: torch.Tensor, cache: torch.Tensor,
                                  indices: torch.Tensor, block_size: int, *,
                                  record: int = PSK_REC_FP8_DS_MLA, rope_dim: int = 64,
                                  is_ue8m0: bool = True) -> torch.Tensor:
    """Gather + dequantize rows ``indices`` [T, C] into ``out`` [T, C, D] bf16
    (``out`` may be a strided view, e.g. a column range of a wider output)."""
    _need_cuda(out, cache, indices)
    _need(out, torch.bfloat16, "out")
    _need(indices, torch.int32, "indices")
    if out.dim() != 3 or out.stride(2) != 1:
        raise ValueError("out must be [T, C, D] with unit inner stride")
    T, C = indices.shape
    if out.shape[0] != T or out.shape[1] != C:
        raise ValueError(f"out {tuple(out.shape)} does not match indices {tuple(indices.shape)}")
    num_pages, page_stride = _pages(cache)
    _call(out.device, "dequantize_and_gather_k_cache", _ptr(out), out.stride(0), out.stride(1),
          _ptr(cache), num_pages, page_stride, block_size, record, out.shape[2],
          rope_dim if record == PSK_REC_FP8_DS_MLA else 0, int(bool(is_ue8m0)),
          _ptr(indices), _rows(indices, "indices"), T, C)
    return out


# ---- prefill workspace path ------------------------------------------------------------

def dequantize_and_gather_k_cache_ranges(out: torch.Tensor, cache: torch.Tensor,
                                         seq_lens: torch.Tensor,
                                         gather_lens: Optional[torch.Tensor],
                                         block_table: torch.Tensor, block_size: int,
                                         offset: int, *, rope_dim: int = 64,
                                         is_ue8m0: bool = True,
                                         base_offsets: Optional[torch.Tensor] = None
                                         ) -> torch.Tensor:
    """Range-form gather into ``out`` [R, rows, D] bf16 (a workspace); see psk.h."""
    _need_cuda(out, cache, seq_lens, gather_lens, block_table, base_offsets)
    _need(out, torch.bfloat16, "out")
    if out.dim() != 3 or out.stride(2) != 1:
        raise ValueError("out must be [R, rows, D] with unit inner stride")
    for t, n in ((seq_lens, "seq_lens"), (block_table, "block_table")):
        _need(t, torch.int32, n)
    num_pages, page_stride = _pages(cache)
    _call(out.device, "dequantize_and_gather_k_cache_ranges",
          _ptr(out), out.stride(0), out.stride(1),
          out.shape[1], _ptr(cache), num_pages, page_stride, block_size,
          PSK_REC_FP8_DS_MLA, out.shape[2], rope_dim, int(bool(is_ue8m0)), _ptr(seq_lens),
          _ptr(gather_lens), _ptr(block_table), _rows(block_table, "block_table"),
          block_table.shape[1], _ptr(base_offsets), seq_lens.shape[0], offset)
    return out


def combine_topk_swa_workspace_indices(topk_indices: torch.Tensor,
                                       query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                                       gather_lens: torch.Tensor, token_to_req: torch.Tensor,
                                       window_size: int, compress_ratio: int,
                                       workspace_width: int, compressed_base: int, *,
                                       is_valid_token: Optional[torch.Tensor] = None,
                                       out: Optional[torch.Tensor] = None,
                                       lens: Optional[torch.Tensor] = None):
    """Workspace-relative index build; returns (indices [T, W + roundup4(K)], lens [T])."""
    _need_cuda(topk_indices, query_start_loc, seq_lens, gather_lens, token_to_req,
               is_valid_token)
    dev = topk_indices.device
    T, K = topk_indices.shape
    width = window_size + (K + 3) // 4 * 4
    if out is None:
        out = torch.empty((T, width), dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=dev)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    _call(dev, "combine_topk_swa_workspace_indices", _ptr(query_start_loc), _ptr(seq_lens),
          _ptr(gather_lens), _ptr(token_to_req), seq_lens.shape[0], T, window_size,
          compress_ratio, _ptr(topk_indices), _rows(topk_indices, "topk_indices"), K,
          workspace_width, compressed_base, _ptr(valid), _ptr(out), _rows(out, "out"),
          _ptr(lens))
    return out, lens


def indexer_mxfp4_paged_gather(cache: torch.Tensor, block_table: torch.Tensor,
                               cu_seq_lens: torch.Tensor, block_size: int, head_dim: int,
                               total_rows: int, values_out: Optional[torch.Tensor] = None,
                               scales_out: Optional[torch.Tensor] = None):
    """Raw MXFP4 rows over request ranges; returns (values [N, D/2], scales [N, D/32]) uint8."""
    _need_cuda(cache, block_table, cu_seq_lens)
    dev = cache.device
    if values_out is None:
        values_out = torch.empty((total_rows, head_dim // 2), dtype=torch.uint8, device=dev)
    if scales_out is None:
        scales_out = torch.empty((total_rows, head_dim // 32), dtype=torch.uint8, device=dev)
    num_pages, page_stride = _pages(cache)
    _call(dev, "indexer_mxfp4_paged_gather", _ptr(values_out), _ptr(scales_out), _ptr(cache),
          num_pages, page_stride, block_size, head_dim, _ptr(block_table),
          _rows(block_table, "block_table"), block_table.shape[1], _ptr(cu_seq_lens),
          cu_seq_lens.shape[0] - 1, total_rows)
    return values_out, scales_out


# ---- dense builders ---------------------------------------------------------------------

def decode_swa_indices_and_lens(query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                                token_to_req: torch.Tensor, block_table: torch.Tensor,
                                block_size: int, window_size: int, *,
                                base_offsets: Optional[torch.Tensor] = None,
                                is_valid_token: Optional[torch.Tensor] = None,
                                out: Optional[torch.Tensor] = None,
                                lens: Optional[torch.Tensor] = None):
    """Window-only slot indices of decode tokens; returns (indices [T, W], lens [T])."""
    _need_cuda(query_start_loc, seq_lens, token_to_req, block_table, base_offsets,
               is_valid_token)
    dev = token_to_req.device
    T = token_to_req.shape[0]
    if out is None:
        out = torch.empty((T, window_size), dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=dev)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    _call(dev, "decode_swa_indices_and_lens", _ptr(query_start_loc), _ptr(seq_lens),
          _ptr(token_to_req), seq_lens.shape[0], T, _ptr(block_table),
          _rows(block_table, "block_table"), block_table.shape[1], _ptr(base_offsets),
          block_size, window_size, _ptr(valid), _ptr(out), _rows(out, "out"), _ptr(lens))
    return out, lens


def compute_dense_compressed_indices_and_lens(positions: torch.Tensor,
                                              token_to_req: torch.Tensor,
                                              block_table: torch.Tensor, block_size: int,
                                              compress_ratio: int, width: int, *,
                                              num_reqs: Optional[int] = None,
                                              base_offsets: Optional[torch.Tensor] = None,
                                              is_valid_token: Optional[torch.Tensor] = None,
                                              out: Optional[torch.Tensor] = None,
                                              lens: Optional[torch.Tensor] = None):
    """Slots of every visible compressed entry; returns (indices [T, width], lens [T])."""
    _need_cuda(positions, token_to_req, block_table, base_offsets, is_valid_token)
    _need(positions, torch.int64, "positions")
    dev = positions.device
    T = positions.shape[0]
    if out is None:
        out = torch.empty((T, width), dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=dev)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    R = block_table.shape[0] if num_reqs is None else num_reqs
    _call(dev, "compute_dense_compressed_indices_and_lens", _ptr(positions), T,
          _ptr(token_to_req), R, _ptr(block_table), _rows(block_table, "block_table"),
          block_table.shape[1], _ptr(base_offsets), block_size, compress_ratio, width,
          _ptr(valid), _ptr(out), _rows(out, "out"), _ptr(lens))
    return out, lens


def build_dense_prefill_local_compressed_indices(positions: torch.Tensor, compress_ratio: int,
                                                 width: int, *,
                                                 out: Optional[torch.Tensor] = None):
    """Request-local dense compressed indices [T, width] (j, or -1 past the visible count)."""
    _need_cuda(positions)
    _need(positions, torch.int64, "positions")
    dev = positions.device
    T = positions.shape[0]
    if out is None:
        out = torch.empty((T, width), dtype=torch.int32, device=dev)
    _call(dev, "build_dense_prefill_local_compressed_indices", _ptr(positions), T,
          compress_ratio, width, _ptr(out), _rows(out, "out"))
    return out


def combine_dense_swa_indices(positions: torch.Tensor, token_to_req: torch.Tensor,
                              seq_lens: torch.Tensor, gather_lens: torch.Tensor,
                              window_size: int, workspace_width: int, compressed_base: int = 0,
                              *, out: Optional[torch.Tensor] = None,
                              lens: Optional[torch.Tensor] = None):
    """Workspace-relative window indices of layers without a compressed cache;
    returns (indices [T, W], lens [T])."""
    _need_cuda(positions, token_to_req, seq_lens, gather_lens)
    _need(positions, torch.int64, "positions")
    dev = positions.device
    T = positions.shape[0]
    if out is None:
        out = torch.empty((T, window_size), dtype=torch.int32, device=dev)
    if lens is None:
        lens = torch.empty((T,), dtype=torch.int32, device=dev)
    _call(dev, "combine_dense_swa_indices", _ptr(positions), _ptr(token_to_req), _ptr(seq_lens),
          _ptr(gather_lens), seq_lens.shape[0], T, window_size, workspace_width,
          compressed_base, _ptr(out), _rows(out, "out"), _ptr(lens))
    return out, lens


# ---- indexer-key variants -------------------------------------------------------------

def write_indexer_fp8_cache(index_k: torch.Tensor, cache: torch.Tensor, slot_mapping: torch.Tensor,
                            block_size: int, *, err_count: Optional[torch.Tensor] = None) -> None:
    """FP8 indexer keys ([values | binary32 power-of-two scale] pages)."""
    _need_cuda(index_k, cache, slot_mapping, err_count)
    _need(index_k, torch.bfloat16, "index_k")
    _need(slot_mapping, torch.int64, "slot_mapping")
    num_pages, page_stride = _pages(cache)
    _call(index_k.device, "write_indexer_fp8_cache", _ptr(index_k), _rows(index_k, "index_k"),
          _ptr(slot_mapping), slot_mapping.shape[0], _ptr(cache), num_pages, page_stride,
          block_size, index_k.shape[1], _ptr(err_count))


def indexer_k_norm_rope_store(k_pre: torch.Tensor, positions: torch.Tensor,
                              cos_sin_cache: torch.Tensor, rms_norm_weight: torch.Tensor,
                              rms_norm_eps: float, k_cache: torch.Tensor,
                              kv_slot_mapping: torch.Tensor, compress_ratio: int,
                              use_fp4_cache: bool, block_size: int, *,
                              err_count: Optional[torch.Tensor] = None) -> None:
    """k_norm -> GPT-J RoPE -> MXFP4 / FP8 indexer record -> paged store of
    128-dim indexer keys (the vLLM op's argument names)."""
    _need_cuda(k_pre, positions, cos_sin_cache, rms_norm_weight, k_cache, kv_slot_mapping,
               err_count)
    _need(k_pre, torch.bfloat16, "k_pre")
    _need(positions, torch.int64, "positions")
    _need(cos_sin_cache, torch.float32, "cos_sin_cache")
    _need(rms_norm_weight, torch.float32, "rms_norm_weight")
    _need(kv_slot_mapping, torch.int64, "kv_slot_mapping")
    if k_pre.dim() != 2 or k_pre.shape[1] != 128:
        raise ValueError("k_pre must be [num_tokens, 128]")
    num_pages, page_stride = _pages(k_cache)
    record = PSK_REC_MXFP4 if use_fp4_cache else PSK_REC_FP8_INDEXER
    _call(k_pre.device, "indexer_k_norm_rope_store",
          _ptr(k_pre), _rows(k_pre, "k_pre"), _ptr(positions),
          _ptr(cos_sin_cache), _rows(cos_sin_cache, "cos_sin_cache"), cos_sin_cache.shape[0],
          _ptr(rms_norm_weight.contiguous()), float(rms_norm_eps), _ptr(kv_slot_mapping),
          kv_slot_mapping.shape[0], compress_ratio, record, _ptr(k_cache), num_pages,
          page_stride, block_size, _ptr(err_count))


# ---- compressed-KV producer -------------------------------------------------------------

def save_compressor_state(kv: torch.Tensor, score: torch.Tensor, ape: torch.Tensor,
                          state_cache: torch.Tensor, slot_mapping: torch.Tensor,
                          positions: torch.Tensor, block_size: int, compress_ratio: int, *,
                          err_count: Optional[torch.Tensor] = None) -> None:
    """state[slot] = [kv, score + ape[pos % ratio]] into the binary32 state cache
    [pages, block_size, 2 * state_width]."""
    _need_cuda(kv, score, ape, state_cache, slot_mapping, positions, err_count)
    for t, n in ((kv, "kv"), (score, "score"), (ape, "ape"), (state_cache, "state_cache")):
        _need(t, torch.float32, n)
    _need(slot_mapping, torch.int64, "slot_mapping")
    _need(positions, torch.int64, "positions")
    if kv.stride() != score.stride():
        raise ValueError("kv and score must share a layout")
    sw = kv.shape[1]
    if state_cache.dim() != 3 or state_cache.shape[1] != block_size or \
            state_cache.shape[2] != 2 * sw or not state_cache.is_contiguous():
        raise ValueError("state_cache must be contiguous [pages, block_size, 2 * state_width]")
    _call(kv.device, "save_compressor_state", _ptr(kv), _ptr(score), _rows(kv, "kv"),
          _ptr(ape.contiguous()), sw, _ptr(slot_mapping), _ptr(positions),
          slot_mapping.shape[0], compress_ratio, _ptr(state_cache), state_cache.shape[0],
          block_size, _ptr(err_count))


def compress_kv_cache_insert(state_cache: torch.Tensor, token_to_req_indices: torch.Tensor,
                             positions: torch.Tensor, compressor_slot_mapping: torch.Tensor,
                             block_table: torch.Tensor, compressor_block_size: int,
                             rms_norm_weight: torch.Tensor, rms_norm_eps: float,
                             cos_sin_cache: torch.Tensor, kv_cache_2d: torch.Tensor,
                             kv_slot_mapping: torch.Tensor, kv_cache_block_size: int,
                             compress_ratio: int, *, overlap: Optional[bool] = None,
                             block_table_base_offsets: Optional[torch.Tensor] = None,
                             err_count: Optional[torch.Tensor] = None) -> None:
    """Window-pooled, normalised, rotated fp8_ds_mla rows of the compressed KV
    cache (ratio 4 with overlap = the CSA insert, ratio 128 = the HCA insert)."""
    _need_cuda(state_cache, token_to_req_indices, positions, compressor_slot_mapping,
               block_table, rms_norm_weight, cos_sin_cache, kv_cache_2d, kv_slot_mapping,
               block_table_base_offsets, err_count)
    _need(state_cache, torch.float32, "state_cache")
    _need(positions, torch.int64, "positions")
    _need(rms_norm_weight, torch.float32, "rms_norm_weight")
    _need(cos_sin_cache, torch.float32, "cos_sin_cache")
    if overlap is None:
        overlap = compress_ratio == 4
    if state_cache.dim() != 3 or not state_cache.is_contiguous():
        raise ValueError("state_cache must be contiguous [pages, block_size, 2 * state_width]")
    num_pages, page_stride = _pages(kv_cache_2d)
    _call(state_cache.device, "compress_kv_cache_insert", _ptr(state_cache), state_cache.shape[0],
          compressor_block_size, state_cache.shape[2] // 2, _ptr(token_to_req_indices),
          _ptr(positions), _ptr(compressor_slot_mapping), _ptr(block_table),
          _rows(block_table, "block_table"), block_table.shape[1],
          _ptr(block_table_base_offsets), block_table.shape[0], positions.shape[0],
          compress_ratio, int(bool(overlap)), _ptr(rms_norm_weight.contiguous()),
          float(rms_norm_eps), _ptr(cos_sin_cache), _rows(cos_sin_cache, "cos_sin_cache"),
          cos_sin_cache.shape[0], _ptr(kv_cache_2d), num_pages, page_stride,
          kv_cache_block_size, _ptr(kv_slot_mapping), _ptr(err_count))


# ---- fused gathers ------------------------------------------------------------------------

def dequantize_and_gather_k_cache_topk(out: torch.Tensor, cache: torch.Tensor,
                                       topk_indices: torch.Tensor,
                                       token_to_req_indices: torch.Tensor,
                                       block_table: torch.Tensor, block_size: int, *,
                                       record: int = PSK_REC_FP8_DS_MLA, rope_dim: int = 64,
                                       num_reqs: Optional[int] = None,
                                       base_offsets: Optional[torch.Tensor] = None,
                                       is_valid_token: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t, j] = the row of topk_indices[t, j] mapped through the request's table
    (= compute_global_topk_indices_and_lens + dequantize_and_gather_k_cache)."""
    _need_cuda(out, cache, topk_indices, token_to_req_indices, block_table, base_offsets,
               is_valid_token)
    _need(out, torch.bfloat16, "out")
    T, K = topk_indices.shape
    if out.dim() != 3 or out.shape[0] != T or out.shape[1] != K or out.stride(2) != 1:
        raise ValueError("out must be [T, K, D] with unit inner stride")
    num_pages, page_stride = _pages(cache)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    R = block_table.shape[0] if num_reqs is None else num_reqs
    _call(out.device, "dequantize_and_gather_k_cache_topk", _ptr(out), out.stride(0), out.stride(1),
          _ptr(cache), num_pages, page_stride, block_size, record, out.shape[2],
          rope_dim if record == PSK_REC_FP8_DS_MLA else 0, _ptr(topk_indices),
          _rows(topk_indices, "topk_indices"), T, K, _ptr(token_to_req_indices),
          _ptr(block_table), _rows(block_table, "block_table"), block_table.shape[1], R,
          _ptr(base_offsets), _ptr(valid))
    return out


def dequantize_and_gather_k_cache_window(out: torch.Tensor, cache: torch.Tensor,
                                         query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                                         token_to_req: torch.Tensor,
                                         replay_start: Optional[torch.Tensor],
                                         block_table: torch.Tensor, block_size: int,
                                         window_size: int, *, rope_dim: int = 64,
                                         base_offsets: Optional[torch.Tensor] = None,
                                         is_valid_token: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t, c] = the row of window column c of token t (= the window columns of
    combine_topk_swa_indices + dequantize_and_gather_k_cache)."""
    _need_cuda(out, cache, query_start_loc, seq_lens, token_to_req, replay_start, block_table,
               base_offsets, is_valid_token)
    _need(out, torch.bfloat16, "out")
    T = token_to_req.shape[0]
    if out.dim() != 3 or out.shape[0] != T or out.shape[1] != window_size or out.stride(2) != 1:
        raise ValueError("out must be [T, window, D] with unit inner stride")
    num_pages, page_stride = _pages(cache)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    _call(out.device, "dequantize_and_gather_k_cache_window",
          _ptr(out), out.stride(0), out.stride(1),
          _ptr(cache), num_pages, page_stride, block_size, out.shape[2], rope_dim,
          _ptr(query_start_loc), _ptr(seq_lens), _ptr(token_to_req), _ptr(replay_start),
          seq_lens.shape[0], T, _ptr(block_table), _rows(block_table, "block_table"),
          block_table.shape[1], _ptr(base_offsets), window_size, _ptr(valid))
    return out


def device_wait_timeouts() -> int:
    """Expired in-kernel bounded waits on the current device (0 in normal operation)."""
    return _abi.device_wait_timeouts()


def device_wait_selftest(limit_ns: int, device: torch.device) -> None:
    """Launch one bounded wait that nothing completes (counted when it expires)."""
    _call(device, "psk_device_wait_selftest", int(limit_ns))


def dequantize_and_gather_k_cache_pair(out: torch.Tensor, cache_a: torch.Tensor, block_size_a: int,
                                       cache_b: torch.Tensor, block_size_b: int,
                                       indices: torch.Tensor, split: int, *,
                                       rope_dim: int = 64) -> torch.Tensor:
    """out[t, j] = row indices[t, j] of cache_a for j < split, of cache_b for
    j >= split (fp8_ds_mla, UE8M0)."""
    _need_cuda(out, cache_a, cache_b, indices)
    _need(out, torch.bfloat16, "out")
    R, C = indices.shape
    if out.dim() != 3 or out.shape[0] != R or out.shape[1] != C or out.stride(2) != 1:
        raise ValueError("out must be [rows, cols, D] with unit inner stride")
    np_a, ps_a = _pages(cache_a)
    np_b, ps_b = _pages(cache_b)
    _call(out.device, "dequantize_and_gather_k_cache_pair", _ptr(out), out.stride(0), out.stride(1),
          _ptr(cache_a), np_a, ps_a, block_size_a, _ptr(cache_b), np_b, ps_b, block_size_b,
          out.shape[2], rope_dim, _ptr(indices), _rows(indices, "indices"), R, C, split)
    return out


def dequantize_and_gather_k_cache_dense(out: torch.Tensor, cache: torch.Tensor,
                                        positions: torch.Tensor, token_to_req: torch.Tensor,
                                        block_table: torch.Tensor, block_size: int,
                                        compress_ratio: int, *, rope_dim: int = 64,
                                        num_reqs: Optional[int] = None,
                                        base_offsets: Optional[torch.Tensor] = None,
                                        is_valid_token: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out[t, c] = compressed entry c of token t when visible (= the dense
    compressed indices followed by the gather)."""
    _need_cuda(out, cache, positions, token_to_req, block_table, base_offsets, is_valid_token)
    _need(out, torch.bfloat16, "out")
    T = positions.shape[0]
    if out.dim() != 3 or out.shape[0] != T or out.stride(2) != 1:
        raise ValueError("out must be [T, width, D] with unit inner stride")
    num_pages, page_stride = _pages(cache)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    R = block_table.shape[0] if num_reqs is None else num_reqs
    _call(out.device, "dequantize_and_gather_k_cache_dense",
          _ptr(out), out.stride(0), out.stride(1),
          _ptr(cache), num_pages, page_stride, block_size, out.shape[2], rope_dim,
          _ptr(positions), T, _ptr(token_to_req), R, _ptr(block_table),
          _rows(block_table, "block_table"), block_table.shape[1], _ptr(base_offsets),
          compress_ratio, out.shape[1], _ptr(valid))
    return out


# ---- batch metadata from request lengths ------------------------------------------------
#
# A decode step makes these calls (and the attention ones) once per layer with
# kernels of a few microseconds, so their argument checks read each property of a
# tensor once.

def _index(t: torch.Tensor) -> int:
    """CUDA device index of the tensor a call takes its device from."""
    i = t.get_device()
    if i < 0:
        raise ValueError("libpsk operates on CUDA tensors only (no CPU fallback)")
    return i


def _same(t: torch.Tensor, index: int, name: str) -> None:
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _vec(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, size: int, index: int):
    """Address of a 1-D contiguous tensor of ``dtype`` with ``size`` entries at least; None for
    None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dim() != 1 or not t.is_contiguous():
        raise ValueError(f"{name} must be 1-D contiguous")
    if t.numel() < size:
        raise ValueError(f"{name} must have at least {size} entries, got {t.numel()}")
    return t.data_ptr()


def _table(t: torch.Tensor, name: str, rows: int, index: int):
    """Address, row stride and width of an int32 block table with ``rows`` rows at least; the
    library refuses a stride below the width (expanded or overlapping rows)."""
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be {torch.int32}, got {t.dtype}")
    _same(t, index, name)
    stride, (n, width) = _rows(t, name), t.shape
    if n < rows:
        raise ValueError(f"{name} must have at least {rows} rows, got {n}")
    return t.data_ptr(), stride, width


def compute_slot_mappings(query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                          block_table: torch.Tensor, block_size: int, num_tokens: int, *,
                          base_offsets: Optional[torch.Tensor] = None,
                          compressed_block_table: Optional[torch.Tensor] = None,
                          compressed_block_size: Optional[int] = None,
                          compressed_base_offsets: Optional[torch.Tensor] = None,
                          compress_ratio: int = 1,
                          positions: Optional[torch.Tensor] = None,
                          token_to_req: Optional[torch.Tensor] = None,
                          slot_mapping: Optional[torch.Tensor] = None,
                          compressed_slot_mapping: Optional[torch.Tensor] = None):
    """Batch metadata from request lengths; returns (positions [T] int64, token_to_req [T]
    int32, slot_mapping [T] int64, compressed_slot_mapping [T] int64), -1 for padding tokens."""
    i, i32, i64 = _index(seq_lens), torch.int32, torch.int64
    dev, T, R = seq_lens.device, int(num_tokens), seq_lens.numel()
    if T < 0:
        raise ValueError("num_tokens must be >= 0")
    if positions is None:
        positions = torch.empty((T,), dtype=i64, device=dev)
    if token_to_req is None:
        token_to_req = torch.empty((T,), dtype=i32, device=dev)
    if slot_mapping is None:
        slot_mapping = torch.empty((T,), dtype=i64, device=dev)
    if compressed_slot_mapping is None:
        compressed_slot_mapping = torch.empty((T,), dtype=i64, device=dev)
    cbt = compressed_block_table
    _call(dev, "compute_slot_mappings",
          _vec(query_start_loc, i32, "query_start_loc", R + 1, i),
          _vec(seq_lens, i32, "seq_lens", R, i), R, T,
          *_table(block_table, "block_table", R, i),
          _vec(base_offsets, i32, "base_offsets", R, i), block_size,
          *((None, 0, 0) if cbt is None else _table(cbt, "compressed_block_table", R, i)),
          _vec(compressed_base_offsets, i32, "compressed_base_offsets", R, i),
          block_size if compressed_block_size is None else compressed_block_size, compress_ratio,
          _vec(positions, i64, "positions", T, i), _vec(token_to_req, i32, "token_to_req", T, i),
          _vec(slot_mapping, i64, "slot_mapping", T, i),
          _vec(compressed_slot_mapping, i64, "compressed_slot_mapping", T, i))
    return positions, token_to_req, slot_mapping, compressed_slot_mapping


def extend_block_tables(seq_lens: torch.Tensor, page_pool: torch.Tensor,
                        block_table: torch.Tensor, block_size: int, *,
                        page_counts: Optional[torch.Tensor] = None,
                        pool_head: Optional[torch.Tensor] = None, compress_ratio: int = 1,
                        page_counts_out: Optional[torch.Tensor] = None,
                        pool_head_out: Optional[torch.Tensor] = None,
                        err_count: Optional[torch.Tensor] = None):
    """Grow ``block_table`` [R, width] int32 (in place) to the pages ``seq_lens`` needs, with
    pages of ``page_pool`` from ``pool_head`` on; returns (block_table, page_counts [R],
    pool_head [1]).  The inputs but the table are left as they were."""
    i, i32 = _index(seq_lens), torch.int32
    dev, R = seq_lens.device, seq_lens.numel()
    table, stride, width = _table(block_table, "block_table", R, i)
    if R > 1 and block_table.stride(0) < width:
        raise ValueError("rows of block_table must not overlap")
    if page_counts_out is None:
        page_counts_out = torch.empty((R,), dtype=i32, device=dev)
    if pool_head_out is None:
        pool_head_out = torch.empty((1,), dtype=i32, device=dev)
    _call(dev, "extend_block_tables", _vec(seq_lens, i32, "seq_lens", R, i), R, block_size,
          compress_ratio, _vec(page_counts, i32, "page_counts", R, i),
          _vec(page_pool, i32, "page_pool", 0, i), page_pool.numel(),
          _vec(pool_head, i32, "pool_head", 1, i), table, stride, width,
          _vec(page_counts_out, i32, "page_counts_out", R, i),
          _vec(pool_head_out, i32, "pool_head_out", 1, i),
          _vec(err_count, i32, "err_count", 1, i))
    if R == 0:  # nothing was launched: the head stays where it is
        if pool_head is None:
            pool_head_out[:1].fill_(0)
        else:
            torch.clamp(pool_head[:1], min=0, out=pool_head_out[:1])
    return block_table, page_counts_out, pool_head_out


# ---- attention over paged fp8_ds_mla caches ------------------------------------------------

def _heads(t: torch.Tensor, name: str, index: int):
    """Address and strides of a [T, H, D] bf16 tensor with unit inner stride (a size-1 dim may
    carry any stride)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    _same(t, index, name)
    if t.dim() != 3 or t.stride(2) != 1:
        raise ValueError(f"{name} must be [T, H, D] with unit inner stride")
    T, H, D = t.shape
    st, sh, _ = t.stride()
    return t.data_ptr(), (st if T > 1 else H * D), (sh if H > 1 else D)


def _cache_of(cache: Optional[torch.Tensor], name: str, index: int):
    if cache is None:
        return None, 0, 0
    _same(cache, index, name)
    return (cache.data_ptr(), *_pages(cache))


def _attention_outputs(q, out, lse, workspace, need, index):
    """Allocated or checked outputs and workspace: (out, lse, the arguments for them)."""
    T, H, D = q.shape
    if out is None:
        out = torch.empty((T, H, D), dtype=torch.bfloat16, device=q.device)
        o = (out.data_ptr(), H * D, D)
    else:
        if out.shape != q.shape:
            raise ValueError(f"out {tuple(out.shape)} does not match q {tuple(q.shape)}")
        o = _heads(out, "out", index)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
        ls = H
    else:
        _need(lse, torch.float32, "lse")
        _same(lse, index, "lse")
        if lse.shape != (T, H) or (H > 1 and lse.stride(1) != 1):
            raise ValueError(f"lse must be [{T}, {H}] with unit inner stride")
        ls = lse.stride(0) if T > 1 else H
    if workspace is None:
        if need > 0:
            workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    else:
        _vec(workspace, torch.uint8, "workspace", 0, index)
    w = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())
    return out, lse, (*o, lse.data_ptr(), ls, *w)


def _on(index: int, fn, *args):
    """A size query that depends on the device: asked with that device current."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return fn(*args)
    return fn(*args)


def sparse_mla_attention_workspace_bytes(device: torch.device, num_tokens: int, num_heads: int,
                                         head_dim: int, cols: int) -> int:
    """Bytes of ``workspace`` a sparse_mla_attention call of these sizes needs on ``device``."""
    index = torch.device(device).index
    return _on(_current_device() if index is None else index,
               _abi.lib().sparse_mla_attention_workspace_bytes, num_tokens, num_heads, head_dim, cols)


def chunk_mla_attention_workspace_bytes(device: torch.device, num_tokens: int, num_reqs: int,
                                        num_heads: int, head_dim: int, table_width: int,
                                        block_size: int, window_size: int = 0) -> int:
    """Bytes of ``workspace`` a chunk_mla_attention call of these sizes needs on ``device``."""
    index = torch.device(device).index
    return _on(_current_device() if index is None else index,
               _abi.lib().chunk_mla_attention_workspace_bytes, num_tokens, num_reqs, num_heads,
               head_dim, table_width, block_size, window_size)


def sparse_mla_attention(q: torch.Tensor, cache: torch.Tensor, indices: torch.Tensor,
                         block_size: int, *, extra_cache: Optional[torch.Tensor] = None,
                         extra_block_size: Optional[int] = None, split: Optional[int] = None,
                         softmax_scale: Optional[float] = None,
                         sink: Optional[torch.Tensor] = None, rope_dim: int = 64,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None):
    """Attention of ``q`` [T, H, D] over the fp8_ds_mla rows ``indices`` [T, C] names (records with
    UE8M0 scales; binary32 ones, is_ue8m0=False at the insert, would be misread): slots of
    ``cache`` in columns [0, split), of ``extra_cache`` in the others (``split`` defaults to all
    columns).  Returns (out [T, H, D] bf16, lse [T, H] binary32); scale defaults to D^-1/2.
    ``workspace`` (uint8) is scratch; two calls that can run at once need one each."""
    i = _index(q)
    qa = _heads(q, "q", i)
    T, H, D = q.shape
    _need(indices, torch.int32, "indices")
    _same(indices, i, "indices")
    if indices.dim() != 2 or indices.shape[0] != T:
        raise ValueError(f"indices must be [{T}, C]")
    C = indices.shape[1]
    need = _on(i, _abi.lib().sparse_mla_attention_workspace_bytes, T, H, D, C)
    out, lse, oa = _attention_outputs(q, out, lse, workspace, need, i)
    _call(q.device, "sparse_mla_attention", *qa, T, H, *_cache_of(cache, "cache", i), block_size,
          *_cache_of(extra_cache, "extra_cache", i),
          block_size if extra_block_size is None else extra_block_size, D, rope_dim,
          indices.data_ptr(), _rows(indices, "indices"), C, C if split is None else split,
          D ** -0.5 if softmax_scale is None else softmax_scale,
          _vec(sink, torch.float32, "sink", H, i), *oa)
    return out, lse


def chunk_mla_attention(q: torch.Tensor, cache: torch.Tensor, query_start_loc: torch.Tensor,
                        seq_lens: torch.Tensor, token_to_req: torch.Tensor,
                        block_table: torch.Tensor, block_size: int, *, window_size: int = 0,
                        replay_start: Optional[torch.Tensor] = None,
                        base_offsets: Optional[torch.Tensor] = None,
                        is_valid_token: Optional[torch.Tensor] = None,
                        softmax_scale: Optional[float] = None,
                        sink: Optional[torch.Tensor] = None, rope_dim: int = 64,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None):
    """Causal attention of a chunk of new tokens ``q`` [T, H, D] over their requests' positions
    through ``block_table`` (whole context, or the last ``window_size`` positions); rows of the
    new tokens must be in the cache (records with UE8M0 scales).  Returns (out [T, H, D] bf16,
    lse [T, H] binary32).  Whole contexts: time and scratch grow with the table's width; where a
    bound on ``seq_lens`` is known, pass ``block_table[:, :ceil(bound / block_size)]``."""
    i, i32 = _index(q), torch.int32
    qa = _heads(q, "q", i)
    T, H, D = q.shape
    R = seq_lens.numel()
    table = _table(block_table, "block_table", R, i)
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    need = _on(i, _abi.lib().chunk_mla_attention_workspace_bytes, T, R, H, D, table[2], block_size,
               window_size)
    out, lse, oa = _attention_outputs(q, out, lse, workspace, need, i)
    _call(q.device, "chunk_mla_attention", *qa, T, H, *_cache_of(cache, "cache", i), block_size, D,
          rope_dim, _vec(query_start_loc, i32, "query_start_loc", R + 1, i),
          _vec(seq_lens, i32, "seq_lens", R, i), _vec(token_to_req, i32, "token_to_req", T, i),
          _vec(replay_start, i32, "replay_start", R, i), R, *table,
          _vec(base_offsets, i32, "base_offsets", R, i), window_size,
          _vec(valid, torch.uint8, "is_valid_token", T, i),
          D ** -0.5 if softmax_scale is None else softmax_scale,
          _vec(sink, torch.float32, "sink", H, i), *oa)
    return out, lse


# ---- rotary positions ------------------------------------------------------------------------

_ROPE_SCALING = {"none": _abi.PSK_ROPE_UNSCALED, "linear": _abi.PSK_ROPE_LINEAR, "yarn": _abi.PSK_ROPE_YARN}
_ROTARY_DTYPES = {torch.bfloat16: _abi.PSK_DTYPE_BF16, torch.float16: _abi.PSK_DTYPE_FP16,
                  torch.float32: _abi.PSK_DTYPE_FP32}


def build_rope_cos_sin_cache(num_positions: int, rope_dim: int, *, theta: float = 10000.0,
                             scaling: str = "none", factor: float = 1.0,
                             original_positions: int = 0, beta_fast: float = 32.0,
                             beta_slow: float = 1.0, attention_factor: float = 1.0,
                             first_position: int = 0, device=None,
                             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Table [num_positions, rope_dim] binary32 of the cosines, then sines, of positions from
    ``first_position`` on; ``scaling`` "none", "linear" (by ``factor``) or "yarn" (by parts, from
    ``original_positions``); every value times ``attention_factor``."""
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(_ROPE_SCALING)}, got {scaling!r}")
    if out is None:
        if num_positions < 0 or rope_dim < 0:
            raise ValueError("num_positions and rope_dim must be >= 0")
        dev = torch.device("cuda" if device is None else device)
        if dev.type != "cuda":
            raise ValueError("libpsk operates on CUDA tensors only (no CPU fallback)")
        out = torch.empty((num_positions, rope_dim), dtype=torch.float32, device=dev)
    else:
        _index(out)
        _need(out, torch.float32, "out")
        if out.shape != (num_positions, rope_dim):
            raise ValueError(f"out must be [{num_positions}, {rope_dim}]")
    _call(out.device, "build_rope_cos_sin_cache", out.data_ptr(), _rows(out, "out"), first_position,
          num_positions, rope_dim, theta, _ROPE_SCALING[scaling], factor, original_positions,
          beta_fast, beta_slow, attention_factor)
    return out


def _rotated(t: torch.Tensor, name: str, T: int, D: int, dtype: torch.dtype, index: int):
    """Address and strides of a [T, H, D] (or, one head, [T, D]) tensor with unit inner stride (a
    size-1 dim may carry any stride), and its heads."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    _same(t, index, name)
    shape, stride = t.shape, t.stride()
    if len(shape) not in (2, 3) or shape[0] != T or shape[-1] != D or (stride[-1] != 1 and D > 1):
        raise ValueError(f"{name} must be [{T}, heads, {D}] or [{T}, {D}] with unit inner stride")
    H, sh = (shape[1], stride[1]) if len(shape) == 3 else (1, D)
    if H == 1:
        sh = D
    return (t.data_ptr(), stride[0] if T > 1 else H * D, sh), H


def apply_rotary_embedding(positions: torch.Tensor, q: torch.Tensor, cos_sin_cache: torch.Tensor,
                           k: Optional[torch.Tensor] = None, *, rope_offset: Optional[int] = None,
                           interleaved: bool = True, inverse: bool = False,
                           q_out: Optional[torch.Tensor] = None,
                           k_out: Optional[torch.Tensor] = None,
                           err_count: Optional[torch.Tensor] = None):
    """Rotate ``rope_dim = cos_sin_cache.shape[1]`` dims from ``rope_offset`` on (default: the last
    ones) of every head of ``q`` [T, H, D] and ``k`` [T, Hk, D] or [T, D] (bf16, fp16 or binary32) by
    ``positions`` [T] int64 (negative: a padding token, not rotated).  Returns (q_out, k_out);
    ``q_out=q`` rotates in place.  ``inverse`` turns back, and is the gradient of the forward
    rotation."""
    i = _index(q)
    if q.dtype not in _ROTARY_DTYPES:
        raise TypeError(f"q must be one of {[str(d) for d in _ROTARY_DTYPES]}, got {q.dtype}")
    dtype, dev, shape = q.dtype, q.device, q.shape
    T, D = shape[0], shape[-1]
    _need(cos_sin_cache, torch.float32, "cos_sin_cache")
    _same(cos_sin_cache, i, "cos_sin_cache")
    qa, H = _rotated(q, "q", T, D, dtype, i)
    if q_out is None:
        q_out = torch.empty(shape, dtype=dtype, device=dev)
        qo = (q_out.data_ptr(), H * D, D)
    elif q_out.shape != shape:
        raise ValueError(f"q_out {tuple(q_out.shape)} does not match q {tuple(shape)}")
    else:
        qo, _ = _rotated(q_out, "q_out", T, D, dtype, i)
    ka, ko, Hk = (None, 0, 0), (None, 0, 0), 0
    if k is not None:
        ka, Hk = _rotated(k, "k", T, D, dtype, i)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=dtype, device=dev)
            ko = (k_out.data_ptr(), Hk * D, D)
        elif k_out.shape != k.shape:
            raise ValueError(f"k_out {tuple(k_out.shape)} does not match k {tuple(k.shape)}")
        else:
            ko, _ = _rotated(k_out, "k_out", T, D, dtype, i)
    elif k_out is not None:
        raise ValueError("k_out without k")
    stride, (rows, rope) = _rows(cos_sin_cache, "cos_sin_cache"), cos_sin_cache.shape
    _call(dev, "apply_rotary_embedding", *qa, H, *ka, Hk, T, _ROTARY_DTYPES[dtype], D,
          D - rope if rope_offset is None else rope_offset, rope, int(bool(interleaved)),
          int(bool(inverse)), _vec(positions, torch.int64, "positions", T, i),
          cos_sin_cache.data_ptr(), stride, rows, *qo, *ko,
          _vec(err_count, torch.int32, "err_count", 1, i))
    return q_out, k_out


# ---- eviction from a cache -------------------------------------------------------------------

def _per_row(t: Optional[torch.Tensor], dtype: torch.dtype, name: str, R: int, width: int, index: int):
    """Address and row stride of a [>= R, >= width] matrix of values per cached row."""
    if t is None:
        return None, 0
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    shape = t.shape
    if len(shape) != 2 or shape[0] < R or shape[1] < width:
        raise ValueError(f"{name} must be at least [{R}, {width}], got {tuple(shape)}")
    stride, inner = t.stride()
    if inner != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name} must have unit inner stride")
    if shape[0] <= 1 or shape[1] == 0:  # a size-1 dim may carry any stride (0 from broadcasting)
        stride = max(stride, shape[1])
    return t.data_ptr(), stride


def _move_list(t: torch.Tensor, R: int, count: int, index: int):
    """Address and row stride of the moves [>= R, >= count, 2] int32."""
    if t.dtype != torch.int32:
        raise TypeError(f"moves must be {torch.int32}, got {t.dtype}")
    _same(t, index, "moves")
    if t.dim() != 3 or t.shape[2] != 2 or t.shape[0] < R or t.shape[1] < count:
        raise ValueError(f"moves must be at least [{R}, {count}, 2], got {tuple(t.shape)}")
    st = t.stride()
    if t.numel() > 0 and (st[2] != 1 or (t.shape[1] > 1 and st[1] != 2)):
        raise ValueError("moves must hold its pairs side by side")
    return t.data_ptr(), (st[0] if t.shape[0] > 1 else 2 * t.shape[1])


def accumulate_attention_weights_workspace_bytes(device: torch.device) -> int:
    """Bytes of ``workspace`` an accumulate_attention_weights call needs on ``device``."""
    index = torch.device(device).index
    return _on(_current_device() if index is None else index,
               _abi.lib().accumulate_attention_weights_workspace_bytes)


_weights_workspace: dict = {}


def accumulate_attention_weights(q: torch.Tensor, lse: torch.Tensor, cache: torch.Tensor,
                                 query_start_loc: torch.Tensor, seq_lens: torch.Tensor,
                                 block_table: torch.Tensor, block_size: int, weights: torch.Tensor, *,
                                 decay: float = 1.0, window_size: int = 0,
                                 replay_start: Optional[torch.Tensor] = None,
                                 base_offsets: Optional[torch.Tensor] = None,
                                 is_valid_token: Optional[torch.Tensor] = None,
                                 softmax_scale: Optional[float] = None,
                                 sink: Optional[torch.Tensor] = None, rope_dim: int = 64,
                                 out: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``decay * weights`` [R, W] plus the attention each cached row got from the new tokens ``q``
    [T, H, D], summed over tokens and heads: a chunk as chunk_mla_attention took it, with the
    ``lse`` [T, H] it returned.  In place unless ``out`` is given; entries past ``seq_lens`` are left
    as they were.  The new tokens' own rows add to what ``weights`` holds there like any other, so the
    caller sets them to 0 first (see select_cache_evictions).  ``window_size`` and ``replay_start`` count
    rows, which after an eviction are not positions.  ``workspace`` (uint8) is scratch; two calls that
    can run at once need one each."""
    i, i32 = _index(q), torch.int32
    qa = _heads(q, "q", i)
    T, H, D = q.shape
    if lse.dtype != torch.float32:
        raise TypeError(f"lse must be {torch.float32}, got {lse.dtype}")
    _same(lse, i, "lse")
    if lse.shape != (T, H) or (H > 1 and lse.stride(1) != 1):
        raise ValueError(f"lse must be [{T}, {H}] with unit inner stride")
    R = seq_lens.numel()
    width = weights.shape[1] if weights.dim() == 2 else 0
    w = _per_row(weights, torch.float32, "weights", R, width, i)
    if out is None:
        out, o = weights, w
    else:
        o = _per_row(out, torch.float32, "out", R, width, i)
    if R > 1 and o[1] < width:
        raise ValueError("rows of weights must not overlap")
    valid = None if is_valid_token is None else is_valid_token.to(torch.uint8)
    if workspace is None:
        need = _weights_workspace.get(i)  # a property of the device
        if need is None:
            need = _weights_workspace[i] = accumulate_attention_weights_workspace_bytes(q.device)
        workspace = torch.empty((need,), dtype=torch.uint8, device=q.device)
    else:
        _vec(workspace, torch.uint8, "workspace", 0, i)
    _call(q.device, "accumulate_attention_weights", *qa, T, H, lse.data_ptr(),
          lse.stride(0) if T > 1 else H, *_cache_of(cache, "cache", i), block_size, D, rope_dim,
          _vec(query_start_loc, i32, "query_start_loc", R + 1, i), _vec(seq_lens, i32, "seq_lens", R, i),
          _vec(replay_start, i32, "replay_start", R, i), R, *_table(block_table, "block_table", R, i),
          _vec(base_offsets, i32, "base_offsets", R, i), window_size,
          _vec(valid, torch.uint8, "is_valid_token", T, i),
          D ** -0.5 if softmax_scale is None else softmax_scale,
          _vec(sink, torch.float32, "sink", H, i), *w, width, decay, *o, workspace.data_ptr(),
          workspace.numel())
    return out


def select_cache_evictions(weights: torch.Tensor, seq_lens: torch.Tensor, keep_lens: torch.Tensor, *,
                           row_positions: Optional[torch.Tensor] = None, num_first: int = 0,
                           num_recent: int = 0, weights_out: Optional[torch.Tensor] = None,
                           positions_out: Optional[torch.Tensor] = None,
                           moves: Optional[torch.Tensor] = None,
                           num_moves: Optional[torch.Tensor] = None,
                           seq_lens_out: Optional[torch.Tensor] = None,
                           err_count: Optional[torch.Tensor] = None):
    """Choose the ``keep_lens`` [R] rows of the greatest ``weights`` [R, W] of each request (with the
    first ``num_first`` positions and the ``num_recent`` newest ones protected) and the moves that
    bring them below the new length.  ``weights`` and ``row_positions`` are updated in place unless
    ``weights_out`` / ``positions_out`` are given.  Returns (moves [R, W // 2, 2] of which
    ``num_moves`` are set, num_moves [R], seq_lens [R], weights, row_positions).

    Entries from the new length on keep what they held, weights and positions of rows that have moved
    or gone: the caller writes those of the rows that new tokens take there.  Rows then stand in no
    order of positions, so calls that take a row for its position (windows, replay starts, top-k and
    sliding-window indices, the positions of compute_slot_mappings) see rows.  A step over a cache of
    at most ``keep`` [R] rows a request, ``lens`` [R] of which are there, with new tokens at ``positions``
    (none of them padding)::

        ops.apply_rotary_embedding(positions, q, cos_sin, k, q_out=q, k_out=k)  # the last 64 dims
        seq_lens = lens + qsl.diff()
        rows, req, slots, _ = ops.compute_slot_mappings(qsl, seq_lens, table, 64, q.shape[0])
        ops.quantize_and_insert_k_cache(k, cache, slots, 64)
        at = req.long(), rows  # of the new rows, over what an evicted row may have left there
        weights[at], row_positions[at] = 0.0, positions.int()
        out, lse = ops.chunk_mla_attention(q, cache, qsl, seq_lens, req, table, 64)
        ops.accumulate_attention_weights(q, lse, cache, qsl, seq_lens, table, 64, weights)
        moves, counts, lens, _, _ = ops.select_cache_evictions(
            weights, seq_lens, keep, row_positions=row_positions, num_first=4, num_recent=64)
        ops.move_cache_rows(cache, table, moves, counts, 64, 512)
    """
    i, i32 = _index(weights), torch.int32
    dev, R = weights.device, seq_lens.numel()
    width = weights.shape[1] if weights.dim() == 2 else 0
    w = _per_row(weights, torch.float32, "weights", R, width, i)
    p = _per_row(row_positions, i32, "row_positions", R, width, i)
    if weights_out is None:
        weights_out, wo = weights, w
    else:
        wo = _per_row(weights_out, torch.float32, "weights_out", R, width, i)
    if positions_out is None:
        positions_out, po = row_positions, p
    else:
        po = _per_row(positions_out, i32, "positions_out", R, width, i)
    for t, a in ((weights_out, wo), (positions_out, po)):
        if t is not None and R > 1 and a[1] < width:
            raise ValueError("rows of weights and row_positions must not overlap")
    if moves is None:
        moves = torch.empty((R, width // 2, 2), dtype=i32, device=dev)
    if num_moves is None:
        num_moves = torch.empty((R,), dtype=i32, device=dev)
    if seq_lens_out is None:
        seq_lens_out = torch.empty((R,), dtype=i32, device=dev)
    _call(dev, "select_cache_evictions", *w, _vec(seq_lens, i32, "seq_lens", R, i),
          _vec(keep_lens, i32, "keep_lens", R, i), R, width, *p, num_first, num_recent, *wo, *po,
          *_move_list(moves, R, width // 2, i), _vec(num_moves, i32, "num_moves", R, i),
          _vec(seq_lens_out, i32, "seq_lens_out", R, i), _vec(err_count, i32, "err_count", 1, i))
    return moves, num_moves, seq_lens_out, weights_out, positions_out


def move_cache_rows(cache: torch.Tensor, block_table: torch.Tensor, moves: torch.Tensor,
                    num_moves: torch.Tensor, block_size: int, head_dim: int, *,
                    record: int = PSK_REC_FP8_DS_MLA, rope_dim: int = 64, is_ue8m0: bool = True,
                    base_offsets: Optional[torch.Tensor] = None,
                    err_count: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Carry out the ``moves`` [R, M, 2] (from, to; ``num_moves`` [R] of them) of
    select_cache_evictions in ``cache``, through ``block_table``."""
    i, i32 = _index(cache), torch.int32
    R = num_moves.numel()
    count = moves.shape[1] if moves.dim() == 3 else 0
    _call(cache.device, "move_cache_rows", cache.data_ptr(), *_pages(cache), block_size, record, head_dim,
          rope_dim if record == PSK_REC_FP8_DS_MLA else 0, int(bool(is_ue8m0)),
          *_table(block_table, "block_table", R, i), _vec(base_offsets, i32, "base_offsets", R, i), R,
          *_move_list(moves, R, count, i), count, _vec(num_moves, i32, "num_moves", R, i),
          _vec(err_count, i32, "err_count", 1, i))
    return cache
