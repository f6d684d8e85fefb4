"""paged_kv_cache_int64_gb300 - attention over a paged KV cache with int64 block addressing, for
NVIDIA GB300 (sm_103a).

A thin Python binding over the C ABI of libpkv.so (include/pkv.h): every function here only
marshals torch tensors into pointers, strides and sizes and calls the library on the current
CUDA stream; all computation runs in the library's CUDA kernels. There is no CPU fallback: if the
library is missing or fails to load, importing this package raises.
"""
from __future__ import annotations

import ctypes as C
import math
import os
import struct

import torch

from . import _build

__all__ = [
    "PKV_OK", "PKV_ERR_INVALID_ARG", "PKV_ERR_UNSUPPORTED", "PKV_ERR_CUDA", "PKV_ERR_DEVICE_BOUNDS",
    "PKV_ERR_TIMEOUT", "PKV_QK_BF16", "PKV_QK_INT8", "PKV_KV_BF16", "PKV_KV_INT8", "PKV_KV_FP8", "PkvError", "lib",
    "library_path", "kv_cache_write", "kv_int8_stats_quant", "paged_prefill_attn_fp8", "kv_fp8_dequant_dense", "paged_prefill_attn", "paged_prefill_workspace_bytes", "spec_verify_workspace_bytes", "spec_verify_pick_split",
    "spec_verify_attn_partial", "spec_verify_attn_partial_fp8", "spec_verify_combine", "EXPORTED_SYMBOLS",
    "kv_cache_write_fp4", "kv_fp4_dequant_dense", "spec_verify_attn_fp4", "spec_verify_fp4_workspace_bytes",
    "PKV_KV_FP4", "spec_verify_accept", "kv_attn_weights", "kv_attn_weights_workspace_bytes", "kv_evict_select",
    "kv_cache_compact", "kv_cache_compact_workspace_bytes",
]

PKV_OK, PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA, PKV_ERR_DEVICE_BOUNDS, PKV_ERR_TIMEOUT = range(6)
PKV_QK_BF16, PKV_QK_INT8 = 0, 1
PKV_KV_BF16, PKV_KV_INT8, PKV_KV_FP8, PKV_KV_FP4 = 0, 1, 2, 3

EXPORTED_SYMBOLS = (
    "pkv_last_error", "pkv_abi_version", "pkv_kv_int8_stats_quant", "pkv_kv_fp8_dequant_dense",
    "pkv_paged_prefill_attn", "pkv_spec_verify_workspace_bytes", "pkv_spec_verify_attn_partial",
    "pkv_spec_verify_combine", "pkv_spec_verify_attn_partial_fp8", "pkv_spec_verify_noalloc_capacity_bytes",
    "pkv_spec_verify_attn_noalloc", "pkv_kv_cache_write", "pkv_paged_prefill_attn_fp8",
    "pkv_paged_prefill_workspace_bytes", "pkv_testing_set_wait_limit_ns", "pkv_spec_verify_pick_split",
    "pkv_kv_cache_write_fp4", "pkv_kv_fp4_dequant_dense", "pkv_spec_verify_fp4_workspace_bytes",
    "pkv_spec_verify_attn_fp4", "pkv_spec_verify_accept", "pkv_kv_attn_weights",
    "pkv_kv_attn_weights_workspace_bytes", "pkv_kv_evict_select", "pkv_kv_cache_compact",
    "pkv_kv_cache_compact_workspace_bytes", "pkv_call_packed",
)

library_path = _build.LIB


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkv status {status}: {message}")
        self.status = status


def _load():
    if not os.path.exists(library_path):
        raise ImportError(f"{library_path} is missing: build it first with "
                          "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc); there is no CPU fallback")
    L = C.CDLL(library_path)
    i32, i64, f32, vp, sz = C.c_int32, C.c_int64, C.c_float, C.c_void_p, C.c_size_t
    L.pkv_last_error.restype = C.c_char_p
    L.pkv_abi_version.restype = i32
    L.pkv_testing_set_wait_limit_ns.argtypes = [C.c_uint64]
    L.pkv_testing_set_wait_limit_ns.restype = None
    L.pkv_kv_int8_stats_quant.argtypes = [vp, i64, i64, i64, i64, vp, i64, i32, vp, vp, i32, i32, i32, i32, i32,
                                          vp, vp, vp, i64, vp, vp]
    L.pkv_kv_fp8_dequant_dense.argtypes = [vp, vp, i64, i64, i64, i64, vp, i64, i32, vp, i32, i32, i32, i32, i32,
                                           vp, vp, vp, vp, vp, vp]
    L.pkv_paged_prefill_attn.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp, i64, i32, vp, vp, i32, i32, i32, i32,
                                         i32, i32, i32, f32, i32, vp, vp, vp, i64, vp, vp, i64, vp, vp]
    L.pkv_paged_prefill_workspace_bytes.argtypes = [i32]
    L.pkv_paged_prefill_workspace_bytes.restype = sz
    L.pkv_spec_verify_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.pkv_spec_verify_workspace_bytes.restype = sz
    L.pkv_spec_verify_pick_split.argtypes = [vp, i32, i32, i32, i32, i32]
    L.pkv_spec_verify_pick_split.restype = i32
    L.pkv_spec_verify_attn_partial.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, i64, i32, vp,
                                               i32, i32, i32, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp]
    L.pkv_spec_verify_combine.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp]
    L.pkv_spec_verify_attn_partial_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i64, i32, vp, i32,
                                                   i32, i32, i32, i32, i32, f32, i32, i32, vp, vp, vp, vp]
    L.pkv_spec_verify_noalloc_capacity_bytes.argtypes = []
    L.pkv_spec_verify_noalloc_capacity_bytes.restype = sz
    L.pkv_spec_verify_attn_noalloc.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, vp, i64, i32, vp,
                                               i32, i32, i32, i32, i32, i32, f32, i32, i32, vp, vp, vp]
    L.pkv_spec_verify_attn_noalloc.restype = i32
    L.pkv_kv_cache_write.argtypes = [vp, vp, i64, vp, i64, i32, vp, vp, i32, i32, i32, vp, vp, i64, i64, i64, i64,
                                     vp, vp, i64, i64, vp, vp, i32, i32, i32, vp, vp]
    L.pkv_paged_prefill_attn_fp8.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i64, i32, vp, vp, i32, i32,
                                             i32, i32, i32, i32, i32, f32, vp, vp, i64, vp, vp]
    cache4 = [i64] * 7  # num_blocks, three code strides, three scale strides
    L.pkv_kv_cache_write_fp4.argtypes = [vp, vp, i64, vp, i64, i32, vp, vp, i32, i32, vp, vp, vp, vp, vp, vp, *cache4,
                                         i32, i32, i32, vp, vp]
    L.pkv_kv_fp4_dequant_dense.argtypes = [vp, vp, vp, vp, vp, vp, *cache4, vp, i64, i32, vp, vp, i32, i32, i32, i32,
                                           i32, vp, vp, i64, vp, vp]
    L.pkv_spec_verify_attn_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, *cache4, vp, i64, i32, vp, i32, i32, i32, i32,
                                           i32, i32, f32, vp, vp, i64, vp, vp]
    L.pkv_spec_verify_fp4_workspace_bytes.argtypes = [i32]
    L.pkv_spec_verify_fp4_workspace_bytes.restype = sz
    L.pkv_spec_verify_accept.argtypes = [vp, i64, i64, vp, i64, i64, i32, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.pkv_kv_attn_weights.argtypes = [vp, vp, i32, vp, *[i64] * 6, vp, i64, i32, vp, vp, *[i32] * 6, f32, vp, i32, i32,
                                      vp, vp, vp, i64, i64, i64, vp, i64, vp, vp]
    L.pkv_kv_evict_select.argtypes = [vp, i64, i64, i64, vp, *[i32] * 5, vp, vp, vp, vp]
    L.pkv_kv_cache_compact.argtypes = [vp, vp, i32, *[i64] * 4, vp, vp, i64, i64, i64, vp, i64, i32, vp, i64, i32, vp, vp,
                                       *[i32] * 5, vp, i64, i64, i64, vp, i64, vp, vp]
    for name in ("pkv_kv_attn_weights_workspace_bytes", "pkv_kv_cache_compact_workspace_bytes"):
        getattr(L, name).argtypes = [i32, i32, i32]
        getattr(L, name).restype = sz
    L.pkv_call_packed.argtypes = [i32, C.c_char_p, i64]
    for name in ("pkv_spec_verify_accept", "pkv_kv_attn_weights", "pkv_kv_evict_select", "pkv_kv_cache_compact", "pkv_call_packed"):
        getattr(L, name).restype = i32
    for name in ("pkv_kv_cache_write_fp4", "pkv_kv_fp4_dequant_dense", "pkv_spec_verify_attn_fp4"):
        getattr(L, name).restype = i32
    for name in ("pkv_paged_prefill_attn_fp8", "pkv_kv_cache_write", "pkv_kv_int8_stats_quant", "pkv_kv_fp8_dequant_dense", "pkv_paged_prefill_attn",
                 "pkv_spec_verify_attn_partial", "pkv_spec_verify_combine", "pkv_spec_verify_attn_partial_fp8"):
        getattr(L, name).restype = i32
    return L


lib = _load()


def _check(status: int):
    if status != PKV_OK:
        raise PkvError(status, lib.pkv_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _cache_strides(cache: torch.Tensor):
    """[num_blocks][block_size][num_kv_heads][head_dim] view with a contiguous last dim."""
    assert cache.dim() == 4 and cache.stride(3) == 1, "cache must be [nb][bs][hkv][D] with contiguous D"
    nb, bs, hkv, d = cache.shape
    return nb, bs, hkv, d, cache.stride(0), cache.stride(1), cache.stride(2)


def _ws_bytes(ws):
    if ws is None:
        return 0
    assert ws.is_cuda and ws.is_contiguous(), "workspace must be a contiguous CUDA tensor"
    return ws.numel() * ws.element_size()


def _i32(t):
    assert t.dtype == torch.int32 and t.is_cuda, "expected a CUDA int32 tensor"
    return t


# ---------------------------------------------------------------------------------------------
# the five calls (names of the C ABI without the pkv_ prefix)
# ---------------------------------------------------------------------------------------------

def kv_cache_write(k_new, v_new, block_table, seq_lens, query_start_loc, max_q_len, k_cache, v_cache,
                   kv_dtype=PKV_KV_BF16, k_scale_cache=None, v_scale_cache=None, k_scale=None, v_scale=None,
                   dev_err=None, stream=None):
    """Store the chunk's new rows k_new / v_new (bf16 [total_q][hkv][D], token stride free) into the paged
    caches ([nb][bs][hkv][D]: bf16, int8 with fp32 scale caches [nb][bs][hkv], or uint8 e4m3 with device
    scalar scales k_scale / v_scale) at positions seq_lens[r] - q_len + i."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_cache)
    assert v_cache.stride() == k_cache.stride() and v_cache.shape == k_cache.shape
    want = {PKV_KV_BF16: torch.bfloat16, PKV_KV_INT8: torch.int8, PKV_KV_FP8: torch.uint8}[kv_dtype]
    assert k_cache.dtype == want and v_cache.dtype == want, f"cache dtype must be {want}"
    assert k_new.dtype == torch.bfloat16 and v_new.dtype == torch.bfloat16 and k_new.stride() == v_new.stride()
    assert k_new.dim() == 3 and k_new.stride(2) == 1 and k_new.stride(1) == d, "new rows: [total][hkv][D], heads contiguous"
    ssb = sst = 0
    if kv_dtype == PKV_KV_INT8:
        assert k_scale_cache.dtype == torch.float32 and k_scale_cache.stride() == v_scale_cache.stride()
        assert k_scale_cache.stride(2) == 1
        ssb, sst = k_scale_cache.stride(0), k_scale_cache.stride(1)
    _i32(block_table)
    R = block_table.shape[0]
    _check(lib.pkv_kv_cache_write(_ptr(k_new), _ptr(v_new), k_new.stride(0), _ptr(block_table), block_table.stride(0),
                                  block_table.shape[1], _ptr(_i32(seq_lens)), _ptr(_i32(query_start_loc)), R,
                                  int(max_q_len), int(kv_dtype), _ptr(k_cache), _ptr(v_cache), nb, sb, st, sh,
                                  _ptr(k_scale_cache), _ptr(v_scale_cache), ssb, sst, _ptr(k_scale), _ptr(v_scale), bs,
                                  hkv, d, _ptr(dev_err), _stream(stream)))


def kv_int8_stats_quant(k_cache, block_table, pos_begin, pos_end, max_tokens, k8, k8_scale, dev_err=None,
                        stream=None, k16=None):
    """Per-token-head int8 quantization of the paged bf16 K cache into k8 [R][max_ctx][hkv][D] int8 and
    k8_scale [R][max_ctx][hkv] fp32 for positions [pos_begin[r], pos_end[r]); k16 (optional, fp16, same
    shape as k8) also receives the codes as fp16 values."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_cache)
    assert k_cache.dtype == torch.bfloat16, "kv_int8_stats_quant reads a bf16 K cache"
    _i32(block_table)
    R = block_table.shape[0]
    assert k8.dtype == torch.int8 and k8.is_contiguous() and k8_scale.dtype == torch.float32
    _check(lib.pkv_kv_int8_stats_quant(_ptr(k_cache), nb, sb, st, sh, _ptr(block_table), block_table.stride(0),
                                       block_table.shape[1], _ptr(_i32(pos_begin)), _ptr(_i32(pos_end)), R,
                                       int(max_tokens), bs, hkv, d, _ptr(k8), _ptr(k8_scale), _ptr(k16), k8.shape[1],
                                       _ptr(dev_err), _stream(stream)))


def kv_fp8_dequant_dense(k_fp8, v_fp8, block_table, seq_lens, k_scale, v_scale, k_dense, v_dense, dev_err=None,
                         stream=None):
    """e4m3 paged K/V (uint8 [nb][bs][hkv][D]) -> dense bf16 [R][max_seq][hkv][D] for pos < seq_lens[r]."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_fp8)
    assert v_fp8.stride() == k_fp8.stride() and v_fp8.shape == k_fp8.shape
    assert k_fp8.dtype == torch.uint8 and v_fp8.dtype == torch.uint8, "e4m3 caches are uint8 tensors"
    _i32(block_table)
    R = block_table.shape[0]
    assert k_dense.is_contiguous() and v_dense.is_contiguous() and k_dense.dtype == torch.bfloat16
    _check(lib.pkv_kv_fp8_dequant_dense(_ptr(k_fp8), _ptr(v_fp8), nb, sb, st, sh, _ptr(block_table),
                                        block_table.stride(0), block_table.shape[1], _ptr(_i32(seq_lens)), R,
                                        k_dense.shape[1], bs, hkv, d, _ptr(k_scale), _ptr(v_scale), _ptr(k_dense),
                                        _ptr(v_dense), _ptr(dev_err), _stream(stream)))


def paged_prefill_attn(q, k_cache, v_cache, block_table, seq_lens, query_start_loc, max_q_len, softmax_scale,
                       out, qk_mode=PKV_QK_BF16, k8=None, k8_scale=None, dev_err=None, stream=None, k16=None,
                       workspace=None):
    """Chunked causal prefill attention. q/out bf16 [total_q][Hq][D]; caches bf16 [nb][bs][hkv][D]
    (k_cache may be None in int8 mode, which reads k8 (or its fp16 copy k16) and k8_scale from
    kv_int8_stats_quant). workspace: None (one CTA per query tile) or a CUDA byte tensor of
    paged_prefill_workspace_bytes() bytes (persistent grid: full waves, last wave cut into key ranges)."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(v_cache)
    assert v_cache.dtype == torch.bfloat16 and (k_cache is None or k_cache.dtype == torch.bfloat16), \
        "paged_prefill_attn reads bf16 caches (e4m3 caches: paged_prefill_attn_fp8)"
    if k_cache is not None:
        assert k_cache.stride() == v_cache.stride() and k_cache.shape == v_cache.shape
    assert q.is_contiguous() and out.is_contiguous() and q.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    _i32(block_table)
    R = block_table.shape[0]
    max_ctx = 0 if k8 is None and k16 is None else (k8 if k8 is not None else k16).shape[1]
    _check(lib.pkv_paged_prefill_attn(_ptr(q), _ptr(k_cache), _ptr(v_cache), nb, sb, st, sh, _ptr(block_table),
                                      block_table.stride(0), block_table.shape[1], _ptr(_i32(seq_lens)),
                                      _ptr(_i32(query_start_loc)), R, q.shape[0], int(max_q_len), q.shape[1],
                                      hkv, d, bs, float(softmax_scale), int(qk_mode), _ptr(k8), _ptr(k8_scale),
                                      _ptr(k16), max_ctx, _ptr(out), _ptr(workspace), _ws_bytes(workspace),
                                      _ptr(dev_err), _stream(stream)))


def paged_prefill_attn_fp8(q, k_fp8, v_fp8, k_scale, v_scale, block_table, seq_lens, query_start_loc, max_q_len,
                           softmax_scale, out, dev_err=None, stream=None, workspace=None):
    """Chunked causal prefill attention read straight from per-tensor e4m3 paged K/V (uint8
    [nb][bs][hkv][D]) with device scalar scales; each tile is dequantized in shared memory."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_fp8)
    assert v_fp8.stride() == k_fp8.stride() and v_fp8.shape == k_fp8.shape
    assert k_fp8.dtype == torch.uint8 and v_fp8.dtype == torch.uint8
    assert q.is_contiguous() and out.is_contiguous() and q.dtype == torch.bfloat16 and out.dtype == torch.bfloat16
    _i32(block_table)
    R = block_table.shape[0]
    _check(lib.pkv_paged_prefill_attn_fp8(_ptr(q), _ptr(k_fp8), _ptr(v_fp8), _ptr(k_scale), _ptr(v_scale), nb, sb, st,
                                          sh, _ptr(block_table), block_table.stride(0), block_table.shape[1],
                                          _ptr(_i32(seq_lens)), _ptr(_i32(query_start_loc)), R, q.shape[0],
                                          int(max_q_len), q.shape[1], hkv, d, bs, float(softmax_scale), _ptr(out),
                                          _ptr(workspace), _ws_bytes(workspace), _ptr(dev_err), _stream(stream)))


def paged_prefill_workspace_bytes(num_ctas=None) -> int:
    """bytes of the persistent prefill workspace for num_ctas CTAs (default: the current device's SM
    count, the persistent grid's size)."""
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(lib.pkv_paged_prefill_workspace_bytes(int(num_ctas)))


def spec_verify_workspace_bytes(num_tokens, num_q_heads, head_dim, max_splits) -> int:
    return int(lib.pkv_spec_verify_workspace_bytes(num_tokens, num_q_heads, head_dim, max_splits))


def spec_verify_pick_split(seq_lens, T, num_q_heads, num_kv_heads, num_sms) -> int:
    """Host-side split_tokens choice for spec_verify_attn_partial from the batch's sequence lengths
    (host values); 0 on a bad argument."""
    import numpy as np
    sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    return int(lib.pkv_spec_verify_pick_split(sl.ctypes.data, int(sl.shape[0]), int(T), int(num_q_heads),
                                               int(num_kv_heads), int(num_sms)))


def spec_verify_attn_partial(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, T, softmax_scale,
                             split_tokens, part_o, part_lse, dev_err=None, stream=None):
    """Split-KV verify partials over an int8 cache ([nb][bs][hkv][D]) with fp32 per-token-head
    scales ([nb][bs][hkv]); part_o [S][R*T][Hq][D], part_lse [S][R*T][Hq] fp32."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_cache)
    assert k_cache.dtype == torch.int8 and v_cache.dtype == torch.int8, "int8 caches"
    assert v_cache.stride() == k_cache.stride() and k_scale.stride() == v_scale.stride()
    assert k_scale.dim() == 3 and k_scale.stride(2) == 1
    _i32(block_table)
    R = block_table.shape[0]
    max_splits = part_o.shape[0]
    _check(lib.pkv_spec_verify_attn_partial(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                            nb, sb, st, sh, k_scale.stride(0), k_scale.stride(1),
                                            _ptr(block_table), block_table.stride(0), block_table.shape[1],
                                            _ptr(_i32(seq_lens)), R, int(T), q.shape[1], hkv, d, bs,
                                            float(softmax_scale), int(split_tokens), max_splits, _ptr(part_o),
                                            _ptr(part_lse), _ptr(dev_err), _stream(stream)))


def spec_verify_attn_partial_fp8(q, k_fp8, v_fp8, k_descale, v_descale, block_table, seq_lens, T, softmax_scale,
                                 split_tokens, part_o, part_lse, dev_err=None, stream=None):
    """Split-KV verify partials over a per-tensor fp8 e4m3 cache (uint8 [nb][bs][hkv][D]); k_descale /
    v_descale: device fp32 scalars."""
    nb, bs, hkv, d, sb, st, sh = _cache_strides(k_fp8)
    assert v_fp8.stride() == k_fp8.stride()
    assert k_fp8.dtype == torch.uint8 and v_fp8.dtype == torch.uint8, "e4m3 caches are uint8 tensors"
    _i32(block_table)
    R = block_table.shape[0]
    _check(lib.pkv_spec_verify_attn_partial_fp8(_ptr(q), _ptr(k_fp8), _ptr(v_fp8), _ptr(k_descale),
                                                _ptr(v_descale), nb, sb, st, sh, _ptr(block_table),
                                                block_table.stride(0), block_table.shape[1], _ptr(_i32(seq_lens)), R,
                                                int(T), q.shape[1], hkv, d, bs, float(softmax_scale),
                                                int(split_tokens), part_o.shape[0], _ptr(part_o), _ptr(part_lse),
                                                _ptr(dev_err), _stream(stream)))


def spec_verify_combine(part_o, part_lse, seq_lens, T, split_tokens, out, stream=None):
    """Log-sum-exp merge of the partials into out bf16 [R*T][Hq][D]."""
    max_splits, rows_t, hq, d = part_o.shape
    R = seq_lens.shape[0]
    _check(lib.pkv_spec_verify_combine(_ptr(part_o), _ptr(part_lse), _ptr(_i32(seq_lens)), R, int(T), hq, d,
                                       int(split_tokens), max_splits, _ptr(out), _stream(stream)))


def splits_needed(max_seq_len: int, split_tokens: int) -> int:
    return max(1, math.ceil(max_seq_len / split_tokens))


# ---------------------------------------------------------------------------------------------
# the 4-bit cache: e2m1 codes uint8 [nb][bs][hkv][128], e4m3 scale bytes uint8 [nb][bs][hkv][16],
# one fp32 scale per tensor
# ---------------------------------------------------------------------------------------------

# The smallest calls run for two or three microseconds on the device, so the checks below keep to few
# attribute reads: one test a property, devices as indices, the raw stream.
_U8, _I32, _F32, _BF16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _cache4(k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale):
    """The checked cache's device index, the ABI's (num_blocks, strides), block_size, heads."""
    shape, cs, ss = k_fp4.shape, k_fp4.stride(), k_bscale.stride()
    nb, bs, hkv, row = shape
    assert row == 128 and v_fp4.shape == shape and k_bscale.shape == v_bscale.shape == (nb, bs, hkv, 16), \
        "codes [nb][bs][hkv][128], scales [nb][bs][hkv][16]"
    assert v_fp4.stride() == cs and v_bscale.stride() == ss and cs[3] == 1 and ss[3] == 1, "K and V strides must agree"
    assert k_fp4.dtype is v_fp4.dtype is k_bscale.dtype is v_bscale.dtype is _U8, "the 4-bit cache is uint8 tensors"
    assert k_scale.dtype is v_scale.dtype is _F32, "k_scale and v_scale are fp32 device scalars"
    dev = k_fp4.get_device()
    assert dev >= 0 and dev == v_fp4.get_device() == k_bscale.get_device() == v_bscale.get_device() == \
        k_scale.get_device() == v_scale.get_device(), "the cache and its scales must be on one CUDA device"
    return dev, (nb, cs[0], cs[1], cs[2], ss[0], ss[1], ss[2]), bs, hkv


def _table(block_table, *vectors):
    """The checked block table's requests, columns and row stride; vectors: its int32 companions."""
    R, cols = block_table.shape
    row, col = block_table.stride()
    assert block_table.dtype is _I32 and (col == 1 or cols == 1), "int32 block_table [R][..], columns contiguous"
    for t in vectors:
        assert t.dtype is _I32 and t.dim() == 1 and t.is_contiguous(), "int32 vectors, contiguous, beside the block table"
    return R, cols, row


def _raw_stream(dev, stream):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _launch(fn, dev, others, args):
    """fn(*args) with device `dev` current; the tensors `others` must be on it."""
    for t in others:
        assert t.get_device() == dev, "tensors of one call must be on one device"
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != PKV_OK:
        _check(rc)


def _packed(call, fn):
    """The call of that number with fn's arguments packed into one array (null pointers as 0): ctypes takes 0.11 us to
    convert an argument (attention weights of one request of 1,024 back to back: 13.0 us, 10.9 packed)."""
    pack = struct.Struct("=" + "".join("d" if t is C.c_float else "q" for t in fn.argtypes)).pack
    entry, size = lib.pkv_call_packed, 8 * len(fn.argtypes)
    return lambda *args: entry(call, pack(*args), size)


_spec_verify_accept = _packed(0, lib.pkv_spec_verify_accept)
_kv_attn_weights = _packed(1, lib.pkv_kv_attn_weights)
_kv_evict_select = _packed(2, lib.pkv_kv_evict_select)
_kv_cache_compact = _packed(3, lib.pkv_kv_cache_compact)


def _err(dev_err, dev):
    if dev_err is None:
        return 0
    assert dev_err.dtype is _I32 and dev_err.get_device() == dev, "dev_err: int32 on the cache's device"
    return dev_err.data_ptr()


def kv_cache_write_fp4(k_new, v_new, block_table, seq_lens, query_start_loc, max_q_len, k_fp4, v_fp4, k_bscale,
                       v_bscale, k_scale, v_scale, dev_err=None, stream=None):
    """Quantize the chunk's new rows k_new / v_new (bf16 [total_q][hkv][256], token stride free) to 4 bits
    and store them into the paged cache at positions seq_lens[r] - q_len + i."""
    dev, cache, bs, hkv = _cache4(k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale)
    st = k_new.stride()
    _, heads, d = k_new.shape
    assert k_new.dtype is v_new.dtype is _BF16 and v_new.shape == k_new.shape and v_new.stride() == st and \
        heads == hkv and st[2] == 1 and st[1] == d, "new rows: bf16 [total][hkv][D], heads contiguous, K and V alike"
    R, cols, row = _table(block_table, seq_lens, query_start_loc)
    assert seq_lens.shape[0] == R and query_start_loc.shape[0] == R + 1, "seq_lens [R], query_start_loc [R + 1]"
    _launch(lib.pkv_kv_cache_write_fp4, dev, (k_new, v_new, block_table, seq_lens, query_start_loc),
            (k_new.data_ptr(), v_new.data_ptr(), st[0], block_table.data_ptr(), row, cols,
             seq_lens.data_ptr(), query_start_loc.data_ptr(), R, int(max_q_len), k_fp4.data_ptr(), v_fp4.data_ptr(),
             k_bscale.data_ptr(), v_bscale.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *cache, bs, hkv, d,
             _err(dev_err, dev), _raw_stream(dev, stream)))


def kv_fp4_dequant_dense(k_fp4, v_fp4, k_bscale, v_bscale, block_table, pos_begin, pos_end, max_tokens, k_scale, v_scale,
                         k_dense, v_dense, dev_err=None, stream=None):
    """Positions [pos_begin[r], pos_end[r]) of the 4-bit cache -> dense bf16 [R][max_ctx][hkv][256], each at
    its own position."""
    dev, cache, bs, hkv = _cache4(k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale)
    R, max_ctx, heads, d = k_dense.shape
    assert k_dense.dtype is v_dense.dtype is _BF16 and v_dense.shape == k_dense.shape and heads == hkv and \
        k_dense.is_contiguous() and v_dense.is_contiguous(), "dense rows: contiguous bf16 [R][max_ctx][hkv][256]"
    reqs, cols, row = _table(block_table, pos_begin, pos_end)
    assert reqs == pos_begin.shape[0] == pos_end.shape[0] == R, "block_table [R][..], pos_begin, pos_end [R]"
    _launch(lib.pkv_kv_fp4_dequant_dense, dev, (block_table, pos_begin, pos_end, k_dense, v_dense),
            (k_fp4.data_ptr(), v_fp4.data_ptr(), k_bscale.data_ptr(), v_bscale.data_ptr(), k_scale.data_ptr(),
             v_scale.data_ptr(), *cache, block_table.data_ptr(), row, cols, pos_begin.data_ptr(), pos_end.data_ptr(), R,
             int(max_tokens), bs, hkv, d, k_dense.data_ptr(), v_dense.data_ptr(), max_ctx, _err(dev_err, dev),
             _raw_stream(dev, stream)))


def spec_verify_fp4_workspace_bytes(num_ctas=None) -> int:
    """bytes of spec_verify_attn_fp4's workspace for num_ctas CTAs (default: the current device's SM count)."""
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(lib.pkv_spec_verify_fp4_workspace_bytes(int(num_ctas)))


def spec_verify_attn_fp4(q, k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale, block_table, seq_lens, T, softmax_scale,
                         out, workspace, dev_err=None, stream=None):
    """Verify (T tokens a request) or decode (T = 1) attention over the 4-bit cache; q / out bf16
    [R*T][Hq][256]. workspace: a CUDA byte tensor of spec_verify_fp4_workspace_bytes() bytes, one for each
    stream or graph whose calls may overlap."""
    dev, cache, bs, hkv = _cache4(k_fp4, v_fp4, k_bscale, v_bscale, k_scale, v_scale)
    R, cols, row = _table(block_table, seq_lens)
    rows, hq, d = q.shape
    assert q.dtype is out.dtype is _BF16 and out.shape == q.shape and rows == R * T and q.is_contiguous() and \
        out.is_contiguous(), "q and out: contiguous bf16 [R*T][Hq][256]"
    assert seq_lens.shape[0] == R, "seq_lens [R]"
    assert workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor"
    _launch(lib.pkv_spec_verify_attn_fp4, dev, (q, block_table, seq_lens, out, workspace),
            (q.data_ptr(), k_fp4.data_ptr(), v_fp4.data_ptr(), k_bscale.data_ptr(), v_bscale.data_ptr(),
             k_scale.data_ptr(), v_scale.data_ptr(), *cache, block_table.data_ptr(), row, cols, seq_lens.data_ptr(), R,
             int(T), hq, hkv, d, bs, float(softmax_scale), out.data_ptr(), workspace.data_ptr(), workspace.nbytes,
             _err(dev_err, dev), _raw_stream(dev, stream)))


# ---------------------------------------------------------------------------------------------
# after the verify attention: which drafts stay, and which keys
# ---------------------------------------------------------------------------------------------

_PROBS = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_KV_TYPES = {PKV_KV_BF16: torch.bfloat16, PKV_KV_INT8: torch.int8, PKV_KV_FP8: torch.uint8, PKV_KV_FP4: torch.uint8}


def _flat(t, dtype, shape):
    """t's pointer; t: contiguous, of that type and shape."""
    assert t.dtype is dtype and t.shape == shape and t.is_contiguous(), f"expected contiguous {dtype} {list(shape)}"
    return t.data_ptr()


def _maybe(t):
    return None if t is None else t.data_ptr()


def spec_verify_accept(target_probs, draft_probs, draft_ids, u_accept, u_sample, out_tokens, num_out, num_drafts=None,
                       dev_err=None, stream=None):
    """Verify drafted tokens against the target's probabilities [R][T][vocab] (fp32, bf16 or fp16, rows contiguous):
    draft_ids int32 [R][T-1] drawn from draft_probs [R][T-1][vocab] (None: proposed by no distribution), uniform
    numbers u_accept [R][T-1] and u_sample [R] fp32; num_drafts int32 [R] (None: T-1 each). out_tokens int32 [R][T]:
    the accepted drafts, the token drawn after them, -1; num_out int32 [R]: how many are tokens."""
    shape = target_probs.shape
    R, T, V = shape
    sr, st, se = target_probs.stride()
    dev = target_probs.get_device()
    dtype = target_probs.dtype
    assert dtype in _PROBS and (se == 1 or V == 1), "target_probs: fp32, bf16 or fp16 [R][T][vocab], rows contiguous"
    assert dev >= 0, "target_probs must be a CUDA tensor"
    others = (draft_ids, u_accept, u_sample, out_tokens, num_out)
    q = qr = qt = 0
    if draft_probs is not None:
        qr, qt, qe = draft_probs.stride()
        assert draft_probs.dtype is dtype and draft_probs.shape == (R, T - 1, V) and (qe == 1 or V == 1), \
            "draft_probs: [R][T-1][vocab], of target_probs' type, rows contiguous"
        q = draft_probs.data_ptr()
        others += (draft_probs,)
    nd = 0
    if num_drafts is not None:
        nd = _flat(num_drafts, _I32, (R,))
        others += (num_drafts,)
    drafts = (R, T - 1)
    _launch(_spec_verify_accept, dev, others,
            (target_probs.data_ptr(), sr, st, q, qr, qt, _PROBS[dtype], _flat(draft_ids, _I32, drafts),
             _flat(u_accept, _F32, drafts), _flat(u_sample, _F32, (R,)), nd, R, T, V, _flat(out_tokens, _I32, (R, T)),
             _flat(num_out, _I32, (R,)), _err(dev_err, dev), _raw_stream(dev, stream)))


def kv_attn_weights_workspace_bytes(num_rows, num_q_heads, num_ctas=None) -> int:
    """bytes of kv_attn_weights' workspace for num_rows = R*T query rows on num_ctas CTAs (default: the current
    device's SM count)."""
    if num_ctas is None:
        num_ctas = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    return int(lib.pkv_kv_attn_weights_workspace_bytes(int(num_rows), int(num_q_heads), int(num_ctas)))


def kv_attn_weights(q, k_cache, block_table, seq_lens, T, softmax_scale, weights, workspace, kv_dtype=PKV_KV_BF16,
                    k_scale=None, prev=None, prev_lens=None, q_valid=None, part_lse=None, split_tokens=0, dev_err=None,
                    stream=None):
    """weights[r][h][pos] (fp32 [R][hkv][max_ctx]) = prev's (positions < prev_lens[r]) + the attention weight that the key
    collects from tokens t < q_valid[r] of the step's T, all query heads of its KV head; q bf16 [R*T][Hq][256]. k_cache:
    bf16, int8 (k_scale fp32 [nb][bs][hkv]) or uint8 e4m3 (k_scale a device scalar), by kv_dtype. part_lse [S][R*T][Hq] with
    its split_tokens: what a verify call left for the same queries (None: computed first)."""
    nb, bs, hkv, d = k_cache.shape
    sb, st, sh, se = k_cache.stride()
    dev = k_cache.get_device()
    assert dev >= 0 and se == 1 and kv_dtype != PKV_KV_FP4 and k_cache.dtype is _KV_TYPES[kv_dtype], \
        "k_cache: a CUDA tensor [nb][bs][hkv][D] of kv_dtype, D contiguous"
    R, cols, row = _table(block_table, seq_lens)
    rows, hq, dq = q.shape
    assert q.dtype is _BF16 and rows == R * T and dq == d and q.is_contiguous(), "q: contiguous bf16 [R*T][Hq][256]"
    shape, (wr, wh, we) = weights.shape, weights.stride()
    max_ctx = shape[2]
    assert weights.dtype is _F32 and shape[0] == R and shape[1] == hkv and (we == 1 or max_ctx == 1), \
        "weights: fp32 [R][hkv][max_ctx], positions contiguous"
    assert seq_lens.shape[0] == R, "seq_lens [R]"
    assert workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor"
    others = (q, block_table, seq_lens, weights, workspace)
    scale = ssb = sst = 0
    if kv_dtype != PKV_KV_BF16:
        if kv_dtype == PKV_KV_INT8:
            ssb, sst, ssh = k_scale.stride()
            assert k_scale.dtype is _F32 and k_scale.shape == (nb, bs, hkv) and (ssh == 1 or hkv == 1), \
                "k_scale: fp32 [nb][bs][hkv], heads contiguous"
        else:
            assert k_scale.dtype is _F32 and k_scale.numel() == 1, "k_scale: an fp32 device scalar"
        scale = k_scale.data_ptr()
        others += (k_scale,)
    old = lens = valid = lse = splits = 0
    if prev is not None:
        assert prev.dtype is _F32 and prev.shape == shape and prev.stride() == (wr, wh, we), "prev: laid out as weights"
        old = prev.data_ptr()
        others += (prev,)
    if prev_lens is not None:
        lens = _flat(prev_lens, _I32, (R,))
        others += (prev_lens,)
    if q_valid is not None:
        valid = _flat(q_valid, _I32, (R,))
        others += (q_valid,)
    if part_lse is not None:
        splits = part_lse.shape[0]
        lse = _flat(part_lse, _F32, (splits, rows, hq))
        others += (part_lse,)
    _launch(_kv_attn_weights, dev, others,
            (q.data_ptr(), k_cache.data_ptr(), kv_dtype, scale, nb, sb, st, sh, ssb, sst, block_table.data_ptr(), row, cols,
             seq_lens.data_ptr(), valid, R, int(T), hq, hkv, d, bs, float(softmax_scale), lse, int(split_tokens), splits, old,
             lens, weights.data_ptr(), wr, wh, max_ctx, workspace.data_ptr(), workspace.nbytes, _err(dev_err, dev),
             _raw_stream(dev, stream)))


def kv_evict_select(scores, seq_lens, sinks, recent, budget, keep, new_lens, dev_err=None, stream=None):
    """keep int32 [R][hkv][budget] := the positions of each (request, KV head) that stay, ascending: the first `sinks`,
    the last `recent`, the highest of scores (fp32 [R][hkv][max_ctx]) in between; new_lens int32 [R] := how many (a buffer of
    its own, not seq_lens)."""
    R, hkv, max_ctx = scores.shape
    sr, sh, se = scores.stride()
    dev = scores.get_device()
    assert dev >= 0 and scores.dtype is _F32 and (se == 1 or max_ctx == 1), "scores: fp32 [R][hkv][max_ctx] on the GPU, positions contiguous"
    budget = int(budget)
    _launch(_kv_evict_select, dev, (seq_lens, keep, new_lens),
            (scores.data_ptr(), sr, sh, max_ctx, _flat(seq_lens, _I32, (R,)), R, hkv, int(sinks), int(recent), budget,
             _flat(keep, _I32, (R, hkv, budget)), _flat(new_lens, _I32, (R,)), _err(dev_err, dev), _raw_stream(dev, stream)))


def kv_cache_compact_workspace_bytes(num_reqs, num_kv_heads, budget) -> int:
    return int(lib.pkv_kv_cache_compact_workspace_bytes(int(num_reqs), int(num_kv_heads), int(budget)))


def kv_cache_compact(k_cache, v_cache, src_table, dst_table, keep, new_lens, workspace, kv_dtype=PKV_KV_BF16, k_scale=None,
                     v_scale=None, weights=None, dev_err=None, stream=None):
    """Row j of (r, h) := row keep[r][h][j] (int32 [R][hkv][budget], ascending), j < new_lens[r], in K, V, the scale
    caches (int8: fp32 [nb][bs][hkv]; 4-bit: uint8 [nb][bs][hkv][16]) and weights (fp32 [R][hkv][max_ctx]). Read through
    src_table, written through dst_table: the same table, or other blocks."""
    shape, strides = k_cache.shape, k_cache.stride()
    nb, bs, hkv, d = shape
    sb, st, sh, se = strides
    dev = k_cache.get_device()
    assert dev >= 0 and se == 1 and k_cache.dtype is v_cache.dtype is _KV_TYPES[kv_dtype], \
        "caches: CUDA tensors [nb][bs][hkv][D] of kv_dtype, D contiguous"
    assert v_cache.shape == shape and v_cache.stride() == strides, "K and V strides must agree"
    R, cols, row = _table(src_table, new_lens)
    reqs, dcols, drow = (R, cols, row) if dst_table is src_table else _table(dst_table)
    budget = keep.shape[2]
    assert reqs == R == new_lens.shape[0], "src_table, dst_table, new_lens: the same requests"
    assert workspace.is_contiguous(), "workspace must be a contiguous CUDA tensor"
    others = (v_cache, src_table, dst_table, keep, new_lens, workspace)
    scale = (0, 0, 0, 0, 0)
    if kv_dtype in (PKV_KV_INT8, PKV_KV_FP4):
        want = (nb, bs, hkv) if kv_dtype == PKV_KV_INT8 else (nb, bs, hkv, 16)
        ss = k_scale.stride()
        assert k_scale.dtype is v_scale.dtype is (_F32 if kv_dtype == PKV_KV_INT8 else _U8) and k_scale.shape == v_scale.shape == want \
            and v_scale.stride() == ss and ss[3:] in ((), (1,)), "scale caches: fp32 [nb][bs][hkv] (int8) or uint8 [nb][bs][hkv][16] (4-bit)"
        scale = (k_scale.data_ptr(), v_scale.data_ptr(), ss[0], ss[1], ss[2])
        others += (k_scale, v_scale)
    w = (0, 0, 0, 0)
    if weights is not None:
        (wR, wh, max_ctx), (wr, whs, we) = weights.shape, weights.stride()
        assert weights.dtype is _F32 and wR == R and wh == hkv and (we == 1 or max_ctx == 1), \
            "weights: fp32 [R][hkv][max_ctx], positions contiguous"
        w = (weights.data_ptr(), wr, whs, max_ctx)
        others += (weights,)
    _launch(_kv_cache_compact, dev, others,
            (k_cache.data_ptr(), v_cache.data_ptr(), kv_dtype, nb, sb, st, sh, *scale, src_table.data_ptr(), row, cols,
             dst_table.data_ptr(), drow, dcols, _flat(keep, _I32, (R, hkv, budget)), new_lens.data_ptr(), R, hkv, budget, bs,
             d * 2 if kv_dtype == PKV_KV_FP4 else d, *w, workspace.data_ptr(), workspace.nbytes, _err(dev_err, dev),
             _raw_stream(dev, stream)))
