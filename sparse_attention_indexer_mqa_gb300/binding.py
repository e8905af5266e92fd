"""Thin ctypes binding of libidx_gb300.so (include/idx.h).

The functions carry the C names and only marshal arguments: torch tensors become raw
pointers, the stream defaults to torch's current stream, and a non-zero status raises
IdxError. All computation runs in the library's CUDA kernels; there is no fallback: if the
library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes as C
import os
import re
import threading

from . import build as _build

IDX_MXFP4, IDX_FP8 = 0, 1
IDX_ROPE_NONE, IDX_ROPE_NEOX, IDX_ROPE_INTERLEAVED = 0, 1, 2
IDX_STATUS_BAD_SLOT, IDX_STATUS_BAD_POS, IDX_STATUS_BAD_PAGE = 0x1, 0x2, 0x4
IDX_STATUS_TIMEOUT, IDX_STATUS_BAD_LEN = 0x8, 0x10
IDX_STATUS_NO_PAGE, IDX_STATUS_BAD_VALUE = 0x20, 0x40
IDX_BF16, IDX_FP16 = 0, 1

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "idx.h")

_lock = threading.Lock()
_lib = None


class IdxError(RuntimeError):
    def __init__(self, fn, status):
        super().__init__(f"{fn} failed with status {status} ({_status_str(status)})")
        self.status = status


class IdxLayout(C.Structure):
    _fields_ = [("page_bytes", C.c_int64), ("code_offset", C.c_int64),
                ("code_bytes", C.c_int64), ("scale_offset", C.c_int64),
                ("scale_bytes", C.c_int64), ("bytes_per_token", C.c_int32),
                ("page_size", C.c_int32)]


class IdxKvLayout(C.Structure):
    _fields_ = [("page_bytes", C.c_int64), ("head_bytes", C.c_int64), ("scale_offset", C.c_int64),
                ("scale_block", C.c_int32), ("page_size", C.c_int32), ("kv_heads", C.c_int32),
                ("head_dim", C.c_int32)]


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load (building first if needed) the CUDA library; raises if that is impossible."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"CUDA library {path} is missing; run build() first")
            lib = C.CDLL(path)
            _declare(lib)
            _lib = lib
    return _lib


def exported_names():
    """Entry points declared in include/idx.h."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|const char\*)\s+(idx_\w+)\(", txt, re.M)))


def _declare(L):
    vp, i64, i32, f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_float
    L.idx_status_string.argtypes = [C.c_int]; L.idx_status_string.restype = C.c_char_p
    L.idx_cache_layout.argtypes = [i32, i32, C.POINTER(IdxLayout)]
    L.idx_k_store.argtypes = [vp, i64, i64, vp, vp, vp, i32, i32, i32, vp, vp, f32, i32, vp, i64,
                              i32, i64, vp, vp]
    L.idx_q_quant.argtypes = [vp, i64, i32, vp, vp, i32, i32, vp, f32, f32, i32, vp, vp, vp, vp,
                              vp]
    L.idx_qk_prep.argtypes = [vp, i64, i64, vp, vp, i32, i32, vp, vp, f32, vp, i64, i32, i64,
                              vp, i64, i32, vp, i32, vp, f32, f32, vp, vp, vp, vp, i32, i32, vp, vp]
    L.idx_mqa_logits_paged.argtypes = [vp, vp, vp, i64, i32, i32, vp, i64, i32, i64, vp, i32, vp,
                                       vp, i32, i32, i32, i32, vp, i64, vp, C.c_size_t, vp, vp]
    L.idx_mqa_logits_workspace_bytes.argtypes = [C.POINTER(C.c_size_t)]
    L.idx_topk.argtypes = [vp, i64, vp, vp, i32, i64, i32, i32, i32, vp, vp, vp]
    L.idx_debug_encode.argtypes = [i32, vp, i64, vp, vp]
    L.idx_mqa_topk_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, C.POINTER(C.c_size_t)]
    L.idx_mqa_topk_paged.argtypes = [vp, vp, vp, i64, i32, i32, vp, i64, i32, i64, vp, i32, vp, vp,
                                     i32, i32, i32, i32, i32, vp, vp, C.c_size_t, vp, vp]
    L.idx_debug_mma_rate.argtypes = [i32, i32, vp, C.POINTER(C.c_double), vp]
    L.idx_mqa_topk_paged_noalloc.argtypes = [vp, vp, vp, i64, i32, i32, vp, i64, i32, i64, vp, i32,
                                             vp, vp, i32, i32, i32, i32, i32, vp, vp, vp]
    L.idx_mqa_topk_cand_workspace_bytes.argtypes = [i64, i32, i32, i32, C.POINTER(C.c_size_t)]
    L.idx_mqa_topk_cand_paged.argtypes = [vp, vp, vp, i64, i32, i32, vp, i64, i32, i64, vp, i32, vp,
                                          vp, i32, i32, i32, i32, vp, i32, vp, i32, i32, vp, vp,
                                          C.c_size_t, vp, vp]
    L.idx_debug_wait_timeout.argtypes = [i32, vp, vp]
    L.idx_compress_k_store.argtypes = [vp, vp, i64, i64, vp, vp, i64, i32, vp, vp, vp, i32, i32, i32,
                                       vp, vp, f32, i32, vp, i64, i32, i64, vp, vp]
    L.idx_step_meta.argtypes = [vp, vp, i32, vp, i32, i32, i32, vp, i32, vp, i64, vp, vp, vp, vp, i64,
                                vp, vp, vp]
    L.idx_kv_layout.argtypes = [i32, i32, i32, C.POINTER(IdxKvLayout)]
    L.idx_kv_store.argtypes = [vp, vp, i32, i64, i32, i32, i64, i64, i64, i64, vp, vp, i64, i32, i64, vp,
                               vp]
    L.idx_attn_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32, C.POINTER(C.c_size_t)]
    L.idx_attn_paged.argtypes = [vp, i32, i64, i32, i32, i32, i64, i64, vp, i64, i32, i64, vp, i32, vp, vp,
                                 i32, i32, i32, i32, vp, i64, i32, f32, vp, i64, i64, vp, vp, C.c_size_t,
                                 vp, vp]
    for n in ("idx_cache_layout", "idx_k_store", "idx_q_quant", "idx_qk_prep", "idx_mqa_logits_paged",
              "idx_topk", "idx_debug_encode", "idx_mqa_topk_workspace_bytes", "idx_mqa_topk_paged",
              "idx_debug_mma_rate", "idx_mqa_topk_paged_noalloc", "idx_compress_k_store",
              "idx_mqa_topk_cand_workspace_bytes", "idx_mqa_topk_cand_paged",
              "idx_mqa_logits_workspace_bytes", "idx_debug_wait_timeout", "idx_step_meta", "idx_kv_layout",
              "idx_kv_store", "idx_attn_workspace_bytes", "idx_attn_paged"):
        getattr(L, n).restype = C.c_int


def _status_str(s):
    try:
        return load(False).idx_status_string(s).decode()
    except Exception:
        return "?"


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn, st):
    if st != 0:
        raise IdxError(fn, st)


def idx_cache_layout(dtype: int, page_size: int) -> IdxLayout:
    out = IdxLayout()
    _check("idx_cache_layout", load().idx_cache_layout(dtype, page_size, C.byref(out)))
    return out


def idx_k_store(k, slot_mapping, positions, cos_sin, rope, apply_norm, dtype, pool, num_pages,
                page_size, page_stride, gamma=None, beta=None, eps=1e-6, dev_status=None,
                stream=None, n_rows=None, k_row_stride=None):
    n = k.shape[0] if n_rows is None else n_rows
    stride = k.stride(0) if k_row_stride is None else k_row_stride
    max_pos = cos_sin.shape[0] if cos_sin is not None else 0
    _check("idx_k_store", load().idx_k_store(
        _ptr(k), n, stride, _ptr(slot_mapping), _ptr(positions), _ptr(cos_sin), max_pos, rope,
        int(apply_norm), _ptr(gamma), _ptr(beta), eps, dtype, _ptr(pool), num_pages, page_size,
        page_stride, _ptr(dev_status), _stream(stream)))


def idx_compress_k_store(k_raw, gate, boundary, first, ratio, slot_mapping, positions, cos_sin, rope,
                         norm, dtype, pool, num_pages, page_size, page_stride, gamma=None, beta=None,
                         eps=1e-6, dev_status=None, stream=None, n_entries=None):
    """k_raw / gate: bf16 (int16/uint16 storage) [n_raw, >=128] sharing one row stride."""
    assert k_raw.stride(0) == gate.stride(0) and k_raw.shape[0] == gate.shape[0]
    n = boundary.shape[0] if n_entries is None else n_entries
    max_pos = cos_sin.shape[0] if cos_sin is not None else 0
    _check("idx_compress_k_store", load().idx_compress_k_store(
        _ptr(k_raw), _ptr(gate), k_raw.shape[0], k_raw.stride(0), _ptr(boundary), _ptr(first), n,
        int(ratio), _ptr(slot_mapping), _ptr(positions), _ptr(cos_sin), max_pos, rope, int(norm),
        _ptr(gamma), _ptr(beta), eps, dtype, _ptr(pool), num_pages, page_size, page_stride,
        _ptr(dev_status), _stream(stream)))


def idx_q_quant(q, positions, cos_sin, rope, w_in, softmax_scale, head_scale, dtype, q_codes,
                q_scales, w_out, dev_status=None, stream=None):
    T, H = q.shape[0], q.shape[1]
    max_pos = cos_sin.shape[0] if cos_sin is not None else 0
    _check("idx_q_quant", load().idx_q_quant(
        _ptr(q), T, H, _ptr(positions), _ptr(cos_sin), max_pos, rope, _ptr(w_in), softmax_scale,
        head_scale, dtype, _ptr(q_codes), _ptr(q_scales), _ptr(w_out), _ptr(dev_status),
        _stream(stream)))


def idx_qk_prep(k, slot_mapping, k_positions, k_rope, apply_norm, pool, num_pages, page_size,
                page_stride, q, q_positions, q_rope, w_in, softmax_scale, head_scale, q_codes,
                q_scales, w_out, cos_sin, dtype, gamma=None, beta=None, eps=1e-6, dev_status=None,
                stream=None):
    n = k.shape[0] if k is not None else 0
    stride = k.stride(0) if k is not None else 128
    T, H = q.shape[0], q.shape[1]
    max_pos = cos_sin.shape[0] if cos_sin is not None else 0
    _check("idx_qk_prep", load().idx_qk_prep(
        _ptr(k), n, stride, _ptr(slot_mapping), _ptr(k_positions), k_rope, int(apply_norm),
        _ptr(gamma), _ptr(beta), eps, _ptr(pool), num_pages, page_size, page_stride, _ptr(q), T, H,
        _ptr(q_positions), q_rope, _ptr(w_in), softmax_scale, head_scale, _ptr(q_codes),
        _ptr(q_scales), _ptr(w_out), _ptr(cos_sin), max_pos, dtype, _ptr(dev_status),
        _stream(stream)))


def idx_mqa_logits_paged(q_codes, q_scales, w, dtype, pool, num_pages, page_size, page_stride,
                         page_table, seq_lens_k, cu_seqlens_q, causal, max_q_len, max_seq_len_k,
                         logits, dev_status=None, stream=None, workspace=None):
    T, H = w.shape
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("idx_mqa_logits_paged", load().idx_mqa_logits_paged(
        _ptr(q_codes), _ptr(q_scales), _ptr(w), T, H, dtype, _ptr(pool), num_pages, page_size,
        page_stride, _ptr(page_table), page_table.shape[1], _ptr(seq_lens_k), _ptr(cu_seqlens_q),
        seq_lens_k.shape[0], int(causal), max_q_len, max_seq_len_k, _ptr(logits),
        logits.stride(0), _ptr(workspace), wsb, _ptr(dev_status), _stream(stream)))


def idx_mqa_logits_workspace_bytes() -> int:
    n = C.c_size_t(0)
    _check("idx_mqa_logits_workspace_bytes", load().idx_mqa_logits_workspace_bytes(C.byref(n)))
    return int(n.value)


def idx_topk(logits, seq_lens_k, cu_seqlens_q, causal, max_seq_len_k, k, out_idx,
             dev_status=None, stream=None, T=None):
    T = logits.shape[0] if T is None else T
    _check("idx_topk", load().idx_topk(
        _ptr(logits), logits.stride(0), _ptr(seq_lens_k), _ptr(cu_seqlens_q),
        seq_lens_k.shape[0], T, int(causal), int(max_seq_len_k), k, _ptr(out_idx),
        _ptr(dev_status), _stream(stream)))


def idx_mqa_topk_workspace_bytes(T, H, B, max_q_len, max_seq_len_k) -> int:
    n = C.c_size_t(0)
    _check("idx_mqa_topk_workspace_bytes",
           load().idx_mqa_topk_workspace_bytes(T, H, B, max_q_len, max_seq_len_k, C.byref(n)))
    return int(n.value)


def idx_mqa_topk_paged(q_codes, q_scales, w, dtype, pool, num_pages, page_size, page_stride,
                       page_table, seq_lens_k, cu_seqlens_q, causal, max_q_len, max_seq_len_k, k,
                       out_idx, workspace, dev_status=None, stream=None):
    T, H = w.shape
    _check("idx_mqa_topk_paged", load().idx_mqa_topk_paged(
        _ptr(q_codes), _ptr(q_scales), _ptr(w), T, H, dtype, _ptr(pool), num_pages, page_size,
        page_stride, _ptr(page_table), page_table.shape[1], _ptr(seq_lens_k), _ptr(cu_seqlens_q),
        seq_lens_k.shape[0], int(causal), max_q_len, max_seq_len_k, k, _ptr(out_idx),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(dev_status),
        _stream(stream)))


def idx_mqa_topk_cand_workspace_bytes(T, max_cand, page_size, max_seq_len_k) -> int:
    n = C.c_size_t(0)
    _check("idx_mqa_topk_cand_workspace_bytes",
           load().idx_mqa_topk_cand_workspace_bytes(T, max_cand, page_size, max_seq_len_k, C.byref(n)))
    return int(n.value)


def idx_mqa_topk_cand_paged(q_codes, q_scales, w, dtype, pool, num_pages, page_size, page_stride,
                            page_table, seq_lens_k, cu_seqlens_q, causal, max_q_len, max_seq_len_k,
                            cand_blocks, n_cand, max_cand, k, out_idx, workspace, dev_status=None,
                            stream=None):
    T, H = w.shape
    _check("idx_mqa_topk_cand_paged", load().idx_mqa_topk_cand_paged(
        _ptr(q_codes), _ptr(q_scales), _ptr(w), T, H, dtype, _ptr(pool), num_pages, page_size,
        page_stride, _ptr(page_table), page_table.shape[1], _ptr(seq_lens_k), _ptr(cu_seqlens_q),
        seq_lens_k.shape[0], int(causal), max_q_len, max_seq_len_k, _ptr(cand_blocks),
        cand_blocks.shape[1], _ptr(n_cand), max_cand, k, _ptr(out_idx), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(dev_status), _stream(stream)))


def idx_debug_encode(kind, x, out, stream=None):
    _check("idx_debug_encode", load().idx_debug_encode(kind, _ptr(x), x.numel(), _ptr(out),
                                                       _stream(stream)))


def idx_debug_wait_timeout(limit_us, dev_status, stream=None):
    _check("idx_debug_wait_timeout", load().idx_debug_wait_timeout(int(limit_us), _ptr(dev_status),
                                                                   _stream(stream)))


def idx_debug_mma_rate(dtype, iters, dev_status=None, stream=None) -> float:
    """Launch the tensor-core rate probe; returns the flops one CTA (SM) performs."""
    f = C.c_double(0.0)
    _check("idx_debug_mma_rate", load().idx_debug_mma_rate(dtype, iters, _ptr(dev_status), C.byref(f),
                                                           _stream(stream)))
    return float(f.value)


def idx_mqa_topk_paged_noalloc(q_codes, q_scales, w, dtype, pool, num_pages, page_size, page_stride,
                               page_table, seq_lens_k, cu_seqlens_q, causal, max_q_len, max_seq_len_k,
                               k, out_idx, dev_status=None, stream=None):
    T, H = w.shape
    _check("idx_mqa_topk_paged_noalloc", load().idx_mqa_topk_paged_noalloc(
        _ptr(q_codes), _ptr(q_scales), _ptr(w), T, H, dtype, _ptr(pool), num_pages, page_size,
        page_stride, _ptr(page_table), page_table.shape[1], _ptr(seq_lens_k), _ptr(cu_seqlens_q),
        seq_lens_k.shape[0], int(causal), max_q_len, max_seq_len_k, k, _ptr(out_idx),
        _ptr(dev_status), _stream(stream)))


def _need(fn, name, x, dtype, ndim=None, contiguous=True):
    """Refuse a tensor whose type or layout the pointer alone would not tell the library, or that
    lies on another device than the current one (where the call is launched)."""
    import torch
    if x.dtype != dtype or (ndim is not None and x.dim() != ndim) or (contiguous and not x.is_contiguous()):
        raise ValueError(f"{fn}: {name} has to be {dtype}"
                         f"{'' if ndim is None else f' with {ndim} dimensions'}"
                         f"{', contiguous' if contiguous else ''}; got {x.dtype}, shape "
                         f"{tuple(x.shape)}, strides {x.stride()}")
    if not x.is_cuda or x.device.index != torch.cuda.current_device():
        raise ValueError(f"{fn}: {name} is on {x.device}, not on the current CUDA device")


def _ftype(fn, x):
    import torch
    if x.dtype == torch.bfloat16:
        return IDX_BF16
    if x.dtype == torch.float16:
        return IDX_FP16
    raise ValueError(f"{fn}: {x.dtype} is neither bfloat16 nor float16")


def idx_step_meta(ctx_lens, q_lens, page_table, page_size, max_seq_len_k, free_pages, free_span, num_pages,
                  cu_seqlens_q, seq_lens_k, positions, slot_mapping, free_next, dev_status=None,
                  stream=None):
    """Page tables, slot map, positions and lengths of a step; T_cap = len(slot_mapping)."""
    import torch
    i32, fn = torch.int32, "idx_step_meta"
    B, T = ctx_lens.shape[0], slot_mapping.shape[0]
    for name, x, d in (("ctx_lens", ctx_lens, 1), ("q_lens", q_lens, 1), ("page_table", page_table, 2),
                       ("free_pages", free_pages, 1), ("free_span", free_span, 1), ("cu_seqlens_q", cu_seqlens_q, 1),
                       ("seq_lens_k", seq_lens_k, 1), ("positions", positions, 1), ("free_next", free_next, 1)):
        _need(fn, name, x, i32, d)
    _need(fn, "slot_mapping", slot_mapping, torch.int64, 1)
    if (q_lens.shape[0] != B or page_table.shape[0] != B or seq_lens_k.shape[0] != B or cu_seqlens_q.shape[0] != B + 1
            or positions.shape[0] != T or free_span.shape[0] != 2 or free_next.shape[0] != 1):
        raise ValueError(f"{fn}: shapes do not belong to {B} requests and {T} rows")
    _check(fn, load().idx_step_meta(
        _ptr(ctx_lens), _ptr(q_lens), B, _ptr(page_table), page_table.shape[1], page_size, max_seq_len_k,
        _ptr(free_pages), free_pages.shape[0], _ptr(free_span), num_pages, _ptr(cu_seqlens_q), _ptr(seq_lens_k),
        _ptr(positions), _ptr(slot_mapping), T, _ptr(free_next), _ptr(dev_status), _stream(stream)))


def idx_kv_layout(kv_heads: int, head_dim: int, page_size: int) -> IdxKvLayout:
    out = IdxKvLayout()
    _check("idx_kv_layout", load().idx_kv_layout(kv_heads, head_dim, page_size, C.byref(out)))
    return out


def idx_kv_store(k, v, slot_mapping, pool, num_pages, page_size, page_stride, dev_status=None, stream=None):
    """k, v: bf16 or fp16 [rows, kv_heads, head_dim], last dimension dense, the others strided."""
    import torch
    fn = "idx_kv_store"
    ft = _ftype(fn, k)
    _need(fn, "k", k, k.dtype, 3, False)
    _need(fn, "v", v, k.dtype, 3, False)
    _need(fn, "slot_mapping", slot_mapping, torch.int64, 1)
    n, H, D = k.shape
    if v.shape != k.shape or slot_mapping.shape[0] != n:
        raise ValueError(f"{fn}: k {tuple(k.shape)}, v {tuple(v.shape)} and {slot_mapping.shape[0]} slots do not match")
    if n > 0 and (k.stride(2) != 1 or v.stride(2) != 1):
        raise ValueError(f"{fn}: the last dimension of k and v has to be dense")
    _check(fn, load().idx_kv_store(
        _ptr(k), _ptr(v), ft, n, H, D, k.stride(0), k.stride(1), v.stride(0), v.stride(1), _ptr(slot_mapping),
        _ptr(pool), num_pages, page_size, page_stride, _ptr(dev_status), _stream(stream)))


def idx_attn_workspace_bytes(T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel=0) -> int:
    n = C.c_size_t(0)
    _check("idx_attn_workspace_bytes", load().idx_attn_workspace_bytes(
        T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel, C.byref(n)))
    return int(n.value)


def idx_attn_paged(q, pool, num_pages, page_size, page_stride, kv_heads, page_table, seq_lens_k, cu_seqlens_q,
                   causal, max_q_len, max_seq_len_k, softmax_scale, out, lse=None, sel_idx=None, workspace=None,
                   dev_status=None, stream=None):
    """q, out: bf16 or fp16 [T, q_heads, head_dim], last dimension dense, the others strided;
    sel_idx: int32 [T, n_sel], rows strided (the top-k's output), or None for every visible key."""
    import torch
    fn, i32 = "idx_attn_paged", torch.int32
    ft = _ftype(fn, q)
    _need(fn, "q", q, q.dtype, 3, False)
    _need(fn, "out", out, q.dtype, 3, False)
    _need(fn, "page_table", page_table, i32, 2)
    _need(fn, "seq_lens_k", seq_lens_k, i32, 1)
    _need(fn, "cu_seqlens_q", cu_seqlens_q, i32, 1)
    T, H, D = q.shape
    B = seq_lens_k.shape[0]
    if out.shape != q.shape or page_table.shape[0] != B or cu_seqlens_q.shape[0] != B + 1:
        raise ValueError(f"{fn}: q {tuple(q.shape)}, out {tuple(out.shape)}, page_table {tuple(page_table.shape)}, "
                         f"seq_lens_k {B} and cu_seqlens_q {cu_seqlens_q.shape[0]} do not match")
    if T > 0 and (q.stride(2) != 1 or out.stride(2) != 1):
        raise ValueError(f"{fn}: the last dimension of q and out has to be dense")
    sel_stride = n_sel = 0
    if lse is not None:
        _need(fn, "lse", lse, torch.float32, 2)
        if lse.shape != (T, H):
            raise ValueError(f"{fn}: lse is {tuple(lse.shape)}, not {(T, H)}")
    if sel_idx is not None:
        _need(fn, "sel_idx", sel_idx, i32, 2, False)
        n_sel, sel_stride = sel_idx.shape[1], max(sel_idx.stride(0), sel_idx.shape[1])
        if sel_idx.shape[0] != T or (T > 0 and n_sel > 1 and sel_idx.stride(1) != 1) or \
                (T > 1 and sel_idx.stride(0) < n_sel):
            raise ValueError(f"{fn}: sel_idx {tuple(sel_idx.shape)} with strides {sel_idx.stride()}")
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(fn, load().idx_attn_paged(
        _ptr(q), ft, T, H, kv_heads, D, q.stride(0), q.stride(1), _ptr(pool), num_pages, page_size, page_stride,
        _ptr(page_table), page_table.shape[1], _ptr(seq_lens_k), _ptr(cu_seqlens_q), B, int(causal), max_q_len,
        max_seq_len_k, _ptr(sel_idx), sel_stride, n_sel, softmax_scale, _ptr(out), out.stride(0), out.stride(1),
        _ptr(lse), _ptr(workspace), wsb, _ptr(dev_status), _stream(stream)))
