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
    if _lib is not None:
        return _lib
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


_torch = None       # the module, once something needs it
_raw_stream = None  # torch's current stream of a device as a handle, without a Stream object


def _load_torch():
    global _torch, _raw_stream
    import torch
    _torch = torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch


def _stream(stream):
    if stream is None:
        torch = _torch or _load_torch()
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
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


def _device():
    torch = _torch or _load_torch()
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):  # no CUDA device: no tensor is on it
        return -2


def _refuse(fn, name, x, dtype, ndim, dense):
    raise ValueError(f"{fn}: {name} has to be {dtype} with {ndim} dimensions{', contiguous' if dense else ''}, on the "
                     f"current CUDA device; got {x.dtype}, shape {tuple(x.shape)}, strides {x.stride()}, {x.device}")


# The checks of a tensor's type, rank, layout and device that its pointer does not tell the library
# (calls are launched on the current device) are written out in each function: a helper per tensor would
# double the host's share of a small call.

def _ftype(fn, x):
    torch = _torch or _load_torch()
    if x.dtype is torch.bfloat16:
        return IDX_BF16
    if x.dtype is torch.float16:
        return IDX_FP16
    raise ValueError(f"{fn}: {x.dtype} is neither bfloat16 nor float16")


def _status(fn, x, dev):
    """The status word's pointer (the kernels write to it), from a tensor or as a number."""
    if x is None or isinstance(x, int):
        return x
    p = x.data_ptr()
    if x.dtype is not _torch.int32 or x.get_device() != dev or not p:  # null: no elements
        _refuse(fn, "dev_status", x, _torch.int32, 1, False)
    return p


def idx_step_meta(ctx_lens, q_lens, page_table, page_size, max_seq_len_k, free_pages, free_span, num_pages,
                  cu_seqlens_q, seq_lens_k, positions, slot_mapping, free_next, dev_status=None,
                  stream=None):
    """Page tables, slot map, positions and lengths of a step; T_cap = len(slot_mapping)."""
    fn, dev = "idx_step_meta", _device()
    i32 = _torch.int32
    for x in (ctx_lens, q_lens, free_pages, free_span, cu_seqlens_q, seq_lens_k, positions, free_next):
        if x.dtype is not i32 or x.get_device() != dev or not x.is_contiguous():
            _refuse(fn, "every list of lengths, pages or positions", x, i32, 1, True)
    if page_table.dtype is not i32 or page_table.dim() != 2 or page_table.get_device() != dev or \
            not page_table.is_contiguous():
        _refuse(fn, "page_table", page_table, i32, 2, True)
    if slot_mapping.dtype is not _torch.int64 or slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
        _refuse(fn, "slot_mapping", slot_mapping, _torch.int64, 1, True)
    B, T = ctx_lens.numel(), slot_mapping.numel()
    rows, width = page_table.shape
    if (q_lens.numel() != B or rows != B or seq_lens_k.numel() != B or cu_seqlens_q.numel() != B + 1
            or positions.numel() != T or free_span.numel() != 2 or free_next.numel() != 1):
        raise ValueError(f"{fn}: shapes do not belong to {B} requests and {T} rows")
    st = (_lib or load()).idx_step_meta(
        ctx_lens.data_ptr(), q_lens.data_ptr(), B, page_table.data_ptr(), width, page_size, max_seq_len_k,
        free_pages.data_ptr(), free_pages.numel(), free_span.data_ptr(), num_pages, cu_seqlens_q.data_ptr(),
        seq_lens_k.data_ptr(), positions.data_ptr(), slot_mapping.data_ptr(), T, free_next.data_ptr(),
        _status(fn, dev_status, dev), _stream(stream))
    if st:
        _check(fn, st)


def idx_kv_layout(kv_heads: int, head_dim: int, page_size: int) -> IdxKvLayout:
    out = IdxKvLayout()
    _check("idx_kv_layout", load().idx_kv_layout(kv_heads, head_dim, page_size, C.byref(out)))
    return out


def _bytes_behind(x):
    """Bytes from a tensor's first element to the end of its memory: more than its own where it is a view with
    gaps, fewer where it repeats elements."""
    return x.untyped_storage().nbytes() - x.storage_offset() * x.element_size()


def _pool_bytes(fn, pool, num_pages, page_stride, page_bytes, dev):
    """The pool holds its pages: the library only sees a pointer."""
    have = pool.nbytes if pool.is_contiguous() else _bytes_behind(pool)
    if pool.get_device() != dev or (num_pages > 0 and have < (num_pages - 1) * page_stride + page_bytes):
        raise ValueError(f"{fn}: the pool ({tuple(pool.shape)}, {pool.dtype}, {pool.device}) does not hold {num_pages} pages "
                         f"{page_stride} bytes apart on the current CUDA device")


def idx_kv_store(k, v, slot_mapping, pool, num_pages, page_size, page_stride, dev_status=None, stream=None):
    """k, v: bf16 or fp16 [rows, kv_heads, head_dim], last dimension dense, the others strided."""
    fn, dev = "idx_kv_store", _device()
    ft = _ftype(fn, k)
    if k.dim() != 3 or k.get_device() != dev:
        _refuse(fn, "k", k, k.dtype, 3, False)
    if v.dtype is not k.dtype or v.get_device() != dev:
        _refuse(fn, "v", v, k.dtype, 3, False)
    if slot_mapping.dtype is not _torch.int64 or slot_mapping.get_device() != dev or not slot_mapping.is_contiguous():
        _refuse(fn, "slot_mapping", slot_mapping, _torch.int64, 1, True)
    n, H, D = shape = k.shape
    if v.shape != shape or slot_mapping.numel() != n:
        raise ValueError(f"{fn}: k {tuple(k.shape)}, v {tuple(v.shape)} and {slot_mapping.numel()} slots do not match")
    kr, kh, kd = k.stride()
    vr, vh, vd = v.stride()
    if n > 0 and (kd != 1 or vd != 1):
        raise ValueError(f"{fn}: the last dimension of k and v has to be dense")
    if n <= 1 or H <= 1:  # the stride of a dimension of one is arbitrary
        kr, vr = (0, 0) if n <= 1 else (kr, vr)
        kh, vh = (0, 0) if H <= 1 else (kh, vh)
    _pool_bytes(fn, pool, num_pages, page_stride, H * (2 * page_size * D + 16), dev)
    st = (_lib or load()).idx_kv_store(
        k.data_ptr(), v.data_ptr(), ft, n, H, D, kr, kh, vr, vh, slot_mapping.data_ptr(), pool.data_ptr(), num_pages,
        page_size, page_stride, _status(fn, dev_status, dev), _stream(stream))
    if st:
        _check(fn, st)


def idx_attn_workspace_bytes(T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel=0) -> int:
    n = C.c_size_t(0)
    _check("idx_attn_workspace_bytes", load().idx_attn_workspace_bytes(
        T, q_heads, kv_heads, head_dim, B, max_q_len, max_seq_len_k, n_sel, C.byref(n)))
    return int(n.value)


def idx_attn_paged(q, pool, num_pages, page_size, page_stride, kv_heads, page_table, seq_lens_k, cu_seqlens_q,
                   causal, max_q_len, max_seq_len_k, softmax_scale, out, lse=None, sel_idx=None, workspace=None,
                   dev_status=None, stream=None):
    """q, out: bf16 or fp16 [T, q_heads, head_dim], last dimension dense, the others strided;
    sel_idx: int32 [T, n_sel], n_sel >= 1, rows strided (the top-k's output), or None for every visible key."""
    fn, dev = "idx_attn_paged", _device()
    i32 = _torch.int32
    ft = _ftype(fn, q)
    if q.dim() != 3 or q.get_device() != dev:
        _refuse(fn, "q", q, q.dtype, 3, False)
    if out.dtype is not q.dtype or out.get_device() != dev:
        _refuse(fn, "out", out, q.dtype, 3, False)
    if page_table.dtype is not i32 or page_table.dim() != 2 or page_table.get_device() != dev or \
            not page_table.is_contiguous():
        _refuse(fn, "page_table", page_table, i32, 2, True)
    for x in (seq_lens_k, cu_seqlens_q):
        if x.dtype is not i32 or x.get_device() != dev or not x.is_contiguous():
            _refuse(fn, "seq_lens_k and cu_seqlens_q", x, i32, 1, True)
    T, H, D = shape = q.shape
    B = seq_lens_k.numel()
    rows, width = page_table.shape
    if out.shape != shape or rows != B or cu_seqlens_q.numel() != B + 1:
        raise ValueError(f"{fn}: q {tuple(q.shape)}, out {tuple(out.shape)}, page_table {tuple(page_table.shape)}, "
                         f"seq_lens_k {B} and cu_seqlens_q {cu_seqlens_q.numel()} do not match")
    qr, qh, qd = q.stride()
    orow, oh, od = out.stride()
    if T > 0 and (qd != 1 or od != 1):
        raise ValueError(f"{fn}: the last dimension of q and out has to be dense")
    if T <= 1 or H <= 1:  # the stride of a dimension of one is arbitrary
        qr, orow = (0, 0) if T <= 1 else (qr, orow)
        qh, oh = (0, 0) if H <= 1 else (qh, oh)
    _pool_bytes(fn, pool, num_pages, page_stride, kv_heads * (2 * page_size * D + 16), dev)
    sel_stride = n_sel = wsb = 0
    lse_p = sel_p = ws_p = None
    if lse is not None:
        if lse.dtype is not _torch.float32 or lse.shape != (T, H) or lse.get_device() != dev or not lse.is_contiguous():
            _refuse(fn, f"lse (of {T} rows and {H} heads)", lse, _torch.float32, 2, True)
        lse_p = lse.data_ptr()
    if sel_idx is not None:
        if sel_idx.dtype is not i32 or sel_idx.dim() != 2 or sel_idx.get_device() != dev:
            _refuse(fn, "sel_idx", sel_idx, i32, 2, False)
        n, n_sel = sel_idx.shape
        s0, s1 = sel_idx.stride()
        sel_stride = max(s0, n_sel)
        # without columns its pointer may be null, which the library takes for no list
        if n != T or (T > 0 and (n_sel < 1 or (n_sel > 1 and s1 != 1))) or (T > 1 and s0 < n_sel):
            raise ValueError(f"{fn}: sel_idx {tuple(sel_idx.shape)} with strides {sel_idx.stride()} for {T} rows")
        sel_p = sel_idx.data_ptr()
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"{fn}: the workspace has to be contiguous, on the current CUDA device; got "
                             f"{tuple(workspace.shape)}, strides {workspace.stride()}, {workspace.device}")
        wsb, ws_p = workspace.nbytes, workspace.data_ptr()
    st = (_lib or load()).idx_attn_paged(
        q.data_ptr(), ft, T, H, kv_heads, D, qr, qh, pool.data_ptr(), num_pages, page_size, page_stride,
        page_table.data_ptr(), width, seq_lens_k.data_ptr(), cu_seqlens_q.data_ptr(), B, 1 if causal else 0, max_q_len,
        max_seq_len_k, sel_p, sel_stride, n_sel, softmax_scale, out.data_ptr(), orow, oh, lse_p, ws_p, wsb,
        _status(fn, dev_status, dev), _stream(stream))
    if st:
        _check(fn, st)
