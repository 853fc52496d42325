"""Python binding of the ts_attn C library (decode attention over a paged KV cache).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels. Tensors are torch tensors on the current CUDA device; their raw
pointers, sizes and the current stream are passed straight to the C ABI in
``include/ts_attn.h``. Functions keep the C names. Output tensors and
workspaces may be passed in; when omitted they are allocated with torch (the C
library itself never allocates device memory).

The shared library is built in-tree by ``paged_kv_cache_46_gb300.build``.
Importing this package does not need a GPU; calling a kernel does, and there
is no CPU fallback: a missing library raises immediately.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libts_attn.so")

TS_OK, TS_ERR_INVALID_ARG, TS_ERR_UNSUPPORTED, TS_ERR_WORKSPACE, TS_ERR_CUDA, TS_ERR_CAPACITY = range(6)
TS_F32, TS_BF16 = 0, 1
TS_DEVERR_PAGE_RANGE, TS_DEVERR_TIMEOUT, TS_DEVERR_SMEM_ALIGN, TS_DEVERR_TREE = 0x1, 0x2, 0x4, 0x8
TS_NOALLOC_SCRATCH_BYTES = 16 * 1024 * 1024   # include/ts_attn.h


class TSError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{status_string(status)}: {detail}")
        self.status = status
        self.detail = detail


class PrefixGroupsC(ctypes.Structure):
    _fields_ = [
        ("num_groups", ctypes.c_int32),
        ("prefix_indptr", ctypes.c_void_p),
        ("prefix_pages", ctypes.c_void_p),
        ("prefix_len", ctypes.c_void_p),
        ("member_indptr", ctypes.c_void_p),
        ("member_ids", ctypes.c_void_p),
        ("group_of", ctypes.c_void_p),
        ("capacity_groups", ctypes.c_int32),
        ("capacity_prefix_pages", ctypes.c_int32),
        ("capacity_members", ctypes.c_int32),
    ]


class PrefixForestC(ctypes.Structure):
    _fields_ = [
        ("num_nodes", ctypes.c_int32),
        ("num_levels", ctypes.c_int32),
        ("level_indptr", ctypes.c_void_p),
        ("parent", ctypes.c_void_p),
        ("prefix_indptr", ctypes.c_void_p),
        ("prefix_pages", ctypes.c_void_p),
        ("prefix_len", ctypes.c_void_p),
        ("member_indptr", ctypes.c_void_p),
        ("member_ids", ctypes.c_void_p),
        ("group_of", ctypes.c_void_p),
        ("capacity_nodes", ctypes.c_int32),
        ("capacity_levels", ctypes.c_int32),
        ("capacity_prefix_pages", ctypes.c_int32),
        ("capacity_members", ctypes.c_int32),
    ]


class LaunchRecordC(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char * 48), ("ms", ctypes.c_float)]


_VP, _I32, _I64, _F32, _SZ, _U32P = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                                     ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32))

_SIGNATURES = {
    "ts_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ts_last_error_detail": (ctypes.c_char_p, []),
    "ts_version": (ctypes.c_char_p, []),
    "ts_kv_append": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                    ctypes.c_int, _VP]),
    "ts_paged_decode_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "ts_paged_decode_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                            _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_paged_decode_attn_noalloc": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32,
                                                    _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP]),
    "ts_paged_decode_window_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                                   _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_paged_decode_sink_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                                 _I32, _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_kv_append_chunk": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _I64, _I32, _I32, _I32, _I32,
                                          _I32, _I32, ctypes.c_int, _VP]),
    "ts_kv_append_chunk_fp8": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _I64, _I32, _I32,
                                              _I32, _I32, _I32, _I32, ctypes.c_int, _VP]),
    "ts_kv_read_fp8": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32,
                                      ctypes.c_int, _VP, _VP, _VP]),
    "ts_paged_prefill_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32]),
    "ts_paged_prefill_attn": (ctypes.c_int, [_VP, _I64, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32,
                                             _I32, _I32, _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_kv_append_chunk_rope": (ctypes.c_int, [_VP, _I64, _VP, _VP, _I64, _VP, _VP, _F32, _VP, _I32, _I32, _VP, _VP,
                                               _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                               ctypes.c_int, _VP, _I64, _VP]),
    "ts_kv_page_bounds": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32,
                                         ctypes.c_int, _VP]),
    "ts_select_pages_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "ts_select_pages": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                       _I32, _I32, ctypes.c_int, _VP, _VP, _SZ, _VP]),
    "ts_paged_decode_sparse_workspace_size": (_SZ, [_I32, _I32, _I32, _I32, _I32, _I32, _I32]),
    "ts_paged_decode_sparse_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32,
                                                   _I32, _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_kv_fork": (ctypes.c_int, [_VP, _VP, _I32, _VP, _I32, _VP, _I32, _VP, _VP, _VP, _I32, _I32, _I32, _VP]),
    "ts_kv_compact_workspace_size": (_SZ, [_I32]),
    "ts_kv_compact": (ctypes.c_int, [_VP, _VP, _I32, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _VP, _VP, _VP, _SZ,
                                     _VP]),
    "ts_paged_decode_multi_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "ts_paged_decode_multi_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                                  _I32, _I32, _F32, ctypes.c_int, _VP, _VP, _VP, _SZ, _VP]),
    "ts_fold_sq_factor": (_I32, [_I32, _I32, _I32]),
    "ts_kv_append_fp8": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32,
                                        _I32, ctypes.c_int, _VP]),
    "ts_paged_decode_fp8_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32,
                                                _I32, _I32, _F32, _VP, _VP, _VP, _SZ, _VP]),
    "ts_merge_states": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _VP, _I64, _I32, ctypes.c_int, _VP]),
    "ts_group_prefixes": (ctypes.c_int, [_VP, _I32, _VP, _I32, _I32, _I32, ctypes.POINTER(PrefixGroupsC)]),
    "ts_group_prefixes_nested": (ctypes.c_int, [_VP, _I32, _VP, _I32, _I32, _I32, ctypes.POINTER(PrefixForestC)]),
    "ts_cascade_decode_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "ts_cascade_nested_decode_attn": (ctypes.c_int, [_VP, _VP, _VP, ctypes.POINTER(PrefixForestC), _VP, _VP, _I32,
                                                     _VP, _I32, _I32, _I32, _I32, _I32, _I32, _F32, ctypes.c_int,
                                                     _VP, _VP, _VP, _SZ, _VP]),
    "ts_cascade_decode_attn": (ctypes.c_int, [_VP, _VP, _VP, ctypes.POINTER(PrefixGroupsC), _VP, _I32, _VP,
                                              _I32, _I32, _I32, _I32, _I32, _I32, _F32, ctypes.c_int,
                                              _VP, _VP, _VP, _SZ, _VP]),
    "ts_mla_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "ts_mla_paged_decode": (ctypes.c_int, [_VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32, _I32,
                                           _F32, _VP, _VP, _VP, _SZ, _VP]),
    "ts_mla_multi_workspace_size": (_SZ, [_I32, _I32, _I32, _I32]),
    "ts_mla_paged_decode_multi": (ctypes.c_int, [_VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32, _I32,
                                                 _I32, _F32, _VP, _VP, _VP, _SZ, _VP]),
    "ts_paged_decode_tree_attn": (ctypes.c_int, [_VP, _VP, _VP, _VP, _I32, _VP, _VP, _I32, _I32, _I32, _I32, _I32,
                                                 _I32, _I32, _F32, _I32, _VP, _VP, _VP, _SZ, _VP]),
    "ts_mla_paged_decode_fp8": (ctypes.c_int, [_VP, _VP, _VP, _VP, _VP, _I32, _VP, _I32, _I32, _I32, _I32, _I32,
                                               _I32, _I32, _F32, _VP, _VP, _VP, _SZ, _VP]),
    "ts_read_device_error": (ctypes.c_int, [_VP, _U32P, _VP]),
    "ts_trace_enable": (ctypes.c_int, [_I32]),
    "ts_trace_collect": (_I32, [ctypes.POINTER(LaunchRecordC), _I32]),
    "ts_clock_stamp": (ctypes.c_int, [_VP, _I32, _VP]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m paged_kv_cache_46_gb300.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().ts_status_string(int(status)).decode()
    except Exception:  # library not loadable: still describe the code
        return {0: "TS_OK"}.get(int(status), f"status {status}")


def _check(status: int):
    if status != TS_OK:
        raise TSError(status, lib().ts_last_error_detail().decode())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return TS_F32
    if t.dtype == torch.bfloat16:
        return TS_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a Stream object (3 us on the
# host of a GB300, as much as a launch), where torch offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


_HERE = contextlib.nullcontext()


def _made_for(stream):
    """Context in which tensors belong to the call's stream: torch hands a freed workspace on
    in the order of the stream it was made for, and zeroes a new one there."""
    if stream is None:
        return _HERE
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def _rows(t: torch.Tensor):
    """Pointer and row step (elements) of a [rows, heads, D] tensor whose rows are contiguous."""
    rows, heads, D = t.shape
    step, head_step, unit = t.stride()
    if (unit != 1 and D > 1) or (head_step != D and heads > 1):
        raise ValueError("the heads of a row must be contiguous")
    return t.data_ptr(), step if rows > 1 else heads * D


def _pointers(*tensors):
    """Pointers of contiguous tensors (None stays None). The library launches on the
    current device: every tensor must live there."""
    device = -2
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        at = t.get_device()
        if at != device:
            if at < 0 or device != -2 or at != torch.cuda.current_device():
                raise ValueError(f"tensors must be on the current CUDA device (got {t.device})")
            device = at
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        out.append(t.data_ptr())
    return out


_get_device, _is_contiguous, _data_ptr = torch.Tensor.get_device, torch.Tensor.is_contiguous, torch.Tensor.data_ptr
_here = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _marshal(stream, *tensors):
    """Pointers of contiguous tensors on the current CUDA device, and the handle of the call's
    stream behind them."""
    devices = set(map(_get_device, tensors))
    at = devices.pop()
    if devices or at < 0 or at != _here():
        raise ValueError(f"tensors must be on the current CUDA device (got {', '.join(str(t.device) for t in tensors)})")
    if not all(map(_is_contiguous, tensors)):
        raise ValueError("tensors must be contiguous")
    return (*map(_data_ptr, tensors), _raw_stream(at) if stream is None and _raw_stream is not None else _stream(stream))


def _optional(like, t):
    """Pointer of an optional tensor on another one's device (None stays None)."""
    if t is None:
        return None
    if t.get_device() != like.get_device() or not t.is_contiguous():
        raise ValueError("tensors must be contiguous and on the current CUDA device")
    return t.data_ptr()


_DTYPES = {torch.float32: TS_F32, torch.bfloat16: TS_BF16}


def _dtype_code(dtype):
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype} (float32 or bfloat16)")
    return code


def _require_batch(seq_lens, indptr, block_table):
    """_require_chunks, and the block table's row length."""
    if seq_lens.dtype != _INT32 or block_table.dtype != _INT32 or (indptr is not None and indptr.dtype != _INT32):
        raise TypeError("block tables, lengths and row offsets must be int32")
    B = seq_lens.numel()
    rows, slots = block_table.shape
    if rows != B or (indptr is not None and indptr.numel() != B + 1):
        raise ValueError("a batch of B sequences has B lengths, B block-table rows and B + 1 row offsets")
    return B, slots


def _row_step(t: torch.Tensor, rows: int, heads: int, D: int) -> int:
    """Row step (elements) of a [rows, heads, D] tensor whose rows are contiguous."""
    step, head_step, unit = t.stride()
    if (unit != 1 and D > 1) or (head_step != D and heads > 1):
        raise ValueError("the heads of a row must be contiguous")
    return step if rows > 1 else heads * D


def _require_i32(*ts):
    for t in ts:
        if t.dtype != torch.int32:
            raise TypeError("block tables, lengths and positions must be int32")


# ---------------------------------------------------------------------------
# Entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def ts_kv_append(k_new, v_new, k_pool, v_pool, block_table, positions, stream=None) -> None:
    """Write k_new/v_new [B, H_kv, D] into the pools at ``positions`` (see ts_attn.h)."""
    _require_i32(block_table, positions)
    B, H_kv, D = k_new.shape
    _check(lib().ts_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                              block_table.shape[1], _ptr(positions), B, H_kv, D, k_pool.shape[1],
                              k_pool.shape[0], _dt(k_pool), _stream(stream)))


def ts_paged_decode_workspace_size(B: int, H_q: int, D: int) -> int:
    return int(lib().ts_paged_decode_workspace_size(B, H_q, D))


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zeroed, 256-byte aligned uint8 workspace (torch's allocator aligns to >= 256)."""
    ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")
    assert ws.data_ptr() % 256 == 0
    return ws


def ts_paged_decode_attn(q, k_pool, v_pool, block_table, seq_lens, scale: float, out=None, lse=None,
                         workspace=None, stream=None, return_lse: bool = False):
    """Decode attention over a paged cache; returns ``out`` (and ``lse``)."""
    _require_i32(block_table, seq_lens)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_paged_decode_workspace_size(B, H_q, D), q.device)
    _check(lib().ts_paged_decode_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                      block_table.shape[1], _ptr(seq_lens), B, H_q, H_kv, D, ps, P,
                                      float(scale), _dt(q), _ptr(out), _ptr(lse), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def ts_paged_decode_window_attn(q, k_pool, v_pool, block_table, seq_lens, scale: float, window: int, out=None,
                                lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Decode attention over a sliding-window KV group (each query attends its
    sequence's last ``window`` tokens); returns ``out`` (and ``lse``)."""
    _require_i32(block_table, seq_lens)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_paged_decode_workspace_size(B, H_q, D), q.device)
    _check(lib().ts_paged_decode_window_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                             block_table.shape[1], _ptr(seq_lens), B, H_q, H_kv, D, ps, P,
                                             int(window), float(scale), _dt(q), _ptr(out), _ptr(lse),
                                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                                             _stream(stream)))
    return (out, lse) if return_lse else out


def ts_paged_decode_sink_attn(q, k_pool, v_pool, block_table, seq_lens, scale: float, window: int, sinks: int,
                              out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Decode attention over a sliding window whose sequence's first ``sinks`` tokens stay
    visible; returns ``out`` (and ``lse``)."""
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    _require_chunks(seq_lens, None, block_table)
    _require_cache(q, k_pool, v_pool)
    if seq_lens.numel() != B:
        raise ValueError("a batch of B sequences has B queries, B lengths and B block-table rows")
    if out is None:
        with _made_for(stream):
            out = torch.empty(B, H_q, D, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        with _made_for(stream):
            lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    _require_result(out, lse, q)
    qp, kp, vp, bt, lens, op, lp, wp = _pointers(q, k_pool, v_pool, block_table, seq_lens, out, lse, workspace)
    if workspace is None:
        with _made_for(stream):
            workspace = new_workspace(ts_paged_decode_workspace_size(B, H_q, D), q.device)
        wp = workspace.data_ptr()
    _check(lib().ts_paged_decode_sink_attn(qp, kp, vp, bt, block_table.shape[1], lens, B, H_q, H_kv, D, ps, P,
                                           int(window), int(sinks), float(scale), _dt(q), op, lp, wp,
                                           workspace.nbytes, _stream(stream)))
    return (out, lse) if return_lse else out


def _require_cache(q, k_pool, v_pool):
    """Queries and pools of one type; pools [num_pages, page_size, H_kv, D] alike."""
    if k_pool.dtype != q.dtype or v_pool.dtype != q.dtype:
        raise TypeError("queries and pools must have one dtype")
    if k_pool.shape != v_pool.shape or k_pool.shape[3] != q.shape[2]:
        raise ValueError("pools must be [num_pages, page_size, H_kv, D] with the queries' D")


def _require_result(out, lse, q):
    if out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must have the queries' shape and dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != q.shape[:2]):
        raise ValueError("lse must be float32 of the queries' rows and heads")


_INT32 = torch.int32


def _require_chunks(seq_lens, indptr, block_table):
    """int32 metadata of B sequences: B lengths, B block-table rows, B + 1 row offsets."""
    if seq_lens.dtype != _INT32 or block_table.dtype != _INT32 or (indptr is not None and indptr.dtype != _INT32):
        raise TypeError("block tables, lengths and row offsets must be int32")
    B = seq_lens.numel()
    if block_table.shape[0] != B or (indptr is not None and indptr.numel() != B + 1):
        raise ValueError("a batch of B sequences has B lengths, B block-table rows and B + 1 row offsets")
    return B


def _chunk_rows(k_new, v_new, k_pool, v_pool):
    """Pointers and common row step of new K and V rows [T, H_kv, D] for pools [P, ps, H_kv, D]."""
    if k_new.dtype != v_new.dtype or k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must be alike")
    if k_pool.shape != v_pool.shape or k_pool.shape[2:] != k_new.shape[1:]:
        raise ValueError("pools must be [num_pages, page_size, H_kv, D] with the new rows' H_kv and D")
    k, step = _rows(k_new)
    v, v_step = _rows(v_new)
    if step != v_step:
        raise ValueError("k_new and v_new rows must be equally far apart")
    if k_new.get_device() != k_pool.get_device() or v_new.get_device() != k_pool.get_device():
        raise ValueError("new rows and pools must be on one device")
    return k, v, step


def ts_kv_append_chunk(k_new, v_new, k_pool, v_pool, block_table, seq_lens, q_indptr, stream=None) -> None:
    """Write the K/V rows [T, H_kv, D] of a ragged batch of prompt chunks into the pools:
    rows ``q_indptr[b]`` .. ``q_indptr[b + 1] - 1`` are sequence b's newest tokens, which
    ``seq_lens[b]`` counts already (see ts_attn.h). Rows may be a part of wider rows."""
    B = _require_chunks(seq_lens, q_indptr, block_table)
    if k_pool.dtype != k_new.dtype or v_pool.dtype != k_new.dtype:
        raise TypeError("new rows and pools must have one dtype")
    k, v, step = _chunk_rows(k_new, v_new, k_pool, v_pool)
    kp, vp, bt, lens, ptr = _pointers(k_pool, v_pool, block_table, seq_lens, q_indptr)
    P, ps, H_kv, D = k_pool.shape
    _check(lib().ts_kv_append_chunk(k, v, kp, vp, bt, block_table.shape[1], lens, ptr, step, k_new.shape[0], B, H_kv,
                                    D, ps, P, _dt(k_new), _stream(stream)))


def ts_kv_append_chunk_fp8(k_new, v_new, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, q_indptr,
                           stream=None) -> None:
    """Quantize the K/V rows of a ragged batch of prompt chunks into fp8 pools and their
    scales: placement as ``ts_kv_append_chunk``, values as ``ts_kv_append_fp8``."""
    B = _require_chunks(seq_lens, q_indptr, block_table)
    _require_fp8_cache(k_pool, v_pool, k_scale, v_scale)
    k, v, step = _chunk_rows(k_new, v_new, k_pool, v_pool)
    kp, vp, ks, vs, bt, lens, ptr = _pointers(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, q_indptr)
    P, ps, H_kv, D = k_pool.shape
    _check(lib().ts_kv_append_chunk_fp8(k, v, kp, vp, ks, vs, bt, block_table.shape[1], lens, ptr, step,
                                        k_new.shape[0], B, H_kv, D, ps, P, _dt(k_new), _stream(stream)))


def ts_kv_read_fp8(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, kv_indptr, k_out, v_out,
                   stream=None) -> None:
    """Read an fp8 cache back: row ``kv_indptr[b] + t`` of k_out / v_out [rows, H_kv, D] (bf16
    or f32) becomes token t of sequence b; other rows stay as they were (see ts_attn.h)."""
    B = _require_chunks(seq_lens, kv_indptr, block_table)
    _require_fp8_cache(k_pool, v_pool, k_scale, v_scale)
    rows, H_kv, D = k_out.shape
    P, ps, H_pool, D_pool = k_pool.shape
    if k_out.dtype != v_out.dtype or k_out.shape != v_out.shape or k_pool.shape != v_pool.shape or \
            H_kv != H_pool or D != D_pool:
        raise ValueError("k_out and v_out must be [rows, H_kv, D] with the pools' H_kv and D")
    kp, vp, ks, vs, bt, lens, ptr, ko, vo = _pointers(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens,
                                                      kv_indptr, k_out, v_out)
    _check(lib().ts_kv_read_fp8(kp, vp, ks, vs, bt, block_table.shape[1], lens, ptr, rows, B, H_kv, D, ps, P,
                                _dt(k_out), ko, vo, _stream(stream)))


def ts_paged_prefill_workspace_size(T: int, B: int, H_q: int, H_kv: int, D: int) -> int:
    return int(lib().ts_paged_prefill_workspace_size(T, B, H_q, H_kv, D))


def ts_paged_prefill_attn(q, k_pool, v_pool, block_table, seq_lens, q_indptr, scale: float, window: int = 0,
                          sinks: int = 0, out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Attention of a ragged batch of prompt chunks, q [T, H_q, D] with rows ``q_indptr[b]`` ..
    ``q_indptr[b + 1] - 1`` of sequence b, over a paged cache that holds their K/V rows
    (``ts_kv_append_chunk``); ``seq_lens`` count them. Causal; ``window`` > 0 keeps the last
    ``window`` tokens of each query and the sequence's first ``sinks``. Returns ``out``
    [T, H_q, D] (and ``lse``); rows of no sequence are left as they were."""
    B = _require_chunks(seq_lens, q_indptr, block_table)
    T, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    _require_cache(q, k_pool, v_pool)
    qp, step = _rows(q)
    if out is None:
        with _made_for(stream):
            out = torch.empty(T, H_q, D, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        with _made_for(stream):
            lse = torch.empty(T, H_q, dtype=torch.float32, device=q.device)
    _require_result(out, lse, q)
    if q.get_device() != k_pool.get_device():
        raise ValueError("queries and pools must be on one device")
    kp, vp, bt, lens, ptr, op, lp, wp = _pointers(k_pool, v_pool, block_table, seq_lens, q_indptr, out, lse,
                                                  workspace)
    if workspace is None:
        with _made_for(stream):
            workspace = new_workspace(ts_paged_prefill_workspace_size(T, B, H_q, H_kv, D), q.device)
        wp = workspace.data_ptr()
    _check(lib().ts_paged_prefill_attn(qp, step, kp, vp, bt, block_table.shape[1], lens, ptr, T, B, H_q, H_kv, D, ps,
                                       P, int(window), int(sinks), float(scale), _dt(q), op, lp, wp,
                                       workspace.nbytes, _stream(stream)))
    return (out, lse) if return_lse else out


def ts_kv_append_chunk_rope(q, k_new, v_new, k_pool, v_pool, block_table, seq_lens, q_indptr, inv_freq=None,
                            q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False, q_out=None,
                            stream=None):
    """Normalise (where weights are given) and rotate the queries [T, H_q, D] and keys [T, H_kv, D]
    of a ragged batch of chunks by their positions, and write K and V into the pools (see
    ts_attn.h). ``inv_freq`` (float32, radians per position) has one entry per rotated pair.
    Rows may be a part of wider rows. Returns the queries, in ``q_out`` (which may be ``q``)."""
    B, slots = _require_batch(seq_lens, q_indptr, block_table)
    q_shape, new_shape, pool_shape = q.shape, k_new.shape, k_pool.shape
    T, H_q, D = q_shape
    P, ps, H_kv, D_pool = pool_shape
    dtype = q.dtype
    if k_new.dtype != dtype or v_new.dtype != dtype or k_pool.dtype != dtype or v_pool.dtype != dtype:
        raise TypeError("queries, new rows and pools must have one dtype")
    if v_pool.shape != pool_shape or D != D_pool or new_shape != (T, H_kv, D) or v_new.shape != new_shape:
        raise ValueError("q must be [T, H_q, D], new rows [T, H_kv, D], pools [num_pages, page_size, H_kv, D]")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != dtype or w.numel() != D):
            raise ValueError("weights must be [D] of the queries' dtype")
    rot = 0
    if inv_freq is not None:
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1:
            raise TypeError("inv_freq must be float32 [rot_dim / 2]")
        rot = 2 * inv_freq.numel()
    step = _row_step(k_new, T, H_kv, D)
    if _row_step(v_new, T, H_kv, D) != step:
        raise ValueError("k_new and v_new rows must be equally far apart")
    q_step = out_step = _row_step(q, T, H_q, D)
    if q_out is None:
        with _made_for(stream):
            q_out = torch.empty(T, H_q, D, dtype=dtype, device=q.device)
        out_step = H_q * D
    elif q_out is not q:
        if q_out.dtype != dtype or q_out.shape != q_shape:
            raise ValueError("q_out must have the queries' shape and dtype")
        out_step = _row_step(q_out, T, H_q, D)
    at = k_pool.get_device()
    if q.get_device() != at or k_new.get_device() != at or v_new.get_device() != at or q_out.get_device() != at:
        raise ValueError("queries, new rows and pools must be on one device")
    kp, vp, bt, lens, ptr, on = _marshal(stream, k_pool, v_pool, block_table, seq_lens, q_indptr)
    _check(lib().ts_kv_append_chunk_rope(q.data_ptr(), q_step, k_new.data_ptr(), v_new.data_ptr(), step,
                                         _optional(k_pool, q_weight), _optional(k_pool, k_weight), eps,
                                         _optional(k_pool, inv_freq), rot, bool(interleaved), kp, vp, bt, slots, lens,
                                         ptr, T, B, H_q, H_kv, D, ps, P, _dtype_code(dtype), q_out.data_ptr(), out_step,
                                         on))
    return q_out


def _require_bounds(bounds, bound_scale, D):
    """Page bounds int8 [num_pages, H_kv, 2, D] and their scales float32 [num_pages, H_kv]: (num_pages, H_kv)."""
    if bounds.dtype != torch.int8 or bound_scale.dtype != torch.float32:
        raise TypeError("page bounds are int8, their scales float32")
    of = bound_scale.shape
    if len(of) != 2 or bounds.shape != (*of, 2, D):
        raise ValueError("page bounds must be [num_pages, H_kv, 2, D], their scales [num_pages, H_kv]")
    return of


def ts_kv_page_bounds(k_pool, bounds, bound_scale, block_table, seq_lens, q_indptr, rows: int, stream=None) -> None:
    """Bounds of the keys of every page that holds one of the newest tokens (those of ``q_indptr``,
    ``rows`` in all), into ``bounds`` int8 [num_pages, H_kv, 2, D] and ``bound_scale`` float32
    [num_pages, H_kv] (see ts_attn.h). Other pages' bounds stay."""
    B, slots = _require_batch(seq_lens, q_indptr, block_table)
    P, ps, H_kv, D = k_pool.shape
    if _require_bounds(bounds, bound_scale, D) != (P, H_kv):
        raise ValueError("page bounds must have the pool's pages and kv heads")
    kp, bp, sp, bt, lens, ptr, on = _marshal(stream, k_pool, bounds, bound_scale, block_table, seq_lens, q_indptr)
    _check(lib().ts_kv_page_bounds(kp, bp, sp, bt, slots, lens, ptr, rows, B, H_kv, D, ps, P,
                                   _dtype_code(k_pool.dtype), on))


def ts_select_pages_workspace_size(B: int, q_len: int, H_kv: int, bt_stride: int) -> int:
    return int(lib().ts_select_pages_workspace_size(B, q_len, H_kv, bt_stride))


def ts_select_pages(q, bounds, bound_scale, block_table, seq_lens, page_size: int, pages: int, first: int = 1,
                    last: int = 1, page_idx=None, workspace=None, stream=None):
    """The ``pages`` slots of each sequence whose page bounds promise most, for every query row and
    kv head: q [B, H_q, D] or [B, q_len, H_q, D] -> int32 [B, (q_len,) H_kv, pages], ascending,
    -1 behind the last; the first ``first`` and last ``last`` pages are always among them
    (see ts_attn.h)."""
    B, slots = _require_batch(seq_lens, None, block_table)
    rows, q_len, H_q, D = _query_rows(q, B)
    P, H_kv = _require_bounds(bounds, bound_scale, D)
    want = (*rows, H_kv, pages)
    if page_idx is None:
        with _made_for(stream):
            page_idx = torch.empty(want, dtype=_INT32, device=q.device)
    elif page_idx.dtype != _INT32 or page_idx.shape != want:
        raise ValueError("page_idx must be int32 [B, (q_len,) H_kv, pages]")
    qp, bp, sp, bt, lens, ip, on = _marshal(stream, q, bounds, bound_scale, block_table, seq_lens, page_idx)
    if workspace is None:
        with _made_for(stream):
            workspace = new_workspace(ts_select_pages_workspace_size(B, q_len, H_kv, slots), q.device)
    _check(lib().ts_select_pages(qp, bp, sp, bt, slots, lens, B, q_len, H_q, H_kv, D, page_size, P, pages, first, last,
                                 _dtype_code(q.dtype), ip, _optional(q, workspace), workspace.nbytes, on))
    return page_idx


def _query_rows(q, B):
    """Leading sizes, q_len, H_q and D of queries [B, H_q, D] or [B, q_len, H_q, D]."""
    shape = q.shape
    if len(shape) == 3:
        n, H_q, D = shape
        rows, q_len = (n,), 1
    elif len(shape) == 4:
        n, q_len, H_q, D = shape
        rows = (n, q_len)
    else:
        n = -1
    if n != B:
        raise ValueError("q must be [B, H_q, D] or [B, q_len, H_q, D]")
    return rows, q_len, H_q, D


def ts_paged_decode_sparse_workspace_size(B: int, q_len: int, H_q: int, H_kv: int, D: int, page_size: int,
                                          pages: int) -> int:
    return int(lib().ts_paged_decode_sparse_workspace_size(B, q_len, H_q, H_kv, D, page_size, pages))


def ts_paged_decode_sparse_attn(q, k_pool, v_pool, block_table, seq_lens, page_idx, scale: float, out=None, lse=None,
                                workspace=None, stream=None, return_lse: bool = False):
    """Decode attention over listed pages: q [B, H_q, D] or [B, q_len, H_q, D], ``page_idx`` int32
    [B, (q_len,) H_kv, pages] of block-table slots (negative: none; see ts_select_pages). Token j of
    a sequence, at position ``seq_lens[b] - q_len + j``, attends the listed pages' tokens up to
    itself. Returns ``out`` (and ``lse``)."""
    B, slots = _require_batch(seq_lens, None, block_table)
    rows, q_len, H_q, D = _query_rows(q, B)
    pool_shape, dtype = k_pool.shape, q.dtype
    P, ps, H_kv, D_pool = pool_shape
    if k_pool.dtype != dtype or v_pool.dtype != dtype:
        raise TypeError("queries and pools must have one dtype")
    if v_pool.shape != pool_shape or D_pool != D:
        raise ValueError("pools must be [num_pages, page_size, H_kv, D] with the queries' D")
    of = page_idx.shape
    pages = of[-1]
    if page_idx.dtype != _INT32 or of != (*rows, H_kv, pages):
        raise ValueError("page_idx must be int32 [B, (q_len,) H_kv, pages]")
    if out is None:
        with _made_for(stream):
            out = torch.empty(*rows, H_q, D, dtype=dtype, device=q.device)
    if lse is None and return_lse:
        with _made_for(stream):
            lse = torch.empty(*rows, H_q, dtype=torch.float32, device=q.device)
    if out.dtype != dtype or out.shape != (*rows, H_q, D):
        raise ValueError("out must have the queries' shape and dtype")
    if lse is not None and (lse.dtype != torch.float32 or lse.shape != (*rows, H_q)):
        raise ValueError("lse must be float32 of the queries' rows and heads")
    qp, kp, vp, bt, lens, ip, op, on = _marshal(stream, q, k_pool, v_pool, block_table, seq_lens, page_idx, out)
    if workspace is None:
        with _made_for(stream):
            size = ts_paged_decode_sparse_workspace_size(B, q_len, H_q, H_kv, D, ps, pages)
            workspace = new_workspace(size, q.device)
    _check(lib().ts_paged_decode_sparse_attn(qp, kp, vp, bt, slots, lens, ip, pages, B, q_len, H_q, H_kv, D, ps, P,
                                             scale, _dtype_code(dtype), op, _optional(q, lse), _optional(q, workspace),
                                             workspace.nbytes, on))
    return (out, lse) if return_lse else out


class KVBuffers:
    """The buffers of a cache that one block table serves, for ts_kv_fork and ts_kv_compact: tensors
    [num_pages, ...], kept alive by this object."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        self.num_pages = self.tensors[0].shape[0] if self.tensors else 0
        for t in self.tensors:
            if t.dim() < 1 or t.shape[0] != self.num_pages:
                raise ValueError("buffers must have one number of pages")
        pointers = _pointers(*self.tensors)
        n = len(pointers)
        self.count = n
        self.device = self.tensors[0].get_device() if n else -1
        self._data = (ctypes.c_void_p * n)(*pointers)
        self._bytes = (ctypes.c_int64 * n)(*(t.nbytes // max(1, self.num_pages) for t in self.tensors))
        self.data, self.page_bytes = ctypes.addressof(self._data), ctypes.addressof(self._bytes)


def kv_buffers(tensors) -> KVBuffers:
    """A cache's tensors [num_pages, ...] (K, V, scales, bounds, of any layers) as one handle."""
    return KVBuffers(tensors)


def _require_buffers(buffers, block_table):
    if not isinstance(buffers, KVBuffers):
        buffers = KVBuffers(buffers)
    if buffers.count == 0:
        raise ValueError("a cache has one buffer at least")
    if buffers.device != block_table.get_device():
        raise ValueError("buffers and block table must be on one device")
    return buffers


def ts_kv_fork(buffers, block_table, seq_lens, parents, children, fresh, page_size: int, stream=None) -> None:
    """Row ``children[i]`` of ``block_table`` and ``seq_lens`` becomes a continuation of row
    ``parents[i]``: whole pages are shared, a partly filled last page is copied to page ``fresh[i]``
    in all ``buffers`` (a list of tensors [num_pages, ...], or kv_buffers of one). See ts_attn.h."""
    B, slots = _require_batch(seq_lens, None, block_table)
    buffers = _require_buffers(buffers, block_table)
    n = parents.numel()
    for t in (parents, children, fresh):
        if t.dtype != _INT32 or t.numel() != n:
            raise TypeError("parents, children and fresh must be int32 of one length")
    bt, lens, pp, cp, fp, on = _marshal(stream, block_table, seq_lens, parents, children, fresh)
    _check(lib().ts_kv_fork(buffers.data, buffers.page_bytes, buffers.count, bt, slots, lens, B, pp, cp, fp, n,
                            page_size, buffers.num_pages, on))


def ts_kv_compact_workspace_size(num_pages: int) -> int:
    return int(lib().ts_kv_compact_workspace_size(num_pages))


def ts_kv_compact(buffers, block_table, seq_lens, page_size: int, table_out=None, page_map=None, used=None,
                  workspace=None, stream=None):
    """Move the pages that the rows of ``block_table`` hold to the front of all ``buffers`` (a list of
    tensors [num_pages, ...], or kv_buffers of one). Returns the new block table (``table_out``, which
    may be ``block_table``), each page's new id (-1: free) and the number of pages in use (int32 [1]):
    the pages from there on are free. See ts_attn.h."""
    B, slots = _require_batch(seq_lens, None, block_table)
    buffers = _require_buffers(buffers, block_table)
    P = buffers.num_pages
    if table_out is None or page_map is None or used is None or workspace is None:
        device = block_table.device
        with _made_for(stream):
            if table_out is None:
                table_out = torch.empty_like(block_table)
            if page_map is None:
                page_map = torch.empty(P, dtype=_INT32, device=device)
            if used is None:
                used = torch.empty(1, dtype=_INT32, device=device)
            if workspace is None:
                workspace = new_workspace(ts_kv_compact_workspace_size(P), device)
    if table_out.dtype != _INT32 or page_map.dtype != _INT32 or used.dtype != _INT32:
        raise TypeError("tables and page ids must be int32")
    if table_out.shape != block_table.shape or page_map.numel() != P or used.numel() != 1:
        raise ValueError("table_out must be the block table's shape, page_map [num_pages], used [1]")
    bt, to, lens, mp, up, wp, on = _marshal(stream, block_table, table_out, seq_lens, page_map, used, workspace)
    _check(lib().ts_kv_compact(buffers.data, buffers.page_bytes, buffers.count, bt, to, slots, lens, B, page_size,
                               P, mp, up, wp, workspace.nbytes, on))
    return table_out, page_map, used


def ts_paged_decode_attn_noalloc(q, k_pool, v_pool, block_table, seq_lens, scale: float, out, lse=None,
                                 stream=None) -> None:
    """ts_paged_decode_attn for callers that cannot allocate device memory.

    The library takes its split-KV scratch from a fixed array in its own device
    image (TS_NOALLOC_SCRATCH_BYTES, one per GPU, kept until exit) instead of a
    caller workspace. ``out`` (and ``lse`` if wanted) must be passed in: this
    wrapper allocates nothing either. Calls that may overlap on one GPU share
    the array and race; see include/ts_attn.h.
    """
    _require_i32(block_table, seq_lens)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    _check(lib().ts_paged_decode_attn_noalloc(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                              block_table.shape[1], _ptr(seq_lens), B, H_q, H_kv, D, ps, P,
                                              float(scale), _dt(q), _ptr(out), _ptr(lse), _stream(stream)))


def ts_paged_decode_multi_workspace_size(B: int, q_len: int, H_q: int, D: int) -> int:
    return int(lib().ts_paged_decode_multi_workspace_size(B, q_len, H_q, D))


def ts_fold_sq_factor(num_heads: int, q_len: int, tile_rows: int = 128) -> int:
    """Query tokens folded into a tile's rows (see include/ts_attn.h)."""
    return int(lib().ts_fold_sq_factor(num_heads, q_len, tile_rows))


def ts_paged_decode_multi_attn(q, k_pool, v_pool, block_table, seq_lens, scale: float, out=None, lse=None,
                               workspace=None, stream=None, return_lse: bool = False):
    """Decode with q_len query tokens per sequence, q [B, q_len, H_q, D]; seq_lens count
    the new tokens (already appended). Returns ``out`` [B, q_len, H_q, D] (and ``lse``)."""
    _require_i32(block_table, seq_lens)
    B, q_len, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, q_len, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_paged_decode_multi_workspace_size(B, q_len, H_q, D), q.device)
    _check(lib().ts_paged_decode_multi_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                            block_table.shape[1], _ptr(seq_lens), B, q_len, H_q, H_kv, D,
                                            ps, P, float(scale), _dt(q), _ptr(out), _ptr(lse),
                                            _ptr(workspace), workspace.numel() * workspace.element_size(),
                                            _stream(stream)))
    return (out, lse) if return_lse else out


def _require_fp8_cache(k_pool, v_pool, k_scale, v_scale):
    if k_pool.dtype != torch.uint8 or v_pool.dtype != torch.uint8:
        raise TypeError("fp8 pools hold e4m3fn codes as uint8")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32:
        raise TypeError("fp8 scales are float32 [num_pages, page_size, H_kv]")
    if k_scale.shape != k_pool.shape[:3] or v_scale.shape != v_pool.shape[:3]:
        raise ValueError("scales must be [num_pages, page_size, H_kv] of their pool")


def ts_kv_append_fp8(k_new, v_new, k_pool, v_pool, k_scale, v_scale, block_table, positions,
                     stream=None) -> None:
    """Quantize k_new/v_new [B, H_kv, D] into fp8 pools and their scales (see ts_attn.h)."""
    _require_i32(block_table, positions)
    _require_fp8_cache(k_pool, v_pool, k_scale, v_scale)
    B, H_kv, D = k_new.shape
    _check(lib().ts_kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale),
                                  _ptr(v_scale), _ptr(block_table), block_table.shape[1], _ptr(positions), B,
                                  H_kv, D, k_pool.shape[1], k_pool.shape[0], _dt(k_new), _stream(stream)))


def ts_paged_decode_fp8_attn(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, scale: float,
                             out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Decode attention over an fp8 (e4m3fn) cache with bf16 queries; returns ``out`` (and ``lse``)."""
    _require_i32(block_table, seq_lens)
    _require_fp8_cache(k_pool, v_pool, k_scale, v_scale)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_paged_decode_workspace_size(B, H_q, D), q.device)
    _check(lib().ts_paged_decode_fp8_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
                                          _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, H_q, H_kv,
                                          D, ps, P, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def ts_merge_states(o_a, lse_a, o_b, lse_b, o_out=None, lse_out=None, stream=None):
    """LSE-merge two states [rows, D] (+ [rows] LSE); returns (o_out, lse_out)."""
    D = o_a.shape[-1]
    rows = o_a.numel() // D
    if o_out is None:
        o_out = torch.empty_like(o_a)
    if lse_out is None:
        lse_out = torch.empty_like(lse_a)
    _check(lib().ts_merge_states(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), _ptr(o_out), _ptr(lse_out),
                                 rows, D, _dt(o_a), _stream(stream)))
    return o_out, lse_out


def ts_group_prefixes(block_table: np.ndarray, seq_lens: np.ndarray, page_size: int, min_group: int = 2):
    """Host greedy longest-shared-prefix grouping; returns a dict of int32 numpy arrays."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = lens.shape[0]
    cap_g = max(1, B // max(2, min_group))
    caps = np.maximum(0, (lens.astype(np.int64) - 1) // page_size)
    cap_pages = max(1, int(min(int(caps.sum()), cap_g * bt.shape[1])))
    # the library writes every entry it reports; nothing needs clearing
    arrays = {
        "prefix_indptr": np.empty(cap_g + 1, np.int32), "prefix_pages": np.empty(cap_pages, np.int32),
        "prefix_len": np.empty(cap_g, np.int32), "member_indptr": np.empty(cap_g + 1, np.int32),
        "member_ids": np.empty(max(1, B), np.int32), "group_of": np.empty(max(1, B), np.int32),
    }
    c = PrefixGroupsC(0, *[arrays[k].ctypes.data for k in
                           ("prefix_indptr", "prefix_pages", "prefix_len", "member_indptr", "member_ids",
                            "group_of")], cap_g, cap_pages, max(1, B))
    _check(lib().ts_group_prefixes(bt.ctypes.data, bt.shape[1], lens.ctypes.data, B, page_size, min_group,
                                   ctypes.byref(c)))
    G = c.num_groups
    return {
        "num_groups": G,
        "prefix_indptr": arrays["prefix_indptr"][:G + 1].copy(),
        "prefix_pages": arrays["prefix_pages"][:arrays["prefix_indptr"][G]].copy(),
        "prefix_len": arrays["prefix_len"][:G].copy(),
        "member_indptr": arrays["member_indptr"][:G + 1].copy(),
        "member_ids": arrays["member_ids"][:arrays["member_indptr"][G]].copy(),
        "group_of": arrays["group_of"][:B].copy(),
    }


def ts_group_prefixes_nested(block_table: np.ndarray, seq_lens: np.ndarray, page_size: int,
                             min_group: int = 2):
    """Host greedy shared-prefix search kept as a tree; returns a dict of int32 numpy arrays
    (nodes level by level, see ts_prefix_forest in ts_attn.h)."""
    bt = np.ascontiguousarray(block_table, dtype=np.int32)
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    B = lens.shape[0]
    caps = np.maximum(0, (lens.astype(np.int64) - 1) // page_size)
    cap_n = max(1, B)               # every node has >= 2 members and its own sequence set
    cap_l = max(1, int(caps.max()) if B else 1)
    cap_pages = max(1, int(caps.sum()))
    cap_members = max(1, int(caps.sum()))  # a sequence is in at most one node per shared page
    while True:
        arrays = {
            "level_indptr": np.empty(cap_l + 1, np.int32), "parent": np.empty(cap_n, np.int32),
            "prefix_indptr": np.empty(cap_n + 1, np.int32), "prefix_pages": np.empty(cap_pages, np.int32),
            "prefix_len": np.empty(cap_n, np.int32), "member_indptr": np.empty(cap_n + 1, np.int32),
            "member_ids": np.empty(cap_members, np.int32), "group_of": np.empty(max(1, B), np.int32),
        }
        c = PrefixForestC(0, 0, *[arrays[k].ctypes.data for k in
                                  ("level_indptr", "parent", "prefix_indptr", "prefix_pages", "prefix_len",
                                   "member_indptr", "member_ids", "group_of")],
                          cap_n, cap_l, cap_pages, cap_members)
        st = lib().ts_group_prefixes_nested(bt.ctypes.data, bt.shape[1], lens.ctypes.data, B, page_size,
                                            min_group, ctypes.byref(c))
        if st != TS_ERR_CAPACITY:
            break
        cap_n, cap_l = max(cap_n, c.num_nodes), max(cap_l, c.num_levels)
        cap_members *= 2
    _check(st)
    N, L = c.num_nodes, c.num_levels
    return {
        "num_nodes": N, "num_levels": L,
        "level_indptr": arrays["level_indptr"][:L + 1].copy() if N else np.zeros(1, np.int32),
        "parent": arrays["parent"][:N].copy(),
        "prefix_indptr": arrays["prefix_indptr"][:N + 1].copy(),
        "prefix_pages": arrays["prefix_pages"][:arrays["prefix_indptr"][N]].copy(),
        "prefix_len": arrays["prefix_len"][:N].copy(),
        "member_indptr": arrays["member_indptr"][:N + 1].copy(),
        "member_ids": arrays["member_ids"][:arrays["member_indptr"][N]].copy(),
        "group_of": arrays["group_of"][:B].copy(),
    }


def forest_to_device(forest: dict, device="cuda") -> dict:
    """Device int32 copies of the arrays of ts_group_prefixes_nested (plus the host level_indptr)."""
    out = {"num_nodes": int(forest["num_nodes"]), "num_levels": int(forest["num_levels"]),
           "level_indptr_host": np.ascontiguousarray(forest["level_indptr"], dtype=np.int32)}
    for k in ("level_indptr", "parent", "prefix_indptr", "prefix_pages", "prefix_len", "member_indptr",
              "member_ids", "group_of"):
        a = forest[k] if len(forest[k]) else np.zeros(1, np.int32)
        out[k] = torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)
    return out


def ts_cascade_nested_decode_attn(q, k_pool, v_pool, forest_dev: dict, block_table, seq_lens, scale: float,
                                  out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Cascade decode over a nested prefix forest (device arrays from forest_to_device)."""
    _require_i32(block_table, seq_lens)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_cascade_decode_workspace_size(B, H_q, D), q.device)
    f = forest_dev
    c = PrefixForestC(f["num_nodes"], f["num_levels"], *[f[k].data_ptr() for k in
                                                         ("level_indptr", "parent", "prefix_indptr", "prefix_pages",
                                                          "prefix_len", "member_indptr", "member_ids", "group_of")],
                      0, 0, 0, 0)
    lvl = f["level_indptr_host"]
    _check(lib().ts_cascade_nested_decode_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), ctypes.byref(c),
                                               lvl.ctypes.data, _ptr(block_table), block_table.shape[1],
                                               _ptr(seq_lens), B, H_q, H_kv, D, ps, P, float(scale), _dt(q),
                                               _ptr(out), _ptr(lse), _ptr(workspace),
                                               workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def groups_to_device(groups: dict, device="cuda") -> dict:
    """Device int32 copies of the CSR arrays of ts_group_prefixes."""
    out = {"num_groups": int(groups["num_groups"])}
    for k in ("prefix_indptr", "prefix_pages", "prefix_len", "member_indptr", "member_ids", "group_of"):
        a = groups[k] if len(groups[k]) else np.zeros(1, np.int32)
        out[k] = torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(device)
    return out


def ts_cascade_decode_workspace_size(B: int, H_q: int, D: int) -> int:
    return int(lib().ts_cascade_decode_workspace_size(B, H_q, D))


def ts_cascade_decode_attn(q, k_pool, v_pool, groups_dev: dict, block_table, seq_lens, scale: float,
                           out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Shared-prefix (cascade) decode attention; ``groups_dev`` from :func:`groups_to_device`."""
    _require_i32(block_table, seq_lens)
    B, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_cascade_decode_workspace_size(B, H_q, D), q.device)
    g = groups_dev
    c = PrefixGroupsC(g["num_groups"], _ptr(g["prefix_indptr"]), _ptr(g["prefix_pages"]), _ptr(g["prefix_len"]),
                      _ptr(g["member_indptr"]), _ptr(g["member_ids"]), _ptr(g["group_of"]), 0, 0, 0)
    _check(lib().ts_cascade_decode_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), ctypes.byref(c), _ptr(block_table),
                                        block_table.shape[1], _ptr(seq_lens), B, H_q, H_kv, D, ps, P,
                                        float(scale), _dt(q), _ptr(out), _ptr(lse), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def ts_mla_workspace_size(B: int, H: int, D_v: int) -> int:
    return int(lib().ts_mla_workspace_size(B, H, D_v))


def ts_mla_paged_decode(q, kv_pool, block_table, seq_lens, scale: float, d_v: int = 512, out=None, lse=None,
                        workspace=None, stream=None, return_lse: bool = False):
    """Absorbed-MLA decode: q [B, H, Dqk] bf16, kv_pool [P, ps, Dqk] bf16 -> out [B, H, d_v]."""
    _require_i32(block_table, seq_lens)
    B, H, Dqk = q.shape
    P, ps, _ = kv_pool.shape
    if out is None:
        out = torch.empty(B, H, d_v, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty(B, H, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_mla_workspace_size(B, H, d_v), q.device)
    _check(lib().ts_mla_paged_decode(_ptr(q), _ptr(kv_pool), _ptr(block_table), block_table.shape[1],
                                     _ptr(seq_lens), B, H, Dqk, d_v, ps, P, float(scale), _ptr(out), _ptr(lse),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)))
    return (out, lse) if return_lse else out


def ts_paged_decode_tree_attn(q, k_pool, v_pool, block_table, seq_lens, parents, scale: float, out=None,
                              lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Tree verification: q [B, n, H_q, D] bf16, parents int32 [B, n] (-1 or an
    earlier draft token) -> out [B, n, H_q, D]."""
    _require_i32(block_table, seq_lens, parents)
    B, n, H_q, D = q.shape
    P, ps, H_kv, _ = k_pool.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty(B, n, H_q, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(256, q.device)
    _check(lib().ts_paged_decode_tree_attn(_ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(block_table),
                                           block_table.shape[1], _ptr(seq_lens), _ptr(parents), B, n, H_q, H_kv, D,
                                           ps, P, float(scale), _dt(q), _ptr(out), _ptr(lse), _ptr(workspace),
                                           workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def ts_mla_multi_workspace_size(B: int, q_len: int, H: int, D_v: int) -> int:
    return int(lib().ts_mla_multi_workspace_size(B, q_len, H, D_v))


def ts_mla_paged_decode_multi(q, kv_pool, block_table, seq_lens, scale: float, d_v: int = 512, out=None,
                              lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Absorbed-MLA decode of q_len tokens per sequence: q [B, q_len, H, Dqk] bf16,
    kv_pool [P, ps, Dqk] bf16 -> out [B, q_len, H, d_v]."""
    _require_i32(block_table, seq_lens)
    B, q_len, H, Dqk = q.shape
    P, ps, _ = kv_pool.shape
    if out is None:
        out = torch.empty(B, q_len, H, d_v, dtype=q.dtype, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty(B, q_len, H, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(ts_mla_multi_workspace_size(B, q_len, H, d_v), q.device)
    _check(lib().ts_mla_paged_decode_multi(_ptr(q), _ptr(kv_pool), _ptr(block_table), block_table.shape[1],
                                           _ptr(seq_lens), B, q_len, H, Dqk, d_v, ps, P, float(scale), _ptr(out),
                                           _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream)))
    return (out, lse) if return_lse else out


def ts_mla_paged_decode_fp8(q_codes, q_scale, kv_codes, kv_scale, block_table, seq_lens, scale: float,
                            d_v: int = 512, out=None, lse=None, workspace=None, stream=None, return_lse: bool = False):
    """Absorbed-MLA decode on e4m3 inputs: q_codes uint8 [B, H, 576] or [B, q_len, H, 576]
    with q_scale float32 [B, (q_len,) H]; kv_codes uint8 [P, ps, 576] with kv_scale
    float32 [P, ps] -> out bf16 [B, (q_len,) H, d_v]."""
    _require_i32(block_table, seq_lens)
    if q_codes.dtype != torch.uint8 or kv_codes.dtype != torch.uint8:
        raise TypeError("fp8 codes travel as uint8 tensors")
    if q_scale.dtype != torch.float32 or kv_scale.dtype != torch.float32:
        raise TypeError("scales must be float32")
    single = q_codes.dim() == 3
    B, q_len, H, Dqk = (q_codes.shape[0], 1, *q_codes.shape[1:]) if single else q_codes.shape
    P, ps, _ = kv_codes.shape
    shape = (B, H) if single else (B, q_len, H)
    if out is None:
        out = torch.empty(*shape, d_v, dtype=torch.bfloat16, device=q_codes.device)
    if lse is None and return_lse:
        lse = torch.empty(*shape, dtype=torch.float32, device=q_codes.device)
    if workspace is None:
        workspace = new_workspace(ts_mla_multi_workspace_size(B, q_len, H, d_v), q_codes.device)
    _check(lib().ts_mla_paged_decode_fp8(_ptr(q_codes), _ptr(q_scale), _ptr(kv_codes), _ptr(kv_scale),
                                         _ptr(block_table), block_table.shape[1], _ptr(seq_lens), B, q_len, H, Dqk,
                                         d_v, ps, P, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))
    return (out, lse) if return_lse else out


def ts_read_device_error(workspace, stream=None) -> int:
    """Sticky device error bits of a workspace; None reads those of the
    allocation-free entry point's static scratch on the current device."""
    v = ctypes.c_uint32(0)
    _check(lib().ts_read_device_error(_ptr(workspace), ctypes.byref(v), _stream(stream)))
    return int(v.value)


def ts_trace_enable(on: bool) -> None:
    _check(lib().ts_trace_enable(1 if on else 0))


def ts_clock_stamp(stamps, stream=None) -> None:
    """Enqueues one clock stamp per row of ``stamps`` (an int64 device tensor
    [n, 3]): SM id, that SM's cycle counter, global timer in ns."""
    if stamps.dtype != torch.int64 or stamps.dim() != 2 or stamps.shape[1] != 3 or not stamps.is_contiguous():
        raise TSError(TS_ERR_INVALID_ARG, "ts_clock_stamp: stamps must be a contiguous int64 tensor [n, 3]")
    _check(lib().ts_clock_stamp(_ptr(stamps), stamps.shape[0], _stream(stream)))


def ts_trace_collect(capacity: int = 4096):
    """[(kernel name, device ms)] of the launches recorded since the last collect."""
    buf = (LaunchRecordC * capacity)()
    n = lib().ts_trace_collect(buf, capacity)
    if n < 0:
        raise TSError(TS_ERR_CUDA, lib().ts_last_error_detail().decode())
    return [(buf[i].kernel.decode(), float(buf[i].ms)) for i in range(min(n, capacity))]
