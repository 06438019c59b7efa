"""Thin ctypes binding of libsatk.so (include/satk.h).

Argument marshalling only: every function checks dtypes and shapes of the
torch tensors it is handed, passes their device pointers, sizes and strides
to the C entry point of the same name on the current CUDA stream, and raises
on a non-zero return.  No computation happens here and there is no fallback:
without the compiled library every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsatk.so")

SATK_F32, SATK_BF16, SATK_F16 = 0, 1, 2
SATK_PAIRS_F32, SATK_PACKED_BF16 = 0, 1
STATUS_SLOTS_EXCEEDED = 1
STATUS_DUPLICATE_KEYS = 2
STATUS_BAD_REQUEST = 4
STATUS_NO_BLOCK = 8
STATUS_TOO_MANY_TOKENS = 16
STATUS_BAD_ROW = 32
STATUS_BAD_POSITION = 64
STATUS_STALLED = 128
TOPK_MAX_K = 4096
MERGE_MAX_CANDIDATES = 32768
TABLES_MAX_REQUESTS = 8192
LATENT_MAX = 512
LATENT_TAIL_MAX = 64
EXPANDED_MAX_QK = 256
EXPANDED_MAX_V = 128
LATENT_MAX_RANKS = 64

EXPORTS = ("satk_topk_rows", "satk_dcp_pack", "satk_dcp_merge_select",
           "satk_dcp_rescue_select", "satk_rescue_recv_words", "satk_status_string",
           "satk_dcp_emit_rows", "satk_topk_rows_sorted", "topk_rows", "topk_rows_sorted",
           "dcp_pack", "dcp_merge_select", "dcp_rescue_select", "dcp_emit_rows",
           "satk_dcp_topk_pack", "dcp_topk_pack", "satk_debug_flags", "satk_step_tables",
           "satk_latent_store", "satk_latent_workspace_bytes", "satk_latent_attend",
           "satk_latent_attend_rows", "satk_latent_attend_expanded", "satk_latent_merge")

_lock = threading.Lock()
_lib = None


class SatkError(RuntimeError):
    pass


def load(path: str) -> ctypes.CDLL:
    """Loads a build of the library at `path` and declares the signatures of
    its entry points (include/satk.h)."""
    if not os.path.exists(path):
        raise SatkError(f"{path} is missing: build it with "
                        "`python -m sparse_attention_indexer_radix_gb300.build`")
    L = ctypes.CDLL(path)
    vp, i32, i64, c_int = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    f32, size = ctypes.c_float, ctypes.c_size_t
    sigs = {
        "satk_topk_rows": [vp, c_int, i64, i64, i64, vp, i32, vp, i64, vp],
        "satk_topk_rows_sorted": [vp, c_int, i64, i64, i64, vp, i32, vp, i64, vp],
        "satk_dcp_pack": [vp, i64, i64, i64, vp, i64, i32, vp, vp, vp],
        "satk_dcp_topk_pack": [vp, i64, i64, i64, vp, i32, vp, vp],
        "satk_dcp_merge_select": [vp, c_int, i32, i64, i32, i32, vp, i64, vp, vp, vp],
        "satk_dcp_rescue_select": [vp, i32, i64, i32, i32, vp, i64, i64, vp, vp, vp, vp,
                                   i64, vp, vp],
        "satk_dcp_emit_rows": [vp, i64, i32, i64, i32, i32, vp, vp, i64, i64, i32, i32,
                               i64, vp, i64, vp, vp, vp],
        "satk_step_tables": [vp, vp, i32, i32, i32, i32, i64, vp, i64, vp, i64, i32, i32, i64,
                             vp, vp, vp, vp, vp, vp, vp, vp, vp],
        "satk_latent_store": [vp, i64, vp, i64, c_int, i64, i32, i32, vp, f32, vp, i64, vp, i32,
                              vp, vp, i64, i64, vp, vp],
        "satk_latent_attend": [vp, c_int, i64, i32, i32, i32, i64, i64, vp, i64, i64, vp, vp,
                               i64, i64, i32, i32, i64, vp, vp, i32, f32, vp, i64, i64, vp, vp,
                               size, vp, vp],
        "satk_latent_attend_rows": [vp, c_int, i64, i32, i32, i32, i64, i64, vp, i64, i64, vp,
                                    i64, i32, vp, f32, vp, i64, i64, vp, vp, size, vp, vp],
        "satk_latent_attend_expanded": [vp, c_int, i64, i32, i32, i32, i64, i64, vp, i64, i64,
                                        i64, vp, i64, vp, i32, i64, i64, vp, vp, i32, vp, f32,
                                        vp, i64, i64, vp, vp],
        "satk_latent_merge": [vp, c_int, i32, i64, i32, i32, i64, i64, i64, vp, vp, i64, i64,
                              vp, vp],
    }
    for name, args in sigs.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = c_int
    L.satk_rescue_recv_words.argtypes = [i64, i32, i32]
    L.satk_rescue_recv_words.restype = ctypes.c_size_t
    L.satk_latent_workspace_bytes.argtypes = [i32, i32]
    L.satk_latent_workspace_bytes.restype = size
    L.satk_status_string.argtypes = [c_int]
    L.satk_status_string.restype = ctypes.c_char_p
    L.satk_debug_flags.argtypes = [c_int]
    L.satk_debug_flags.restype = ctypes.c_uint
    return L


_routed = threading.local()


def lib() -> ctypes.CDLL:
    """The library the calls of this module go to: libsatk.so, loaded on
    first use (raises if it has not been built), or the one `routed_to`
    selects for the current thread."""
    global _lib
    r = getattr(_routed, "lib", None)
    if r is not None:
        return r
    with _lock:
        if _lib is None:
            _lib = load(LIB_PATH)
    return _lib


@contextlib.contextmanager
def routed_to(L: ctypes.CDLL):
    """Within the block, this thread's calls go to the library L (another
    build of the same sources, e.g. the bounds-checking debug build)."""
    prev = getattr(_routed, "lib", None)
    _routed.lib = L
    try:
        yield L
    finally:
        _routed.lib = prev


# Stands in for the data pointer of a zero-size tensor (torch gives 0) in a
# call whose batch is empty: the entry points check it is non-null and
# aligned, then return before any launch, so it is never dereferenced.
_EMPTY_BATCH_PTR = 256


def _ptr(t, empty_batch: bool = False):
    if t is None:
        return None
    if empty_batch and t.data_ptr() == 0:
        return ctypes.c_void_p(_EMPTY_BATCH_PTR)
    return ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(rc: int, name: str):
    if rc != 0:
        msg = lib().satk_status_string(rc).decode()
        raise SatkError(f"{name} returned {rc}: {msg}")


def _need_cuda(*ts) -> int:
    """The CUDA device of the first tensor; every one must live on a CUDA device."""
    for t in ts:
        if t is not None and not t.is_cuda:
            raise SatkError("every tensor must live on a CUDA device")
    return ts[0].get_device()


def _on(device: int, f, *args):
    """f(*args) with `device` current: launches, a kernel's attributes and the
    number of SMs go by the current device, not by the tensors'."""
    if device == torch.cuda.current_device():
        return f(*args)
    with torch.cuda.device(device):
        return f(*args)


def _int32_or_none(t, name):
    if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
        raise SatkError(f"{name} must be contiguous int32")


def _rowmajor_2d(t, name):
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise SatkError(f"{name} must be 2-D with unit column stride, got "
                        f"{tuple(t.shape)} {t.stride()}")


def _table_columns(max_blocks, width: int) -> int:
    """How many columns of a block table count: of the tensor's own at most,
    although the library would take any number below the row stride."""
    if max_blocks is None:
        return width
    if max_blocks > width:
        raise SatkError(f"max_blocks {max_blocks} is more than block_table's {width} columns")
    return max_blocks


def topk_rows(logits: torch.Tensor, k: int, row_ends: torch.Tensor | None = None,
              out: torch.Tensor | None = None, *, sorted: bool = False) -> torch.Tensor:
    """Exact top-k column ids of each row of ``logits`` ([rows, cols] float32
    or bfloat16, any row stride).  ``out`` (int32 [rows, >= k], any row
    stride) receives the ids in columns [0, k); columns past k are never
    written.  ``sorted`` orders them by descending score, ties by ascending
    column (satk_topk_rows_sorted).  Returns ``out`` (allocated [rows, k]
    when not given)."""
    dev = _need_cuda(logits, row_ends, out)
    _rowmajor_2d(logits, "logits")
    if logits.dtype == torch.float32:
        dt = SATK_F32
    elif logits.dtype == torch.bfloat16:
        dt = SATK_BF16
    else:
        raise SatkError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    rows, cols = logits.shape
    if out is None:
        out = torch.empty((rows, k), dtype=torch.int32, device=logits.device)
    _rowmajor_2d(out, "out")
    if out.dtype != torch.int32 or out.shape[0] != rows or out.shape[1] < k:
        raise SatkError(f"out must be int32 [{rows}, >= {k}]")
    if row_ends is not None and (row_ends.dtype != torch.int32 or not row_ends.is_contiguous()
                                 or row_ends.numel() < rows):
        raise SatkError("row_ends must be contiguous int32 [rows]")
    ld = logits.stride(0) if rows > 1 else max(cols, 1)
    ld_out = out.stride(0) if rows > 1 else out.shape[1]
    f = lib().satk_topk_rows_sorted if sorted else lib().satk_topk_rows
    e = rows == 0
    rc = _on(dev, f, _ptr(logits, e), dt, rows, cols, ld, _ptr(row_ends, e), k, _ptr(out, e),
             ld_out, _stream(logits.device))
    _check(rc, "satk_topk_rows_sorted" if sorted else "satk_topk_rows")
    return out


def packed_row_words(n: int) -> int:
    return n + n // 32


def rescue_slots(k: int, n: int) -> int:
    return (k - 1) // n


def rescue_recv_words(T: int, n: int, k: int) -> int:
    return int(lib().satk_rescue_recv_words(T, n, k))


def dcp_pack(logits: torch.Tensor, local_idx: torch.Tensor,
             row_ends: torch.Tensor | None = None,
             out: torch.Tensor | None = None) -> torch.Tensor:
    """Pack a local top-n (``local_idx`` int32 [rows, n], -1 padded) of the
    bf16 ``logits`` [rows, S] into B' rows ``out`` (int32 [rows, n + n/32],
    contiguous)."""
    dev = _need_cuda(logits, local_idx, row_ends, out)
    _rowmajor_2d(logits, "logits")
    _rowmajor_2d(local_idx, "local_idx")
    if logits.dtype != torch.bfloat16 or local_idx.dtype != torch.int32:
        raise SatkError("dcp_pack takes bfloat16 logits and int32 local_idx")
    rows, S = logits.shape
    n = local_idx.shape[1]
    if out is None:
        out = torch.empty((rows, packed_row_words(n)), dtype=torch.int32, device=logits.device)
    if out.dtype != torch.int32 or not out.is_contiguous() or \
            out.numel() != rows * packed_row_words(n):
        raise SatkError(f"out must be contiguous int32 [{rows}, {packed_row_words(n)}]")
    ld = logits.stride(0) if rows > 1 else max(S, 1)
    ld_idx = local_idx.stride(0) if rows > 1 else n
    e = rows == 0
    rc = _on(dev, lib().satk_dcp_pack,
             _ptr(logits, e), rows, S, ld, _ptr(local_idx, e), ld_idx, n, _ptr(row_ends, e),
             _ptr(out, e), _stream(logits.device))
    _check(rc, "satk_dcp_pack")
    return out


def dcp_topk_pack(logits: torch.Tensor, n: int, row_ends: torch.Tensor | None = None,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """The local top-n of each bf16 row of ``logits`` [rows, S] written
    straight as B' rows ``out`` (int32 [rows, n + n/32], contiguous): what
    dcp_pack makes of topk_rows(logits, n)."""
    dev = _need_cuda(logits, row_ends, out)
    _rowmajor_2d(logits, "logits")
    if logits.dtype != torch.bfloat16:
        raise SatkError("dcp_topk_pack takes bfloat16 logits")
    rows, S = logits.shape
    if out is None:
        out = torch.empty((rows, packed_row_words(n)), dtype=torch.int32, device=logits.device)
    if out.dtype != torch.int32 or not out.is_contiguous() or \
            out.numel() != rows * packed_row_words(n):
        raise SatkError(f"out must be contiguous int32 [{rows}, {packed_row_words(n)}]")
    if row_ends is not None and (row_ends.dtype != torch.int32 or not row_ends.is_contiguous()):
        raise SatkError("row_ends must be contiguous int32")
    ld = logits.stride(0) if rows > 1 else max(S, 1)
    e = rows == 0
    rc = _on(dev, lib().satk_dcp_topk_pack,
             _ptr(logits, e), rows, S, ld, _ptr(row_ends, e), n, _ptr(out, e),
             _stream(logits.device))
    _check(rc, "satk_dcp_topk_pack")
    return out


def dcp_merge_select(cand: torch.Tensor, k: int, *, packed: bool,
                     ids_out: torch.Tensor | None = None,
                     sat_word: torch.Tensor | None = None,
                     status: torch.Tensor | None = None) -> torch.Tensor:
    """Top-k merge over a rank-major candidate buffer read in place.

    packed=False: ``cand`` is [W, T, n, 2] int32 (float32 score bits, global
    id).  packed=True: ``cand`` is int32 [W, T, n + n/32] B' rows; then
    ``sat_word`` (int32 [T]) may receive the saturation words."""
    dev = _need_cuda(cand, ids_out, sat_word, status)
    if cand.dtype != torch.int32 or not cand.is_contiguous():
        raise SatkError("cand must be contiguous int32")
    if packed:
        if cand.dim() != 3:
            raise SatkError("packed cand must be [W, T, n + n/32]")
        W, T, words = cand.shape
        n = words * 32 // 33
        if packed_row_words(n) != words:
            raise SatkError(f"packed rows of {words} words are not n + n/32")
        fmt = SATK_PACKED_BF16
    else:
        if cand.dim() != 4 or cand.shape[3] != 2:
            raise SatkError("pairs cand must be [W, T, n, 2]")
        W, T, n, _ = cand.shape
        fmt = SATK_PAIRS_F32
    if ids_out is None:
        ids_out = torch.empty((T, k), dtype=torch.int32, device=cand.device)
    _rowmajor_2d(ids_out, "ids_out")
    if ids_out.dtype != torch.int32 or ids_out.shape[0] != T or ids_out.shape[1] < k:
        raise SatkError(f"ids_out must be int32 [{T}, >= {k}]")
    _int32_or_none(sat_word, "sat_word")
    _int32_or_none(status, "status")
    if sat_word is not None and sat_word.numel() < T:
        raise SatkError("sat_word must hold T words")
    ld_out = ids_out.stride(0) if T > 1 else ids_out.shape[1]
    e = T == 0
    rc = _on(dev, lib().satk_dcp_merge_select,
             _ptr(cand, e), fmt, W, T, n, k, _ptr(ids_out, e), ld_out, _ptr(sat_word, e),
             _ptr(status), _stream(cand.device))
    _check(rc, "satk_dcp_merge_select")
    return ids_out


def dcp_rescue_select(packed: torch.Tensor, logits: torch.Tensor, sat_word: torch.Tensor,
                      ids_out: torch.Tensor, k: int, *, recv: torch.Tensor | None = None,
                      row_ends: torch.Tensor | None = None,
                      status: torch.Tensor | None = None) -> torch.Tensor:
    """Second round of the packed merge: pushes of the saturated ranks into
    ``recv`` and the re-select of the saturated rows of ``ids_out`` (in
    place).  ``logits`` is bf16 [W, T, S] (unit column stride, rows at a
    common stride); ``row_ends`` int32 [W, T].  Returns ``recv``."""
    dev = _need_cuda(packed, logits, sat_word, ids_out, recv, row_ends, status)
    if packed.dtype != torch.int32 or packed.dim() != 3 or not packed.is_contiguous():
        raise SatkError("packed must be contiguous int32 [W, T, n + n/32]")
    W, T, words = packed.shape
    n = words * 32 // 33
    if logits.dtype != torch.bfloat16 or logits.dim() != 3 or tuple(logits.shape[:2]) != (W, T):
        raise SatkError(f"logits must be bfloat16 [{W}, {T}, S]")
    S = logits.shape[2]
    if S > 1 and logits.stride(2) != 1:
        raise SatkError("logits rows need unit column stride")
    ld = logits.stride(1) if T > 1 else (logits.stride(0) if W > 1 else max(S, 1))
    if W > 1 and T > 1 and logits.stride(0) != ld * T:
        raise SatkError("logits rows must sit at one common stride (rank-major)")
    _int32_or_none(status, "status")
    words_needed = rescue_recv_words(T, n, k)
    if recv is None:
        recv = torch.zeros(max(words_needed, 1), dtype=torch.int32, device=packed.device)
    if recv.dtype != torch.int32 or not recv.is_contiguous() or recv.numel() < words_needed:
        raise SatkError(f"recv must be contiguous int32 with >= {words_needed} words")
    _rowmajor_2d(ids_out, "ids_out")
    ld_out = ids_out.stride(0) if T > 1 else ids_out.shape[1]
    e = T == 0
    rc = _on(dev, lib().satk_dcp_rescue_select,
             _ptr(packed, e), W, T, n, k, _ptr(logits, e), S, ld, _ptr(row_ends, e),
             _ptr(sat_word, e), _ptr(recv, e), _ptr(ids_out, e), ld_out, _ptr(status),
             _stream(packed.device))
    _check(rc, "satk_dcp_rescue_select")
    return recv


def dcp_emit_rows(ids: torch.Tensor, W: int, dcp_rank: int, req_id: torch.Tensor,
                  block_table: torch.Tensor, block_size: int, stride_rows: int, *,
                  k: int | None = None, max_blocks: int | None = None,
                  rows_out: torch.Tensor | None = None,
                  valid_out: torch.Tensor | None = None,
                  status: torch.Tensor | None = None):
    """This rank's physical KV rows of the selected global ids ``ids``
    ([T, >= k] int32, as a merge writes them): ``block_table`` is int32
    [R, width] (unit column stride; ``max_blocks`` defaults to its width),
    ``req_id`` int32 [T].  Returns (rows_out [T, >= k] int32, valid_out [T]
    int32)."""
    dev = _need_cuda(ids, req_id, block_table, rows_out, valid_out, status)
    _rowmajor_2d(ids, "ids")
    _rowmajor_2d(block_table, "block_table")
    if ids.dtype != torch.int32 or req_id.dtype != torch.int32 or block_table.dtype != torch.int32:
        raise SatkError("ids, req_id and block_table must be int32")
    T = ids.shape[0]
    k = ids.shape[1] if k is None else k
    if not req_id.is_contiguous() or req_id.numel() < T:
        raise SatkError("req_id must be contiguous int32 with T entries")
    R, width = block_table.shape
    max_blocks = _table_columns(max_blocks, width)
    if rows_out is None:
        rows_out = torch.empty((T, k), dtype=torch.int32, device=ids.device)
    if valid_out is None:
        valid_out = torch.empty(T, dtype=torch.int32, device=ids.device)
    _rowmajor_2d(rows_out, "rows_out")
    if rows_out.dtype != torch.int32 or rows_out.shape[0] != T or rows_out.shape[1] < k:
        raise SatkError(f"rows_out must be int32 [{T}, >= {k}]")
    if valid_out.dtype != torch.int32 or not valid_out.is_contiguous() or valid_out.numel() < T:
        raise SatkError("valid_out must be contiguous int32 with T entries")
    _int32_or_none(status, "status")
    ld_ids = ids.stride(0) if T > 1 else ids.shape[1]
    ld_rows = rows_out.stride(0) if T > 1 else rows_out.shape[1]
    ld_table = block_table.stride(0) if R > 1 else max(width, 1)
    e = T == 0
    rc = _on(dev, lib().satk_dcp_emit_rows,
             _ptr(ids, e), T, k, ld_ids, W, dcp_rank, _ptr(req_id, e), _ptr(block_table, e), R,
             ld_table, max_blocks, block_size, stride_rows, _ptr(rows_out, e), ld_rows,
             _ptr(valid_out, e), _ptr(status), _stream(ids.device))
    _check(rc, "satk_dcp_emit_rows")
    return rows_out, valid_out


# The latent-cache operators are called once a layer and step with little work
# each, so their marshalling reads every tensor property once (a handful of
# 0.1 us calls) and hands plain integers to ctypes.

_DTYPE16 = {torch.bfloat16: SATK_BF16, torch.float16: SATK_F16}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dtype16(t, name: str) -> int:
    code = _DTYPE16.get(t.dtype)
    if code is None:
        raise SatkError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return code


def _stream_on(device: int) -> int:
    if _raw_stream is not None:
        return _raw_stream(device)
    return torch.cuda.current_stream(device).cuda_stream


def _device_of(*ts) -> int:
    """The CUDA device that holds every tensor."""
    dev = None
    for t in ts:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise SatkError("every tensor must live on a CUDA device")
        if dev is None:
            dev = d
        elif d != dev:
            raise SatkError(f"tensors on two devices: {dev} and {d}")
    return dev


def _addr(t):
    """A tensor's address for ctypes: None stays NULL, a tensor without
    elements gets the stand-in that is checked and never dereferenced."""
    if t is None:
        return None
    return t.data_ptr() or _EMPTY_BATCH_PTR


def _int32_vec(t, n: int, name: str):
    if t.dtype is not torch.int32 or t.numel() < n or not t.is_contiguous():
        raise SatkError(f"{name} must be contiguous int32 with {n} entries")


def _status_addr(status):
    """The address of the nullable status word: kernels OR bits into four bytes."""
    if status is None:
        return None
    _int32_vec(status, 1, "status")
    return status.data_ptr()


def _bad_layout(t, name: str, dims: int):
    raise SatkError(f"{name} must be {dims}-D with unit stride in its last dimension, got "
                    f"{tuple(t.shape)} {t.stride()}")


def _matrix(t, name: str):
    """(rows, cols, row stride) of a 2-D tensor with unit column stride."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (shape[1] > 1 and stride[1] != 1):
        _bad_layout(t, name, 2)
    rows, cols = shape
    return rows, cols, stride[0] if rows > 1 else (cols or 1)


def _heads(t, name: str):
    """(rows, heads, width, row stride, head stride) of a 3-D tensor with unit
    stride inside; strides of dimensions of one as if it were contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (shape[2] > 1 and stride[2] != 1):
        _bad_layout(t, name, 3)
    n, h, w = shape
    return n, h, w, stride[0] if n > 1 else h * w, stride[1] if h > 1 else w


def _lse_out(lse, T: int, H: int, like):
    if lse is None:
        return torch.empty((T, H), dtype=torch.float32, device=like.device)
    if lse.dtype is not torch.float32 or lse.shape != (T, H) or not lse.is_contiguous():
        raise SatkError(f"lse must be contiguous float32 [{T}, {H}]")
    return lse


def _heads_out(out, T: int, H: int, width: int, like):
    """The output tensor, with its row and head strides."""
    if out is None:
        return (torch.empty((T, H, width), dtype=like.dtype, device=like.device), H * width, width)
    n, h, w, ld_t, ld_h = _heads(out, "out")
    if out.dtype is not like.dtype or (n, h, w) != (T, H, width):
        raise SatkError(f"out must be {like.dtype} [{T}, {H}, {width}]")
    return out, ld_t, ld_h


class StepTables(NamedTuple):
    """What step_tables writes: token_starts [R + 1], lens [R], blocks_used [1]
    and the per-token req_id, positions, row_ends, slots [tokens], all int32."""
    token_starts: torch.Tensor
    lens: torch.Tensor
    req_id: torch.Tensor
    positions: torch.Tensor
    row_ends: torch.Tensor
    slots: torch.Tensor
    blocks_used: torch.Tensor


def step_tables(context_lens: torch.Tensor, new_lens: torch.Tensor, free_blocks: torch.Tensor,
                block_table: torch.Tensor, *, tokens: int, block_size: int, stride_rows: int,
                W: int = 1, dcp_rank: int = 0, drafted: bool = False,
                max_blocks: int | None = None, out: StepTables | None = None,
                status: torch.Tensor | None = None) -> StepTables:
    """One step's metadata from request lengths: extends ``block_table``
    (int32 [R, width], in place) with blocks taken from the front of
    ``free_blocks`` and returns the per-token arrays that topk_rows
    (row_ends), dcp_emit_rows (req_id), latent_store (positions, slots) and
    latent_attend take.  ``tokens`` is their capacity; entries past the last
    new token are padding (row_end 0, slot -1).  ``drafted`` gives every new
    token its request's context as row_end."""
    dev = _device_of(context_lens, new_lens, free_blocks, block_table, status)
    R, width, ld = _matrix(block_table, "block_table")
    if block_table.dtype is not torch.int32:
        raise SatkError("block_table must be int32")
    _int32_vec(context_lens, R, "context_lens")
    _int32_vec(new_lens, R, "new_lens")
    _int32_vec(free_blocks, 0, "free_blocks")
    if tokens < 0:
        raise SatkError("tokens must not be negative")
    sizes = (R + 1, R, tokens, tokens, tokens, tokens, 1)
    if out is None:
        # one allocation, one after the other
        buf = torch.empty(2 * R + 4 * tokens + 2, dtype=torch.int32, device=block_table.device)
        out = StepTables(*buf.split(sizes))
        base = buf.data_ptr()
        at = [base, base + 4 * (R + 1), base + 4 * (2 * R + 1)]
        for _ in range(4):
            at.append(at[-1] + 4 * tokens)
    else:
        _device_of(block_table, *out)
        for name, t, n in zip(StepTables._fields, out, sizes):
            _int32_vec(t, n, name)
        at = [_addr(t) for t in out]
    rc = _on(
        dev, lib().satk_step_tables,
        _addr(context_lens), _addr(new_lens), R, W, dcp_rank, block_size, stride_rows,
        _addr(free_blocks), free_blocks.numel(), _addr(block_table), ld,
        _table_columns(max_blocks, width), 1 if drafted else 0, tokens, *at,
        _status_addr(status), _stream_on(dev))
    if rc:
        _check(rc, "satk_step_tables")
    return out


def latent_store(latent: torch.Tensor, tail: torch.Tensor | None, slots: torch.Tensor,
                 cache: torch.Tensor, *, weight: torch.Tensor | None = None, eps: float = 1e-6,
                 cos_sin: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 interleaved: bool = False, status: torch.Tensor | None = None) -> torch.Tensor:
    """Writes rows [norm(latent) * weight | rotated tail] of new tokens into
    ``cache`` ([rows, >= dl + dr] bfloat16 or float16, in place) at ``slots``
    (int32 [T], negative: skipped, others distinct: tokens that share a slot
    leave parts of each).  ``weight`` float32 [dl] or None (no norm);
    ``cos_sin`` float32 [P, dr] (cosines, then sines) with ``positions``
    int32 [T], or None (no rotation).  Returns ``cache``."""
    dev = _device_of(latent, tail, slots, cache, weight, cos_sin, positions, status)
    T, dl, ld = _matrix(latent, "latent")
    rows, width, ld_cache = _matrix(cache, "cache")
    dt = _dtype16(cache, "cache")
    dr = ld_tail = 0
    if tail is not None:
        n, dr, ld_tail = _matrix(tail, "tail")
        if tail.dtype is not cache.dtype or n != T:
            raise SatkError(f"tail must be {cache.dtype} [{T}, dr]")
    if latent.dtype is not cache.dtype or width < dl + dr:
        raise SatkError(f"latent must be {cache.dtype} and cache at least {dl + dr} wide")
    _int32_vec(slots, T, "slots")
    if weight is not None and (weight.dtype is not torch.float32 or weight.numel() != dl
                               or not weight.is_contiguous()):
        raise SatkError(f"weight must be contiguous float32 [{dl}]")
    P = 0
    if cos_sin is not None:
        shape = cos_sin.shape
        if cos_sin.dtype is not torch.float32 or len(shape) != 2 or shape[1] != dr or \
                not cos_sin.is_contiguous():
            raise SatkError(f"cos_sin must be contiguous float32 [P, {dr}]")
        if positions is None:
            raise SatkError("cos_sin needs positions")
        _int32_vec(positions, T, "positions")
        P = shape[0]
    rc = _on(
        dev, lib().satk_latent_store,
        _addr(latent), ld, _addr(tail) if dr else None, ld_tail, dt, T, dl, dr, _addr(weight),
        eps, _addr(cos_sin) if dr else None, P, _addr(positions), 1 if interleaved else 0,
        _addr(slots), _addr(cache), rows, ld_cache, _status_addr(status), _stream_on(dev))
    if rc:
        _check(rc, "satk_latent_store")
    return cache


def latent_workspace_bytes(heads: int, latent_dim: int) -> int:
    """Bytes of the scratch of latent_attend and latent_attend_rows on the
    current device."""
    return int(lib().satk_latent_workspace_bytes(heads, latent_dim))


def _latent_call(dev, q, cache, latent_dim, out, lse, workspace):
    """Shared checks of the two attentions over cache rows: the tokens, the
    arguments before and after the keys', and the results."""
    T, H, D, ld_t, ld_h = _heads(q, "q")
    rows, width, ld_cache = _matrix(cache, "cache")
    dt = _dtype16(q, "q")
    if cache.dtype is not q.dtype or width < D:
        raise SatkError(f"cache must be {q.dtype} and at least {D} wide")
    if not 0 < latent_dim <= D:
        raise SatkError(f"latent_dim must be in 1..{D}")
    out, lo_t, lo_h = _heads_out(out, T, H, latent_dim, q)
    lse = _lse_out(lse, T, H, q)
    if workspace is None:
        size = max(_on(dev, lib().satk_latent_workspace_bytes, H, latent_dim), 16)
        workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    else:
        if not workspace.is_contiguous():
            raise SatkError("workspace must be contiguous")
        size = workspace.numel() * workspace.element_size()
    head = (_addr(q), dt, T, H, latent_dim, D - latent_dim, ld_t, ld_h, _addr(cache), rows,
            ld_cache)
    end = (_addr(out), lo_t, lo_h, _addr(lse), _addr(workspace), size)
    return T, head, end, out, lse


def latent_attend(q: torch.Tensor, cache: torch.Tensor, req_id: torch.Tensor,
                  block_table: torch.Tensor, row_ends: torch.Tensor, *, block_size: int,
                  stride_rows: int, latent_dim: int, scale: float,
                  tree: torch.Tensor | None = None, max_blocks: int | None = None,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None):
    """Attention of ``q`` ([T, H, D] bfloat16 or float16) over the requests'
    paged latent caches: token t sees its request's local tokens
    [0, row_ends[t]) and, with ``tree`` (int32 [T, words]), local token
    row_ends[t] + b for each set bit b.  Keys are whole cache rows, values
    their first ``latent_dim`` columns.  Returns (out [T, H, latent_dim], lse
    float32 [T, H])."""
    dev = _device_of(q, cache, req_id, block_table, row_ends, tree, out, lse, workspace, status)
    T, head, end, out, lse = _latent_call(dev, q, cache, latent_dim, out, lse, workspace)
    R, width, ld_table = _matrix(block_table, "block_table")
    if block_table.dtype is not torch.int32:
        raise SatkError("block_table must be int32")
    _int32_vec(req_id, T, "req_id")
    _int32_vec(row_ends, T, "row_ends")
    words = 0
    if tree is not None:
        shape = tree.shape
        if tree.dtype is not torch.int32 or len(shape) != 2 or shape[0] != T or shape[1] < 1 or \
                not tree.is_contiguous():
            raise SatkError(f"tree must be contiguous int32 [{T}, >= 1]")
        words = shape[1]
    rc = _on(
        dev, lib().satk_latent_attend,
        *head, _addr(req_id), _addr(block_table), R, ld_table,
        _table_columns(max_blocks, width), block_size, stride_rows, _addr(row_ends),
        _addr(tree), words, scale, *end, _status_addr(status), _stream_on(dev))
    if rc:
        _check(rc, "satk_latent_attend")
    return out, lse


def latent_attend_rows(q: torch.Tensor, cache: torch.Tensor, rows: torch.Tensor, *,
                       latent_dim: int, scale: float, counts: torch.Tensor | None = None,
                       k: int | None = None, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       status: torch.Tensor | None = None):
    """Attention of ``q`` ([T, H, D]) over each token's selected cache rows:
    ``rows`` int32 [T, >= k] and ``counts`` int32 [T] as dcp_emit_rows writes
    them (negative entries and those past the count are skipped).  Returns
    (out [T, H, latent_dim], lse float32 [T, H])."""
    dev = _device_of(q, cache, rows, counts, out, lse, workspace, status)
    T, head, end, out, lse = _latent_call(dev, q, cache, latent_dim, out, lse, workspace)
    n, width, ld_rows = _matrix(rows, "rows")
    k = width if k is None else k
    if rows.dtype is not torch.int32 or n != T or width < k:
        raise SatkError(f"rows must be int32 [{T}, >= {k}]")
    if counts is not None:
        _int32_vec(counts, T, "counts")
    rc = _on(
        dev, lib().satk_latent_attend_rows,
        *head, _addr(rows), ld_rows, k, _addr(counts), scale, *end, _status_addr(status),
        _stream_on(dev))
    if rc:
        _check(rc, "satk_latent_attend_rows")
    return out, lse


def latent_attend_expanded(q: torch.Tensor, k: torch.Tensor, tail: torch.Tensor | None,
                           v: torch.Tensor, token_starts: torch.Tensor, key_starts: torch.Tensor,
                           row_ends: torch.Tensor, *, scale: float,
                           out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """Prompt attention with per-head keys and values: ``q`` [T, H, dn + dr],
    ``k`` [S, H, dn], ``tail`` [S, dr] (shared by the heads, or None), ``v``
    [S, H, dv]; request r owns tokens token_starts[r:r+2] and keys
    key_starts[r:r+2]; token t sees its request's first row_ends[t] keys.
    Returns (out [T, H, dv], lse float32 [T, H])."""
    dev = _device_of(q, k, tail, v, token_starts, key_starts, row_ends, out, lse)
    T, H, D, q_t, q_h = _heads(q, "q")
    S, hk, dn, k_s, k_h = _heads(k, "k")
    sv, hv, dv, v_s, v_h = _heads(v, "v")
    dt = _dtype16(q, "q")
    if k.dtype is not q.dtype or v.dtype is not q.dtype:
        raise SatkError(f"k and v must be {q.dtype}")
    dr = ld_tail = 0
    if tail is not None:
        n, dr, ld_tail = _matrix(tail, "tail")
        if tail.dtype is not q.dtype or n != S:
            raise SatkError(f"tail must be {q.dtype} [{S}, dr]")
    if hk != H or (sv, hv) != (S, H) or D != dn + dr:
        raise SatkError(f"k, v and q must be [{S}, {H}, dn], [{S}, {H}, dv] and [T, {H}, dn + dr]")
    R = token_starts.numel() - 1
    if R < 0:
        raise SatkError("token_starts must have at least one entry")
    _int32_vec(token_starts, R + 1, "token_starts")
    _int32_vec(key_starts, R + 1, "key_starts")
    _int32_vec(row_ends, T, "row_ends")
    out, o_t, o_h = _heads_out(out, T, H, dv, q)
    lse = _lse_out(lse, T, H, q)
    rc = _on(
        dev, lib().satk_latent_attend_expanded,
        _addr(q), dt, T, H, dn, dr, q_t, q_h, _addr(k), S, k_s, k_h, _addr(tail) if dr else None,
        ld_tail, _addr(v), dv, v_s, v_h, _addr(token_starts), _addr(key_starts), R,
        _addr(row_ends), scale, _addr(out), o_t, o_h, _addr(lse), _stream_on(dev))
    if rc:
        _check(rc, "satk_latent_attend_expanded")
    return out, lse


def latent_merge(parts: torch.Tensor, lse: torch.Tensor, *, out: torch.Tensor | None = None,
                 lse_out: torch.Tensor | None = None):
    """Joins W partial attention results over disjoint keys: ``parts``
    [W, T, H, dv] bfloat16 or float16, ``lse`` float32 [W, T, H] contiguous.
    Returns (out [T, H, dv], lse float32 [T, H])."""
    dev = _device_of(parts, lse, out, lse_out)
    shape, stride = parts.shape, parts.stride()
    if len(shape) != 4 or (shape[3] > 1 and stride[3] != 1):
        _bad_layout(parts, "parts", 4)
    W, T, H, dv = shape
    dt = _dtype16(parts, "parts")
    if lse.dtype is not torch.float32 or lse.shape != (W, T, H) or not lse.is_contiguous():
        raise SatkError(f"lse must be contiguous float32 [{W}, {T}, {H}]")
    out, o_t, o_h = _heads_out(out, T, H, dv, parts)
    lse_out = _lse_out(lse_out, T, H, parts)
    rc = _on(
        dev, lib().satk_latent_merge,
        _addr(parts), dt, W, T, H, dv, stride[0] if W > 1 else T * H * dv,
        stride[1] if T > 1 else H * dv, stride[2] if H > 1 else dv, _addr(lse), _addr(out), o_t,
        o_h, _addr(lse_out), _stream_on(dev))
    if rc:
        _check(rc, "satk_latent_merge")
    return out, lse_out
