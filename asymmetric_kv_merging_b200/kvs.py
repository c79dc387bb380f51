"""ctypes binding of libkvs.so -- argument marshalling only.

Every function here turns torch tensors into raw pointers, calls the C entry point
of the same name (declared in include/kvs.h) on the current CUDA stream, and
raises KvsError on a non-OK status. All computation happens in the library's
CUDA kernels. Importing this module fails if the library is missing: there is
no other implementation to fall back to.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkvs.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libkvs.so not built ({_LIB_PATH}); run python -m asymmetric_kv_merging_b200.build")
_lib = ctypes.CDLL(_LIB_PATH)

F32, BF16 = 0, 1
OP_SCORE, OP_MERGE, OP_DECODE, OP_PREFILL, OP_PAGES = 0, 1, 2, 3, 4
SCOPE_HEAD, SCOPE_POOLED = 0, 1
_DTYPES = {F32: torch.float32, BF16: torch.bfloat16}
FORM_FULL, FORM_DIAGONAL, FORM_PER_QUERY = 0, 1, 2
FLAG_BAD_LENGTH, FLAG_OUT_CAPACITY, FLAG_INPLACE_SPAN, FLAG_NONFINITE_STATS = 1, 2, 4, 8
FLAG_TIMEOUT, FLAG_BUDGET, FLAG_NO_PAGES, FLAG_BAD_PAGE = 16, 32, 64, 128
PAGE_ROWS = 32

STATUS = {0: "KVS_OK", 1: "KVS_ERR_INVALID_ARG", 2: "KVS_ERR_UNSUPPORTED", 3: "KVS_ERR_BUDGET",
          4: "KVS_ERR_WORKSPACE", 5: "KVS_ERR_ALIAS", 6: "KVS_ERR_CUDA"}

EXPORTS = ("kvs_workspace_size", "kvs_score_pairs", "kvs_merge_compact", "kvs_decode_attn",
           "kvs_device_flags", "kvs_status_str", "kvs_version", "kvs_launch_count",
           "kvs_decode_attn_static", "kvs_static_scratch_bytes", "kvs_score_pairs_form",
           "kvs_prefill_chunk", "kvs_plan_rounds", "kvs_static_device_flags",
           "kvs_stream_read", "kvs_page_bytes", "kvs_page_assign", "kvs_page_store",
           "kvs_page_load", "kvs_page_decode_attn")


class CacheDesc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("H_q", ctypes.c_int32),
                ("d", ctypes.c_int32), ("T_cap", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class PagePool(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


class KvsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({_lib.kvs_status_str(status).decode()})")


_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_P = ctypes.POINTER(CacheDesc)
_lib.kvs_version.restype = _i32
_lib.kvs_launch_count.restype = ctypes.c_int64
_lib.kvs_status_str.restype = ctypes.c_char_p
_lib.kvs_status_str.argtypes = [ctypes.c_int]
_lib.kvs_workspace_size.restype = _sz
_lib.kvs_workspace_size.argtypes = [_P, _i32, _i32]
_lib.kvs_score_pairs.restype = ctypes.c_int
_lib.kvs_score_pairs.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
_lib.kvs_score_pairs_form.restype = ctypes.c_int
_lib.kvs_score_pairs_form.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _i32,
                                      _vp, _sz, _vp]
_lib.kvs_prefill_chunk.restype = ctypes.c_int
_lib.kvs_prefill_chunk.argtypes = [_P, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i32,
                                   _i32, _i32, ctypes.POINTER(_i32), _vp, _sz, _vp]
_lib.kvs_plan_rounds.restype = ctypes.c_int
_lib.kvs_plan_rounds.argtypes = [_i32, _i32, _i32, _i32, ctypes.POINTER(_i32), _i32,
                                 ctypes.POINTER(_i32)]
_lib.kvs_merge_compact.restype = ctypes.c_int
_lib.kvs_merge_compact.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp, _i32, _i32,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.kvs_decode_attn.restype = ctypes.c_int
_lib.kvs_decode_attn.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.kvs_decode_attn_static.restype = ctypes.c_int
_lib.kvs_decode_attn_static.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.kvs_static_scratch_bytes.restype = _sz
_lib.kvs_device_flags.restype = ctypes.c_int
_lib.kvs_stream_read.restype = ctypes.c_int
_lib.kvs_stream_read.argtypes = [_vp, ctypes.c_int64, _i32, _i32, _vp, _sz, _vp]
_lib.kvs_static_device_flags.restype = ctypes.c_int
_lib.kvs_static_device_flags.argtypes = [ctypes.POINTER(_i32), _i32, _vp]
_PP = ctypes.POINTER(PagePool)
_lib.kvs_page_bytes.restype = _sz
_lib.kvs_page_bytes.argtypes = [_i32]
_lib.kvs_page_assign.restype = ctypes.c_int
_lib.kvs_page_assign.argtypes = [_PP, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _sz, _vp]
_lib.kvs_page_store.restype = ctypes.c_int
_lib.kvs_page_store.argtypes = [_P, _vp, _vp, _vp, _vp, _PP, _vp, _sz, _vp]
_lib.kvs_page_load.restype = ctypes.c_int
_lib.kvs_page_load.argtypes = [_P, _PP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.kvs_page_decode_attn.restype = ctypes.c_int
_lib.kvs_page_decode_attn.argtypes = [_P, _vp, _PP, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.kvs_device_flags.argtypes = [_vp, ctypes.POINTER(_i32), _i32, _vp]

if _lib.kvs_version() != 1:
    raise ImportError("libkvs.so version mismatch; rebuild it")


def library_path() -> str:
    return _LIB_PATH


def dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return F32
    if t == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported cache dtype {t}")


def make_desc(B: int, H_kv: int, H_q: int, d: int, T_cap: int, dtype) -> CacheDesc:
    code = dtype if isinstance(dtype, int) else dtype_code(dtype)
    return CacheDesc(int(B), int(H_kv), int(H_q), int(d), int(T_cap), int(code))


def desc_of(K: torch.Tensor, H_q: int) -> CacheDesc:
    """Descriptor of a [B, H_kv, T_cap, d] cache tensor."""
    B, H_kv, T_cap, d = K.shape
    return make_desc(B, H_kv, H_q, d, T_cap, K.dtype)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# the handle of a device's current stream without building a Stream object (3 us a call), where torch
# has it: one without CUDA does not, and sizes and plans need no device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)
_current_device = torch.cuda.current_device


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        raise KvsError(status, where)


def workspace_size(desc: CacheDesc, W: int, op: int) -> int:
    return int(_lib.kvs_workspace_size(ctypes.byref(desc), int(W), int(op)))


def workspace(desc: CacheDesc, W: int = 32, ops=(OP_SCORE, OP_MERGE, OP_DECODE), device=None) -> torch.Tensor:
    """A zero-filled workspace large enough for every op in `ops` (uint8 tensor)."""
    n = max(workspace_size(desc, W, op) for op in ops)
    if n == 0:
        raise ValueError("invalid cache shape for the workspace")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def score_pairs(desc, K, V, logn, lens, cand_begin, n_recent, Q_win, W, score, w_b, ws, stream=None,
                form=None):
    """kvs_score_pairs, or kvs_score_pairs_form when `form` is given."""
    if form is None:
        _check(_lib.kvs_score_pairs(ctypes.byref(desc), _ptr(K), _ptr(V), _ptr(logn), _ptr(lens),
                                    _ptr(cand_begin), int(n_recent), _ptr(Q_win), int(W),
                                    _ptr(score), _ptr(w_b), _ptr(ws), ws.numel(), _stream(stream)),
               "kvs_score_pairs")
        return
    _check(_lib.kvs_score_pairs_form(ctypes.byref(desc), _ptr(K), _ptr(V), _ptr(logn), _ptr(lens),
                                     _ptr(cand_begin), int(n_recent), _ptr(Q_win), int(W),
                                     _ptr(score), _ptr(w_b), int(form), _ptr(ws), ws.numel(),
                                     _stream(stream)),
           "kvs_score_pairs_form")


def merge_compact(desc, K, V, logn, lens, cand_begin, n_recent, score, w_b, target, scope,
                  T_cap_out, K_out, V_out, logn_out, len_out, ws, dbg_selected=None,
                  dbg_out_offset=None, dbg_kmerged=None, stream=None):
    _check(_lib.kvs_merge_compact(ctypes.byref(desc), _ptr(K), _ptr(V), _ptr(logn), _ptr(lens),
                                  _ptr(cand_begin), int(n_recent), _ptr(score), _ptr(w_b),
                                  _ptr(target), int(scope), int(T_cap_out), _ptr(K_out),
                                  _ptr(V_out), _ptr(logn_out), _ptr(len_out), _ptr(dbg_selected),
                                  _ptr(dbg_out_offset), _ptr(dbg_kmerged), _ptr(ws), ws.numel(),
                                  _stream(stream)),
           "kvs_merge_compact")


def decode_attn(desc, q, K, V, logn, lens, out, ws, k_new=None, v_new=None, stream=None):
    _check(_lib.kvs_decode_attn(ctypes.byref(desc), _ptr(q), _ptr(K), _ptr(V), _ptr(logn),
                                _ptr(lens), _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(ws),
                                ws.numel(), _stream(stream)),
           "kvs_decode_attn")


def device_flags(ws: torch.Tensor, clear: bool = False, stream=None) -> int:
    out = _i32(0)
    _check(_lib.kvs_device_flags(_ptr(ws), ctypes.byref(out), int(bool(clear)), _stream(stream)),
           "kvs_device_flags")
    return int(out.value)


def status_str(code: int) -> str:
    return _lib.kvs_status_str(int(code)).decode()


def launch_count() -> int:
    """Kernels launched through the library by this process (host-side count)."""
    return int(_lib.kvs_launch_count())


def decode_attn_static(desc, q, K, V, logn, lens, out, k_new=None, v_new=None, stream=None):
    """kvs_decode_attn on the library's built-in scratch buffer: allocates nothing."""
    _check(_lib.kvs_decode_attn_static(ctypes.byref(desc), _ptr(q), _ptr(K), _ptr(V), _ptr(logn),
                                       _ptr(lens), _ptr(k_new), _ptr(v_new), _ptr(out),
                                       _stream(stream)),
           "kvs_decode_attn_static")


def static_device_flags(clear: bool = False, stream=None) -> int:
    """kvs_static_device_flags: the flag word of the built-in scratch buffer."""
    out = _i32(0)
    _check(_lib.kvs_static_device_flags(ctypes.byref(out), int(bool(clear)), _stream(stream)),
           "kvs_static_device_flags")
    return int(out.value)


def stream_read(buf: torch.Tensor, d: int, ctas: int, ws: torch.Tensor, stream=None):
    """kvs_stream_read: stream a bf16 [rows, d] buffer with the decode's loads (timing
    helper)."""
    _check(_lib.kvs_stream_read(_ptr(buf), buf.numel() // d, int(d), int(ctas), _ptr(ws),
                                ws.numel(), _stream(stream)), "kvs_stream_read")


def static_scratch_bytes() -> int:
    return int(_lib.kvs_static_scratch_bytes())


def prefill_chunk(desc, K, V, logn, lens, L, k_chunk, v_chunk, Q_win, W, budget, sink, ws,
                  form=FORM_FULL, stream=None) -> int:
    """kvs_prefill_chunk: append a [B, H_kv, n, d] chunk at row L of every head and merge
    back to `budget`; returns the new length of every head."""
    n = 0 if k_chunk is None else int(k_chunk.shape[2])
    out = _i32(0)
    _check(_lib.kvs_prefill_chunk(ctypes.byref(desc), _ptr(K), _ptr(V), _ptr(logn), _ptr(lens),
                                  int(L), _ptr(k_chunk), _ptr(v_chunk), n, _ptr(Q_win), int(W),
                                  int(budget), int(sink), int(form), ctypes.byref(out), _ptr(ws),
                                  ws.numel(), _stream(stream)),
           "kvs_prefill_chunk")
    return int(out.value)


def plan_rounds(length: int, target: int, cand_begin: int, n_recent: int, max_lens: int = 64):
    """kvs_plan_rounds: the per-head lengths [len, ..., target] of the merge rounds."""
    buf = (_i32 * int(max_lens))()
    n = _i32(0)
    _check(_lib.kvs_plan_rounds(int(length), int(target), int(cand_begin), int(n_recent), buf,
                                int(max_lens), ctypes.byref(n)), "kvs_plan_rounds")
    return [int(buf[i]) for i in range(n.value + 1)]


def page_bytes(d: int) -> int:
    """Bytes of a page of 32 rows of d channels (0: head dim not built)."""
    return int(_lib.kvs_page_bytes(int(d)))


def page_pool(pages: torch.Tensor, table: torch.Tensor) -> PagePool:
    """The pool of `pages` [n_pages, page_bytes(d)] (uint8) with the page tables `table`
    [units, max_pages] (int32). It keeps both tensors alive."""
    if pages.dim() != 2 or pages.dtype != torch.uint8 or pages.shape[1] not in (page_bytes(64), page_bytes(128)):
        raise ValueError("pages must be uint8 [n_pages, page_bytes(d)]")
    if table.dim() != 2 or table.dtype != torch.int32 or table.device != pages.device:
        raise ValueError("table must be int32 [units, max_pages] on the pages' device")
    pool = PagePool(_ptr(pages), _ptr(table), pages.shape[0], table.shape[1])
    pool.tensors = (pages, table)
    pool.device, pool.units = pages.get_device(), table.shape[0]
    pool.head_dim = 64 if pages.shape[1] == page_bytes(64) else 128
    return pool


_I32, _U8, _FP32 = torch.int32, torch.uint8, torch.float32


def _arg(t, dtype, n, device):
    """Raw pointer of a tensor that the library reads or writes as n elements of dtype; a wrong
    type, size, device or layout would be read as something else, so it raises."""
    if t is None:
        return None
    if t.dtype is dtype and t.numel() == n and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"expected a contiguous {dtype} tensor of {n} elements on cuda:{device}, "
                     f"not {t.dtype} of {tuple(t.shape)} on {t.device}")


def _pool_device(pool: PagePool, units: int, d: Optional[int] = None) -> int:
    """The device of a call on `pool`, which has to be the current one (kernels launch there)."""
    device = pool.device
    if device != _current_device():
        raise ValueError(f"the pool is on {pool.tensors[0].device}, which is not the current device")
    if pool.units < units:
        raise ValueError(f"the pool has tables of {pool.units} units, not {units}")
    if d is not None and d != pool.head_dim:
        raise ValueError(f"the pool's pages are of head dim {pool.head_dim}, not {d}")
    return device


def page_assign(pool, rows, held, free_pages, n_free, ws, slots=None, slot_begin=None, stream=None):
    """kvs_page_assign: every unit of rows [units] holds the pages of its rows; with slots
    [units, stride], the slots of its rows from slot_begin on."""
    units = rows.numel()
    dev = _pool_device(pool, units)
    stride = 0 if slots is None else slots.shape[-1]
    nws = ws.numel()
    st = _lib.kvs_page_assign(
        pool, units, _arg(rows, _I32, units, dev), _arg(held, _I32, units, dev),
        _arg(free_pages, _I32, pool.n_pages, dev), _arg(n_free, _I32, 1, dev),
        _arg(slot_begin, _I32, units, dev), _arg(slots, _I32, units * stride, dev), stride,
        _arg(ws, _U8, nws, dev), nws, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise KvsError(st, "kvs_page_assign")


def _dtype(desc: CacheDesc, where: str) -> torch.dtype:
    dtype = _DTYPES.get(desc.dtype)
    if dtype is None:
        raise KvsError(2, where)                             # KVS_ERR_UNSUPPORTED, as the library says
    return dtype


def page_store(desc, K, V, logn, slots, pool, ws, stream=None):
    """kvs_page_store: the rows of K, V [B, H_kv, T_cap, d] into the pages at `slots`."""
    d, dtype = desc.d, _dtype(desc, "kvs_page_store")
    rows = desc.B * desc.H_kv * desc.T_cap
    dev = _pool_device(pool, 0, d)
    nws = ws.numel()
    st = _lib.kvs_page_store(
        desc, _arg(K, dtype, rows * d, dev), _arg(V, dtype, rows * d, dev),
        _arg(logn, _FP32, rows, dev), _arg(slots, _I32, rows, dev), pool, _arg(ws, _U8, nws, dev), nws,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise KvsError(st, "kvs_page_store")


def page_load(desc, pool, slots, K, V, logn, ws, stream=None):
    """kvs_page_load: the rows at `slots` back into K, V [B, H_kv, T_cap, d] and logn."""
    d, dtype = desc.d, _dtype(desc, "kvs_page_load")
    rows = desc.B * desc.H_kv * desc.T_cap
    dev = _pool_device(pool, 0, d)
    nws = ws.numel()
    st = _lib.kvs_page_load(
        desc, pool, _arg(slots, _I32, rows, dev), _arg(K, dtype, rows * d, dev),
        _arg(V, dtype, rows * d, dev), _arg(logn, _FP32, rows, dev), _arg(ws, _U8, nws, dev), nws,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise KvsError(st, "kvs_page_load")


def page_decode_attn(desc, q, pool, lens, out, ws, k_new=None, v_new=None, stream=None):
    """kvs_page_decode_attn: one decode step over the pages of every unit."""
    d, dtype, units = desc.d, _dtype(desc, "kvs_page_decode_attn"), desc.B * desc.H_kv
    dev = _pool_device(pool, units, d)
    n, nws = desc.B * desc.H_q * d, ws.numel()
    st = _lib.kvs_page_decode_attn(
        desc, _arg(q, dtype, n, dev), pool, _arg(lens, _I32, units, dev),
        _arg(k_new, dtype, units * d, dev), _arg(v_new, dtype, units * d, dev), _arg(out, dtype, n, dev),
        _arg(ws, _U8, nws, dev), nws, _raw_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        raise KvsError(st, "kvs_page_decode_attn")
