"""Python binding of libckv (the GB300 KV compressor) over its C ABI.

Argument marshalling only: every step runs in the library's CUDA kernels.
Functions take CUDA ``torch.Tensor`` arguments, pass their device pointers and
the current CUDA stream to the C entry point of the same name, and raise
``CkvError`` for a non-zero return code.  There is no CPU path: without the
built library (``build()`` / ``__graft_entry__.build()``) every call raises.

Layouts (see include/ckv.h): kv_score rows are C4 ``[kv-ovl|kv|score-ovl|score]``
(4*hd) or C128 ``[kv|score]`` (2*hd); the state is ``[rows, width]`` in the
input dtype with 8 rows per request (C4) or 128 (C128); plans are uint8
tensors of 16-byte (compress, decode) or 8-byte (write) records.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional, Tuple

import torch

from . import build as _build

F32 = 0
BF16 = 1
OUT_TOKEN = 0
OUT_COMPACT = 1

STATUS_BAD_LENGTH = 1
STATUS_BAD_TOTAL = 2
STATUS_CAPACITY = 4
STATUS_BAD_INDEX = 8
STATUS_TIMEOUT = 16

_lock = threading.Lock()
_lib = None


class CkvError(RuntimeError):
    def __init__(self, code: int, func: str, msg: str):
        super().__init__(f"{func}: {msg} (code {code})")
        self.code = code


def library_path() -> str:
    return _build.LIB


def load_library():
    """Loads libckv.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libckv.so is not built ({path}); run "
                               "compressed_kv_attention_compressplan_gb300.build.build() first")
        lib = ctypes.CDLL(path)
        vp, u32, i32, u64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int, ctypes.c_uint64
        lib.ckv_capacity_compress.argtypes = [i32, u32, u32]
        lib.ckv_capacity_compress.restype = u32
        lib.ckv_capacity_write.argtypes = [i32, u32, u32]
        lib.ckv_capacity_write.restype = u32
        lib.ckv_plan_decode.argtypes = [i32, vp, vp, u32, vp, vp, vp, vp]
        i64 = ctypes.c_int64
        lib.ckv_capacity_write_paged.argtypes = [i32, u32, u32, i32]
        lib.ckv_capacity_write_paged.restype = u32
        lib.ckv_plan_prefill_paged.argtypes = [i32, vp, vp, i64, u32, vp, u64, i32, i32, vp, vp, u32, u32, u32, u32,
                                               i32, vp, vp, vp, vp, vp]
        lib.ckv_plan_decode_paged.argtypes = [i32, vp, vp, i64, u32, vp, u64, i32, i32, vp, u32, vp, vp, vp, vp]
        lib.ckv_plan_prefill.argtypes = [i32, vp, vp, vp, u32, u32, u32, u32, i32, vp, vp, vp, vp, vp]
        lib.ckv_compress_write.argtypes = [i32, i32, i32, vp, u64, vp, u32, vp, vp, u32, vp, vp]
        lib.ckv_compress_pool_prefill.argtypes = [i32, i32, i32, i32, vp, u64, vp, u32, vp, vp, vp, u32, i32, vp,
                                                  ctypes.POINTER(PrefillHints), vp, vp]
        lib.ckv_compress_prefill.argtypes = [i32, i32, i32, i32, vp, u64, vp, u32, vp, vp, vp, vp, u32, u32, i32,
                                             vp, ctypes.POINTER(PrefillHints), vp, vp]
        lib.ckv_compress_decode.argtypes = [i32, i32, i32, i32, vp, u64, vp, vp, vp, vp, vp, vp, u32, vp, vp, vp]
        f32 = ctypes.c_float
        lib.ckv_capacity_online_units.argtypes = [u32, u32]
        lib.ckv_capacity_online_units.restype = u32
        lib.ckv_plan_online_prefill.argtypes = [vp, vp, vp, u32, u32, i64, u32, i32, vp, vp, vp, vp]
        lib.ckv_plan_online_decode.argtypes = [vp, vp, u32, i64, vp, vp, vp]
        lib.ckv_compress_online_prefill.argtypes = [i32, i32, i32, vp, u64, vp, u32, vp, vp, vp, u32, i32, u32, vp,
                                                    vp, vp]
        lib.ckv_compress_online_decode.argtypes = [i32, i32, i32, vp, u64, vp, vp, vp, u32, vp, vp, vp]
        lib.ckv_norm_rope_store_prefill.argtypes = [i32, i32, i32, i32, vp, i32, u64, vp, vp, u32, vp, f32, vp, u32,
                                                    vp, u64, i32, vp, u64, vp, vp]
        lib.ckv_norm_rope_store_decode.argtypes = [i32, i32, i32, i32, vp, vp, u32, vp, f32, vp, u32, vp, i32, vp,
                                                   u64, vp, vp]
        lib.ckv_compress_decode_norm_rope_store.argtypes = [i32, i32, i32, i32, vp, u64, vp, vp, vp, vp, vp, u32, vp,
                                                            f32, vp, u32, vp, i32, vp, u64, vp, vp]
        qc = ctypes.POINTER(Q8CacheArg)
        lib.ckv_capacity_q8_store.argtypes = [u32, u32, u32]
        lib.ckv_capacity_q8_store.restype = u32
        lib.ckv_plan_q8_store.argtypes = [qc, vp, vp, vp, u32, u32, vp, u64, u32, u32, i32, vp, vp, vp, vp]
        lib.ckv_q8_store.argtypes = [qc, i32, vp, vp, u32, vp, vp, u32, vp, vp]
        lib.ckv_q8_store_reset.argtypes = [qc, i32, vp, vp, u32, vp, vp, u32, vp, vp, vp]
        for f in (lib.ckv_q8_attn_plan_bytes, lib.ckv_q8_attn_workspace_bytes):
            f.argtypes = [qc, u32, u32, u32]
            f.restype = u64
        lib.ckv_plan_q8_attn.argtypes = [qc, u32, u32, vp, vp, vp, vp, u32, u32, vp, u64, vp, vp]
        lib.ckv_q8_attn.argtypes = [qc, u32, u32, f32, vp, u32, u32, vp, u64, u32, vp, u64, i32, vp, vp, vp, u64, vp,
                                    vp]
        lib.ckv_q8_weigh.argtypes = [qc, u32, u32, f32, f32, vp, vp, u32, vp, vp, vp, vp, u32, vp, u64, u32, vp, vp,
                                     vp]
        lib.ckv_q8_evict.argtypes = [qc, vp, vp, vp, u32, vp, u64, vp, u64, u32, u32, u32, u32, vp, vp, vp, vp]
        lib.ckv_q8_rope_store.argtypes = [qc, i32, vp, u64, vp, u64, u32, vp, vp, f32, vp, u32, u32, u32, i32, vp, vp, u32,
                                          vp, vp, vp]
        lib.ckv_q8_bounds.argtypes = [qc, vp, vp, vp, vp, u32, vp, u64, u32, vp, vp]
        lib.ckv_q8_block_scores.argtypes = [qc, vp, u32, u32, f32, vp, u32, vp, vp, vp, vp, u32, vp, u64, u32, u32, vp, vp,
                                            vp]
        lib.ckv_q8_block_select.argtypes = [vp, u32, u32, u32, u32, u32, vp, vp, vp, u32, u32, u32, u32, vp, vp, vp]
        lib.ckv_q8_attn_blocks_workspace_bytes.argtypes = [qc, u32, u32, u32]
        lib.ckv_q8_attn_blocks_workspace_bytes.restype = u64
        lib.ckv_q8_attn_blocks.argtypes = [qc, u32, u32, f32, vp, u32, vp, u32, vp, vp, vp, vp, u32, vp, u64, u32, i32, vp,
                                           vp, vp, u64, vp, vp]
        lib.ckv_error_string.argtypes = [i32]
        lib.ckv_error_string.restype = ctypes.c_char_p
        lib.ckv_version.restype = i32
        lib.ckv_set_wait_limit_ns.argtypes = [u64]
        lib.ckv_set_wait_limit_ns.restype = u64
        _lib = lib
        return lib


def _check(rc: int, func: str):
    if rc != 0:
        msg = load_library().ckv_error_string(rc).decode()
        raise CkvError(rc, func, msg)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libckv takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libckv takes contiguous tensors only")
    return ctypes.c_void_p(t.data_ptr())


def _lengths(*ts: Optional[torch.Tensor]) -> int:
    """Checks the per-request arrays (rid, seq_lens, extend_lens): int64, one
    dimension, all of one length (the batch), which is returned.  The library
    reads them as raw int64 arrays, so another dtype would be misread."""
    batch = None
    for t in ts:
        if t is None:
            continue
        if t.dtype != torch.int64 or t.dim() != 1:
            raise ValueError(f"per-request arrays must be 1-D int64 tensors (got {t.dtype}, {t.dim()}-D)")
        if batch is None:
            batch = t.numel()
        elif t.numel() != batch:
            raise ValueError(f"per-request arrays differ in length ({t.numel()} != {batch})")
    return batch or 0


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return F32
    if dt == torch.bfloat16:
        return BF16
    raise ValueError(f"unsupported dtype {dt}")


def width_of(ratio: int, head_dim: int) -> int:
    return 4 * head_dim if ratio == 4 else 2 * head_dim


def window_of(ratio: int) -> int:
    return 8 if ratio == 4 else ratio


def capacity_compress(ratio: int, batch: int, num_q_tokens: int) -> int:
    return int(load_library().ckv_capacity_compress(ratio, batch, num_q_tokens))


def capacity_write(ratio: int, batch: int, num_q_tokens: int) -> int:
    return int(load_library().ckv_capacity_write(ratio, batch, num_q_tokens))


def set_wait_limit_ns(limit_ns: int) -> int:
    """Sets the time limit of the staged kernels' waits on their copies for later launches
    (0 restores the 2 s default) and returns the previous limit."""
    if not 0 <= int(limit_ns) < 1 << 64:
        raise ValueError("limit_ns must fit an unsigned 64-bit integer")
    return int(load_library().ckv_set_wait_limit_ns(int(limit_ns)))


def new_status(device=None) -> torch.Tensor:
    """A zeroed device status word (uint32 bits, stored in an int32 tensor)."""
    return torch.zeros(4, dtype=torch.int32, device=device or "cuda")


# ------------------------------------------------------------------------------ plans
def new_decode_order(batch: int, device=None) -> torch.Tensor:
    """Storage for a decode batch's boundary-row list: ``[batch + 1, 8]`` uint8 (``ckv_decode_order_t``)."""
    return torch.empty(batch + 1, 8, dtype=torch.uint8, device=device or "cuda")


def _order(order: Optional[torch.Tensor], batch: int):
    if order is None:
        return None
    if order.dtype != torch.uint8 or order.dim() != 2 or order.shape[1] != 8 or order.shape[0] < batch + 1:
        raise ValueError("a decode order is a uint8 tensor [batch + 1, 8] (new_decode_order)")
    return _ptr(order)


def plan_decode(ratio: int, rid: torch.Tensor, seq_lens: torch.Tensor, plan_d: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, stream=None, order: Optional[torch.Tensor] = None) -> torch.Tensor:
    """DecodePlan records ``[batch, 16]`` uint8.  With ``order`` (``new_decode_order``), the batch's
    page-boundary rows are also written there, in row order."""
    batch = _lengths(rid, seq_lens)
    if plan_d is None:
        plan_d = torch.empty(max(batch, 1), 16, dtype=torch.uint8, device=rid.device)
    _check(load_library().ckv_plan_decode(ratio, _ptr(rid), _ptr(seq_lens), batch, _ptr(plan_d),
                                          _order(order, batch), _ptr(status), _stream(stream)), "ckv_plan_decode")
    return plan_d[:batch]


def plan_prefill(ratio: int, rid: torch.Tensor, seq_lens: torch.Tensor, extend_lens: torch.Tensor,
                 num_q_tokens: int, capacity_c: Optional[int] = None, capacity_w: Optional[int] = None,
                 pad_invalid: bool = False, plan_c: Optional[torch.Tensor] = None,
                 plan_w: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Returns ``(plan_c [cap_c,16] u8, plan_w [cap_w,8] u8, counts [4] int32)``; counts stay on the device:
    ``{num_c, num_w, min extend_len, max extend_len}``."""
    batch = _lengths(rid, seq_lens, extend_lens)
    dev = rid.device
    if capacity_c is None:
        capacity_c = capacity_compress(ratio, batch, num_q_tokens)
    if capacity_w is None:
        capacity_w = capacity_write(ratio, batch, num_q_tokens)
    if plan_c is None:
        plan_c = torch.empty(max(capacity_c, 1), 16, dtype=torch.uint8, device=dev)
    if plan_w is None:
        plan_w = torch.empty(max(capacity_w, 1), 8, dtype=torch.uint8, device=dev)
    if counts is None:
        counts = torch.empty(4, dtype=torch.int32, device=dev)
    _check(load_library().ckv_plan_prefill(ratio, _ptr(rid), _ptr(seq_lens), _ptr(extend_lens), batch, num_q_tokens,
                                           capacity_c, capacity_w, int(pad_invalid), _ptr(plan_c), _ptr(plan_w),
                                           _ptr(counts), _ptr(status), _stream(stream)), "ckv_plan_prefill")
    return plan_c[:capacity_c], plan_w[:capacity_w], counts


def capacity_write_paged(ratio: int, batch: int, num_q_tokens: int, swa_page_size: int) -> int:
    return int(load_library().ckv_capacity_write_paged(ratio, batch, num_q_tokens, swa_page_size))


def _paged_maps(req_to_token: Optional[torch.Tensor], full_to_state: Optional[torch.Tensor]):
    """(pointer, stride, rows) of req_to_token and (pointer, size) of full_to_state; C128 takes None for both."""
    if req_to_token is None:
        return None, 0, 0, None, 0
    if req_to_token.dtype != torch.int32 or full_to_state.dtype != torch.int64 or req_to_token.dim() != 2:
        raise ValueError("req_to_token must be 2-D int32 and full_to_state int64")
    return (_ptr(req_to_token), req_to_token.shape[1], req_to_token.shape[0], _ptr(full_to_state),
            full_to_state.numel())


def plan_prefill_paged(ratio: int, rid: torch.Tensor, req_to_token: torch.Tensor, full_to_state: torch.Tensor,
                       swa_page_size: int, ring_size: int, seq_lens: torch.Tensor, extend_lens: torch.Tensor,
                       num_q_tokens: int, capacity_c: Optional[int] = None, capacity_w: Optional[int] = None,
                       pad_invalid: bool = False, counts: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None, plan_c: Optional[torch.Tensor] = None,
                       plan_w: Optional[torch.Tensor] = None):
    """SWA-paged prefill plans; req_to_token is ``[num_reqs, stride]`` int32, full_to_state int64."""
    batch = _lengths(rid, seq_lens, extend_lens)
    dev = rid.device
    if capacity_c is None:
        capacity_c = capacity_compress(ratio, batch, num_q_tokens)
    if capacity_w is None:
        capacity_w = capacity_write_paged(ratio, batch, num_q_tokens, swa_page_size)
    if plan_c is None:
        plan_c = torch.empty(max(capacity_c, 1), 16, dtype=torch.uint8, device=dev)
    if plan_w is None:
        plan_w = torch.empty(max(capacity_w, 1), 8, dtype=torch.uint8, device=dev)
    if counts is None:
        counts = torch.empty(4, dtype=torch.int32, device=dev)
    r2t, stride, nreq, f2s, nfull = _paged_maps(req_to_token, full_to_state)
    _check(load_library().ckv_plan_prefill_paged(ratio, _ptr(rid), r2t, stride, nreq, f2s, nfull, swa_page_size,
                                                 ring_size, _ptr(seq_lens), _ptr(extend_lens), batch, num_q_tokens, capacity_c,
                                                 capacity_w, int(pad_invalid), _ptr(plan_c), _ptr(plan_w),
                                                 _ptr(counts), _ptr(status), _stream(stream)),
           "ckv_plan_prefill_paged")
    return plan_c[:capacity_c], plan_w[:capacity_w], counts


def plan_decode_paged(ratio: int, rid: torch.Tensor, req_to_token: torch.Tensor, full_to_state: torch.Tensor,
                      swa_page_size: int, ring_size: int, seq_lens: torch.Tensor,
                      status: Optional[torch.Tensor] = None, stream=None,
                      order: Optional[torch.Tensor] = None) -> torch.Tensor:
    batch = _lengths(rid, seq_lens)
    plan_d = torch.empty(max(batch, 1), 16, dtype=torch.uint8, device=rid.device)
    r2t, stride, nreq, f2s, nfull = _paged_maps(req_to_token, full_to_state)
    _check(load_library().ckv_plan_decode_paged(ratio, _ptr(rid), r2t, stride, nreq, f2s, nfull, swa_page_size,
                                                ring_size, _ptr(seq_lens), batch, _ptr(plan_d), _order(order, batch),
                                                _ptr(status), _stream(stream)),
           "ckv_plan_decode_paged")
    return plan_d[:batch]


# ------------------------------------------------------------------------------ compute
def _state_rows(state: torch.Tensor, ratio: int, head_dim: int) -> int:
    w = width_of(ratio, head_dim)
    if state.numel() % w:
        raise ValueError("state width does not match ratio / head_dim")
    return state.numel() // w


def compress_write(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, plan_w: torch.Tensor,
                   counts: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    _check(load_library().ckv_compress_write(ratio, head_dim, dtype_code(state.dtype), _ptr(state),
                                             _state_rows(state, ratio, head_dim), _ptr(kv_score),
                                             kv_score.shape[0], _ptr(plan_w), _ptr(counts), plan_w.shape[0],
                                             _ptr(status), _stream(stream)), "ckv_compress_write")


class PrefillHints(ctypes.Structure):
    """ckv_prefill_hints_t: the planner's rid / seq_lens / extend_lens (device pointers) and batch."""
    _fields_ = [("rid", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p), ("extend_lens", ctypes.c_void_p),
                ("batch", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _hints(hints):
    """``None`` or ``(rid, seq_lens, extend_lens)`` device tensors -> a ctypes pointer (or None)."""
    if hints is None:
        return None
    rid, sl, el = hints
    batch = _lengths(rid, sl, el)
    return ctypes.pointer(PrefillHints(_ptr(rid), _ptr(sl), _ptr(el), batch, 0))


def compress_pool_prefill(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                          plan_c: torch.Tensor, counts: Optional[torch.Tensor] = None,
                          out_layout: int = OUT_TOKEN, out_dtype: torch.dtype = torch.float32,
                          out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                          stream=None, hints=None) -> torch.Tensor:
    """``hints``: ``None`` or the ``(rid, seq_lens, extend_lens)`` the planner read (prefetch only)."""
    nq = kv_score.shape[0]
    rows = nq if out_layout == OUT_TOKEN else plan_c.shape[0]
    if out is None:
        out = torch.empty(max(rows, 1), head_dim, dtype=out_dtype, device=kv_score.device)
    _check(load_library().ckv_compress_pool_prefill(ratio, head_dim, dtype_code(kv_score.dtype), dtype_code(out.dtype),
                                                    _ptr(state), _state_rows(state, ratio, head_dim), _ptr(kv_score),
                                                    nq, _ptr(ape), _ptr(plan_c), _ptr(counts), plan_c.shape[0],
                                                    out_layout, _ptr(out), _hints(hints), _ptr(status),
                                                    _stream(stream)),
           "ckv_compress_pool_prefill")
    return out[:rows]


def compress_prefill(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                     plan_c: torch.Tensor, plan_w: torch.Tensor, counts: Optional[torch.Tensor] = None,
                     out_layout: int = OUT_TOKEN, out_dtype: torch.dtype = torch.float32,
                     out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None, hints=None) -> torch.Tensor:
    """Pool, then write the state (one stream, in that order).  ``hints`` as compress_pool_prefill."""
    nq = kv_score.shape[0]
    rows = nq if out_layout == OUT_TOKEN else plan_c.shape[0]
    if out is None:
        out = torch.empty(max(rows, 1), head_dim, dtype=out_dtype, device=kv_score.device)
    _check(load_library().ckv_compress_prefill(ratio, head_dim, dtype_code(kv_score.dtype), dtype_code(out.dtype),
                                               _ptr(state), _state_rows(state, ratio, head_dim), _ptr(kv_score), nq,
                                               _ptr(ape), _ptr(plan_c), _ptr(plan_w), _ptr(counts), plan_c.shape[0],
                                               plan_w.shape[0], out_layout, _ptr(out), _hints(hints), _ptr(status),
                                               _stream(stream)), "ckv_compress_prefill")
    return out[:rows]


def compress_decode(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                    plan_d: torch.Tensor, out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None, order: Optional[torch.Tensor] = None,
                    rid_hint: Optional[torch.Tensor] = None, seq_lens_hint: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Decode step over ``plan_d``; ``order`` is the boundary-row list plan_decode wrote for it (optional);
    ``rid_hint`` / ``seq_lens_hint`` are the arrays plan_decode read (optional, both or neither): the decode
    prefetches its windows from them before its dependency wait."""
    batch = plan_d.shape[0]
    if (rid_hint is None) != (seq_lens_hint is None):
        raise ValueError("rid_hint and seq_lens_hint go together")
    if rid_hint is not None and _lengths(rid_hint, seq_lens_hint) != batch:
        raise ValueError("the hints need one entry per batch row")
    if out is None:
        out = torch.empty(max(batch, 1), head_dim, dtype=out_dtype, device=kv_score.device)
    _check(load_library().ckv_compress_decode(ratio, head_dim, dtype_code(kv_score.dtype), dtype_code(out.dtype),
                                              _ptr(state), _state_rows(state, ratio, head_dim), _ptr(kv_score),
                                              _ptr(ape), _ptr(plan_d), _order(order, batch), _ptr(rid_hint),
                                              _ptr(seq_lens_hint), batch, _ptr(out), _ptr(status), _stream(stream)),
           "ckv_compress_decode")
    return out[:batch]


# ------------------------------------------------------------------------------ online C128 state
def capacity_online_units(batch: int, num_q_tokens: int) -> int:
    return int(load_library().ckv_capacity_online_units(batch, num_q_tokens))


def plan_online_prefill(rid: torch.Tensor, seq_lens: torch.Tensor, extend_lens: torch.Tensor, num_q_tokens: int,
                        slot_offset: int = 0, capacity_u: Optional[int] = None, pad_invalid: bool = False,
                        units: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None):
    """Returns ``(units [cap_u, 16] u8, counts [4] int32)``; counts = {num_c, num_units, min el, max el}."""
    batch = _lengths(rid, seq_lens, extend_lens)
    if capacity_u is None:
        capacity_u = capacity_online_units(batch, num_q_tokens)
    if units is None:
        units = torch.empty(max(capacity_u, 1), 16, dtype=torch.uint8, device=rid.device)
    if counts is None:
        counts = torch.empty(4, dtype=torch.int32, device=rid.device)
    _check(load_library().ckv_plan_online_prefill(_ptr(rid), _ptr(seq_lens), _ptr(extend_lens), batch, num_q_tokens,
                                                  slot_offset, capacity_u, int(pad_invalid), _ptr(units),
                                                  _ptr(counts), _ptr(status), _stream(stream)),
           "ckv_plan_online_prefill")
    return units[:capacity_u], counts


def plan_online_decode(rid: torch.Tensor, seq_lens: torch.Tensor, slot_offset: int = 0,
                       plan_d: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    batch = _lengths(rid, seq_lens)
    if plan_d is None:
        plan_d = torch.empty(max(batch, 1), 16, dtype=torch.uint8, device=rid.device)
    _check(load_library().ckv_plan_online_decode(_ptr(rid), _ptr(seq_lens), batch, slot_offset, _ptr(plan_d),
                                                 _ptr(status), _stream(stream)), "ckv_plan_online_decode")
    return plan_d[:batch]


def _online_state(state: torch.Tensor, head_dim: int) -> int:
    if state.dtype != torch.float32 or state.numel() % (3 * head_dim):
        raise ValueError("the online state is fp32 [slots, 3 * head_dim]")
    return state.numel() // (3 * head_dim)


def compress_online_prefill(head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                            units: torch.Tensor, counts: Optional[torch.Tensor], out_layout: int = OUT_TOKEN,
                            out_dtype: torch.dtype = torch.float32, out_rows: Optional[int] = None,
                            out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Folds the units' tokens into the state; token layout out [num_q_tokens, hd], compact [out_rows, hd]."""
    nq = kv_score.shape[0]
    if out is None:
        rows = nq if out_layout == OUT_TOKEN else int(out_rows)
        out = torch.empty(max(rows, 1), head_dim, dtype=out_dtype, device=kv_score.device)
    rows = out.shape[0] if out_layout == OUT_COMPACT else nq
    _check(load_library().ckv_compress_online_prefill(head_dim, dtype_code(kv_score.dtype), dtype_code(out.dtype),
                                                      _ptr(state), _online_state(state, head_dim), _ptr(kv_score),
                                                      nq, _ptr(ape), _ptr(units), _ptr(counts), units.shape[0],
                                                      out_layout, rows, _ptr(out), _ptr(status), _stream(stream)),
           "ckv_compress_online_prefill")
    return out


def compress_online_decode(head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                           plan_d: torch.Tensor, out_dtype: torch.dtype = torch.float32,
                           out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    batch = plan_d.shape[0]
    if out is None:
        out = torch.empty(max(batch, 1), head_dim, dtype=out_dtype, device=kv_score.device)
    _check(load_library().ckv_compress_online_decode(head_dim, dtype_code(kv_score.dtype), dtype_code(out.dtype),
                                                     _ptr(state), _online_state(state, head_dim), _ptr(kv_score),
                                                     _ptr(ape), _ptr(plan_d), batch, _ptr(out), _ptr(status),
                                                     _stream(stream)), "ckv_compress_online_decode")
    return out[:batch]


# ------------------------------------------------------------------------------ norm, RoPE, store
def _nr_common(rows: torch.Tensor, norm_weight: torch.Tensor, freqs: torch.Tensor, kv_cache: torch.Tensor):
    if norm_weight.dtype != torch.float32 or freqs.dtype != torch.float32 or freqs.dim() != 3 or freqs.shape[2] != 2:
        raise ValueError("norm_weight must be fp32 [head_dim] and freqs fp32 [max_pos, rope_dim/2, 2]")
    head_dim = kv_cache.shape[-1]
    return head_dim, 2 * freqs.shape[1], dtype_code(rows.dtype), dtype_code(kv_cache.dtype)


def norm_rope_store_prefill(ratio: int, rows: torch.Tensor, plan_c: torch.Tensor, counts: Optional[torch.Tensor],
                            norm_weight: torch.Tensor, eps: float, freqs: torch.Tensor, out_loc: torch.Tensor,
                            kv_cache: torch.Tensor, in_layout: int = OUT_COMPACT, status: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """RMSNorm + RoPE of the pooled prefill rows, stored into ``kv_cache`` at ``out_loc[ragged_id]``."""
    hd, rope_dim, ci, cc = _nr_common(rows, norm_weight, freqs, kv_cache)
    _check(load_library().ckv_norm_rope_store_prefill(ratio, hd, rope_dim, ci, _ptr(rows), in_layout, rows.shape[0],
                                                      _ptr(plan_c), _ptr(counts), plan_c.shape[0], _ptr(norm_weight),
                                                      float(eps), _ptr(freqs), freqs.shape[0], _ptr(out_loc),
                                                      out_loc.numel(), cc, _ptr(kv_cache), kv_cache.shape[0],
                                                      _ptr(status), _stream(stream)),
           "ckv_norm_rope_store_prefill")


def norm_rope_store_decode(ratio: int, rows: torch.Tensor, plan_d: torch.Tensor, norm_weight: torch.Tensor,
                           eps: float, freqs: torch.Tensor, out_loc: torch.Tensor, kv_cache: torch.Tensor,
                           status: Optional[torch.Tensor] = None, stream=None) -> None:
    """RMSNorm + RoPE of the decode output rows (non-boundary rows stored as zeros) at ``out_loc[b]``."""
    hd, rope_dim, ci, cc = _nr_common(rows, norm_weight, freqs, kv_cache)
    if out_loc.numel() < plan_d.shape[0]:
        raise ValueError("out_loc needs one entry per batch row")
    _check(load_library().ckv_norm_rope_store_decode(ratio, hd, rope_dim, ci, _ptr(rows), _ptr(plan_d),
                                                     plan_d.shape[0], _ptr(norm_weight), float(eps), _ptr(freqs),
                                                     freqs.shape[0], _ptr(out_loc), cc, _ptr(kv_cache),
                                                     kv_cache.shape[0], _ptr(status), _stream(stream)),
           "ckv_norm_rope_store_decode")


def compress_decode_norm_rope_store(head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                                    plan_d: torch.Tensor, norm_weight: torch.Tensor, eps: float, freqs: torch.Tensor,
                                    out_loc: torch.Tensor, kv_cache: torch.Tensor,
                                    status: Optional[torch.Tensor] = None, stream=None,
                                    rid_hint: Optional[torch.Tensor] = None,
                                    seq_lens_hint: Optional[torch.Tensor] = None) -> None:
    """The C4 decode fused with norm + RoPE + store: the state write, and each row's pooled row (+0.0 off a
    group boundary) normalised, rotated and stored into ``kv_cache`` at ``out_loc[b]``."""
    if norm_weight.dtype != torch.float32 or freqs.dtype != torch.float32 or freqs.dim() != 3 or freqs.shape[2] != 2:
        raise ValueError("norm_weight must be fp32 [head_dim] and freqs fp32 [max_pos, rope_dim/2, 2]")
    if (rid_hint is None) != (seq_lens_hint is None):
        raise ValueError("rid_hint and seq_lens_hint go together")
    batch = plan_d.shape[0]
    if out_loc.dtype != torch.int64 or out_loc.numel() < batch:
        raise ValueError("out_loc must be int64 with one entry per batch row")
    _lengths(rid_hint, seq_lens_hint)
    _check(load_library().ckv_compress_decode_norm_rope_store(
        4, head_dim, 2 * freqs.shape[1], dtype_code(kv_score.dtype), _ptr(state), _state_rows(state, 4, head_dim),
        _ptr(kv_score), _ptr(ape), _ptr(plan_d), _ptr(rid_hint), _ptr(seq_lens_hint), batch, _ptr(norm_weight),
        float(eps), _ptr(freqs), freqs.shape[0], _ptr(out_loc), dtype_code(kv_cache.dtype), _ptr(kv_cache),
        kv_cache.shape[0], _ptr(status), _stream(stream)), "ckv_compress_decode_norm_rope_store")


# ------------------------------------------------------------------------------ 8-bit paged cache
class Q8CacheArg(ctypes.Structure):
    """ckv_q8_cache_t."""
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_uint32), ("block_tokens", ctypes.c_uint32),
                ("n_kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32)]


class Q8Cache(NamedTuple):
    """A paged cache in 8 bits: ``k`` (and ``v``) ``[num_blocks, n_kv_heads, block_tokens, head_dim]``
    float8_e4m3fn, ``k_scale`` (and ``v_scale``) fp32 ``[num_blocks, n_kv_heads]``; the value held is
    ``k * k_scale``.  Without ``v`` the entries are keys and values at once (a latent cache)."""
    k: torch.Tensor
    k_scale: torch.Tensor
    v: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def new_q8_cache(num_blocks: int, n_kv_heads: int, block_tokens: int, head_dim: int, latent: bool = False,
                 device=None) -> Q8Cache:
    """An empty cache (zeros, scales 1); ``latent``: no separate values."""
    dev = device or "cuda"

    def side():
        pool = torch.zeros(num_blocks, n_kv_heads, block_tokens, head_dim, dtype=torch.uint8, device=dev)
        return pool.view(torch.float8_e4m3fn), torch.ones(num_blocks, n_kv_heads, device=dev)

    k, ks = side()
    v, vs = (None, None) if latent else side()
    return Q8Cache(k, ks, v, vs)


# Calls that make tensors make them on the stream that they run on: memory of the current stream could still be in use
# there, and a workspace is free again when the call returns.
#
# These calls are made once a layer on few microseconds of work, so what they check is checked in few Python steps:
# a tensor's address is taken, with the checks that make it usable, by _at(); lengths by _lens().
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_E4M3, _FP32 = torch.float8_e4m3fn, torch.float32


def _at(device: int, t: Optional[torch.Tensor]) -> Optional[int]:
    """The address of a contiguous tensor on the given CUDA device."""
    if t is None:
        return None
    if t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise ValueError("libckv takes CUDA tensors of one device only" if t.get_device() != device else
                     "libckv takes contiguous tensors only")


def _stream_of(device: int, stream):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _lens(device: int, *ts: torch.Tensor):
    """The batch and the addresses of per-request arrays: int64, one dimension, one length."""
    shape, at = ts[0].shape, []
    for t in ts:
        if t.dtype is not torch.int64 or t.shape != shape:
            _lengths(*ts)
        at.append(_at(device, t))
    if len(shape) != 1:
        _lengths(*ts)
    return shape[0], at


def _q8(cache: Q8Cache) -> Tuple[Q8CacheArg, int]:
    """ckv_q8_cache_t, and the device: the cache's, which must be the current one."""
    k, ks, v, vs = cache
    shape = k.shape
    if k.dtype is not _E4M3 or len(shape) != 4:
        raise ValueError("a q8 cache's k is float8_e4m3fn [num_blocks, n_kv_heads, block_tokens, head_dim]")
    blocks, heads, tokens, dim = shape
    if ks.dtype is not _FP32 or ks.shape != (blocks, heads):
        raise ValueError("a q8 cache's scales are fp32 [num_blocks, n_kv_heads]")
    device = k.get_device()
    if device < 0:
        raise ValueError("libckv takes CUDA tensors only")
    v_at = vs_at = None
    if v is not None or vs is not None:
        if v is None or vs is None:
            raise ValueError("v and v_scale go together")
        if v.dtype is not _E4M3 or v.shape != shape or vs.dtype is not _FP32 or vs.shape != (blocks, heads):
            raise ValueError("a q8 cache's v and v_scale are shaped like its k and k_scale")
        v_at, vs_at = _at(device, v), _at(device, vs)
    arg = Q8CacheArg(_at(device, k), _at(device, ks), v_at, vs_at, blocks, tokens, heads, dim)
    if device != _current_device():
        raise ValueError("the q8 cache is not on the current device")
    return arg, device


def _table(device: int, table: torch.Tensor):
    """(address, stride, rows) of a block table ``[num_reqs, blocks]`` int32."""
    shape = table.shape
    if table.dtype is not torch.int32 or len(shape) != 2:
        raise ValueError("a block table is int32 [num_reqs, blocks]")
    return _at(device, table), shape[1], shape[0]


def _is(t: torch.Tensor, what: str, dtype: torch.dtype, *shape: int) -> None:
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} {list(shape)} (got {t.dtype} {list(t.shape)})")


def _bytes_of(t: torch.Tensor, what: str) -> int:
    if t.dtype is not torch.uint8:
        raise ValueError(f"{what} is a uint8 tensor")
    return t.numel()


def _store_plan(plan: torch.Tensor, capacity: int) -> None:
    if plan.dtype is not torch.uint8 or plan.dim() != 2 or plan.shape[1] != 16 or plan.shape[0] < capacity:
        raise ValueError("a store plan is a uint8 tensor [capacity, 16]")


def _counts(**counts: int) -> None:
    """For counts of which one is negative or past 32 bits, which ctypes would take modulo 2^32."""
    raise ValueError("counts must be from 0 to 2^32 - 1 (got %s)" % ", ".join(f"{k} {v}" for k, v in counts.items()))


def _q8_error(rc: int, func: str):
    raise CkvError(rc, func, load_library().ckv_error_string(rc).decode())


def capacity_q8_store(batch: int, num_rows: int, block_tokens: int) -> int:
    if (batch | num_rows | block_tokens) >> 32:
        _counts(batch=batch, num_rows=num_rows, block_tokens=block_tokens)
    return int(load_library().ckv_capacity_q8_store(batch, num_rows, block_tokens))


def plan_q8_store(cache: Q8Cache, rid: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor, num_rows: int,
                  block_table: torch.Tensor, capacity: Optional[int] = None, pad_invalid: bool = False,
                  plan: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The blocks that a step's new rows touch: ``(plan [cap, 16] u8, counts [4] int32)``.  ``kv_lens`` counts the
    new entries (``new_lens``, 0 allowed); the plan serves every layer of the step."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return plan_q8_store(cache, rid, kv_lens, new_lens, num_rows, block_table, capacity, pad_invalid, plan, counts,
                                 status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, kv_at, new_at) = _lens(dev, rid, kv_lens, new_lens)
    if (num_rows | (capacity or 0)) >> 32:
        _counts(num_rows=num_rows, capacity=capacity or 0)
    if capacity is None:
        capacity = lib.ckv_capacity_q8_store(batch, num_rows, arg.block_tokens)
    if plan is None:
        plan = torch.empty((capacity, 16), dtype=torch.uint8, device=rid.device)
    _store_plan(plan, capacity)
    if counts is None:
        counts = torch.empty(4, dtype=torch.int32, device=rid.device)
    _is(counts, "counts", torch.int32, 4)
    table, stride, reqs = _table(dev, block_table)
    rc = lib.ckv_plan_q8_store(arg, rid_at, kv_at, new_at, batch, num_rows, table, stride, reqs, capacity,
                               int(pad_invalid), _at(dev, plan), _at(dev, counts), _at(dev, status),
                               _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_plan_q8_store")
    return (plan if plan.shape[0] == capacity else plan[:capacity]), counts


def q8_store(cache: Q8Cache, k_rows: torch.Tensor, v_rows: Optional[torch.Tensor], plan: torch.Tensor,
             counts: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None,
             weights: Optional[torch.Tensor] = None) -> None:
    """Quantises rows ``[num_rows, n_kv_heads, head_dim]`` into the cache; ``v_rows`` is None for a latent cache.
    ``weights`` (as ``q8_weigh`` takes them): set to 0 where rows are stored, so that a slot that is used again does not keep
    its last owner's."""
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    n = k_rows.shape[0]
    _is(k_rows, "k_rows", k_rows.dtype, n, arg.n_kv_heads, arg.head_dim)
    if (v_rows is None) != (cache.v is None):
        raise ValueError("v_rows go with a cache that has v")
    if v_rows is not None:
        _is(v_rows, "v_rows", k_rows.dtype, n, arg.n_kv_heads, arg.head_dim)
    _store_plan(plan, 0)
    if counts is not None:
        _is(counts, "counts", torch.int32, 4)
    args = (arg, dtype_code(k_rows.dtype), _at(dev, k_rows), _at(dev, v_rows), n, _at(dev, plan), _at(dev, counts),
            plan.shape[0])
    if weights is None:
        rc = lib.ckv_q8_store(*args, _at(dev, status), _stream_of(dev, stream))
    else:
        _is(weights, "weights", _FP32, arg.num_blocks, arg.block_tokens)
        rc = lib.ckv_q8_store_reset(*args, _at(dev, weights), _at(dev, status), _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_store")


class Q8AttnPlan(NamedTuple):
    """What ``plan_q8_attn`` made (device memory) and the shape it holds for."""
    buffer: torch.Tensor
    n_heads: int
    ratio: int
    batch: int
    num_q: int


def plan_q8_attn(cache: Q8Cache, n_heads: int, ratio: int, rid: torch.Tensor, seq_lens: torch.Tensor,
                 extend_lens: torch.Tensor, kv_lens: torch.Tensor, num_q: int, buffer: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, stream=None) -> Q8AttnPlan:
    """Shares a step's attention out over the SMs.  Request b's ``extend_lens[b]`` queries are the last tokens of
    ``seq_lens[b]``; it has ``kv_lens[b]`` entries of ``ratio`` tokens each.  Serves every layer of the step."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return plan_q8_attn(cache, n_heads, ratio, rid, seq_lens, extend_lens, kv_lens, num_q, buffer, status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, seq_at, ext_at, kv_at) = _lens(dev, rid, seq_lens, extend_lens, kv_lens)
    if (n_heads | ratio | num_q) >> 32:
        _counts(n_heads=n_heads, ratio=ratio, num_q=num_q)
    if buffer is None:
        size = max(lib.ckv_q8_attn_plan_bytes(arg, n_heads, batch, num_q), 16)
        buffer = torch.empty(size, dtype=torch.uint8, device=rid.device)
        buffer_at = buffer.data_ptr()
    else:
        size, buffer_at = _bytes_of(buffer, "a plan buffer"), _at(dev, buffer)
    rc = lib.ckv_plan_q8_attn(arg, n_heads, ratio, rid_at, seq_at, ext_at, kv_at, batch, num_q, buffer_at, size,
                              _at(dev, status), _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_plan_q8_attn")
    return Q8AttnPlan(buffer, n_heads, ratio, batch, num_q)


def q8_attn_workspace(cache: Q8Cache, n_heads: int, batch: int, num_q: int) -> torch.Tensor:
    """Workspace for ``q8_attn`` calls of this shape; calls that may run at the same time need one each."""
    if (n_heads | batch | num_q) >> 32:
        _counts(n_heads=n_heads, batch=batch, num_q=num_q)
    n = load_library().ckv_q8_attn_workspace_bytes(_q8(cache)[0], n_heads, batch, num_q)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k.device)


def q8_attn(cache: Q8Cache, q: torch.Tensor, plan: Q8AttnPlan, block_table: torch.Tensor, scale: float,
            out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
            out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
            status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax attention of ``q`` (bf16 ``[num_q, n_heads, head_dim]``) over the cache: ``(out, lse)``, ``lse`` fp32
    ``[num_q, n_heads]``.  Queries that see nothing get zeros and -inf."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q8_attn(cache, q, plan, block_table, scale, out, lse, out_dtype, workspace, status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    buffer, n_heads, ratio, batch, num_q = plan
    _is(q, "q", torch.bfloat16, num_q, n_heads, arg.head_dim)
    where = q.device  # what is made here is contiguous and on it
    if out is None:
        out = torch.empty_like(q) if out_dtype is torch.bfloat16 else torch.empty(q.shape, dtype=out_dtype, device=where)
        out_at = out.data_ptr()
    else:
        _is(out, "out", out.dtype, num_q, n_heads, arg.head_dim)
        out_at = _at(dev, out)
    if lse is None:
        lse = torch.empty((num_q, n_heads), dtype=_FP32, device=where)
        lse_at = lse.data_ptr()
    else:
        _is(lse, "lse", _FP32, num_q, n_heads)
        lse_at = _at(dev, lse)
    if workspace is None:
        size = max(lib.ckv_q8_attn_workspace_bytes(arg, n_heads, batch, num_q), 16)
        workspace = torch.empty(size, dtype=torch.uint8, device=where)
        space_at = workspace.data_ptr()
    else:
        size, space_at = _bytes_of(workspace, "a workspace"), _at(dev, workspace)
    table, stride, reqs = _table(dev, block_table)
    rc = lib.ckv_q8_attn(arg, n_heads, ratio, scale, _at(dev, q), batch, num_q, table, stride, reqs,
                         _at(dev, buffer), buffer.numel(), dtype_code(out.dtype), out_at, lse_at, space_at, size,
                         _at(dev, status), _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_attn")
    return out, lse


def q8_weigh(cache: Q8Cache, q: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor, ratio: int,
             rid: torch.Tensor, seq_lens: torch.Tensor, extend_lens: torch.Tensor, kv_lens: torch.Tensor,
             block_table: torch.Tensor, scale: float, decay: float = 1.0, status: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """``weights[slot] = decay * weights[slot] +`` the softmax weight that the step's queries gave the entry, over all
    heads; ``weights`` fp32 ``[num_blocks, block_tokens]``, ``lse`` as ``q8_attn`` returned it."""
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, seq_at, ext_at, kv_at) = _lens(dev, rid, seq_lens, extend_lens, kv_lens)
    if q.dim() != 3:
        raise ValueError("q is bf16 [num_q, n_heads, head_dim]")
    if ratio >> 32:
        _counts(ratio=ratio)
    num_q, n_heads, _ = q.shape
    _is(q, "q", torch.bfloat16, num_q, n_heads, arg.head_dim)
    _is(lse, "lse", torch.float32, num_q, n_heads)
    _is(weights, "weights", torch.float32, arg.num_blocks, arg.block_tokens)
    table, stride, reqs = _table(dev, block_table)
    rc = lib.ckv_q8_weigh(arg, n_heads, ratio, scale, decay, _at(dev, q), _at(dev, lse), num_q, rid_at, seq_at, ext_at,
                          kv_at, batch, table, stride, reqs, _at(dev, weights), _at(dev, status),
                          _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_weigh")
    return weights


def q8_evict(cache: Q8Cache, weights: torch.Tensor, rid: torch.Tensor, kv_lens: torch.Tensor,
             block_table: torch.Tensor, dst_table: torch.Tensor, budget: int, sinks: int = 0, recent: int = 0,
             kept: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Keeps each request's ``budget`` entries of largest weight, its first ``sinks`` and newest ``recent`` among
    them, and moves them (with their weights) into the blocks of ``dst_table``, which must be no source's.  Returns
    ``(kept [batch, budget] int32 old positions, -1 past the end, new_lens [batch] int64)``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q8_evict(cache, weights, rid, kv_lens, block_table, dst_table, budget, sinks, recent, kept, new_lens,
                            status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, kv_at) = _lens(dev, rid, kv_lens)
    if (budget | sinks | recent) >> 32:
        _counts(budget=budget, sinks=sinks, recent=recent)
    _is(weights, "weights", torch.float32, arg.num_blocks, arg.block_tokens)
    src, stride, reqs = _table(dev, block_table)
    dst, dst_stride, dst_reqs = _table(dev, dst_table)
    if dst_reqs != reqs:
        raise ValueError("block_table and dst_table have a row for each request")
    if kept is None:
        kept = torch.empty((batch, budget), dtype=torch.int32, device=rid.device)
    else:
        _is(kept, "kept", torch.int32, batch, budget)
    if new_lens is None:
        new_lens = torch.empty(batch, dtype=torch.int64, device=rid.device)
    else:
        _is(new_lens, "new_lens", torch.int64, batch)
    rc = lib.ckv_q8_evict(arg, _at(dev, weights), rid_at, kv_at, batch, src, stride, dst, dst_stride, reqs, budget,
                          sinks, recent, _at(dev, kept), _at(dev, new_lens), _at(dev, status),
                          _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_evict")
    return kept, new_lens


def _rows_at(device: int, t: torch.Tensor, what: str, dtype: torch.dtype, *shape: int) -> Tuple[int, int]:
    """Address and row stride of rows ``[n, heads, dim]`` whose rows are contiguous but may lie apart."""
    _is(t, what, dtype, *shape)
    n, heads, dim = shape
    s0, s1, s2 = t.stride()
    if t.get_device() != device:
        raise ValueError("libckv takes CUDA tensors of one device only")
    if (s2 != 1 and dim > 1) or (s1 != dim and heads > 1):
        raise ValueError(f"{what}: a row's heads and channels must be contiguous")
    return t.data_ptr(), s0 if n > 1 else heads * dim


def q8_rope_store(cache: Q8Cache, k_rows: torch.Tensor, v_rows: Optional[torch.Tensor], plan: torch.Tensor,
                  positions: Optional[torch.Tensor], freqs: Optional[torch.Tensor],
                  counts: Optional[torch.Tensor] = None, rope_begin: int = 0, halves: bool = False,
                  norm_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                  weights: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """``q8_store`` with the keys' norm and rotation on the way.  ``k_rows`` and ``v_rows`` ``[num_rows, n_kv_heads,
    head_dim]`` may be slices of wider rows.  Channels from ``rope_begin`` on, two for each entry of a row of ``freqs``
    (fp32 ``[max_pos, rope_dim/2, 2]``: cos, sin), turn by row ``positions[row]`` (int64) of it, as pairs of neighbours or, with
    ``halves``, of channels ``rope_dim/2`` apart; no ``freqs``: none does.  ``norm_weight`` (fp32 ``[head_dim]``): RMSNorm before that."""
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    n, dt = k_rows.shape[0], k_rows.dtype
    k_at, k_stride = _rows_at(dev, k_rows, "k_rows", dt, n, arg.n_kv_heads, arg.head_dim)
    if (v_rows is None) != (cache.v is None):
        raise ValueError("v_rows go with a cache that has v")
    v_at, v_stride = None, 0
    if v_rows is not None:
        v_at, v_stride = _rows_at(dev, v_rows, "v_rows", dt, n, arg.n_kv_heads, arg.head_dim)
    _store_plan(plan, 0)
    if counts is not None:
        _is(counts, "counts", torch.int32, 4)
    max_pos = rope_dim = 0
    if freqs is not None:
        if positions is None:
            raise ValueError("freqs need positions")
        _is(positions, "positions", torch.int64, n)
        if freqs.dtype is not _FP32 or freqs.dim() != 3 or freqs.shape[2] != 2:
            raise ValueError("freqs is fp32 [max_pos, rope_dim/2, 2]")
        max_pos, rope_dim = freqs.shape[0], 2 * freqs.shape[1]
    if (rope_begin | max_pos) >> 32:
        _counts(rope_begin=rope_begin, max_pos=max_pos)
    if norm_weight is not None:
        _is(norm_weight, "norm_weight", _FP32, arg.head_dim)
    if weights is not None:
        _is(weights, "weights", _FP32, arg.num_blocks, arg.block_tokens)
    rc = lib.ckv_q8_rope_store(arg, dtype_code(dt), k_at, k_stride, v_at, v_stride, n, _at(dev, positions),
                               _at(dev, norm_weight), eps, _at(dev, freqs), max_pos, rope_begin, rope_dim, int(halves),
                               _at(dev, plan), _at(dev, counts), plan.shape[0], _at(dev, weights), _at(dev, status),
                               _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_rope_store")


def new_q8_bounds(cache: Q8Cache) -> torch.Tensor:
    """Storage for a cache's bounds: float8_e4m3fn ``[num_blocks, n_kv_heads, 2, head_dim]`` (zeros)."""
    blocks, heads, _, dim = cache.k.shape
    return torch.zeros(blocks, heads, 2, dim, dtype=torch.uint8, device=cache.k.device).view(_E4M3)


def q8_bounds(cache: Q8Cache, bounds: torch.Tensor, rid: torch.Tensor, kv_lens: torch.Tensor, new_lens: torch.Tensor,
              block_table: torch.Tensor, status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Renews the bounds (the largest and smallest k code of each channel) of the blocks that each request's last
    ``new_lens`` of ``kv_lens`` entries lie in."""
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, kv_at, new_at) = _lens(dev, rid, kv_lens, new_lens)
    _is(bounds, "bounds", _E4M3, arg.num_blocks, arg.n_kv_heads, 2, arg.head_dim)
    table, stride, reqs = _table(dev, block_table)
    rc = lib.ckv_q8_bounds(arg, _at(dev, bounds), rid_at, kv_at, new_at, batch, table, stride, reqs, _at(dev, status),
                           _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_bounds")
    return bounds


def q8_block_scores(cache: Q8Cache, bounds: torch.Tensor, q: torch.Tensor, ratio: int, rid: torch.Tensor,
                    seq_lens: torch.Tensor, extend_lens: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                    scale: float, width: Optional[int] = None, scores: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """What a score of each query (bf16 ``[num_q, n_heads, head_dim]``) with an entry of each block is at most, over the
    heads of a kv head: fp32 ``[num_q, n_kv_heads, width]`` (by default the table's), -inf for blocks that it does not see."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q8_block_scores(cache, bounds, q, ratio, rid, seq_lens, extend_lens, kv_lens, block_table, scale, width,
                                   scores, status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, seq_at, ext_at, kv_at) = _lens(dev, rid, seq_lens, extend_lens, kv_lens)
    if q.dim() != 3:
        raise ValueError("q is bf16 [num_q, n_heads, head_dim]")
    num_q, n_heads, _ = q.shape
    _is(q, "q", torch.bfloat16, num_q, n_heads, arg.head_dim)
    _is(bounds, "bounds", _E4M3, arg.num_blocks, arg.n_kv_heads, 2, arg.head_dim)
    table, stride, reqs = _table(dev, block_table)
    if width is None:
        width = stride if scores is None else scores.shape[-1]
    if (ratio | width) >> 32:
        _counts(ratio=ratio, width=width)
    if scores is None:
        scores = torch.empty((num_q, arg.n_kv_heads, width), dtype=_FP32, device=q.device)
        scores_at = scores.data_ptr()
    else:
        _is(scores, "scores", _FP32, num_q, arg.n_kv_heads, width)
        scores_at = _at(dev, scores)
    rc = lib.ckv_q8_block_scores(arg, _at(dev, bounds), n_heads, ratio, scale, _at(dev, q), num_q, rid_at, seq_at, ext_at,
                                 kv_at, batch, table, stride, reqs, width, scores_at, _at(dev, status),
                                 _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_block_scores")
    return scores


def q8_block_select(scores: torch.Tensor, block_tokens: int, ratio: int, seq_lens: torch.Tensor,
                    extend_lens: torch.Tensor, kv_lens: torch.Tensor, budget: int, sinks: int = 0, recent: int = 0,
                    blocks: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The blocks that each query reads for each kv head, int32 ``[num_q, n_kv_heads, budget]``, ascending, -1 behind the
    last: the first ``sinks`` and the last ``recent`` that it sees, and of the others those of largest score (fp32
    ``[num_q, n_kv_heads, width]``), the lower of equal ones."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q8_block_select(scores, block_tokens, ratio, seq_lens, extend_lens, kv_lens, budget, sinks, recent,
                                   blocks, status)
    lib = _lib or load_library()
    dev = scores.get_device()
    if scores.dtype is not _FP32 or scores.dim() != 3:
        raise ValueError("scores is fp32 [num_q, n_kv_heads, width]")
    if dev < 0:
        raise ValueError("libckv takes CUDA tensors only")
    if dev != _current_device():
        raise ValueError("the scores are not on the current device")
    num_q, heads, width = scores.shape
    batch, (seq_at, ext_at, kv_at) = _lens(dev, seq_lens, extend_lens, kv_lens)
    if (num_q | width | block_tokens | ratio | budget | sinks | recent) >> 32:
        _counts(num_q=num_q, width=width, block_tokens=block_tokens, ratio=ratio, budget=budget, sinks=sinks, recent=recent)
    if blocks is None:
        blocks = torch.empty((num_q, heads, budget), dtype=torch.int32, device=scores.device)
        blocks_at = blocks.data_ptr()
    else:
        _is(blocks, "blocks", torch.int32, num_q, heads, budget)
        blocks_at = _at(dev, blocks)
    rc = lib.ckv_q8_block_select(_at(dev, scores), heads, width, block_tokens, ratio, num_q, seq_at, ext_at, kv_at, batch,
                                 budget, sinks, recent, blocks_at, _at(dev, status), _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_block_select")
    return blocks


def q8_attn_blocks_workspace(cache: Q8Cache, n_heads: int, num_q: int, budget: int) -> torch.Tensor:
    """Workspace for ``q8_attn_blocks`` calls of this shape; calls that may run at the same time need one each."""
    if (n_heads | num_q | budget) >> 32:
        _counts(n_heads=n_heads, num_q=num_q, budget=budget)
    n = load_library().ckv_q8_attn_blocks_workspace_bytes(_q8(cache)[0], n_heads, num_q, budget)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=cache.k.device)


def q8_attn_blocks(cache: Q8Cache, q: torch.Tensor, blocks: torch.Tensor, ratio: int, rid: torch.Tensor,
                   seq_lens: torch.Tensor, extend_lens: torch.Tensor, kv_lens: torch.Tensor, block_table: torch.Tensor,
                   scale: float, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   out_dtype: torch.dtype = torch.bfloat16, workspace: Optional[torch.Tensor] = None,
                   status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``q8_attn`` of each query over the entries that it sees in its listed blocks (int32 ``[num_q, n_kv_heads, budget]``,
    ascending, negative ones passed over): ``(out, lse)``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return q8_attn_blocks(cache, q, blocks, ratio, rid, seq_lens, extend_lens, kv_lens, block_table, scale, out,
                                  lse, out_dtype, workspace, status)
    lib = _lib or load_library()
    arg, dev = _q8(cache)
    batch, (rid_at, seq_at, ext_at, kv_at) = _lens(dev, rid, seq_lens, extend_lens, kv_lens)
    if q.dim() != 3 or blocks.dim() != 3:
        raise ValueError("q is bf16 [num_q, n_heads, head_dim], blocks int32 [num_q, n_kv_heads, budget]")
    num_q, n_heads, _ = q.shape
    budget = blocks.shape[2]
    _is(q, "q", torch.bfloat16, num_q, n_heads, arg.head_dim)
    _is(blocks, "blocks", torch.int32, num_q, arg.n_kv_heads, budget)
    if (ratio | budget) >> 32:
        _counts(ratio=ratio, budget=budget)
    where = q.device
    if out is None:
        out = torch.empty_like(q) if out_dtype is torch.bfloat16 else torch.empty(q.shape, dtype=out_dtype, device=where)
        out_at = out.data_ptr()
    else:
        _is(out, "out", out.dtype, num_q, n_heads, arg.head_dim)
        out_at = _at(dev, out)
    if lse is None:
        lse = torch.empty((num_q, n_heads), dtype=_FP32, device=where)
        lse_at = lse.data_ptr()
    else:
        _is(lse, "lse", _FP32, num_q, n_heads)
        lse_at = _at(dev, lse)
    if workspace is None:
        size = max(lib.ckv_q8_attn_blocks_workspace_bytes(arg, n_heads, num_q, budget), 16)
        workspace = torch.empty(size, dtype=torch.uint8, device=where)
        space_at = workspace.data_ptr()
    else:
        size, space_at = _bytes_of(workspace, "a workspace"), _at(dev, workspace)
    table, stride, reqs = _table(dev, block_table)
    rc = lib.ckv_q8_attn_blocks(arg, n_heads, ratio, scale, _at(dev, q), num_q, _at(dev, blocks), budget, rid_at, seq_at,
                                ext_at, kv_at, batch, table, stride, reqs, dtype_code(out.dtype), out_at, lse_at,
                                space_at, size, _at(dev, status), _stream_of(dev, stream))
    if rc:
        _q8_error(rc, "ckv_q8_attn_blocks")
    return out, lse


# ------------------------------------------------------------------------------ convenience
def prefill_step(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                 rid: torch.Tensor, seq_lens: torch.Tensor, extend_lens: torch.Tensor, out_layout: int = OUT_TOKEN,
                 out_dtype: torch.dtype = torch.float32, status: Optional[torch.Tensor] = None, stream=None):
    """plan_prefill -> pool -> write.  Returns ``(out, plan_c, plan_w, counts)`` (all on the device)."""
    plan_c, plan_w, counts = plan_prefill(ratio, rid, seq_lens, extend_lens, kv_score.shape[0], status=status,
                                          stream=stream)
    out = compress_prefill(ratio, head_dim, state, kv_score, ape, plan_c, plan_w, counts, out_layout, out_dtype,
                           status=status, stream=stream, hints=(rid, seq_lens, extend_lens))
    return out, plan_c, plan_w, counts


def decode_step(ratio: int, head_dim: int, state: torch.Tensor, kv_score: torch.Tensor, ape: torch.Tensor,
                rid: torch.Tensor, seq_lens: torch.Tensor, out_dtype: torch.dtype = torch.float32,
                status: Optional[torch.Tensor] = None, stream=None):
    """plan_decode (with the boundary-row list) -> decode.  Returns ``(out, plan_d)``."""
    order = new_decode_order(rid.numel(), rid.device)
    plan_d = plan_decode(ratio, rid, seq_lens, status=status, stream=stream, order=order)
    out = compress_decode(ratio, head_dim, state, kv_score, ape, plan_d, out_dtype, status=status, stream=stream,
                          order=order, rid_hint=rid, seq_lens_hint=seq_lens)
    return out, plan_d
