"""Python binding of libdsa (include/dsa.h): index-selected sparse attention on B200.

Argument marshalling only (what runs on every call is native: csrc/binding.cpp).
Every step of the path runs in libdsa's CUDA
kernels; torch provides device memory and the current stream.  There is no
fallback: if libdsa.so is missing and cannot be built, importing this package
raises.

Functions carry the C names (``dsa_index_scores`` ...).  Outputs not passed in
are allocated with torch on the inputs' device; workspaces are allocated
zeroed and cached per (device, stream, op), unless one is passed in.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

from . import build as _build
from .rope import RopeTable

# ---------------------------------------------------------------------------
# Library loading
# ---------------------------------------------------------------------------

if _build.is_stale():
    _build.build_library()
_lib = ctypes.CDLL(_build.LIB)
LIB_PATH = _build.LIB
from . import _binding  # noqa: E402  (linked to the library just loaded)

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, DSA_ERR_BAD_INDEX, \
    DSA_ERR_TIMEOUT = range(7)
DSA_KI_BF16, DSA_KI_FP8_E4M3, DSA_KI_MXFP8, DSA_KI_MXFP4 = range(4)
DSA_KV_BF16, DSA_KV_FP8_E4M3 = 0, 1
DSA_OUT_BF16, DSA_OUT_F32 = 0, 1
DSA_NOALLOC_SCRATCH_BYTES = 32 << 20
DSA_OP_QUANTIZE_INDEX_QUERY, DSA_OP_INDEX_SCORES, DSA_OP_TOPK, DSA_OP_SPARSE_MLA, DSA_OP_INDEX_TOPK_ATTN, \
    DSA_OP_INDEX_TOPK_ATTN_FUSED, DSA_OP_APPEND_INDEX_KEYS, DSA_OP_ATTN_MASS, DSA_OP_EVICT_SELECT, \
    DSA_OP_EVICT_COMPACT = range(10)
DSA_SELECT_IN_INDEXER = 1
DSA_MASS_FRACTION_BITS, DSA_MAX_POOLS = 40, 8
DSA_ROPE_BF16, DSA_ROPE_F16, DSA_ROPE_F32 = range(3)
DSA_ROPE_HALF, DSA_ROPE_TRANSPOSE, DSA_ROPE_POS64, DSA_ROPE_MAX_DIM = 1, 2, 4, 1024

# Names the C header declares (checked against include/dsa.h by the tests).
EXPORTS = ("dsa_workspace_size",
           "dsa_quantize_index_query", "dsa_quantize_index_query_mx", "dsa_quantize_index_query_mx4",
           "dsa_append_index_keys_mx4", "dsa_dequantize_mx4",
           "dsa_index_scores", "dsa_topk",
           "dsa_sparse_mla_fwd", "dsa_sparse_mla_fwd_ex", "dsa_sparse_mla_fwd_noalloc",
           "dsa_index_topk_attn", "dsa_index_topk_attn_ex",
           "dsa_attn_mass", "dsa_evict_select", "dsa_evict_compact",
           "dsa_rope",
           "dsa_check_error", "dsa_check_error_noalloc", "dsa_set_wait_limit_ns",
           "dsa_launches_in_last_call", "dsa_launch_timing", "dsa_last_launch_times", "dsa_status_string")


class DsaSeqsC(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_tokens", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("num_phys_pages", ctypes.c_int32), ("max_ctx", ctypes.c_int32),
                ("q_seq_start", ctypes.c_void_p), ("ctx_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p)]


class DsaPoolC(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("row_bytes", ctypes.c_int32)]


_P = ctypes.c_void_p
_I32, _I64, _SZ, _F = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
_SEQ = ctypes.POINTER(DsaSeqsC)
_sig = {
    "dsa_workspace_size": (_SZ, [ctypes.c_int, _SEQ, ctypes.c_int, ctypes.c_int]),
    "dsa_quantize_index_query": (ctypes.c_int, [_P, _P, ctypes.c_int, _P, _P, _P]),
    "dsa_quantize_index_query_mx": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P]),
    "dsa_quantize_index_query_mx4": (ctypes.c_int, [_P, ctypes.c_int, _P, _P, _P]),
    "dsa_append_index_keys_mx4": (ctypes.c_int, [_SEQ, _P, _P, _P, _P, _SZ, _P]),
    "dsa_dequantize_mx4": (ctypes.c_int, [_P, _P, _I64, _P, _P]),
    "dsa_index_scores": (ctypes.c_int, [_SEQ, _P, _P, _P, _P, ctypes.c_int, _P, _I64, _P, _SZ, _P]),
    "dsa_topk": (ctypes.c_int, [_P, _I64, ctypes.c_int, _P, ctypes.c_int, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_fwd": (ctypes.c_int, [_SEQ, _P, _P, _P, ctypes.c_int, ctypes.c_int, _F, _P, ctypes.c_int, _P, _P,
                                          _SZ, _P]),
    "dsa_sparse_mla_fwd_ex": (ctypes.c_int, [_SEQ, _P, _P, _P, ctypes.c_int, _P, ctypes.c_int, ctypes.c_int, _F, _P,
                                             ctypes.c_int, _P, _P, _SZ, _P]),
    "dsa_sparse_mla_fwd_noalloc": (ctypes.c_int, [_SEQ, _P, _P, _P, ctypes.c_int, ctypes.c_int, _F, _P, ctypes.c_int,
                                                  _P, _P]),
    "dsa_index_topk_attn": (ctypes.c_int, [_SEQ, _P, _P, _P, _P, ctypes.c_int, _P, _P, ctypes.c_int, ctypes.c_int,
                                           _F, _P, ctypes.c_int, _P, _P, _P, _SZ, _P]),
    "dsa_index_topk_attn_ex": (ctypes.c_int, [_SEQ, _P, _P, _P, _P, ctypes.c_int, _P, _P, _P, ctypes.c_int,
                                              ctypes.c_int, ctypes.c_int, _F, _P, ctypes.c_int, _P, _P, _P, _SZ,
                                              ctypes.c_uint, _P, _P]),
    "dsa_attn_mass": (ctypes.c_int, [_SEQ, _P, _P, _P, ctypes.c_int, _P, ctypes.c_int, ctypes.c_int, _F, _P, _P, _I64,
                                     _P, _SZ, _P]),
    "dsa_evict_select": (ctypes.c_int, [_P, ctypes.c_int, ctypes.c_int, _P, _I64, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, _P, _P, _P, _SZ, _P]),
    "dsa_evict_compact": (ctypes.c_int, [_SEQ, _P, _P, ctypes.c_int, _P, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(DsaPoolC), ctypes.c_int, _P, _I64, _P, _I64, _P, _SZ, _P]),
    "dsa_rope": (ctypes.c_int, [_P, _P, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _I64, _I64, _I64, _I64,
                                _P, _P, ctypes.c_int, ctypes.c_int, _F, ctypes.c_uint, _P]),
    "dsa_check_error": (ctypes.c_int, [_P, _P]),
    "dsa_check_error_noalloc": (ctypes.c_int, [_P]),
    "dsa_set_wait_limit_ns": (ctypes.c_int, [ctypes.c_uint64]),
    "dsa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "dsa_launches_in_last_call": (ctypes.c_int, []),
    "dsa_launch_timing": (ctypes.c_int, [ctypes.c_int]),
    "dsa_last_launch_times": (ctypes.c_int, [ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_char_p),
                                             ctypes.c_int]),
}
for _name, (_res, _args) in _sig.items():
    _fn = getattr(_lib, _name)
    _fn.restype, _fn.argtypes = _res, _args


class DsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_lib.dsa_status_string(status).decode()}")


def _check(status: int, where: str):
    if status != DSA_OK:
        raise DsaError(status, where)


def status_string(status: int) -> str:
    return _lib.dsa_status_string(status).decode()


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(device: torch.device):
    """The device's current stream, as the integer that ctypes passes on."""
    index = device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


# Refuses, before any C call, a tensor the kernels would misread: need(t, name,
# dtypes, shape, device, min_rows=0) wants a contiguous tensor on `device` with
# one of `dtypes`, a shape matching `shape` (None matches any size) and at least
# `min_rows` rows.  The kernels take bare pointers, so a wrong dtype, a strided
# view or a short pool would otherwise be read out of bounds.
_need = _binding.need
_need_seqs = _binding.need_seqs
_cuda_device = _binding.cuda_device
_empty = _binding.empty


def _refuse(t, name, dtypes, shape, device, min_rows):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")
    if t.dim() != len(shape) or any(w is not None and w != g for g, w in zip(t.shape, shape)):
        want = "[" + ", ".join("*" if w is None else str(w) for w in shape) + "]"
        raise ValueError(f"{name}: shape {list(t.shape)}, expected {want}")
    if t.shape[0] < min_rows:
        raise ValueError(f"{name}: {t.shape[0]} rows, the page pool needs at least {min_rows}")
    raise ValueError(f"{name}: must be contiguous")


_I32T, _F32T, _BF16T = (torch.int32,), (torch.float32,), (torch.bfloat16,)
_FP8T, _U8T = (torch.uint8, torch.float8_e4m3fn), (torch.uint8,)


def _refuse_seqs(seqs, dev: torch.device):
    _need(seqs.q_seq_start, "seqs.q_seq_start", _I32T, (seqs.batch + 1,), dev)
    _need(seqs.ctx_len, "seqs.ctx_len", _I32T, (None,), dev)
    _need(seqs.page_table, "seqs.page_table", _I32T, (seqs.batch, None), dev)


_binding.refusals(_refuse, _refuse_seqs)


def _need_ws(ws, dev: torch.device):
    _need(ws, "ws", (torch.uint8,), (None,), dev)


def _space(ws, nbytes: int, dev: torch.device, key) -> torch.Tensor:
    """The caller's workspace, checked, or the cached one."""
    if ws is None:
        return workspace(nbytes, dev, key)
    _need(ws, "ws", _U8T, (None,), dev)
    return ws


def _need_index_inputs(seqs: "Seqs", qI, w, kI, kI_scale, check_seqs: bool = True) -> torch.device:
    dev = _cuda_device(qI, "qI")
    T, rows = seqs.num_q_tokens, seqs.num_phys_pages * 64
    if check_seqs:
        _need_seqs(seqs, dev)
    _need(qI, "qI", _BF16T, (T, 64, 128), dev)
    _need(w, "w", _F32T, (T, 64), dev)
    if _is_mx4(kI, kI_scale):
        _need(kI, "kI", _U8T, (None, 64), dev, rows)
    else:
        _need(kI, "kI", _FP8T if kI_scale is not None else _BF16T, (None, 128), dev, rows)
    if _is_mx(kI_scale):
        _need(kI_scale, "kI_scale", _U8T, (None, 4), dev, rows)
    elif kI_scale is not None:
        _need(kI_scale, "kI_scale", _F32T, (None,), dev, rows)
    return dev


def _is_mx(kI_scale) -> bool:
    """An MXFP8 or MXFP4 index cache carries E8M0 group scales (uint8 [R, 4])."""
    return kI_scale is not None and kI_scale.dtype == torch.uint8


def _is_mx4(kI, kI_scale) -> bool:
    """Rows of 64 bytes with group scales hold packed 4-bit codes."""
    return _is_mx(kI_scale) and isinstance(kI, torch.Tensor) and kI.dim() == 2 and kI.shape[1] == 64


def _ki_dtype(kI_scale, kI=None) -> int:
    if kI_scale is None:
        return DSA_KI_BF16
    if _is_mx4(kI, kI_scale):
        return DSA_KI_MXFP4
    return DSA_KI_MXFP8 if _is_mx(kI_scale) else DSA_KI_FP8_E4M3


def _need_attn_inputs(seqs: "Seqs", q, kv, out, lse, kv_scale=None) -> torch.device:
    dev = _cuda_device(q, "q")
    _need_seqs(seqs, dev)
    _need(q, "q", _BF16T, (seqs.num_q_tokens, None, 576), dev)
    T, H = q.shape[0], q.shape[1]
    rows = seqs.num_phys_pages * 64
    if kv_scale is None:
        _need(kv, "kv", _BF16T, (None, 576), dev, rows)
    else:  # FP8 latent cache: E4M3 codes and per-row tile-scale bytes
        _need(kv, "kv", _FP8T, (None, 576), dev, rows)
        _need(kv_scale, "kv_scale", (torch.uint8,), (None, 8), dev, rows)
    _need(out, "out", (torch.bfloat16, torch.float32), (T, H, 512), dev)
    if lse is not None:
        _need(lse, "lse", _F32T, (T, H), dev)
    return dev


# ---------------------------------------------------------------------------
# Batch geometry
# ---------------------------------------------------------------------------


@dataclass
class Seqs:
    """Batch geometry on the device (see dsa_seqs_t in include/dsa.h)."""
    q_seq_start: torch.Tensor   # int32 [B+1]
    ctx_len: torch.Tensor       # int32 [B]
    page_table: torch.Tensor    # int32 [B, max_pages]
    num_phys_pages: int
    max_ctx: int
    num_q_tokens: int

    @staticmethod
    def from_host(q_seq_start, ctx_len, page_table, num_phys_pages: int, device="cuda") -> "Seqs":
        qs = torch.as_tensor(q_seq_start, dtype=torch.int32)
        cl = torch.as_tensor(ctx_len, dtype=torch.int32)
        pt = torch.as_tensor(page_table, dtype=torch.int32)
        return Seqs(qs.to(device), cl.to(device), pt.contiguous().to(device), int(num_phys_pages),
                    int(cl.max()), int(qs[-1]))

    @property
    def batch(self) -> int:
        return self.ctx_len.shape[0]

    def c(self) -> DsaSeqsC:
        B, max_pages = self.page_table.shape
        return DsaSeqsC(B, self.num_q_tokens, 64, max_pages, self.num_phys_pages, self.max_ctx,
                        self.q_seq_start.data_ptr(), self.ctx_len.data_ptr(), self.page_table.data_ptr())


def dsa_workspace_size(op: int, seqs: Seqs | None = None, K: int = 1, H: int = 16, *, rows: int = 0,
                       ld: int = 0) -> int:
    c = seqs.c() if seqs is not None else DsaSeqsC(1, rows, 64, 1, 1, ld, None, None, None)
    return int(_lib.dsa_workspace_size(op, ctypes.byref(c), K, H))


_ws_cache: dict = {}            # (device, stream, key) -> buffer
_ws_newest: dict = {}           # (device, key) -> the buffer made last, for whatever stream
_ws_captured: dict = {}


def workspace(nbytes: int, device, key=None) -> torch.Tensor:
    """A zeroed device workspace of at least nbytes, cached per (device, key) for
    the device's current stream.

    The calls' keys: "index_scores", "topk", "sparse_mla", "index_topk_attn",
    "append_index_keys", "attn_mass", "evict_select" and "evict_compact".
    workspace(0, device, key) is the buffer whose error flag dsa_check_error
    reads: that of the current stream, or the newest if it has none.

    Every call that is not given `ws` uses this buffer, so that calls on two
    streams do not share one (the library requires that of concurrent calls:
    scratch and sticky error flag are in it).  Calls of several host threads on
    one stream share one in turn: the binding launches each call as a whole.

    During stream capture another stream's buffer serves where the capturing one has
    none that is large enough, and one that has to be made belongs to the graph
    alone (its zeroing is part of the graph and has not run), so it is not
    cached.  A graph that is replayed beside other calls or graphs, or whose error
    flag is to be read, is captured with a workspace of its own.  A cached buffer
    that a capture uses stays alive when a larger one replaces it: the graph still
    writes to it."""
    if not isinstance(device, torch.device):
        device = torch.device(device)
    capturing = False
    if device.type == "cuda":
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        stream = _binding.stream_of(device)
        if stream is None:
            capturing, stream = True, _stream(device)
        k = (device.index, stream, key)
    else:
        k = (device, None, key)
    ws = _ws_cache.get(k)
    if ws is None and nbytes == 0:
        ws = _ws_newest.get((device, key))
    if capturing and (ws is None or ws.numel() < nbytes):
        ws = max((b for (d, _, name), b in list(_ws_cache.items()) if d == device.index and name == key),
                 key=lambda b: b.numel(), default=None)
    if ws is None or ws.numel() < nbytes:
        small, ws = ws, torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device)
        if not capturing:
            if small is not None:
                ws[:4].copy_(small[:4])     # an error that was not read yet
            _ws_cache[k] = _ws_newest[device, key] = ws
    elif capturing:
        _ws_captured[ws.data_ptr()] = ws
    return ws


# ---------------------------------------------------------------------------
# Entry points
# ---------------------------------------------------------------------------


def dsa_quantize_index_query(qI: torch.Tensor, w: torch.Tensor, codes=None, w_scaled=None):
    dev = _cuda_device(qI, "qI")
    T = qI.shape[0]
    codes = codes if codes is not None else torch.empty((T, 64, 128), dtype=torch.uint8, device=qI.device)
    w_scaled = w_scaled if w_scaled is not None else torch.empty((T, 64), dtype=torch.float32, device=qI.device)
    _need(qI, "qI", _BF16T, (T, 64, 128), dev)
    _need(w, "w", _F32T, (T, 64), dev)
    _need(codes, "codes", _FP8T, (T, 64, 128), dev)
    _need(w_scaled, "w_scaled", _F32T, (T, 64), dev)
    _check(_binding.dsa_quantize_index_query(dev, qI, w, T, codes, w_scaled), "dsa_quantize_index_query")
    return codes, w_scaled


def dsa_quantize_index_query_mx(qI: torch.Tensor, codes=None, scales=None):
    dev = _cuda_device(qI, "qI")
    T = qI.shape[0]
    codes = codes if codes is not None else torch.empty((T, 64, 128), dtype=torch.uint8, device=qI.device)
    scales = scales if scales is not None else torch.empty((T, 64, 4), dtype=torch.uint8, device=qI.device)
    _need(qI, "qI", _BF16T, (T, 64, 128), dev)
    _need(codes, "codes", _FP8T, (T, 64, 128), dev)
    _need(scales, "scales", (torch.uint8,), (T, 64, 4), dev)
    _check(_binding.dsa_quantize_index_query_mx(dev, qI, T, codes, scales), "dsa_quantize_index_query_mx")
    return codes, scales


def dsa_quantize_index_query_mx4(qI: torch.Tensor, codes=None, scales=None):
    """MXFP4: qI [T, 64, 128] bf16 to packed E2M1 codes uint8 [T, 64, 64] and
    E8M0 scales uint8 [T, 64, 4]."""
    dev = _cuda_device(qI, "qI")
    _need(qI, "qI", _BF16T, (qI.shape[0], 64, 128), dev)
    T = qI.shape[0]
    if codes is None:
        codes = _empty((T, 64, 64), torch.uint8, dev)
    else:
        _need(codes, "codes", _U8T, (T, 64, 64), dev)
    if scales is None:
        scales = _empty((T, 64, 4), torch.uint8, dev)
    else:
        _need(scales, "scales", _U8T, (T, 64, 4), dev)
    _check(_binding.dsa_quantize_index_query_mx4(dev, qI, T, codes, scales), "dsa_quantize_index_query_mx4")
    return codes, scales


def dsa_append_index_keys_mx4(seqs: Seqs, k: torch.Tensor, kI: torch.Tensor, kI_scale: torch.Tensor, ws=None):
    """Quantizes the new tokens' index keys k [T, 128] bf16 into the rows of
    their positions of an MXFP4 cache: kI uint8 [R, 64], kI_scale uint8 [R, 4]."""
    dev = _cuda_device(k, "k")
    _need_seqs(seqs, dev)
    _need(k, "k", _BF16T, (seqs.num_q_tokens, 128), dev)
    rows = seqs.num_phys_pages * 64
    _need(kI, "kI", _U8T, (None, 64), dev, rows)
    _need(kI_scale, "kI_scale", _U8T, (None, 4), dev, rows)
    ws = _space(ws, 256, dev, "append_index_keys")
    _check(_binding.dsa_append_index_keys_mx4(dev, seqs, k, kI, kI_scale, ws, ws.numel()),
           "dsa_append_index_keys_mx4")


def dsa_dequantize_mx4(codes: torch.Tensor, scales: torch.Tensor, out=None) -> torch.Tensor:
    """The bf16 values [..., 128] that MXFP4 codes [..., 64] with scales [..., 4]
    stand for (exact)."""
    dev = _cuda_device(codes, "codes")
    if codes.dim() < 1 or codes.shape[-1] != 64:
        raise ValueError(f"codes: shape {list(codes.shape)}, expected [..., 64]")
    lead = codes.shape[:-1]
    _need(codes, "codes", _U8T, codes.shape, dev)
    _need(scales, "scales", _U8T, (*lead, 4), dev)
    if out is None:
        out = _empty((*lead, 128), torch.bfloat16, dev)
    else:
        _need(out, "out", _BF16T, (*lead, 128), dev)
    _check(_binding.dsa_dequantize_mx4(dev, codes, scales, codes.numel() // 64, out), "dsa_dequantize_mx4")
    return out


def dsa_index_scores(seqs: Seqs, qI, w, kI, kI_scale=None, scores=None, ld=None, ws=None):
    """Scores into `scores` [T, ld] fp32 (allocated zeroed when None).  The index
    cache's format follows kI and kI_scale: bf16 [R, 128] without scales; E4M3
    [R, 128] with fp32 [R]; MXFP8 [R, 128] or MXFP4 [R, 64] with uint8 [R, 4].  When
    `scores` is given, ld defaults to its row stride and must equal it."""
    dev = _need_index_inputs(seqs, qI, w, kI, kI_scale)
    T = seqs.num_q_tokens
    if scores is None:
        ld = ld or (seqs.max_ctx + 3) // 4 * 4
        scores = torch.zeros((T, ld), dtype=torch.float32, device=qI.device)
    else:
        _need(scores, "scores", _F32T, (T, None), dev)
        if ld is not None and ld != scores.stride(0):
            raise ValueError(f"ld={ld} differs from the row stride {scores.stride(0)} of scores")
        ld = scores.stride(0)
    ki_dtype = _ki_dtype(kI_scale, kI)
    ws = _space(ws, _binding.workspace_size(DSA_OP_INDEX_SCORES, seqs, 1, 16), dev, "index_scores")
    _check(_binding.dsa_index_scores(dev, seqs, qI, w, kI, kI_scale, ki_dtype, scores, ld, ws, ws.numel()),
           "dsa_index_scores")
    return scores


def dsa_topk(scores: torch.Tensor, row_len: torch.Tensor, K: int, idx=None, ws=None):
    """Top-K of each fp32 row of `scores` [T, ld] (contiguous) over its first
    row_len[t] entries, into idx [T, K] int32."""
    dev = _cuda_device(scores, "scores")
    _need(scores, "scores", _F32T, (None, None), dev)
    T, ld = scores.shape
    idx = idx if idx is not None else torch.empty((T, K), dtype=torch.int32, device=scores.device)
    _need(row_len, "row_len", _I32T, (T,), dev)
    _need(idx, "idx", _I32T, (T, K), dev)
    c = DsaSeqsC(1, T, 64, 1, 1, ld, None, None, None)
    need = _lib.dsa_workspace_size(DSA_OP_TOPK, ctypes.byref(c), K, 16)
    ws = ws if ws is not None else workspace(need, scores.device, "topk")
    _need_ws(ws, dev)
    _check(_binding.dsa_topk(dev, scores, ld, T, row_len, K, idx, ws, ws.numel()), "dsa_topk")
    return idx


def _out_dtype(out: torch.Tensor) -> int:
    if out.dtype == torch.bfloat16:
        return DSA_OUT_BF16
    if out.dtype == torch.float32:
        return DSA_OUT_F32
    raise TypeError("out must be bfloat16 or float32")


def dsa_sparse_mla_fwd(seqs: Seqs, q, kv, idx, scale: float, out=None, lse=None, want_lse=True, ws=None,
                       out_dtype=torch.bfloat16, kv_scale=None):
    """Sparse MLA over the selected rows.  kv_scale (uint8 [R, 8]) marks an FP8
    latent cache: kv then holds E4M3 codes [R, 576] (dsa_sparse_mla_fwd_ex)."""
    T, H, _ = q.shape
    K = idx.shape[1]
    out = out if out is not None else torch.empty((T, H, 512), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    dev = _need_attn_inputs(seqs, q, kv, out, lse, kv_scale)
    _need(idx, "idx", _I32T, (T, K), dev)
    need = _binding.workspace_size(DSA_OP_SPARSE_MLA, seqs, K, H)
    ws = ws if ws is not None else workspace(need, q.device, "sparse_mla")
    _need_ws(ws, dev)
    kv_dtype = DSA_KV_BF16 if kv_scale is None else DSA_KV_FP8_E4M3
    _check(_binding.dsa_sparse_mla_fwd_ex(dev, seqs, q, kv, kv_scale, kv_dtype, idx, K, H, scale, out,
                                          _out_dtype(out), lse, ws, ws.numel()), "dsa_sparse_mla_fwd")
    return out, lse


def dsa_sparse_mla_fwd_noalloc(seqs: Seqs, q, kv, idx, scale: float, out=None, lse=None, want_lse=True,
                               out_dtype=torch.bfloat16):
    """dsa_sparse_mla_fwd without a workspace: the library's built-in scratch
    array is used (for callers that cannot allocate device memory; see
    include/dsa.h).  Outputs not passed in are allocated here for convenience."""
    T, H, _ = q.shape
    K = idx.shape[1]
    out = out if out is not None else torch.empty((T, H, 512), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    dev = _need_attn_inputs(seqs, q, kv, out, lse)
    _need(idx, "idx", _I32T, (T, K), dev)
    _check(_binding.dsa_sparse_mla_fwd_noalloc(dev, seqs, q, kv, idx, K, H, scale, out, _out_dtype(out), lse),
           "dsa_sparse_mla_fwd_noalloc")
    return out, lse


def dsa_index_topk_attn(seqs: Seqs, qI, w, kI, kI_scale, q, kv, K: int, scale: float, out=None, lse=None,
                        idx_out=None, want_lse=True, ws=None, out_dtype=torch.bfloat16, q_ready=None,
                        select_in_indexer=False, kv_scale=None):
    """The whole path.  q_ready (a torch.cuda.Event, optional): the attention
    launch waits on it, so q may still be in flight on another stream.
    select_in_indexer: decode rows that fit are selected inside the indexer
    kernel (DSA_SELECT_IN_INDEXER).  kv_scale (uint8 [R, 8]) marks an FP8
    latent cache (kv = E4M3 codes [R, 576])."""
    T, H, _ = q.shape
    out = out if out is not None else torch.empty((T, H, 512), dtype=out_dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    dev = _need_attn_inputs(seqs, q, kv, out, lse, kv_scale)
    if _need_index_inputs(seqs, qI, w, kI, kI_scale, check_seqs=False) != dev:
        raise ValueError("qI and q are on different devices")
    if idx_out is not None:
        _need(idx_out, "idx_out", _I32T, (T, K), dev)
    ki_dtype = _ki_dtype(kI_scale, kI)
    op = DSA_OP_INDEX_TOPK_ATTN_FUSED if select_in_indexer else DSA_OP_INDEX_TOPK_ATTN
    need = _binding.workspace_size(op, seqs, K, H)
    ws = ws if ws is not None else workspace(need, q.device, "index_topk_attn")
    _need_ws(ws, dev)
    ev = None if q_ready is None else q_ready.cuda_event
    kv_dtype = DSA_KV_BF16 if kv_scale is None else DSA_KV_FP8_E4M3
    _check(_binding.dsa_index_topk_attn_ex(dev, seqs, qI, w, kI, kI_scale, ki_dtype, q, kv, kv_scale, kv_dtype, K, H,
                                           scale, out, _out_dtype(out), lse, idx_out, ws, ws.numel(),
                                           DSA_SELECT_IN_INDEXER if select_in_indexer else 0, ev),
           "dsa_index_topk_attn")
    return out, lse


_I64T = (torch.int64,)


def dsa_attn_mass(seqs: Seqs, q, kv, idx, lse, scale: float, mass, kv_scale=None, ws=None):
    """Adds to mass [B, at least max_ctx] int64 the attention weight that this
    call's tokens give each selected position, averaged over heads, in units of
    2^-DSA_MASS_FRACTION_BITS: q, kv, idx, scale, kv_scale as dsa_sparse_mla_fwd
    took them, lse [T, H] as it returned it.  Returns mass."""
    dev = _cuda_device(q, "q")
    _need_seqs(seqs, dev)
    T, rows = seqs.num_q_tokens, seqs.num_phys_pages * 64
    _need(q, "q", _BF16T, (T, None, 576), dev)
    H = q.shape[1]
    if kv_scale is None:
        _need(kv, "kv", _BF16T, (None, 576), dev, rows)
    else:
        _need(kv, "kv", _FP8T, (None, 576), dev, rows)
        _need(kv_scale, "kv_scale", _U8T, (None, 8), dev, rows)
    _need(idx, "idx", _I32T, (T, None), dev)
    _need(lse, "lse", _F32T, (T, H), dev)
    _need(mass, "mass", _I64T, (seqs.batch, None), dev)
    if mass.shape[1] < seqs.max_ctx:
        raise ValueError(f"mass: {mass.shape[1]} positions per sequence, max_ctx is {seqs.max_ctx}")
    ws = _space(ws, 256, dev, "attn_mass")
    _check(_binding.dsa_attn_mass(dev, seqs, q, kv, kv_scale, DSA_KV_BF16 if kv_scale is None else DSA_KV_FP8_E4M3, idx,
                                  idx.shape[1], H, scale, lse, mass, mass.shape[1], ws, ws.numel()), "dsa_attn_mass")
    return mass


def dsa_evict_select(ctx_len, mass, budget: int, recent: int = 0, sink: int = 0, keep=None, keep_len=None, ws=None):
    """(keep [B, budget] int32, keep_len [B] int32): the positions each
    sequence keeps when its cache is cut back to `budget` rows -- all if it has
    no more, else the first `sink`, the last `recent` and those of the largest
    mass [B, *] int64 -- ascending, -1 behind them."""
    dev = _cuda_device(mass, "mass")
    _need(mass, "mass", _I64T, (None, None), dev)
    B, ld = mass.shape
    _need(ctx_len, "ctx_len", _I32T, (B,), dev)
    if budget < 1 or recent < 0 or sink < 0 or recent + sink > budget:
        raise ValueError(f"budget={budget}, recent={recent}, sink={sink}: expected recent + sink <= budget, budget >= 1")
    if keep is None:
        keep = _empty((B, budget), torch.int32, dev)
    else:
        _need(keep, "keep", _I32T, (B, budget), dev)
    if keep_len is None:
        keep_len = _empty((B,), torch.int32, dev)
    else:
        _need(keep_len, "keep_len", _I32T, (B,), dev)
    ws = _space(ws, 256, dev, "evict_select")
    _check(_binding.dsa_evict_select(dev, ctx_len, B, ld, mass, ld, budget, recent, sink, keep, keep_len, ws, ws.numel()),
           "dsa_evict_select")
    return keep, keep_len


def dsa_evict_compact(seqs: Seqs, keep, keep_len, new_page_table, pools, mass=None, new_mass=None, ws=None):
    """Moves the kept rows of each pool to the new pages.  `pools`: up to
    DSA_MAX_POOLS pools [R, ...], each compacted inside itself (its new pages
    must not be pages that seqs reads), or pairs (pool, destination pool).
    mass, new_mass int64 [B, *] move alike.  Afterwards the batch is
    Seqs(..., ctx_len=keep_len, page_table=new_page_table, ...)."""
    dev = _cuda_device(keep, "keep")
    _need_seqs(seqs, dev)
    B = seqs.batch
    _need(keep, "keep", _I32T, (B, None), dev)
    _need(keep_len, "keep_len", _I32T, (B,), dev)
    _need(new_page_table, "new_page_table", _I32T, (B, None), dev)
    packed = _binding.pools(pools, seqs.num_phys_pages, dev)
    if packed is None:
        _refuse_pools(pools, seqs.num_phys_pages, dev)
    c_pools, new_pages = packed
    ld = new_ld = 0
    if mass is not None or new_mass is not None:
        _need(mass, "mass", _I64T, (B, None), dev)
        _need(new_mass, "new_mass", _I64T, (B, None), dev)
        ld, new_ld = mass.shape[1], new_mass.shape[1]
    need = 256 + (3 * ((new_pages + 31) // 32) * 4 + 255) // 256 * 256
    ws = _space(ws, need, dev, "evict_compact")
    _check(_binding.dsa_evict_compact(dev, seqs, keep, keep_len, keep.shape[1], new_page_table, new_page_table.shape[1],
                                      new_pages, c_pools, len(pools), mass, ld, new_mass, new_ld, ws, ws.numel()),
           "dsa_evict_compact")


def _refuse_pools(pools, pages: int, dev: torch.device):
    if len(pools) > DSA_MAX_POOLS:
        raise ValueError(f"{len(pools)} pools, at most {DSA_MAX_POOLS}")
    for i, p in enumerate(pools):
        src, dst = p if isinstance(p, (tuple, list)) else (p, p)
        for t in (src, dst):
            if not isinstance(t, torch.Tensor) or t.dim() < 1:
                raise TypeError(f"pools[{i}]: expected a tensor of rows")
        _need(src, f"pools[{i}]", (src.dtype,), tuple(src.shape), dev, pages * 64)
        if dst is not src:
            _need(dst, f"pools[{i}] destination", (src.dtype,), (dst.shape[0], *src.shape[1:]), dev, 64)
    raise ValueError("pools: expected a list of tensors or pairs of tensors whose rows have less than 2^31 bytes")


_ROPE_DTYPES = {torch.bfloat16: DSA_ROPE_BF16, torch.float16: DSA_ROPE_F16, torch.float32: DSA_ROPE_F32}


_POS_T = (torch.int64, torch.int32)


def _rope_view(t, name: str, dev: torch.device, dtype):
    """[T, H, D] sizes and [T, H] strides of a [T, H, D] or [T, D] tensor
    whose last dim is contiguous (the stride of a dim of one entry is 0)."""
    return _binding.rows(t, dtype, dev) or _refuse_rows(t, name, dev, dtype)


def _refuse_rows(t, name: str, dev: torch.device, dtype):
    """Says why t is no [T, H, D] or [T, D] tensor with a contiguous last dim."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != dev:
        raise ValueError(f"{name}: on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    sz = t.shape
    if len(sz) not in (2, 3):
        raise ValueError(f"{name}: shape {list(sz)}, expected [T, H, D] or [T, D]")
    if 0 in sz[1:]:
        raise ValueError(f"{name}: shape {list(sz)} has no heads or no dims")
    raise ValueError(f"{name}: the last dim must be contiguous")


def _rope_disjoint(x, out, T, H, D, xt, xh, ot, oh) -> bool:
    """x and out are one view, or share no element (two slices of the rows of
    one buffer among them)."""
    px, po, size = x.data_ptr(), out.data_ptr(), x.element_size()
    if px == po and (xt, xh) == (ot, oh):
        return True
    if px + ((T - 1) * xt + (H - 1) * xh + D) * size <= po or po + ((T - 1) * ot + (H - 1) * oh + D) * size <= px:
        return True
    inner = oh if H > 1 else ot                     # the rows' pitch
    if (xt, xh) != (ot, oh) or inner < D or (H > 1 and T > 1 and ot % oh):
        return False
    delta = (po - px) // size % inner
    return (po - px) % size == 0 and D <= delta <= inner - D


def dsa_rope(x: torch.Tensor, positions: torch.Tensor, table: RopeTable, offset: int = 0, out=None, transpose=False):
    """Rotates dims offset .. offset + table.rot_dim - 1 of every row of x
    ([T, H, D], or [T, D] for rows without heads; bf16, fp16 or fp32; any
    strides over tokens and heads) by its token's position (int32 or int64
    [T], negative ones too) and copies the other dims.

    out: x itself (in place, the other dims untouched), a tensor or view of x's
    shape that shares no element with x, or None for a new contiguous tensor.
    transpose: the transposed map, which takes the gradient of the output to
    that of x (with amplitude 1 it undoes the rotation).  The call records no
    autograd graph and refuses an x that would need one."""
    dev = _cuda_device(x, "x")
    dtype = x.dtype
    kind = _ROPE_DTYPES.get(dtype)
    if kind is None:
        raise TypeError(f"x: dtype {dtype}, expected one of {[str(d) for d in _ROPE_DTYPES]}")
    if x.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("dsa_rope records no gradients: call it under torch.no_grad() and rotate the output's "
                           "gradient with transpose=True")
    T, H, D, xt, xh = _rope_view(x, "x", dev, dtype)
    if not isinstance(table, RopeTable):
        raise TypeError(f"table: expected a RopeTable, got {type(table).__name__}")
    turns, rot_dim = table.turns, table.rot_dim
    _need(turns, "table.turns", _I64T, (rot_dim // 2,), dev)
    _need(positions, "positions", _POS_T, (T,), dev)
    if out is None:
        out = _empty(tuple(x.shape), dtype, dev)
        ot, oh = H * D if T > 1 else 0, D if H > 1 else 0
    elif out is x:
        ot, oh = xt, xh
    else:
        ot, oh = _rope_view(out, "out", dev, dtype)[3:]
        if out.shape != x.shape:
            raise ValueError(f"out: shape {list(out.shape)}, expected {list(x.shape)}")
        if out.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("out: dsa_rope records no gradients")
        if T and not _rope_disjoint(x, out, T, H, D, xt, xh, ot, oh):
            raise ValueError("x and out overlap without being the same view")
    flags = (0 if table.interleaved else DSA_ROPE_HALF) | (DSA_ROPE_TRANSPOSE if transpose else 0) \
        | (DSA_ROPE_POS64 if positions.dtype is torch.int64 else 0)
    _check(_binding.dsa_rope(dev, x, out, kind, T, H, D, xt, xh, ot, oh, positions, turns, rot_dim, offset,
                             table.amplitude, flags), "dsa_rope")
    return out


def dsa_check_error(ws: torch.Tensor) -> int:
    """Synchronise the current stream and return (and clear) the device error status."""
    return int(_lib.dsa_check_error(_ptr(ws), _stream(ws.device)))


def dsa_check_error_noalloc(device=None) -> int:
    """dsa_check_error for the built-in scratch of dsa_sparse_mla_fwd_noalloc
    (synchronises the current stream of `device`)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return int(_lib.dsa_check_error_noalloc(_stream(dev)))


def dsa_set_wait_limit_ns(ns: int) -> None:
    """Limit of every bounded in-kernel wait of this thread's later calls (0 = the 2 s default)."""
    _check(_lib.dsa_set_wait_limit_ns(int(ns)), "dsa_set_wait_limit_ns")


def dsa_launches_in_last_call() -> int:
    """Kernels launched by this thread's most recent entry-point call."""
    return int(_lib.dsa_launches_in_last_call())


def dsa_launch_timing(enable: bool) -> None:
    """Record device events around every kernel of this thread's later calls."""
    _check(_lib.dsa_launch_timing(1 if enable else 0), "dsa_launch_timing")


def dsa_last_launch_times() -> list:
    """[(kernel name, device ms)] of this thread's last call made with timing on."""
    cap = 16
    ms = (ctypes.c_float * cap)()
    names = (ctypes.c_char_p * cap)()
    n = int(_lib.dsa_last_launch_times(ms, names, cap))
    if n < 0:
        raise DsaError(DSA_ERR_CUDA, "dsa_last_launch_times")
    return [(names[i].decode(), float(ms[i])) for i in range(min(n, cap))]


def raw():
    """The ctypes handle of libdsa (for tests that call the C ABI directly)."""
    return _lib
