"""Thin Python binding of libidx (ctypes).  Argument marshalling only: every
step of the computation runs in the library's CUDA kernels.

The functions carry the C names (idx_score, idx_topk, idx_topk_scores,
dosa_topk, witness_merge, witness_indices, block_select) and take torch CUDA
tensors; torch provides device memory and streams, nothing else.  A non-zero
status raises IdxError with the library's message.  If libidx.so has not been
built the import fails loudly: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libidx.so")

IDX_OK = 0
STATUS_NAMES = {1: "ROWS_MISMATCH", 2: "SEGMENTS_OUT_OF_RANGE", 3: "KEEP_OUT_OF_RANGE", 4: "INVALID_ARG",
                5: "UNSUPPORTED", 6: "WORKSPACE_TOO_SMALL", 7: "CUDA"}
IDX_F32, IDX_BF16, IDX_FP8_E4M3, IDX_F16 = 0, 1, 2, 3
IDX_MAX_PLANES = 8
IDX_MAX_SEGMENTS, IDX_MAX_K = 64, 4096
DEVERR_WAIT_TIMEOUT, DEVERR_BAD_ROW, DEVERR_CAPACITY = 1, 2, 4


class IdxError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))


class idx_problem(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_dtype", ctypes.c_int32), ("w", ctypes.c_void_p),
                ("M", ctypes.c_int64), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
                ("keys", ctypes.c_void_p), ("k_dtype", ctypes.c_int32), ("key_scale", ctypes.c_void_p),
                ("n_keys", ctypes.c_int64), ("key_off", ctypes.c_void_p), ("key_len", ctypes.c_void_p),
                ("max_key_len", ctypes.c_int32)]


class dosa_params(ctypes.Structure):
    _fields_ = [("n_seed", ctypes.c_int32), ("retained_heads", ctypes.c_int32), ("n_sample", ctypes.c_int32),
                ("act_freq_min", ctypes.c_float), ("margin_gamma", ctypes.c_float),
                ("candidate_capacity", ctypes.c_int32), ("group_stream", ctypes.c_int32)]


class dosa_stats(ctypes.Structure):
    _fields_ = [("pairs", ctypes.c_ulonglong), ("seeds", ctypes.c_ulonglong), ("candidates", ctypes.c_ulonglong),
                ("survivors", ctypes.c_ulonglong), ("fallback_rows", ctypes.c_ulonglong),
                ("skipped_rows", ctypes.c_ulonglong), ("group_keys", ctypes.c_ulonglong),
                ("solo_keys", ctypes.c_ulonglong)]

DOSA_STATS_FIELDS = len(dosa_stats._fields_)   # int64 counters of a device dosa_stats


class dosa_ws_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("seed_list", "seed_count", "rep_count", "rep_scores", "tau", "status",
                                             "plan_head", "plan_beta", "plan_dnorm", "wfold", "coef", "qprep",
                                             "seed_ld", "rep_ld", "seed_rows")] + \
               [("group_layout", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class topk_prior_stats(ctypes.Structure):
    _fields_ = [("rows_filtered", ctypes.c_ulonglong), ("candidates", ctypes.c_ulonglong),
                ("dense_rows", ctypes.c_ulonglong)]


class block_select_stats(ctypes.Structure):
    _fields_ = [("pairs", ctypes.c_ulonglong), ("blocks_bounded", ctypes.c_ulonglong),
                ("blocks_rescored", ctypes.c_ulonglong), ("fallback_pairs", ctypes.c_ulonglong),
                ("max_bound_use", ctypes.c_float), ("reserved", ctypes.c_float)]


def block_select_stats_tensor(device="cuda") -> torch.Tensor:
    """Zeroed device storage for one block_select_stats (40 bytes)."""
    return torch.zeros(5, dtype=torch.int64, device=device)


def block_select_stats_read(t: torch.Tensor) -> dict:
    """block_select_stats storage -> dict (copies to the host)."""
    h = t.detach().cpu()
    u = h.tolist()
    f = h[4:5].view(torch.float32).tolist()
    return {"pairs": u[0], "blocks_bounded": u[1], "blocks_rescored": u[2], "fallback_pairs": u[3],
            "max_bound_use": f[0]}


class block_sparse_config(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int32), ("top_blocks", ctypes.c_int32), ("init_blocks", ctypes.c_int32),
                ("local_blocks", ctypes.c_int32)]


class attn_problem(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("B", ctypes.c_int32),
                ("T", ctypes.c_int32), ("Hq", ctypes.c_int32), ("n_kv", ctypes.c_int32), ("D", ctypes.c_int32),
                ("q_stride_b", ctypes.c_int64), ("q_stride_t", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("S", ctypes.c_int64),
                ("k_stride_b", ctypes.c_int64), ("k_stride_s", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
                ("v_stride_b", ctypes.c_int64), ("v_stride_s", ctypes.c_int64), ("v_stride_h", ctypes.c_int64),
                ("len", ctypes.c_void_p), ("len_per_head", ctypes.c_int32), ("ids_per_head", ctypes.c_int32),
                ("pk", ctypes.c_void_p), ("pv", ctypes.c_void_p), ("P", ctypes.c_int64),
                ("pk_stride_s", ctypes.c_int64), ("pk_stride_h", ctypes.c_int64), ("pv_stride_s", ctypes.c_int64),
                ("pv_stride_h", ctypes.c_int64), ("prefix_len", ctypes.c_void_p), ("ids", ctypes.c_void_p),
                ("W", ctypes.c_int64)]


class evict_plane(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_bytes", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class evict_problem(ctypes.Structure):
    _fields_ = [("mass", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("len", ctypes.c_void_p),
                ("cur", ctypes.c_void_p), ("B", ctypes.c_int32), ("mass_heads", ctypes.c_int32),
                ("S", ctypes.c_int64), ("stride", ctypes.c_int64), ("n_keep", ctypes.c_int64),
                ("n_first", ctypes.c_int32), ("n_last", ctypes.c_int32), ("planes", ctypes.POINTER(evict_plane)),
                ("n_planes", ctypes.c_int32)]


EXPORTS = {
    "idx_last_error_string": (ctypes.c_char_p, []),
    "idx_device_error": (ctypes.c_uint32, []),
    "idx_set_wait_limit_ns": (ctypes.c_int32, [ctypes.c_uint64]),
    "idx_score": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "idx_topk_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(idx_problem), ctypes.c_int32]),
    "idx_topk": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "idx_topk_scores_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]),
    "idx_topk_scores": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "dosa_topk_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(idx_problem), ctypes.c_int32,
                                                   ctypes.POINTER(dosa_params), ctypes.c_int32]),
    "dosa_topk": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_int32, ctypes.POINTER(dosa_params),
                                   ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                   ctypes.c_void_p]),
    "dosa_workspace_layout": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_int32,
                                               ctypes.POINTER(dosa_params), ctypes.c_int32,
                                               ctypes.POINTER(dosa_ws_layout)]),
    "witness_merge": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_void_p]),
    "witness_indices": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    "block_select_workspace_size": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int32, ctypes.c_int64,
                                                      ctypes.POINTER(block_sparse_config)]),
    "block_select": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_int32, ctypes.c_int32, ctypes.c_int64,
                                      ctypes.POINTER(block_sparse_config), ctypes.c_void_p, ctypes.c_int32,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                      ctypes.c_void_p]),
    "block_select_events": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int64,
                                             ctypes.POINTER(block_sparse_config), ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                             ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "idx_topk_prior_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(idx_problem), ctypes.c_int32, ctypes.c_int32,
                                                        ctypes.c_int32]),
    "idx_topk_prior": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                                        ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "idx_topk_prior_events": (ctypes.c_int32, [ctypes.POINTER(idx_problem), ctypes.c_int32, ctypes.c_void_p,
                                               ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                               ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p]),
    "block_positions": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                         ctypes.c_int32, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                         ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]),
    "block_select_static": (ctypes.c_int32, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                             ctypes.c_int32, ctypes.c_int32, ctypes.c_int64,
                                             ctypes.POINTER(block_sparse_config), ctypes.c_void_p, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "attn_shared_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(attn_problem), ctypes.c_int32]),
    "attn_shared": (ctypes.c_int32, [ctypes.POINTER(attn_problem), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cache_evict": (ctypes.c_int32, [ctypes.POINTER(evict_problem), ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libidx.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libidx.so not built ({LIB_PATH}); run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(st: int) -> None:
    if st != IDX_OK:
        raise IdxError(st, lib().idx_last_error_string().decode(errors="replace"))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _buf(t: Optional[torch.Tensor], dtype: torch.dtype, numel: int, name: str):
    """A caller's device buffer that the library writes or reads as `numel`
    elements of `dtype` (the C ABI takes plain pointers, so this is the last
    place where a short or mistyped buffer can be caught)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")
    return _ptr(t)


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# torch.cuda.current_stream() builds a Stream object; a decode step of a few
# microseconds asks for the handle alone
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)


_DT = {torch.float32: IDX_F32, torch.bfloat16: IDX_BF16, torch.uint8: IDX_FP8_E4M3,
       torch.float8_e4m3fn: IDX_FP8_E4M3}


@dataclass
class Problem:
    """Device tensors of one indexer batch (see idx_problem in include/idx.h)."""
    q: torch.Tensor                     # [M, H, D] float32 or bfloat16
    w: torch.Tensor                     # [M, H] float32
    keys: torch.Tensor                  # [n_keys, D] float32 / bfloat16 / uint8 (e4m3 codes)
    key_len: torch.Tensor               # [M] int32
    max_key_len: int
    key_off: Optional[torch.Tensor] = None   # [M] int64 or None (shared keys)
    key_scale: Optional[torch.Tensor] = None  # [n_keys] float32 for FP8 keys

    def c(self) -> idx_problem:
        M, H, D = self.q.shape
        return idx_problem(_ptr(self.q), _DT[self.q.dtype], _ptr(self.w), M, H, D, _ptr(self.keys),
                           _DT[self.keys.dtype], _ptr(self.key_scale), self.keys.shape[0], _ptr(self.key_off),
                           _ptr(self.key_len), int(self.max_key_len))


def device_error() -> int:
    """Synchronise and return (then clear) the library's device error word."""
    return int(lib().idx_device_error())


DEFAULT_WAIT_LIMIT_NS = 2_000_000_000


def set_wait_limit_ns(ns: int) -> None:
    """Limit of every pipeline wait in the library's kernels (current device)."""
    _check(lib().idx_set_wait_limit_ns(int(ns)))


def _rows_need(M: int, ld: int, width: int) -> int:
    """Elements that M rows of `width` values at row stride `ld` span."""
    return 0 if M <= 0 or width <= 0 else (M - 1) * ld + width


def idx_score(p: Problem, scores: torch.Tensor, ld: Optional[int] = None, stream=None) -> torch.Tensor:
    cp = p.c()
    ld = int(ld if ld is not None else scores.shape[-1])
    need = _rows_need(p.q.shape[0], ld, int(p.max_key_len))
    _check(lib().idx_score(ctypes.byref(cp), _buf(scores, torch.float32, need, "scores"), ld, _stream(stream)))
    return scores


def idx_topk_workspace_size(p: Problem, K: int) -> int:
    cp = p.c()
    return int(lib().idx_topk_workspace_size(ctypes.byref(cp), K))


def idx_topk(p: Problem, K: int, out_ids: torch.Tensor, out_scores: Optional[torch.Tensor], ws: torch.Tensor,
             stream=None):
    cp = p.c()
    MK = p.q.shape[0] * K
    _check(lib().idx_topk(ctypes.byref(cp), K, _buf(out_ids, torch.int32, MK, "out_ids"),
                          _buf(out_scores, torch.float32, MK, "out_scores"), _ptr(ws), ws.numel() * ws.element_size(),
                          _stream(stream)))
    return out_ids, out_scores


def idx_topk_prior_workspace_size(p: Problem, K: int, prior_ld: int, capacity: int) -> int:
    cp = p.c()
    return int(lib().idx_topk_prior_workspace_size(ctypes.byref(cp), K, prior_ld, capacity))


def idx_topk_prior(p: Problem, K: int, prior_ids: torch.Tensor, capacity: int, out_ids: torch.Tensor,
                   out_scores: Optional[torch.Tensor], ws: torch.Tensor, row_status: Optional[torch.Tensor] = None,
                   stats: Optional[torch.Tensor] = None, stream=None):
    """Top-K with the previous step's selection prior_ids [M, prior_ld] as a prior.
    stats: torch.zeros(3, dtype=torch.int64) storage for topk_prior_stats, or None."""
    cp = p.c()
    M = p.q.shape[0]
    _check(lib().idx_topk_prior(ctypes.byref(cp), K, _buf(prior_ids, torch.int32, M * prior_ids.shape[1], "prior_ids"),
                                prior_ids.shape[1], capacity, _buf(out_ids, torch.int32, M * K, "out_ids"),
                                _buf(out_scores, torch.float32, M * K, "out_scores"),
                                _buf(row_status, torch.int32, M, "row_status"), _buf(stats, torch.int64, 3, "stats"),
                                _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return out_ids, out_scores


def idx_topk_prior_events(p: Problem, K: int, prior_ids: torch.Tensor, capacity: int, out_ids: torch.Tensor,
                          out_scores: Optional[torch.Tensor], ws: torch.Tensor, events, stream=None):
    """idx_topk_prior recording 6 torch.cuda.Event (already created) between its stages."""
    cp = p.c()
    M = p.q.shape[0]
    handles = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(e.cuda_event) for e in events[:6]])
    _check(lib().idx_topk_prior_events(ctypes.byref(cp), K,
                                       _buf(prior_ids, torch.int32, M * prior_ids.shape[1], "prior_ids"),
                                       prior_ids.shape[1], capacity, _buf(out_ids, torch.int32, M * K, "out_ids"),
                                       _buf(out_scores, torch.float32, M * K, "out_scores"), None, None, _ptr(ws),
                                       ws.numel() * ws.element_size(), handles, 6, _stream(stream)))
    return out_ids, out_scores


def idx_topk_scores_workspace_size(M: int, max_len: int, K: int) -> int:
    return int(lib().idx_topk_scores_workspace_size(M, max_len, K))


def idx_topk_scores(scores: torch.Tensor, lens: torch.Tensor, max_len: int, K: int, out_ids: torch.Tensor,
                    out_scores: Optional[torch.Tensor] = None, ld: Optional[int] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    M = lens.shape[0]
    ld = int(ld if ld is not None else scores.shape[-1])
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().idx_topk_scores(_buf(scores, torch.float32, _rows_need(M, ld, int(max_len)), "scores"), ld,
                                 _buf(lens, torch.int32, M, "lens"), M, int(max_len), K,
                                 _buf(out_ids, torch.int32, M * K, "out_ids"),
                                 _buf(out_scores, torch.float32, M * K, "out_scores"), _ptr(ws), ws_bytes,
                                 _stream(stream)))
    return out_ids, out_scores


def make_dosa_params(n_seed=12288, retained_heads=16, n_sample=128, act_freq_min=0.5, margin_gamma=2.0 ** -10,
                     candidate_capacity=16384, group_stream=1) -> dosa_params:
    return dosa_params(n_seed, retained_heads, n_sample, act_freq_min, margin_gamma, candidate_capacity,
                       group_stream)


def dosa_topk_workspace_size(p: Problem, K: int, dp: dosa_params, seed_ld: int = 0) -> int:
    cp = p.c()
    return int(lib().dosa_topk_workspace_size(ctypes.byref(cp), K, ctypes.byref(dp), seed_ld))


def dosa_topk(p: Problem, K: int, dp: dosa_params, out_ids: torch.Tensor, out_scores: Optional[torch.Tensor],
              ws: torch.Tensor, seed_ids: Optional[torch.Tensor] = None, row_status: Optional[torch.Tensor] = None,
              stats: Optional[torch.Tensor] = None, stream=None):
    cp = p.c()
    M = p.q.shape[0]
    seed_ld = int(seed_ids.shape[1]) if seed_ids is not None else 0
    _check(lib().dosa_topk(ctypes.byref(cp), K, ctypes.byref(dp), _buf(seed_ids, torch.int32, M * seed_ld, "seed_ids"),
                           seed_ld, _buf(out_ids, torch.int32, M * K, "out_ids"),
                           _buf(out_scores, torch.float32, M * K, "out_scores"),
                           _buf(row_status, torch.int32, M, "row_status"),
                           _buf(stats, torch.int64, DOSA_STATS_FIELDS, "stats"), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream)))
    return out_ids, out_scores


def dosa_workspace_layout(p: Problem, K: int, dp: dosa_params, seed_ld: int = 0) -> dict:
    """Byte offsets (and row strides) of dosa_topk's intermediate arrays in its workspace."""
    cp = p.c()
    out = dosa_ws_layout()
    _check(lib().dosa_workspace_layout(ctypes.byref(cp), K, ctypes.byref(dp), seed_ld, ctypes.byref(out)))
    return {n: int(getattr(out, n)) for n, _ in dosa_ws_layout._fields_}


def witness_merge(topk_ids: torch.Tensor, context_lens: torch.Tensor, keep: int, num_segments: int,
                  max_replacements: int, rows: Optional[int] = None, topk: Optional[int] = None, stream=None):
    rows = topk_ids.shape[0] if rows is None else rows
    topk = topk_ids.shape[1] if topk is None else topk
    _check(lib().witness_merge(_ptr(topk_ids), rows, topk, _ptr(context_lens), context_lens.shape[0], keep,
                               num_segments, max_replacements, _stream(stream)))
    return topk_ids


def witness_indices(learned: torch.Tensor, context_lens: torch.Tensor, num_segments: int, out: torch.Tensor,
                    stream=None):
    rows, topk = learned.shape
    _check(lib().witness_indices(_ptr(learned), rows, topk, _ptr(context_lens), context_lens.shape[0], num_segments,
                                 _ptr(out), _stream(stream)))
    return out


def block_select_workspace_size(Q: int, n_kv: int, L: int, cfg: block_sparse_config) -> int:
    return int(lib().block_select_workspace_size(Q, n_kv, L, ctypes.byref(cfg)))


def block_select(index_q: torch.Tensor, index_k: torch.Tensor, query_pos: torch.Tensor, cfg: block_sparse_config,
                 out: torch.Tensor, out_count: Optional[torch.Tensor], ws: Optional[torch.Tensor], stream=None,
                 stats: Optional[torch.Tensor] = None):
    """stats: block_select_stats_tensor() storage or None."""
    Q, n_kv, D = index_q.shape
    L = index_k.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    if stats is not None and stats.numel() * stats.element_size() < ctypes.sizeof(block_select_stats):
        raise ValueError("stats needs 40 bytes")
    _check(lib().block_select(_ptr(index_q), _ptr(index_k), _ptr(query_pos), Q, n_kv, D, L, ctypes.byref(cfg),
                              _ptr(out), out.shape[-1], _ptr(out_count), _ptr(stats), _ptr(ws), ws_bytes,
                              _stream(stream)))
    return out, out_count


def block_select_events(index_q: torch.Tensor, index_k: torch.Tensor, query_pos: torch.Tensor,
                        cfg: block_sparse_config, out: torch.Tensor, out_count: Optional[torch.Tensor],
                        ws: Optional[torch.Tensor], events, stream=None, stats: Optional[torch.Tensor] = None):
    """block_select recording 6 torch.cuda.Event (already created: recorded once)
    between its kernels on `stream` (profiling)."""
    Q, n_kv, D = index_q.shape
    L = index_k.shape[0]
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    handles = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(e.cuda_event) for e in events[:6]])
    _check(lib().block_select_events(_ptr(index_q), _ptr(index_k), _ptr(query_pos), Q, n_kv, D, L, ctypes.byref(cfg),
                                     _ptr(out), out.shape[-1], _ptr(out_count), _ptr(stats), _ptr(ws), ws_bytes,
                                     handles, 6, _stream(stream)))
    return out, out_count


def block_positions(blocks: torch.Tensor, counts: Optional[torch.Tensor], query_pos: torch.Tensor, L: int,
                    block_size: int, out: torch.Tensor, out_count: Optional[torch.Tensor], stream=None):
    """blocks [Q, n_kv, W] int32 (as block_select writes them) -> covered positions
    [Q, n_kv, out_width] (ascending, -1 padded)."""
    Q, n_kv, W = blocks.shape
    _check(lib().block_positions(_ptr(blocks), _ptr(counts), Q, n_kv, W, _ptr(query_pos), L, block_size, _ptr(out),
                                 out.shape[-1], _ptr(out_count), _stream(stream)))
    return out, out_count


def problem_to_device(wp, device="cuda") -> Problem:
    """Copy a workloads.IndexerProblem (numpy, storage formats) to the device
    without changing a byte."""
    import numpy as np
    if wp.dtype == "f32":
        q = torch.from_numpy(np.ascontiguousarray(wp.q)).to(device)
        keys = torch.from_numpy(np.ascontiguousarray(wp.keys)).to(device)
    else:
        q = torch.from_numpy(np.ascontiguousarray(wp.q).view(np.int16)).to(device).view(torch.bfloat16)
        if wp.dtype == "bf16":
            keys = torch.from_numpy(np.ascontiguousarray(wp.keys).view(np.int16)).to(device).view(torch.bfloat16)
        else:
            keys = torch.from_numpy(np.ascontiguousarray(wp.keys)).to(device)
    w = torch.from_numpy(np.ascontiguousarray(wp.w, dtype=np.float32)).to(device)
    key_len = torch.from_numpy(np.ascontiguousarray(wp.key_len, dtype=np.int32)).to(device)
    key_off = None if wp.key_off is None else torch.from_numpy(np.ascontiguousarray(wp.key_off, dtype=np.int64)).to(device)
    key_scale = None if wp.key_scale is None else torch.from_numpy(np.ascontiguousarray(wp.key_scale)).to(device)
    return Problem(q, w, keys, key_len, int(np.max(wp.key_len)) if len(wp.key_len) else 0, key_off, key_scale)


def block_select_static(index_q: torch.Tensor, index_k: torch.Tensor, query_pos: torch.Tensor,
                        cfg: block_sparse_config, out: torch.Tensor, out_count: Optional[torch.Tensor], stream=None):
    """block_select without a workspace: the scratch is a fixed array inside the
    library (for callers that cannot allocate device memory)."""
    Q, n_kv, D = index_q.shape
    L = index_k.shape[0]
    _check(lib().block_select_static(_ptr(index_q), _ptr(index_k), _ptr(query_pos), Q, n_kv, D, L,
                                     ctypes.byref(cfg), _ptr(out), out.shape[-1], _ptr(out_count), _stream(stream)))
    return out, out_count


_ATTN_DT = {torch.bfloat16: IDX_BF16, torch.float16: IDX_F16}


def _need(ok: bool, msg: str) -> None:
    if not ok:
        raise ValueError(msg)


def _strided(t: torch.Tensor, name: str, shape, dtype):
    """A strided device tensor whose last dimension is contiguous: its address
    and the strides of the others (0 where a dimension has one element)."""
    _need(t.is_cuda, f"{name}: expected a CUDA tensor")
    _need(t.dtype == dtype, f"{name}: expected {dtype}, got {t.dtype}")
    _need(tuple(t.shape) == tuple(shape), f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    _need(t.shape[-1] <= 1 or t.stride(-1) == 1, f"{name}: the last dimension must be contiguous")
    return t.data_ptr(), [0 if n <= 1 else st for n, st in zip(t.shape[:-1], t.stride()[:-1])]


def _dense(t: torch.Tensor, name: str, shapes, dtype):
    """A contiguous device tensor of one of `shapes`."""
    _need(t.is_cuda, f"{name}: expected a CUDA tensor")
    _need(t.dtype == dtype, f"{name}: expected {dtype}, got {t.dtype}")
    _need(tuple(t.shape) in shapes, f"{name}: shape {tuple(t.shape)} is none of {shapes}")
    _need(t.is_contiguous(), f"{name}: expected a contiguous tensor")
    return t.data_ptr()


class _Described:
    """A problem whose C struct is built, with all its checks, when it is first
    used and again after a field was assigned or one of its tensors got other
    memory, another shape, strides or type; a decode loop that only changes the
    tensors' contents builds it once.  Lists of tensors are kept as tuples, so
    that none of theirs is replaced unnoticed."""

    def __setattr__(self, name, value):
        self.__dict__[name] = tuple(value) if isinstance(value, list) else value
        self.__dict__.pop("_desc", None)

    def _tensors(self):
        for v in list(self.__dict__.values()):
            if isinstance(v, torch.Tensor):
                yield v
            elif isinstance(v, tuple):
                yield from (t for t in v if isinstance(t, torch.Tensor))

    def desc(self):
        """(reference to the struct, index of the tensors' device, what the call
        compares its outputs with)"""
        d = self.__dict__.get("_desc")
        if d is not None:
            for t, at, shape, dtype in d[1]:
                if t.data_ptr() != at or t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
                    break
            else:
                for t, at, shape, dtype, strides in d[2]:
                    if t.data_ptr() != at or t.shape != shape or t.dtype is not dtype or t.stride() != strides:
                        break
                else:
                    return d[0]
        self.__dict__.pop("_desc", None)
        c = self.c()
        # The contiguous ones, whose shape says all, are asked for less (a call of
        # 9 us is as long on the host).
        dense, strided = [], []
        for t in self._tensors():
            if t.is_contiguous():
                dense.append((t, t.data_ptr(), t.shape, t.dtype))
            else:
                strided.append((t, t.data_ptr(), t.shape, t.dtype, t.stride()))
        use = (ctypes.byref(c), self._device(), self._shapes(c))
        self.__dict__["_desc"] = (use, dense, strided)
        return use


@dataclass
class AttnProblem(_Described):
    """Device tensors of one attn_shared call (see attn_problem in include/idx.h).
    Caches are indexed [request, slot, KV head, D]; a head-major cache is passed
    as its transposed view."""
    q: torch.Tensor                              # [B, T, Hq, D] bfloat16 or float16
    scale: float
    k: Optional[torch.Tensor] = None             # [B, S, n_kv, D] private caches
    v: Optional[torch.Tensor] = None
    lens: Optional[torch.Tensor] = None          # [B], [B, 1] or [B, n_kv] int32 filled slots
    pk: Optional[torch.Tensor] = None            # [P, n_kv, D] shared prefix
    pv: Optional[torch.Tensor] = None
    prefix_len: Optional[torch.Tensor] = None    # [B] int32
    ids: Optional[torch.Tensor] = None           # [B, T, W] or [B, T, n_kv, W] int32; W == 0 selects no slot

    def _device(self):
        return self.q.device.index

    def _shapes(self, c):
        """Shape and type of out, shape of lse, and of mass with one and with n_kv
        mass heads."""
        q = self.q.shape
        one, each = (torch.Size((c.B, h, c.S)) for h in (1, c.n_kv))
        return q, self.q.dtype, q[:3], one if c.S else None, each if c.S else None

    def c(self) -> attn_problem:
        q = self.q
        _need(q.dim() == 4, "q: expected [B, T, Hq, D]")
        _need(q.dtype in _ATTN_DT, f"q: expected bfloat16 or float16, got {q.dtype}")
        B, T, Hq, D = q.shape
        some = self.k if self.k is not None else self.pk
        _need(some is not None, "neither a private cache nor a prefix")
        _need(some.dim() >= 2, "caches: expected [..., n_kv, D]")
        n_kv = some.shape[-2]
        a = attn_problem(dtype=_ATTN_DT[q.dtype], scale=float(self.scale), B=B, T=T, Hq=Hq, n_kv=n_kv, D=D)
        a.q, (a.q_stride_b, a.q_stride_t, a.q_stride_h) = _strided(q, "q", q.shape, q.dtype)
        if self.k is not None:
            _need(self.v is not None and self.lens is not None, "k needs v and lens")
            _need(self.k.dim() == 4, "k: expected [B, S, n_kv, D]")
            S = self.k.shape[1]
            a.S = S
            a.k, (a.k_stride_b, a.k_stride_s, a.k_stride_h) = _strided(self.k, "k", (B, S, n_kv, D), q.dtype)
            a.v, (a.v_stride_b, a.v_stride_s, a.v_stride_h) = _strided(self.v, "v", (B, S, n_kv, D), q.dtype)
            a.len = _dense(self.lens, "lens", ((B,), (B, 1), (B, n_kv)), torch.int32)
            a.len_per_head = int(self.lens.dim() == 2 and self.lens.shape[1] == n_kv)
        if self.pk is not None:
            _need(self.pv is not None and self.pk.dim() == 3, "pk: expected [P, n_kv, D] with pv")
            P = self.pk.shape[0]
            a.P = P
            a.pk, (a.pk_stride_s, a.pk_stride_h) = _strided(self.pk, "pk", (P, n_kv, D), q.dtype)
            a.pv, (a.pv_stride_s, a.pv_stride_h) = _strided(self.pv, "pv", (P, n_kv, D), q.dtype)
            if self.prefix_len is not None:
                a.prefix_len = _dense(self.prefix_len, "prefix_len", ((B,),), torch.int32)
        if self.ids is not None:
            W = self.ids.shape[-1]
            ids = _dense(self.ids, "ids", ((B, T, W), (B, T, n_kv, W)), torch.int32)
            if W or a.S:  # (an empty list of an empty cache says nothing)
                # An empty tensor's address is 0, which would say that there is no
                # list (every slot) instead of one that holds nothing.  With W == 0
                # nothing is read through it, so any address does: the queries'.
                a.W, a.ids, a.ids_per_head = W, ids or a.q, int(self.ids.dim() == 4)
        return a


def attn_shared_workspace_size(p: AttnProblem, mass: bool = True) -> int:
    return int(lib().attn_shared_workspace_size(p.desc()[0], int(mass)))


def _out(t: torch.Tensor, name: str, shape, dtype):
    """_dense for one shape, quick where the tensor is right."""
    if t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.is_cuda:
        return t.data_ptr()
    return _dense(t, name, (tuple(shape),), dtype)


def attn_shared(p: AttnProblem, out: torch.Tensor, lse: Optional[torch.Tensor], mass: Optional[torch.Tensor],
                ws: torch.Tensor, stream=None):
    """out [B, T, Hq, D]; lse [B, T, Hq] float32 or None; mass [B, n_kv or 1, S]
    float32 (added to) or None."""
    ref, device, (so, dt, sl, s1, sh) = p.desc()
    po = _out(out, "out", so, dt)
    pl = None if lse is None else _out(lse, "lse", sl, torch.float32)
    pm, heads = None, 1
    if mass is not None:
        if s1 is None:
            raise ValueError("mass: there is no private cache")
        s = mass.shape
        if s != s1:
            heads = sh[1]
        if (s == s1 or s == sh) and mass.dtype is torch.float32 and mass.is_contiguous() and mass.is_cuda:
            pm = mass.data_ptr()
        else:
            _dense(mass, "mass", (tuple(s1), tuple(sh)), torch.float32)  # raises
    if not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("ws: expected a contiguous CUDA tensor")
    st = (_lib or lib()).attn_shared(ref, po, pl, pm, heads, ws.data_ptr(), ws.nbytes,
                                     _current_raw_stream(device) if stream is None else stream.cuda_stream)
    if st:
        _check(st)
    return out, lse, mass


@dataclass
class EvictProblem(_Described):
    """Device tensors of one cache_evict call (see evict_problem in include/idx.h).
    planes are indexed [B, S, heads, row] or [B, S, row]; they are compacted in
    place."""
    mass: torch.Tensor                           # [B, mass_heads, S] float32
    lens: torch.Tensor                           # [B, mass_heads] int32
    n_keep: int
    n_first: int = 0
    n_last: int = 0
    pos: Optional[torch.Tensor] = None           # [B, mass_heads, S] int32
    cur: Optional[torch.Tensor] = None           # [B] int32
    planes: tuple = ()

    def _device(self):
        return self.mass.device.index

    def _shapes(self, c):
        """Shapes of out_src (and of outputs beside it), and of out_len."""
        return torch.Size((c.B, c.mass_heads, c.n_keep)), torch.Size((c.B, c.mass_heads))

    def c(self) -> evict_problem:
        _need(self.mass.dim() == 3, "mass: expected [B, mass_heads, S]")
        B, Hm, S = self.mass.shape
        e = evict_problem(B=B, mass_heads=Hm, S=S, stride=S, n_keep=int(self.n_keep), n_first=int(self.n_first),
                          n_last=int(self.n_last))
        e.mass = _dense(self.mass, "mass", ((B, Hm, S),), torch.float32)
        e.len = _dense(self.lens, "lens", ((B, Hm),), torch.int32)
        if self.pos is not None:
            e.pos = _dense(self.pos, "pos", ((B, Hm, S),), torch.int32)
        if self.cur is not None:
            e.cur = _dense(self.cur, "cur", ((B,),), torch.int32)
        n = len(self.planes)
        _need(n <= IDX_MAX_PLANES, f"planes: at most {IDX_MAX_PLANES}")
        arr = (evict_plane * max(n, 1))()
        for i, t in enumerate(self.planes):
            _need(t.dim() in (3, 4) and t.shape[0] == B and t.shape[1] == S,
                  f"planes[{i}]: expected [B, S, heads, row] or [B, S, row], got {tuple(t.shape)}")
            heads = t.shape[2] if t.dim() == 4 else 1
            _need(Hm == 1 or heads == Hm, f"planes[{i}]: {heads} heads for {Hm} mass heads")
            size = t.element_size()
            ptr, st = _strided(t, f"planes[{i}]", t.shape, t.dtype)
            arr[i] = evict_plane(ptr, t.shape[-1] * size, heads, 0, st[0] * size, st[1] * size,
                                 st[2] * size if t.dim() == 4 else 0)
        e.planes, e.n_planes = arr, n
        return e


def cache_evict(p: EvictProblem, out_src: torch.Tensor, out_len: Optional[torch.Tensor] = None,
                out_pos: Optional[torch.Tensor] = None, out_mass: Optional[torch.Tensor] = None, stream=None):
    """out_src [B, mass_heads, n_keep] int32; out_len [B, mass_heads] int32;
    out_pos / out_mass [B, mass_heads, n_keep], or the problem's pos / mass
    themselves."""
    ref, device, (ss, sl) = p.desc()
    ps = _out(out_src, "out_src", ss, torch.int32)
    pl = None if out_len is None else _out(out_len, "out_len", sl, torch.int32)
    ld, pp, pm = ss[2], None, None
    if out_pos is not None or out_mass is not None:
        wide = (out_pos if out_pos is not None else out_mass).shape
        so = ss if wide == ss else torch.Size((ss[0], ss[1], wide[-1]))
        ld = so[2]
        _need(ld >= ss[2], "out_pos and out_mass: rows shorter than n_keep")
        if out_pos is not None:
            pp = _out(out_pos, "out_pos", so, torch.int32)
        if out_mass is not None:
            pm = _out(out_mass, "out_mass", so, torch.float32)
    st = (_lib or lib()).cache_evict(ref, ps, pl, pp, pm, ld,
                                     _current_raw_stream(device) if stream is None else stream.cuda_stream)
    if st:
        _check(st)
    return out_src, out_len, out_pos, out_mass
