"""Python binding of the fpx C ABI (``include/fpx.h``): dynamic block-sparse pooled prefill
attention on B200.

Argument marshalling only: PyTorch supplies device memory and the current CUDA stream; every
step of the path (pooling, scoring, thresholding, CSR compression, sparse attention) runs in the
CUDA kernels of ``libfpx.so``.  There is no CPU fallback: if the library is missing, ``load()``
raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfpx.so")

F32, BF16, E4M3 = 0, 1, 2
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3}

STATUS = {0: "ok", -1: "invalid argument", -2: "unsupported", -3: "misaligned pointer",
          -4: "capacity too small", -5: "CUDA error", -6: "device-side wait timed out",
          -7: "malformed device input"}

# every symbol include/fpx.h declares
EXPORTS = ("fpx_num_blocks", "fpx_scores_elems", "fpx_rows", "fpx_max_nnz", "fpx_workspace_bytes",
           "fpx_clear_status", "fpx_query_status", "fpx_status_string", "fpx_block_scores",
           "fpx_select", "fpx_sparse_prefill", "fpx_attention_path", "fpx_select_noalloc",
           "fpx_select_noalloc_max_bytes", "fpx_diag_bounded_wait", "fpx_block_scores_paged",
           "fpx_sparse_prefill_paged", "fpx_block_scores_rescue", "fpx_select_rescue",
           "fpx_diag_exp2", "fpx_pattern_words", "fpx_vs_workspace_bytes", "fpx_probe_patterns",
           "fpx_vs_select", "fpx_vs_prefill", "fpx_spans", "fpx_span_select", "fpx_span_prefill",
           "fpx_page_workspace_bytes", "fpx_page_resize", "fpx_kv_append",
           "fpx_decode_workspace_bytes", "fpx_decode")


class FpxError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: fpx status {code} ({STATUS.get(code, 'unknown')})")
        self.code = code


class Problem(ctypes.Structure):
    """Mirror of ``fpx_problem``."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("cu_seqlens_d", ctypes.c_void_p),
                ("cu_seqlens_h", ctypes.c_void_p), ("total_tokens", ctypes.c_int32),
                ("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("block", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("q_scale_d", ctypes.c_void_p), ("k_scale_d", ctypes.c_void_p),
                ("v_scale_d", ctypes.c_void_p), ("softmax_scale", ctypes.c_float)]


class PagedKV(ctypes.Structure):
    """Mirror of ``fpx_paged_kv``."""
    _fields_ = [("block_table_d", ctypes.c_void_p), ("pages_per_seq", ctypes.c_int32),
                ("num_pages", ctypes.c_int32)]


class ScoreRule(ctypes.Structure):
    """Mirror of ``fpx_score_rule``."""
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes_d", ctypes.c_void_p), ("key_lo_d", ctypes.c_void_p),
                ("key_hi_d", ctypes.c_void_p)]


class DecodeProblem(ctypes.Structure):
    """Mirror of ``fpx_decode_problem``."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("q_len", ctypes.c_int32), ("hq", ctypes.c_int32),
                ("hkv", ctypes.c_int32), ("d", ctypes.c_int32), ("page", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("softmax_scale", ctypes.c_float),
                ("k_scale_d", ctypes.c_void_p), ("v_scale_d", ctypes.c_void_p),
                ("ctx_lens_d", ctypes.c_void_p), ("block_table_d", ctypes.c_void_p),
                ("pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("num_groups", ctypes.c_int32), ("group_ptr_d", ctypes.c_void_p),
                ("prefix_pages_d", ctypes.c_void_p)]


def paged_kv(block_table: torch.Tensor, num_pages: int) -> PagedKV:
    """Describes a page table: device int32 [num_seqs, pages_per_seq] of page indices."""
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous():
        raise ValueError("block_table must be a contiguous int32 [num_seqs, pages_per_seq] tensor")
    kv = PagedKV(block_table.data_ptr(), block_table.shape[1], int(num_pages))
    kv._keep = block_table  # the table must outlive the calls that use it
    return kv


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libfpx.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m dynamic_block_sparse_pooled_b200.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER(Problem)
    vp, sz, i32, i64, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, \
        ctypes.c_float
    for name in ("fpx_num_blocks", "fpx_scores_elems", "fpx_rows", "fpx_max_nnz"):
        getattr(lib, name).argtypes = [P]
        getattr(lib, name).restype = sz
    lib.fpx_workspace_bytes.argtypes = [P, ctypes.c_int]
    lib.fpx_workspace_bytes.restype = sz
    lib.fpx_clear_status.argtypes = [vp, vp]
    lib.fpx_clear_status.restype = ctypes.c_int
    lib.fpx_query_status.argtypes = [vp, vp]
    lib.fpx_query_status.restype = ctypes.c_int
    lib.fpx_status_string.argtypes = [ctypes.c_int]
    lib.fpx_status_string.restype = ctypes.c_char_p
    lib.fpx_attention_path.argtypes = [P]
    lib.fpx_attention_path.restype = ctypes.c_int
    lib.fpx_block_scores.argtypes = [P, vp, vp, vp, vp, sz, vp]
    lib.fpx_block_scores.restype = ctypes.c_int
    lib.fpx_select.argtypes = [P, vp, f32, i32, i32, vp, vp, i64, vp, vp, sz, vp]
    lib.fpx_select.restype = ctypes.c_int
    lib.fpx_sparse_prefill.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fpx_sparse_prefill.restype = ctypes.c_int
    lib.fpx_select_noalloc.argtypes = [P, vp, f32, i32, i32, vp, vp, i64, vp, vp]
    lib.fpx_select_noalloc.restype = ctypes.c_int
    lib.fpx_select_noalloc_max_bytes.argtypes = []
    lib.fpx_select_noalloc_max_bytes.restype = sz
    lib.fpx_diag_bounded_wait.argtypes = [vp, ctypes.c_uint64, vp]
    lib.fpx_diag_bounded_wait.restype = ctypes.c_int
    lib.fpx_diag_exp2.argtypes = [vp, vp, i64, vp]
    lib.fpx_diag_exp2.restype = ctypes.c_int
    lib.fpx_pattern_words.argtypes = [P]
    lib.fpx_pattern_words.restype = sz
    lib.fpx_vs_workspace_bytes.argtypes = [P, i32]
    lib.fpx_vs_workspace_bytes.restype = sz
    lib.fpx_probe_patterns.argtypes = [P, vp, vp, i32, f32, f32, vp, vp, vp, sz, vp]
    lib.fpx_probe_patterns.restype = ctypes.c_int
    lib.fpx_vs_select.argtypes = [P, vp, vp, vp, vp, i64, vp, vp, sz, vp]
    lib.fpx_vs_select.restype = ctypes.c_int
    lib.fpx_vs_prefill.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fpx_vs_prefill.restype = ctypes.c_int
    K = ctypes.POINTER(PagedKV)
    lib.fpx_block_scores_paged.argtypes = [P, vp, vp, K, vp, vp, sz, vp]
    lib.fpx_block_scores_paged.restype = ctypes.c_int
    lib.fpx_sparse_prefill_paged.argtypes = [P, vp, vp, vp, K, vp, vp, vp, vp, vp, sz, vp]
    lib.fpx_sparse_prefill_paged.restype = ctypes.c_int
    lib.fpx_block_scores_rescue.argtypes = [P, vp, vp, K, vp, vp, vp, vp, sz, vp]
    lib.fpx_block_scores_rescue.restype = ctypes.c_int
    lib.fpx_select_rescue.argtypes = [P, vp, vp, vp, f32, f32, i32, i32, vp, vp, i64, vp, vp, sz,
                                      vp]
    lib.fpx_select_rescue.restype = ctypes.c_int
    RU = ctypes.POINTER(ScoreRule)
    D = ctypes.POINTER(DecodeProblem)
    lib.fpx_spans.argtypes = [P, i32, vp, vp, vp, vp, vp]
    lib.fpx_spans.restype = ctypes.c_int
    lib.fpx_span_select.argtypes = [P, RU, vp, vp, i64, vp, vp, sz, vp]
    lib.fpx_span_select.restype = ctypes.c_int
    lib.fpx_span_prefill.argtypes = [P, vp, vp, vp, K, RU, vp, vp, vp, vp, vp, sz, vp]
    lib.fpx_span_prefill.restype = ctypes.c_int
    lib.fpx_page_workspace_bytes.argtypes = [i32]
    lib.fpx_page_workspace_bytes.restype = sz
    lib.fpx_page_resize.argtypes = [i32, i32, i32, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                    i32, vp, sz, vp]
    lib.fpx_page_resize.restype = ctypes.c_int
    lib.fpx_kv_append.argtypes = [ctypes.c_int, i32, i32, i32, vp, i64, vp, i64, vp, vp, vp, i32,
                                  vp, vp, vp, sz, vp]
    lib.fpx_kv_append.restype = ctypes.c_int
    lib.fpx_decode_workspace_bytes.argtypes = [D]
    lib.fpx_decode_workspace_bytes.restype = sz
    lib.fpx_decode.argtypes = [D, vp, vp, vp, RU, vp, vp, vp, sz, vp]
    lib.fpx_decode.restype = ctypes.c_int
    _lib = lib
    return lib


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def check(code: int, where: str) -> None:
    if code != 0:
        raise FpxError(code, where)


@dataclass
class Prefill:
    """One prefill problem bound to device tensors (keeps the marshalled struct alive)."""
    struct: Problem
    cu_d: Optional[torch.Tensor]
    cu_h: Optional[np.ndarray]
    scales: tuple
    nb: int
    rows: int
    tri: int

    @property
    def ptr(self):
        return ctypes.byref(self.struct)


def problem(q: torch.Tensor, k: torch.Tensor, block: int,
            cu_seqlens: Optional[Sequence[int]] = None, softmax_scale: float = 0.0,
            q_scale: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
            v_scale: Optional[torch.Tensor] = None) -> Prefill:
    """Describes Q [T, Hq, D] / K [T, Hkv, D] (packed by cu_seqlens, host ints) to the library."""
    lib = load()
    t, hq, d = q.shape
    hkv = k.shape[1]
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    s = Problem()
    cu_h = cu_d = None
    if cu_seqlens is not None:
        cu_h = np.ascontiguousarray(np.asarray(cu_seqlens, dtype=np.int32))
        cu_d = torch.from_numpy(cu_h).to(q.device)
        s.num_seqs = len(cu_h) - 1
        s.cu_seqlens_d = cu_d.data_ptr()
        s.cu_seqlens_h = cu_h.ctypes.data
    else:
        s.num_seqs = 1
    s.total_tokens, s.hq, s.hkv, s.d, s.block = t, hq, hkv, d, block
    s.dtype = _DTYPES[q.dtype]
    scales = (q_scale, k_scale, v_scale)
    if s.dtype == E4M3:
        s.q_scale_d, s.k_scale_d, s.v_scale_d = (x.data_ptr() for x in scales)
    s.softmax_scale = softmax_scale
    ref = ctypes.byref(s)
    nb, rows, tri = lib.fpx_num_blocks(ref), lib.fpx_rows(ref), lib.fpx_scores_elems(ref) // hq
    return Prefill(s, cu_d, cu_h, scales, nb, rows, tri)


def workspace(pf: Prefill, which: int = -1, device=None) -> torch.Tensor:
    """A zeroed device workspace (status block cleared) for stage `which` (-1: all stages)."""
    n = load().fpx_workspace_bytes(pf.ptr, which)
    if n == 0:
        raise FpxError(-1, "fpx_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def status(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the device-side status recorded in `ws`."""
    return load().fpx_query_status(_ptr(ws), _stream(stream))


def clear_status(ws: torch.Tensor, stream=None) -> None:
    check(load().fpx_clear_status(_ptr(ws), _stream(stream)), "fpx_clear_status")


def attention_path(pf: Prefill) -> int:
    return load().fpx_attention_path(pf.ptr)


def block_scores(pf: Prefill, q: torch.Tensor, k: torch.Tensor, ws: torch.Tensor,
                 scores: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fpx_block_scores -> fp32 [Hq * TRI] triangular-packed pooled block scores."""
    if scores is None:
        scores = torch.empty(pf.struct.hq * pf.tri, dtype=torch.float32, device=q.device)
    check(load().fpx_block_scores(pf.ptr, _ptr(q), _ptr(k), _ptr(scores), _ptr(ws), ws.numel(),
                                  _stream(stream)), "fpx_block_scores")
    return scores


def _check_csr_outputs(pf: Prefill, row_ptr: torch.Tensor, col_idx: torch.Tensor,
                       nnz: torch.Tensor, capacity: int) -> None:
    """The library writes up to `capacity` col_idx entries and R + 1 row_ptr entries: refuse
    buffers that cannot hold them (the device would write past the tensors)."""
    if row_ptr.dtype != torch.int32 or col_idx.dtype != torch.int32 or nnz.dtype != torch.int64:
        raise ValueError("row_ptr and col_idx must be int32 and nnz int64")
    if not (row_ptr.is_contiguous() and col_idx.is_contiguous()):
        raise ValueError("row_ptr and col_idx must be contiguous")
    if row_ptr.numel() < pf.rows + 1:
        raise ValueError(f"row_ptr holds {row_ptr.numel()} entries, needs {pf.rows + 1}")
    if capacity < 0 or capacity > col_idx.numel():
        raise ValueError(f"capacity {capacity} exceeds col_idx ({col_idx.numel()} entries)")
    if nnz.numel() < 1:
        raise ValueError("nnz needs one int64 entry")


def select(pf: Prefill, scores: torch.Tensor, alpha: float, ws: torch.Tensor,
           sink_blocks: int = 1, window_blocks: int = 1, row_ptr=None, col_idx=None,
           nnz=None, capacity: Optional[int] = None, stream=None):
    """fpx_select -> (row_ptr int32 [R+1], col_idx int32 [capacity], nnz int64 [1])."""
    dev = scores.device
    if row_ptr is None:
        row_ptr = torch.empty(pf.rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        cap = pf.struct.hq * pf.tri if capacity is None else capacity
        col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    cap = col_idx.numel() if capacity is None else capacity
    if nnz is None:
        nnz = torch.empty(1, dtype=torch.int64, device=dev)
    _check_csr_outputs(pf, row_ptr, col_idx, nnz, cap)
    check(load().fpx_select(pf.ptr, _ptr(scores), float(alpha), sink_blocks, window_blocks,
                            _ptr(row_ptr), _ptr(col_idx), cap, _ptr(nnz), _ptr(ws), ws.numel(),
                            _stream(stream)), "fpx_select")
    return row_ptr, col_idx, nnz


def select_noalloc(pf: Prefill, scores: torch.Tensor, alpha: float, sink_blocks: int = 1,
                   window_blocks: int = 1, row_ptr=None, col_idx=None, nnz=None,
                   capacity: Optional[int] = None, stream=None):
    """fpx_select_noalloc: fpx_select for callers that cannot provide a workspace (the scratch
    is a fixed device array inside the library; concurrent calls on one device race on it)."""
    dev = scores.device
    if row_ptr is None:
        row_ptr = torch.empty(pf.rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        cap = pf.struct.hq * pf.tri if capacity is None else capacity
        col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    cap = col_idx.numel() if capacity is None else capacity
    if nnz is None:
        nnz = torch.empty(1, dtype=torch.int64, device=dev)
    _check_csr_outputs(pf, row_ptr, col_idx, nnz, cap)
    check(load().fpx_select_noalloc(pf.ptr, _ptr(scores), float(alpha), sink_blocks,
                                    window_blocks, _ptr(row_ptr), _ptr(col_idx), cap, _ptr(nnz),
                                    _stream(stream)), "fpx_select_noalloc")
    return row_ptr, col_idx, nnz


def sparse_prefill(pf: Prefill, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   row_ptr: torch.Tensor, col_idx: torch.Tensor, ws: torch.Tensor,
                   o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   want_lse: bool = True, stream=None):
    """fpx_sparse_prefill -> (O [T, Hq, D] (bf16, fp32 for fp32 inputs), LSE fp32 [Hq, T])."""
    if o is None:
        odt = torch.float32 if q.dtype == torch.float32 else torch.bfloat16
        o = torch.empty(q.shape, dtype=odt, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    check(load().fpx_sparse_prefill(pf.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(row_ptr),
                                    _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                    _stream(stream)), "fpx_sparse_prefill")
    return o, lse


def block_scores_paged(pf: Prefill, q: torch.Tensor, k_cache: torch.Tensor, kv: PagedKV,
                       ws: torch.Tensor, scores: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """fpx_block_scores_paged: K from the paged cache [num_pages, block, Hkv, D]."""
    if scores is None:
        scores = torch.empty(pf.struct.hq * pf.tri, dtype=torch.float32, device=q.device)
    check(load().fpx_block_scores_paged(pf.ptr, _ptr(q), _ptr(k_cache), ctypes.byref(kv),
                                        _ptr(scores), _ptr(ws), ws.numel(), _stream(stream)),
          "fpx_block_scores_paged")
    return scores


def sparse_prefill_paged(pf: Prefill, q: torch.Tensor, k_cache: torch.Tensor,
                         v_cache: torch.Tensor, kv: PagedKV, row_ptr: torch.Tensor,
                         col_idx: torch.Tensor, ws: torch.Tensor,
                         o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         stream=None):
    """fpx_sparse_prefill_paged: K and V from the paged caches -> (O, LSE)."""
    if o is None:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    check(load().fpx_sparse_prefill_paged(pf.ptr, _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                          ctypes.byref(kv), _ptr(row_ptr), _ptr(col_idx),
                                          _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                                          _stream(stream)), "fpx_sparse_prefill_paged")
    return o, lse


def block_scores_rescue(pf: Prefill, q: torch.Tensor, k: torch.Tensor, ws: torch.Tensor,
                        kv: Optional[PagedKV] = None, stream=None):
    """fpx_block_scores_rescue -> (scores [Hq * TRI], qnorm [Hq, NB], radius [Hkv, NB])."""
    nb = pf.rows // pf.struct.hq
    scores = torch.empty(pf.struct.hq * pf.tri, dtype=torch.float32, device=q.device)
    qnorm = torch.empty((pf.struct.hq, nb), dtype=torch.float32, device=q.device)
    radius = torch.empty((pf.struct.hkv, nb), dtype=torch.float32, device=q.device)
    check(load().fpx_block_scores_rescue(pf.ptr, _ptr(q), _ptr(k),
                                         ctypes.byref(kv) if kv is not None else None,
                                         _ptr(scores), _ptr(qnorm), _ptr(radius), _ptr(ws),
                                         ws.numel(), _stream(stream)), "fpx_block_scores_rescue")
    return scores, qnorm, radius


def select_rescue(pf: Prefill, scores: torch.Tensor, qnorm: torch.Tensor, radius: torch.Tensor,
                  alpha: float, alpha_rescue: float, ws: torch.Tensor, sink_blocks: int = 1,
                  window_blocks: int = 1, stream=None):
    """fpx_select_rescue -> (row_ptr, col_idx, nnz) of the base OR rescue selection."""
    dev = scores.device
    row_ptr = torch.empty(pf.rows + 1, dtype=torch.int32, device=dev)
    cap = pf.struct.hq * pf.tri
    col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    nnz = torch.empty(1, dtype=torch.int64, device=dev)
    check(load().fpx_select_rescue(pf.ptr, _ptr(scores), _ptr(qnorm), _ptr(radius), float(alpha),
                                   float(alpha_rescue), sink_blocks, window_blocks, _ptr(row_ptr),
                                   _ptr(col_idx), cap, _ptr(nnz), _ptr(ws), ws.numel(),
                                   _stream(stream)), "fpx_select_rescue")
    return row_ptr, col_idx, nnz


def prefill(q, k, v, block: int, alpha: float, cu_seqlens=None, sink_blocks: int = 1,
            window_blocks: int = 1, softmax_scale: float = 0.0, q_scale=None, k_scale=None,
            v_scale=None, stream=None) -> dict:
    """The whole path on one stream: scores -> CSR -> O, LSE.  Raises on any recorded error."""
    with torch.cuda.stream(stream):  # the workspace's zeros and the outputs are that stream's too
        pf = problem(q, k, block, cu_seqlens, softmax_scale, q_scale, k_scale, v_scale)
        ws = workspace(pf, -1, q.device)
        scores = block_scores(pf, q, k, ws, stream=stream)
        row_ptr, col_idx, nnz = select(pf, scores, alpha, ws, sink_blocks, window_blocks,
                                       stream=stream)
        o, lse = sparse_prefill(pf, q, k, v, row_ptr, col_idx, ws, stream=stream)
        check(status(ws, stream), "device status")
    return dict(problem=pf, scores=scores, row_ptr=row_ptr, col_idx=col_idx, nnz=nnz, o=o,
                lse=lse)


# ---- query-probe vertical / slash path ------------------------------------------------------

def pattern_words(pf: Prefill) -> int:
    """uint32 words per head of the vertical / slash bitmasks (ceil(T / 32))."""
    return load().fpx_pattern_words(pf.ptr)


def vs_workspace(pf: Prefill, n_probe: int, device=None) -> torch.Tensor:
    """A zeroed workspace for fpx_probe_patterns, fpx_vs_select and fpx_vs_prefill."""
    n = load().fpx_vs_workspace_bytes(pf.ptr, int(n_probe))
    if n == 0:
        raise FpxError(-2, "fpx_vs_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def probe_patterns(pf: Prefill, q: torch.Tensor, k: torch.Tensor, n_probe: int, alpha_v: float,
                   alpha_s: float, ws: torch.Tensor, vert=None, slash=None, stream=None):
    """fpx_probe_patterns -> (vert_bits, slash_bits): int32 [Hq, words] holding the uint32
    bitmasks (bit cu[s] + x of head h: key token / offset x of sequence s)."""
    shape = (pf.struct.hq, max(1, pattern_words(pf)))
    vert = torch.empty(shape, dtype=torch.int32, device=q.device) if vert is None else vert
    slash = torch.empty(shape, dtype=torch.int32, device=q.device) if slash is None else slash
    for t in (vert, slash):
        if t.dtype != torch.int32 or t.numel() < shape[0] * shape[1] or not t.is_contiguous():
            raise ValueError(f"bitmask must be a contiguous int32 tensor of {shape} words")
    check(load().fpx_probe_patterns(pf.ptr, _ptr(q), _ptr(k), int(n_probe), float(alpha_v),
                                    float(alpha_s), _ptr(vert), _ptr(slash), _ptr(ws), ws.numel(),
                                    _stream(stream)), "fpx_probe_patterns")
    return vert, slash


def vs_select(pf: Prefill, vert: torch.Tensor, slash: torch.Tensor, ws: torch.Tensor,
              row_ptr=None, col_idx=None, nnz=None, capacity: Optional[int] = None, stream=None):
    """fpx_vs_select -> (row_ptr, col_idx, nnz): key blocks that can hold an allowed key."""
    dev = vert.device
    if row_ptr is None:
        row_ptr = torch.empty(pf.rows + 1, dtype=torch.int32, device=dev)
    if col_idx is None:
        cap = pf.struct.hq * pf.tri if capacity is None else capacity
        col_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    cap = col_idx.numel() if capacity is None else capacity
    if nnz is None:
        nnz = torch.empty(1, dtype=torch.int64, device=dev)
    _check_csr_outputs(pf, row_ptr, col_idx, nnz, cap)
    check(load().fpx_vs_select(pf.ptr, _ptr(vert), _ptr(slash), _ptr(row_ptr), _ptr(col_idx), cap,
                               _ptr(nnz), _ptr(ws), ws.numel(), _stream(stream)), "fpx_vs_select")
    return row_ptr, col_idx, nnz


def vs_prefill(pf: Prefill, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
               vert: torch.Tensor, slash: torch.Tensor, row_ptr: torch.Tensor,
               col_idx: torch.Tensor, ws: torch.Tensor, o=None, lse=None, stream=None):
    """fpx_vs_prefill -> (O, LSE) under the vertical / slash token mask."""
    if o is None:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    check(load().fpx_vs_prefill(pf.ptr, _ptr(q), _ptr(k), _ptr(v), _ptr(vert), _ptr(slash),
                                _ptr(row_ptr), _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(ws),
                                ws.numel(), _stream(stream)), "fpx_vs_prefill")
    return o, lse


def vs_path(q, k, v, block: int, n_probe: int, alpha_v: float, alpha_s: float, cu_seqlens=None,
            softmax_scale: float = 0.0, q_scale=None, k_scale=None, v_scale=None,
            stream=None) -> dict:
    """The query-probe path on one stream: probes -> vertical / slash bitmasks -> candidate
    blocks -> masked attention.  Raises on any recorded device-side error."""
    with torch.cuda.stream(stream):  # the workspace's zeros and the outputs are that stream's too
        pf = problem(q, k, block, cu_seqlens, softmax_scale, q_scale, k_scale, v_scale)
        ws = vs_workspace(pf, n_probe, q.device)
        vert, slash = probe_patterns(pf, q, k, n_probe, alpha_v, alpha_s, ws, stream=stream)
        row_ptr, col_idx, nnz = vs_select(pf, vert, slash, ws, stream=stream)
        o, lse = vs_prefill(pf, q, k, v, vert, slash, row_ptr, col_idx, ws, stream=stream)
        check(status(ws, stream), "device status")
    return dict(problem=pf, vert=vert, slash=slash, row_ptr=row_ptr, col_idx=col_idx, nnz=nnz,
                o=o, lse=lse)


# ---- attention under a score rule -----------------------------------------------------------

def _expect(name: str, t: Optional[torch.Tensor], dtype, device: int = -2, numel: int = 0,
            shape=None) -> None:
    """Refuses a tensor that the device code would misread (None passes; device: its index)."""
    if t is None or (t.dtype is dtype and (device == -2 or t.get_device() == device) and
                     t.is_contiguous() and t.numel() >= numel and
                     (shape is None or t.shape == shape)):
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device != -2 and t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, expected device {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} holds {t.numel()} entries, needs {numel}")


def _call(name: str, device: int, stream, *args) -> None:
    """Calls entry point `name` with the stream as its last argument (default: the device's current
    one) and the device current.  Host tensors (device -1) are refused: a kernel would read their
    addresses."""
    if device < 0:
        raise ValueError(f"{name}: tensors must be on a GPU")
    fn = getattr(_lib or load(), name)
    handle = stream.cuda_stream if stream is not None else \
        torch._C._cuda_getCurrentRawStream(device)
    if torch._C._cuda_getDevice() == device:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            code = fn(*args, handle)
    if code != 0:
        raise FpxError(code, name)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a launch on `stream`: its memory belongs to that stream's pool."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def score_rule(softcap: float = 0.0, slopes: Optional[torch.Tensor] = None, window: int = 0,
               key_lo: Optional[torch.Tensor] = None,
               key_hi: Optional[torch.Tensor] = None) -> ScoreRule:
    """What a layer does to its scores: a tanh cap, a bias -slopes[h] * |i - j| (fp32 [Hq]), the
    last `window` positions only, and key spans (int32 [query tokens] each, as ``spans`` writes
    them; None: keys 0 .. i).  The tensors must live as long as the rule is used."""
    _expect("slopes", slopes, torch.float32)
    _expect("key_lo", key_lo, torch.int32)
    _expect("key_hi", key_hi, torch.int32)
    if (key_lo is None) != (key_hi is None):
        raise ValueError("key_lo and key_hi come together")
    r = ScoreRule(float(softcap), int(window), _ptr(slopes), _ptr(key_lo), _ptr(key_hi))
    r._keep = (slopes, key_lo, key_hi)
    return r


def _check_rule(rule: ScoreRule, hq: int, tokens: int, device: int) -> None:
    slopes, lo, hi = getattr(rule, "_keep", (None, None, None))
    _expect("slopes", slopes, torch.float32, device, hq)
    _expect("key_lo", lo, torch.int32, device, tokens)
    _expect("key_hi", hi, torch.int32, device, tokens)


def _check_problem(pf: Prefill, device: int) -> None:
    """The problem's own tensors (offsets, e4m3 scales) must lie where the call's do."""
    if pf.cu_d is not None and pf.cu_d.get_device() != device:
        _expect("cu_seqlens", pf.cu_d, torch.int32, device)
    if pf.struct.dtype == E4M3:
        for name, t in zip(("q_scale", "k_scale", "v_scale"), pf.scales):
            heads = pf.struct.hq if name == "q_scale" else pf.struct.hkv
            _expect(name, t, torch.float32, device, heads)


def spans(pf: Prefill, doc_cu: Optional[torch.Tensor] = None,
          prefix: Optional[torch.Tensor] = None, key_lo: Optional[torch.Tensor] = None,
          key_hi: Optional[torch.Tensor] = None, device=None, stream=None):
    """fpx_spans -> (key_lo, key_hi) int32 [T]: each document (doc_cu int32 [documents + 1] token
    offsets; None: each sequence) attends itself, causally but for its first prefix[document]
    tokens.  `device` is needed only where no tensor names one."""
    given = [t for t in (key_lo, key_hi, doc_cu, prefix, pf.cu_d) if t is not None]
    on = given[0].device if given else torch.device(device or "cuda")
    if on.type != "cuda":
        raise ValueError("fpx_spans: tensors must be on a GPU")
    dev = on.index if on.index is not None else torch.cuda.current_device()
    total = pf.struct.total_tokens
    docs = 0 if doc_cu is None else doc_cu.numel() - 1
    if doc_cu is not None and docs < 1:
        raise ValueError("doc_cu needs at least one document")
    _check_problem(pf, dev)
    _expect("doc_cu", doc_cu, torch.int32, dev)
    _expect("prefix", prefix, torch.int32, dev, docs if doc_cu is not None else pf.struct.num_seqs)
    key_lo = _empty(total, torch.int32, on, stream) if key_lo is None else key_lo
    key_hi = _empty(total, torch.int32, on, stream) if key_hi is None else key_hi
    _expect("key_lo", key_lo, torch.int32, dev, total)
    _expect("key_hi", key_hi, torch.int32, dev, total)
    _call("fpx_spans", dev, stream, pf.ptr, docs, _ptr(doc_cu), _ptr(prefix), _ptr(key_lo),
          _ptr(key_hi))
    return key_lo, key_hi


def span_capacity(pf: Prefill) -> int:
    """CSR entries that a rule can need at most: Hq * sum of (blocks of a sequence)^2, or as many as
    a call takes, 2^31 - 1.  (Selections that pass it are recorded as any that pass their capacity.)"""
    b = pf.struct.block
    lens = np.diff(pf.cu_h.astype(np.int64)) if pf.cu_h is not None else \
        np.array([pf.struct.total_tokens], dtype=np.int64)
    return min(int(pf.struct.hq * ((-(-lens // b)) ** 2).sum()), 2 ** 31 - 1)


def span_select(pf: Prefill, rule: ScoreRule, ws: torch.Tensor, row_ptr=None, col_idx=None,
                nnz=None, capacity: Optional[int] = None, stream=None):
    """fpx_span_select -> (row_ptr, col_idx, nnz): the key blocks that the rule's spans reach."""
    dev, index = ws.device, ws.get_device()
    _expect("ws", ws, torch.uint8, index)
    _check_problem(pf, index)
    _check_rule(rule, pf.struct.hq, pf.struct.total_tokens, index)
    if row_ptr is None:
        row_ptr = _empty(pf.rows + 1, torch.int32, dev, stream)
    if col_idx is None:
        if capacity is not None:
            cap = capacity
        else:  # without key spans no block lies above the diagonal
            cap = span_capacity(pf) if rule.key_lo_d else pf.struct.hq * pf.tri
        col_idx = _empty(max(cap, 1), torch.int32, dev, stream)
    cap = col_idx.numel() if capacity is None else capacity
    if nnz is None:
        nnz = _empty(1, torch.int64, dev, stream)
    _check_csr_outputs(pf, row_ptr, col_idx, nnz, cap)
    if not row_ptr.get_device() == col_idx.get_device() == nnz.get_device() == index:
        raise ValueError(f"row_ptr is on {row_ptr.device}, col_idx is on {col_idx.device} and nnz "
                         f"is on {nnz.device}, expected device {index}")
    _call("fpx_span_select", index, stream, pf.ptr, ctypes.byref(rule), _ptr(row_ptr),
          _ptr(col_idx), cap, _ptr(nnz), _ptr(ws), ws.numel())
    return row_ptr, col_idx, nnz


def span_prefill(pf: Prefill, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rule: ScoreRule,
                 row_ptr: torch.Tensor, col_idx: torch.Tensor, ws: torch.Tensor,
                 kv: Optional[PagedKV] = None, o: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """fpx_span_prefill -> (O, LSE): attention over the listed blocks under the rule.  K and V are
    packed, or with `kv` the page caches."""
    p, dev = pf.struct, q.get_device()
    _expect("q", q, q.dtype, dev, shape=(p.total_tokens, p.hq, p.d))
    rows = kv.num_pages * p.block if kv is not None else p.total_tokens
    for name, t in (("k", k), ("v", v)):
        _expect(name, t, q.dtype, dev)
        if t.numel() != rows * p.hkv * p.d:
            raise ValueError(f"{name} must hold {rows} rows of [{p.hkv}, {p.d}]")
    if _DTYPES[q.dtype] != p.dtype:
        raise TypeError(f"q is {q.dtype}, the problem was described with another type")
    _check_problem(pf, dev)
    if kv is not None:
        _expect("block_table", getattr(kv, "_keep", None), torch.int32, dev)
    _check_rule(rule, p.hq, p.total_tokens, dev)
    _expect("row_ptr", row_ptr, torch.int32, dev, pf.rows + 1)
    _expect("col_idx", col_idx, torch.int32, dev)
    odt = torch.float32 if q.dtype == torch.float32 else torch.bfloat16
    o = _empty(q.shape, odt, q.device, stream) if o is None else o
    if lse is None and want_lse:
        lse = _empty((p.hq, p.total_tokens), torch.float32, q.device, stream)
    _expect("o", o, odt, dev, shape=q.shape)
    _expect("lse", lse, torch.float32, dev, p.hq * p.total_tokens)
    _expect("ws", ws, torch.uint8, dev)
    _call("fpx_span_prefill", dev, stream, pf.ptr, _ptr(q), _ptr(k), _ptr(v),
          ctypes.byref(kv) if kv is not None else None, ctypes.byref(rule), _ptr(row_ptr),
          _ptr(col_idx), _ptr(o), _ptr(lse), _ptr(ws), ws.numel())
    return o, lse


def span_path(q, k, v, block: int, cu_seqlens=None, doc_cu=None, prefix=None, softcap: float = 0.0,
              slopes=None, window: int = 0, softmax_scale: float = 0.0, q_scale=None, k_scale=None,
              v_scale=None, stream=None) -> dict:
    """The whole path under a rule on one stream: spans -> blocks -> O, LSE.  Raises on any
    recorded error."""
    with torch.cuda.device(q.device):
        if stream is None:
            stream = torch.cuda.current_stream(q.device)
        with torch.cuda.stream(stream):  # the workspace's zeros and the offsets are that stream's too
            pf = problem(q, k, block, cu_seqlens, softmax_scale, q_scale, k_scale, v_scale)
            ws = workspace(pf, -1, q.device)
            lo, hi = spans(pf, doc_cu, prefix, device=q.device, stream=stream)
            rule = score_rule(softcap, slopes, window, lo, hi)
            row_ptr, col_idx, nnz = span_select(pf, rule, ws, stream=stream)
            o, lse = span_prefill(pf, q, k, v, rule, row_ptr, col_idx, ws, stream=stream)
            check(status(ws, stream), "device status")
    return dict(problem=pf, rule=rule, row_ptr=row_ptr, col_idx=col_idx, nnz=nnz, o=o, lse=lse)


# ---- paged cache and decode -----------------------------------------------------------------

def page_workspace(num_seqs: int, device=None) -> torch.Tensor:
    """A zeroed workspace for fpx_page_resize (up to num_seqs requests) and fpx_kv_append."""
    n = load().fpx_page_workspace_bytes(int(num_seqs))
    if n == 0:
        raise FpxError(-1, "fpx_page_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def page_resize(lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                free_pages: torch.Tensor, free_count: torch.Tensor, page: int, num_pages: int,
                token_capacity: int, ws: torch.Tensor, keep_pages=None, count_out=None,
                cu_new=None, slots=None, positions=None, stream=None):
    """fpx_page_resize: requests grow or shrink from lens to new_lens -> (cu_new int32 [S + 1],
    slots int32 [token_capacity], positions int32 [token_capacity]).  block_table, free_pages and
    the count (count_out, by default free_count itself) are updated."""
    dev, n = lens.get_device(), lens.numel()
    count_out = free_count if count_out is None else count_out
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table must be [num_seqs, pages_per_seq]")
    i32 = torch.int32
    _expect("lens", lens, i32, dev)
    _expect("new_lens", new_lens, i32, dev, n)
    _expect("keep_pages", keep_pages, i32, dev, n)
    _expect("block_table", block_table, i32, dev)
    _expect("free_pages", free_pages, i32, dev, num_pages)
    _expect("free_count", free_count, i32, dev, 1)
    _expect("count_out", count_out, i32, dev, 1)
    _expect("ws", ws, torch.uint8, dev)
    if cu_new is None:
        cu_new = _empty(n + 1, i32, lens.device, stream)
    else:
        _expect("cu_new", cu_new, i32, dev, n + 1)
    if slots is None:
        slots = _empty(token_capacity, i32, lens.device, stream)
    else:
        _expect("slots", slots, i32, dev, token_capacity)
    if positions is None:
        positions = _empty(token_capacity, i32, lens.device, stream)
    else:
        _expect("positions", positions, i32, dev, token_capacity)
    _call("fpx_page_resize", dev, stream, n, page, num_pages, lens.data_ptr(),
          new_lens.data_ptr(), _ptr(keep_pages), block_table.data_ptr(), block_table.shape[1],
          free_pages.data_ptr(), free_count.data_ptr(), count_out.data_ptr(), cu_new.data_ptr(),
          slots.data_ptr(), positions.data_ptr(), token_capacity, ws.data_ptr(), ws.numel())
    return cu_new, slots, positions


def _cache_rows(name: str, t: torch.Tensor, hkv: int, d: int, device: int) -> int:
    if t.dim() < 3 or t.shape[-1] != d or t.shape[-2] != hkv:
        raise ValueError(f"{name} must be [.., {hkv}, {d}], got {tuple(t.shape)}")
    _expect(name, t, t.dtype, device)
    return t.numel() // (hkv * d)


def kv_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
              v_cache: torch.Tensor, ws: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
              v_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """fpx_kv_append: rows k, v [n, Hkv, D] (each row contiguous; the rows may be strided, as slices
    of a projection's output are) into cache rows slots[n].  e4m3 caches take bf16 rows and the
    heads' scales (fp32 [Hkv])."""
    dev, (n, hkv, d) = k.get_device(), k.shape
    if k_cache.dtype not in _DTYPES:
        raise TypeError(f"unsupported cache type {k_cache.dtype}")
    src = torch.float32 if k_cache.dtype is torch.float32 else torch.bfloat16
    strides = []
    for name, t in (("k", k), ("v", v)):
        if t.dtype is not src or t.get_device() != dev or t.shape != k.shape:
            raise ValueError(f"{name} must be {src} {(n, hkv, d)} on device {dev}")
        step, head, one = t.stride()
        if n > 0 and (one != 1 or (hkv > 1 and head != d)):
            raise ValueError(f"a row of {name} must be contiguous")
        strides.append(step if n > 1 else hkv * d)
    rows = _cache_rows("k_cache", k_cache, hkv, d, dev)
    if _cache_rows("v_cache", v_cache, hkv, d, dev) != rows or v_cache.dtype is not k_cache.dtype:
        raise ValueError("k_cache and v_cache must have the same rows and type")
    _expect("slots", slots, torch.int32, dev, n)
    _expect("k_scale", k_scale, torch.float32, dev, hkv)
    _expect("v_scale", v_scale, torch.float32, dev, hkv)
    _expect("ws", ws, torch.uint8, dev)
    _call("fpx_kv_append", dev, stream, _DTYPES[k_cache.dtype], hkv, d, n, k.data_ptr(),
          strides[0], v.data_ptr(), strides[1], slots.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), rows, _ptr(k_scale), _ptr(v_scale), ws.data_ptr(), ws.numel())


@dataclass
class Decode:
    """One decode problem bound to device tensors (keeps them and the struct alive)."""
    struct: DecodeProblem
    keep: tuple
    q_shape: torch.Size
    q_dtype: torch.dtype
    device: torch.device

    @property
    def ptr(self):
        return ctypes.byref(self.struct)


def decode_problem(q: torch.Tensor, k_cache: torch.Tensor, ctx_lens: torch.Tensor,
                   block_table: torch.Tensor, q_len: int = 1, softmax_scale: float = 0.0,
                   k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                   group_ptr: Optional[torch.Tensor] = None,
                   prefix_pages: Optional[torch.Tensor] = None) -> Decode:
    """Describes Q [S * q_len, Hq, D] against caches [num_pages, page, Hkv, D] (page tables int32
    [S, pages_per_seq], lengths int32 [S]); group_ptr int32 [G + 1] and prefix_pages int32 [G] name
    runs of requests that share their first pages."""
    if k_cache.dtype not in _DTYPES:
        raise TypeError(f"unsupported cache type {k_cache.dtype}")
    if k_cache.dim() != 4 or q.dim() != 3:
        raise ValueError("k_cache must be [num_pages, page, Hkv, D] and q [tokens, Hq, D]")
    dev, n = q.get_device(), ctx_lens.numel()
    num_pages, page, hkv, d = k_cache.shape
    if q.shape[0] != n * q_len or q.shape[2] != d:
        raise ValueError(f"q must be [{n} * {q_len}, Hq, {d}], got {tuple(q.shape)}")
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError("block_table must be [num_seqs, pages_per_seq]")
    if (group_ptr is None) != (prefix_pages is None):
        raise ValueError("group_ptr and prefix_pages come together")
    groups = 0 if group_ptr is None else group_ptr.numel() - 1
    if group_ptr is not None and groups < 1:
        raise ValueError("group_ptr needs at least one group")
    for name, t, dt, need in (("ctx_lens", ctx_lens, torch.int32, n),
                              ("block_table", block_table, torch.int32, 0),
                              ("k_scale", k_scale, torch.float32, hkv),
                              ("v_scale", v_scale, torch.float32, hkv),
                              ("group_ptr", group_ptr, torch.int32, 0),
                              ("prefix_pages", prefix_pages, torch.int32, groups)):
        _expect(name, t, dt, dev, need)
    s = DecodeProblem(n, int(q_len), q.shape[1], hkv, d, page, _DTYPES[k_cache.dtype],
                      float(softmax_scale), _ptr(k_scale), _ptr(v_scale), _ptr(ctx_lens),
                      _ptr(block_table), block_table.shape[1], num_pages, groups, _ptr(group_ptr),
                      _ptr(prefix_pages))
    qdt = torch.float32 if k_cache.dtype == torch.float32 else torch.bfloat16
    return Decode(s, (ctx_lens, block_table, k_scale, v_scale, group_ptr, prefix_pages),
                  q.shape, qdt, q.device)


def decode_workspace(dp: Decode) -> torch.Tensor:
    """A zeroed workspace for fpx_decode."""
    n = load().fpx_decode_workspace_bytes(dp.ptr)
    if n == 0:
        raise FpxError(-2, "fpx_decode_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=dp.device)


def decode(dp: Decode, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
           ws: torch.Tensor, rule: Optional[ScoreRule] = None, o: Optional[torch.Tensor] = None,
           lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """fpx_decode -> (O [S * q_len, Hq, D], LSE fp32 [Hq, S * q_len])."""
    p, dev = dp.struct, dp.keep[0].get_device()
    tokens = dp.q_shape[0]
    _expect("q", q, dp.q_dtype, dev, shape=dp.q_shape)
    shape = (p.num_pages, p.page, p.hkv, p.d)
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if _DTYPES.get(t.dtype) != p.dtype:
            raise TypeError(f"{name} is {t.dtype}, the problem was described with another type")
        _expect(name, t, t.dtype, dev, shape=shape)
    if rule is not None:
        _check_rule(rule, p.hq, tokens, dev)
    if o is None:
        o = _empty(dp.q_shape, dp.q_dtype, dp.device, stream)
    else:
        _expect("o", o, dp.q_dtype, dev, shape=dp.q_shape)
    if lse is not None:
        _expect("lse", lse, torch.float32, dev, p.hq * tokens)
    elif want_lse:
        lse = _empty((p.hq, tokens), torch.float32, dp.device, stream)
    _expect("ws", ws, torch.uint8, dev)
    _call("fpx_decode", dev, stream, dp.ptr, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          ctypes.byref(rule) if rule is not None else None, o.data_ptr(), _ptr(lse),
          ws.data_ptr(), ws.numel())
    return o, lse
