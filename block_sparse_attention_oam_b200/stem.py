"""Thin binding of libstem (include/stem.h): ctypes, and for the operators that run once per
layer and token (stem_decode, stem_evict) a native module, csrc/stem_binding.cpp.

Argument marshalling only: torch tensors provide device memory and the current
CUDA stream; every step of the path runs in libstem's CUDA kernels.  There is no
fallback: if the library is missing, every call raises.

A call runs on `stream`, or on the current stream where none is given; its arguments have to be
ready there, and to live until it has run.  What its caller leaves out (outputs, a workspace) is
allocated on that stream too.
A workspace that was left out is gone when the call returns, and with it the status of the call:
pass one to read it with query_status.
"""
from __future__ import annotations

import ctypes
import dataclasses
import importlib.util
import os
import re
from typing import Optional, Sequence

import numpy as np
import torch

from . import build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libstem.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "stem.h")

STEM_OK, STEM_ERR_INVALID, STEM_ERR_UNSUPPORTED, STEM_ERR_WORKSPACE, STEM_ERR_CUDA, STEM_ERR_TIMEOUT, STEM_ERR_BOUNDS = range(7)
DT_BF16, DT_FP8 = 0, 1
PAGE_SIZE = 64


class StemError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libstem status {status}: {message}")
        self.status = status


class _Problem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("block_size", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("q_scale", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("beta", ctypes.c_float),
        ("keep", ctypes.c_double),
        ("mu", ctypes.c_double),
        ("shared_lists", ctypes.c_int),
    ]


class _Paged(ctypes.Structure):
    _fields_ = [
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("page_size", ctypes.c_int),
        ("max_pages_per_seq", ctypes.c_int),
        ("num_slots", ctypes.c_int),
    ]


class _Decode(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("q_len", ctypes.c_int),
        ("num_q_heads", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("q_scale", ctypes.c_float),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("softmax_scale", ctypes.c_float),
        ("max_kv_len", ctypes.c_int),
        ("prefix_len", ctypes.c_int),
        ("collect_weights", ctypes.c_int),
    ]


class _Evict(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int),
        ("num_kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("max_kv_len", ctypes.c_int),
        ("budget", ctypes.c_int),
        ("sink", ctypes.c_int),
        ("recent", ctypes.c_int),
    ]


class _Sizes(ctypes.Structure):
    _fields_ = [
        ("num_rows", ctypes.c_int64),
        ("scores_per_head", ctypes.c_int64),
        ("nnz_per_head", ctypes.c_int64),
        ("total_tokens", ctypes.c_int64),
        ("workspace_bytes", ctypes.c_size_t),
        ("list_heads", ctypes.c_int64),
    ]


_lib = None
_P = ctypes.c_void_p


def lib() -> ctypes.CDLL:
    """Load libstem.so (built in-tree by build.py).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_oam_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    pp = ctypes.POINTER(_Problem)
    pg = ctypes.POINTER(_Paged)
    sig = {
        "stem_query_sizes": ([pp, ctypes.POINTER(_Sizes)], ctypes.c_int),
        "stem_workspace_size": ([pp], ctypes.c_size_t),
        "stem_tpd_plan": ([ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.POINTER(ctypes.c_double),
                           ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
        "stem_score": ([pp, _P, _P, _P, pg, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "stem_select": ([pp, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "stem_score_select": ([pp, _P, _P, _P, pg, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "bsa_prefill": ([pp, _P, _P, _P, pg, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "bsa_dense_prefill": ([pp, _P, _P, _P, pg, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "stem_attention": ([pp, _P, _P, _P, pg, _P, _P, _P, _P, _P, ctypes.c_size_t, _P], ctypes.c_int),
        "stem_attention_noalloc": ([pp, _P, _P, _P, pg, _P, _P, _P, _P, _P, _P], ctypes.c_int),
        "stem_attention_host": ([pp, _P, _P, _P, _P, _P, _P, pg, _P, _P, _P, _P, _P, ctypes.c_int, _P,
                                 ctypes.c_size_t, _P], ctypes.c_int),
        "stem_decode_workspace_size": ([ctypes.POINTER(_Decode)], ctypes.c_size_t),
        "stem_decode": ([ctypes.POINTER(_Decode), _P, pg, _P, _P, _P, _P, ctypes.c_int64, _P, _P, _P, ctypes.c_size_t,
                         _P], ctypes.c_int),
        "stem_evict_workspace_size": ([ctypes.POINTER(_Evict)], ctypes.c_size_t),
        "stem_evict": ([ctypes.POINTER(_Evict), pg, _P, _P, ctypes.c_int64, pg, _P, _P, ctypes.c_int64, _P, _P,
                        ctypes.c_size_t, _P], ctypes.c_int),
        "stem_query_status": ([_P, _P], ctypes.c_int),
        "stem_reset_status": ([_P, _P], ctypes.c_int),
        "stem_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "stem_last_error": ([], ctypes.c_char_p),
        "stem_debug_inject": ([ctypes.c_int], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def header_functions() -> list:
    """Names of the functions include/stem.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*STEM_API\s+(?:const\s+)?[A-Za-z_][\w]*\s*\*?\s+\**([a-z_][a-z0-9_]*)\s*\(", text, flags=re.M)


def _check(status: int) -> None:
    if status != STEM_OK:
        msg = lib().stem_last_error().decode()
        raise StemError(status, msg or lib().stem_status_string(status).decode())


@dataclasses.dataclass
class Problem:
    cu_seqlens: Sequence[int]
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    block_size: int
    dtype: str = "bf16"
    q_scale: float = 1.0
    k_scale: float = 1.0
    v_scale: float = 1.0
    softmax_scale: float = 0.0
    beta: float = 0.2
    keep: float = 0.25
    mu: float = 0.7
    shared_lists: bool = False   # one selection per KV group (an extension, not in the pages)

    def __post_init__(self):
        self._cu = np.ascontiguousarray(np.asarray(self.cu_seqlens, dtype=np.int32))
        self._c = _Problem(len(self._cu) - 1, self._cu.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                           self.num_q_heads, self.num_kv_heads, self.head_dim, self.block_size,
                           DT_FP8 if self.dtype == "fp8_e4m3" else DT_BF16,
                           self.q_scale, self.k_scale, self.v_scale, self.softmax_scale, self.beta,
                           self.keep, self.mu, 1 if self.shared_lists else 0)

    @property
    def c(self):
        return ctypes.byref(self._c)

    def sizes(self) -> dict:
        s = _Sizes()
        _check(lib().stem_query_sizes(self.c, ctypes.byref(s)))
        return dict(num_rows=s.num_rows, scores_per_head=s.scores_per_head, nnz_per_head=s.nnz_per_head,
                    total_tokens=s.total_tokens, workspace_bytes=s.workspace_bytes, list_heads=s.list_heads)


@dataclasses.dataclass
class PagedKV:
    k_cache: torch.Tensor       # [num_slots, 64, Hkv, d]
    v_cache: torch.Tensor
    block_table: torch.Tensor   # int32 [num_seqs, max_pages] on the device

    def c(self):
        return ctypes.byref(_Paged(self.k_cache.data_ptr(), self.v_cache.data_ptr(), self.block_table.data_ptr(),
                                   PAGE_SIZE, self.block_table.shape[1], self.k_cache.shape[0]))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("libstem takes dense row-major tensors; got a non-contiguous one")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _allocate(device, stream, make) -> torch.Tensor:
    """make(), a new tensor on `device`, in the order of the call's stream: a workspace's zeroing
    goes before the kernels, and what is freed when the call returns is used again behind them."""
    if stream is None:
        return make()
    if stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    with torch.cuda.stream(stream):
        return make()


def _output(device, stream, shape, dtype) -> torch.Tensor:
    """An output that the caller left out.  Its current stream may read it and let go of it there."""
    t = _allocate(device, stream, lambda: torch.empty(shape, dtype=dtype, device=device))
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _workspace(prob: Problem, device, ws, stream):
    return _allocate(device, stream, lambda: workspace(prob, device)) if ws is None else ws


def _paged(paged: Optional[PagedKV]):
    return None if paged is None else paged.c()


def tpd_plan(n_blocks: int, keep: float, mu: float):
    r = ctypes.c_double()
    t = ctypes.c_int64()
    _check(lib().stem_tpd_plan(n_blocks, keep, mu, ctypes.byref(r), ctypes.byref(t)))
    return r.value, t.value


def workspace(prob: Problem, device="cuda") -> torch.Tensor:
    n = prob.sizes()["workspace_bytes"]
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    return ws


def stem_score(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, scores=None, ws=None, stream=None):
    sz = prob.sizes()
    if scores is None:
        scores = _output(q.device, stream, (prob.num_q_heads, sz["scores_per_head"]), torch.float32)
    ws = _workspace(prob, q.device, ws, stream)
    _check(lib().stem_score(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(scores), _ptr(ws),
                            ws.numel(), _stream(stream)))
    return scores


def _lists(sz, dev, row_ptr, col_idx, stream):
    if row_ptr is None:
        row_ptr = _output(dev, stream, sz["num_rows"] + 1, torch.int32)
    if col_idx is None:
        col_idx = _output(dev, stream, (sz["list_heads"], sz["nnz_per_head"]), torch.int32)
    return row_ptr, col_idx


def stem_select(prob: Problem, scores, row_ptr=None, col_idx=None, ws=None, stream=None):
    sz = prob.sizes()
    dev = scores.device
    row_ptr, col_idx = _lists(sz, dev, row_ptr, col_idx, stream)
    ws = _workspace(prob, dev, ws, stream)
    _check(lib().stem_select(prob.c, _ptr(scores), _ptr(row_ptr), _ptr(col_idx), _ptr(ws), ws.numel(),
                             _stream(stream)))
    return row_ptr, col_idx


def stem_score_select(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, row_ptr=None, col_idx=None, ws=None,
                      stream=None):
    """Pool, score and select in one pass (no score matrix): returns (row_ptr, col_idx)."""
    sz = prob.sizes()
    dev = q.device
    row_ptr, col_idx = _lists(sz, dev, row_ptr, col_idx, stream)
    ws = _workspace(prob, dev, ws, stream)
    _check(lib().stem_score_select(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(row_ptr), _ptr(col_idx),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return row_ptr, col_idx


def _out(prob, q, out, stream=None):
    if out is None:
        out = _output(q.device, stream, (q.shape[0], prob.num_q_heads, prob.head_dim), torch.bfloat16)
    return out


def bsa_prefill(prob: Problem, q, k, v, row_ptr, col_idx, paged: Optional[PagedKV] = None, out=None, lse=None,
                ws=None, stream=None):
    out = _out(prob, q, out, stream)
    ws = _workspace(prob, q.device, ws, stream)
    _check(lib().bsa_prefill(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(row_ptr), _ptr(col_idx),
                             _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def bsa_dense_prefill(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, out=None, lse=None, ws=None,
                      stream=None):
    out = _out(prob, q, out, stream)
    ws = _workspace(prob, q.device, ws, stream)
    _check(lib().bsa_dense_prefill(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(out), _ptr(lse),
                                   _ptr(ws), ws.numel(), _stream(stream)))
    return out


def stem_attention(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, out=None, lse=None, row_ptr=None,
                   col_idx=None, ws=None, stream=None):
    out = _out(prob, q, out, stream)
    ws = _workspace(prob, q.device, ws, stream)
    _check(lib().stem_attention(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(out), _ptr(lse),
                                _ptr(row_ptr), _ptr(col_idx), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def capture_attention(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, out=None, lse=None, row_ptr=None,
                      col_idx=None, ws=None):
    """Capture one stem_attention call (pooling, scoring, selection, BSA: every kernel of
    the path) into a CUDA graph on these buffers.  `graph.replay()` re-runs the whole path
    on whatever the buffers hold at replay time, with one launch from the host.  The
    problem (sequence lengths, heads, knobs) is fixed by the capture.  Returns (graph, out); the
    buffers have to live as long as the graph, which holds the workspace (graph.workspace)."""
    out = _out(prob, q, out)
    ws = workspace(prob, q.device) if ws is None else ws
    side = torch.cuda.Stream(device=q.device)
    side.wait_stream(torch.cuda.current_stream(q.device))
    with torch.cuda.stream(side):  # one eager call first: kernel attributes and the budget plan
        stem_attention(prob, q, k, v, paged, out, lse, row_ptr, col_idx, ws)
    torch.cuda.current_stream(q.device).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stem_attention(prob, q, k, v, paged, out, lse, row_ptr, col_idx, ws)
    graph.workspace = ws  # every replay writes it
    return graph, out


def stem_attention_host(prob: Problem, q_host, k_host, v_host, q, k, v, paged: Optional[PagedKV] = None,
                        out_host=None, out=None, lse=None, row_ptr=None, col_idx=None, out_groups: int = 0, ws=None,
                        stream=None):
    """The whole path from host tensors: q_host / k_host / v_host (CPU, ideally pinned)
    go to the device and O comes back into out_host (CPU bf16 [T, Hq, d]), one group of
    kv-heads at a time, the copies of each group overlapping the work of the others.
    q / k / v / out (a paged cache: paged.k_cache / paged.v_cache) are device scratch
    of the full sizes, overwritten with the inputs staged group by group.  Returns
    out_host; the work is asynchronous on `stream` (synchronise before reading it)."""
    out = _out(prob, q, out, stream)
    if out_host is None:
        out_host = torch.empty(tuple(out.shape), dtype=torch.bfloat16, pin_memory=True)
    for t, name in ((q_host, "q_host"), (k_host, "k_host"), (v_host, "v_host"), (out_host, "out_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    ws = _workspace(prob, q.device, ws, stream)
    _check(lib().stem_attention_host(prob.c, _ptr(q_host), _ptr(k_host), _ptr(v_host), _ptr(q), _ptr(k), _ptr(v),
                                     _paged(paged), _ptr(out_host), _ptr(out), _ptr(lse), _ptr(row_ptr),
                                     _ptr(col_idx), int(out_groups), _ptr(ws), ws.numel(), _stream(stream)))
    return out_host


def stem_attention_noalloc(prob: Problem, q, k, v, paged: Optional[PagedKV] = None, out=None, lse=None,
                           row_ptr=None, col_idx=None, status=None, stream=None):
    """stem_attention with the library's static scratch instead of a workspace
    (for callers that cannot allocate device memory).  `status`: optional device
    int32 tensor of one element that receives the call's device status word."""
    out = _out(prob, q, out, stream)
    _check(lib().stem_attention_noalloc(prob.c, _ptr(q), _ptr(k), _ptr(v), _paged(paged), _ptr(out), _ptr(lse),
                                        _ptr(row_ptr), _ptr(col_idx), _ptr(status), _stream(stream)))
    return out


@dataclasses.dataclass(frozen=True)
class Decode:
    """One decoding step: the newest q_len tokens of num_seqs sequences over a paged cache
    (stem_decode_t).  Not to be changed: dataclasses.replace makes one of other numbers (the scale
    of a step's queries, say)."""
    num_seqs: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int
    max_kv_len: int
    q_len: int = 1
    dtype: str = "bf16"
    q_scale: float = 1.0
    k_scale: float = 1.0
    v_scale: float = 1.0
    softmax_scale: float = 0.0
    prefix_len: int = 0          # tokens of a prefix that all sequences share
    weights: bool = False        # also add up the softmax weights of every cached token

    def __post_init__(self):
        c = _Decode(self.num_seqs, self.q_len, self.num_q_heads, self.num_kv_heads, self.head_dim,
                    _dtype_code(self.dtype), self.q_scale, self.k_scale, self.v_scale, self.softmax_scale,
                    self.max_kv_len, self.prefix_len, 1 if self.weights else 0)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_torch", _TORCH_DTYPES[self.dtype])

    @property
    def c(self):
        return ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        n = lib().stem_decode_workspace_size(self.c)
        if n == 0:
            raise StemError(STEM_ERR_INVALID, lib().stem_last_error().decode())
        return n


_TORCH_DTYPES = {"bf16": torch.bfloat16, "fp8_e4m3": torch.float8_e4m3fn}


def _dtype_code(name: str) -> int:
    if name not in _TORCH_DTYPES:
        raise ValueError(f"dtype {name!r} (supported: {', '.join(_TORCH_DTYPES)})")
    return DT_FP8 if name == "fp8_e4m3" else DT_BF16


def _tensor(name: str, t, shape, dtype, device):
    """Address of a dense tensor of this shape (None: any length), type and device."""
    if t.dtype is dtype and t.device == device and t.is_contiguous():
        got = t.shape
        if got == shape or (len(got) == len(shape) and all(w is None or w == g for w, g in zip(shape, got))):
            return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}; got "
                     f"{t.dtype} {tuple(t.shape)} on {t.device}, contiguous: {t.is_contiguous()}")


def _pages(name: str, c: PagedKV, num_seqs: int, Hkv: int, d: int, dtype, device):
    k, v, table = c.k_cache, c.v_cache, c.block_table
    slots, width = k.shape[0], table.shape[-1]
    shape = (slots, PAGE_SIZE, Hkv, d)
    return _Paged(_tensor(f"{name}.k_cache", k, shape, dtype, device), _tensor(f"{name}.v_cache", v, shape, dtype, device),
                  _tensor(f"{name}.block_table", table, (num_seqs, width), torch.int32, device), PAGE_SIZE, width, slots)


_native = None


def _binding():
    """The native module and libstem's entry points for it.  Raises if it is missing, or built
    for another torch or Python."""
    global _native
    if _native is None:
        path = build.BINDING
        if not os.path.exists(path) or not build.binding_fits():
            why = "built for another torch or Python" if os.path.exists(path) else "missing"
            raise RuntimeError(f"{path} is {why}: build it with `python -m block_sparse_attention_oam_b200.build`")
        spec = importlib.util.spec_from_file_location("stem_binding", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        entry = [ctypes.cast(getattr(lib(), f), _P).value for f in ("stem_decode", "stem_evict")]
        _native = (m.decode, entry[0], m.evict, entry[1])
    return _native


def decode_workspace(dec: Decode, device="cuda") -> torch.Tensor:
    return torch.zeros(dec.workspace_bytes(), dtype=torch.uint8, device=device)


def stem_decode(dec: Decode, q, cache: PagedKV, kv_lens, prefix_table=None, weights_in=None, weights_out=None,
                out=None, lse=None, ws=None, stream=None):
    """Attention of the newest tokens q [num_seqs * q_len, Hq, d] over the paged cache, of
    which sequence b holds kv_lens[b] tokens (device int32, the new ones among them), after
    the shared prefix of prefix_table's pages where dec.prefix_len > 0.  dec.weights:
    weights_out [num_seqs, Hkv, stride] = weights_in + the softmax weights of each token.
    Returns out (bf16); lse: float [Hq, num_seqs * q_len], written if given."""
    B, n, Hq, Hkv, d, dev = dec.num_seqs, dec.q_len, dec.num_q_heads, dec.num_kv_heads, dec.head_dim, q.device
    if dev.type != "cuda":
        raise ValueError("stem_decode takes CUDA tensors")
    if out is None:
        out = _output(dev, stream, (B * n, Hq, d), torch.bfloat16)
    if ws is None:
        ws = _allocate(dev, stream, lambda: decode_workspace(dec, dev))
    if dec.weights != (weights_out is not None) or (weights_in is not None and weights_out is None):
        raise ValueError("weights_out goes with Decode(weights=True), weights_in with weights_out")
    call, entry, _, _ = _native or _binding()
    status = call(entry, dec._c, q, cache.k_cache, cache.v_cache, cache.block_table, kv_lens, prefix_table, weights_in,
                  weights_out, out, lse, ws, None if stream is None else stream.cuda_stream)
    if status < 0:  # which tensor it is
        i32, f32, T = torch.int32, torch.float32, B * n
        _tensor("q", q, (T, Hq, d), dec._torch, dev)
        _pages("cache", cache, B, Hkv, d, dec._torch, dev)
        _tensor("kv_lens", kv_lens, (B,), i32, dev)
        if prefix_table is not None:
            _tensor("prefix_table", prefix_table, (-(-dec.prefix_len // PAGE_SIZE),), i32, dev)
        if weights_out is not None:
            _tensor("weights_out", weights_out, (B, Hkv, None), f32, dev)
        if weights_in is not None:
            _tensor("weights_in", weights_in, (B, Hkv, weights_out.shape[-1]), f32, dev)
        _tensor("out", out, (T, Hq, d), torch.bfloat16, dev)
        if lse is not None:
            _tensor("lse", lse, (Hq, T), f32, dev)
        _tensor("ws", ws, (None,), torch.uint8, dev)
        raise ValueError("an argument does not fit the problem")
    if status != STEM_OK:
        _check(status)
    return out


@dataclasses.dataclass(frozen=True)
class Evict:
    """One eviction: every (sequence, kv-head) cut to `budget` tokens (stem_evict_t).  Not to
    be changed, as Decode."""
    num_seqs: int
    num_kv_heads: int
    head_dim: int
    max_kv_len: int
    budget: int
    sink: int = 0
    recent: int = 0
    dtype: str = "bf16"

    def __post_init__(self):
        c = _Evict(self.num_seqs, self.num_kv_heads, self.head_dim, _dtype_code(self.dtype), self.max_kv_len,
                   self.budget, self.sink, self.recent)
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_torch", _TORCH_DTYPES[self.dtype])

    @property
    def c(self):
        return ctypes.byref(self._c)

    def workspace_bytes(self) -> int:
        n = lib().stem_evict_workspace_size(self.c)
        if n == 0:
            raise StemError(STEM_ERR_INVALID, lib().stem_last_error().decode())
        return n


def evict_workspace(ev: Evict, device="cuda") -> torch.Tensor:
    return torch.zeros(ev.workspace_bytes(), dtype=torch.uint8, device=device)


def stem_evict(ev: Evict, src: PagedKV, kv_lens, weights, dst: PagedKV, kv_lens_out=None, weights_out=None, keep=None,
               ws=None, stream=None):
    """Keep the first ev.sink, the last ev.recent and the heaviest other tokens of every
    (sequence, kv-head), ev.budget in all, by weights [num_seqs, Hkv, stride >= max_kv_len];
    their K/V rows go in order to dst's pages, which must be others than those read.
    Returns (keep, kv_lens_out): kept positions [num_seqs, Hkv, budget], -1 behind the last,
    and the new lengths; weights_out [num_seqs, Hkv, stride >= budget] is written if given."""
    B, Hkv, d, dev = ev.num_seqs, ev.num_kv_heads, ev.head_dim, weights.device
    if dev.type != "cuda":
        raise ValueError("stem_evict takes CUDA tensors")
    if kv_lens_out is None:
        kv_lens_out = _output(dev, stream, B, torch.int32)
    if keep is None:
        keep = _output(dev, stream, (B, Hkv, ev.budget), torch.int32)
    if ws is None:
        ws = _allocate(dev, stream, lambda: evict_workspace(ev, dev))
    _, _, call, entry = _native or _binding()
    status = call(entry, ev._c, weights, src.k_cache, src.v_cache, src.block_table, dst.k_cache, dst.v_cache,
                  dst.block_table, kv_lens, kv_lens_out, weights_out, keep, ws,
                  None if stream is None else stream.cuda_stream)
    if status < 0:  # which tensor it is
        i32, f32 = torch.int32, torch.float32
        _tensor("weights", weights, (B, Hkv, None), f32, dev)
        _pages("src", src, B, Hkv, d, ev._torch, dev)
        _pages("dst", dst, B, Hkv, d, ev._torch, dev)
        _tensor("kv_lens", kv_lens, (B,), i32, dev)
        _tensor("kv_lens_out", kv_lens_out, (B,), i32, dev)
        if weights_out is not None:
            _tensor("weights_out", weights_out, (B, Hkv, None), f32, dev)
        _tensor("keep", keep, (B, Hkv, ev.budget), i32, dev)
        _tensor("ws", ws, (None,), torch.uint8, dev)
        raise ValueError("an argument does not fit the problem")
    if status != STEM_OK:
        _check(status)
    return keep, kv_lens_out


def debug_inject(mode: int) -> None:
    """Failure-detection test hook: mode 1 makes the next BSA launch stall one CTA
    until its bounded wait reports STEM_ERR_TIMEOUT."""
    _check(lib().stem_debug_inject(mode))


def query_status(ws, stream=None) -> int:
    """Synchronise, read and clear the device status word; raises on a device error."""
    st = lib().stem_query_status(_ptr(ws), _stream(stream))
    _check(st)
    return st


def problem_for(wl, inputs=None, keep=None) -> Problem:
    """Problem description of a workload (workloads.Workload) and its inputs."""
    cu = np.zeros(len(wl.seqlens) + 1, dtype=np.int32)
    cu[1:] = np.cumsum(wl.seqlens)
    kw = {}
    if inputs is not None and wl.dtype == "fp8_e4m3":
        kw = dict(q_scale=inputs.q_scale, k_scale=inputs.k_scale, v_scale=inputs.v_scale)
    return Problem(cu, wl.num_q_heads, wl.num_kv_heads, wl.head_dim, wl.block, wl.dtype, beta=wl.beta,
                   keep=wl.keep if keep is None else keep, mu=wl.mu, shared_lists=wl.shared_lists, **kw)
