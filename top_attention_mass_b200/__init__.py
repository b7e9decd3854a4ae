"""Python binding of libtam.so: the B200 attention-mass top-k path.

Thin ctypes marshalling over the C ABI declared in ``include/tam.h``; every
step of the path runs in the library's CUDA kernels.  PyTorch only provides
device memory (output tensors, the workspace) and the current CUDA stream.
There is no CPU path: if ``libtam.so`` has not been built, or there is no CUDA
device, every call raises.

Functions (same names as the C entry points, without the ``tam_`` prefix):

* ``mass_oracle_prefill``      passes 1-3 of the attention-mass top-k oracle
* ``attention_lse``            pass 1 alone (per-head log-sum-exp)
* ``mass_select``              pass 2 alone (mass + top-k support, given pass 1's lse)
* ``indexer_topk``             head-collapsed indexer support
* ``sparse_support_attention`` pass 3 alone (attention on a given support)
* ``dense_gqa_prefill``        dense causal GQA attention (comparator)
* ``mass_oracle_prefill_varlen``, ``dense_gqa_prefill_varlen``, ``indexer_topk_varlen``,
  ``sparse_support_attention_varlen``
                               the same over a packed batch of sequences
* ``kv_cache_write``, ``kv_cache_read``
                               rows of new tokens into the pages of a ``PagedKVCache`` (as they
                               are, or quantised to e4m3), and rows back out of them
* ``paged_gqa_attention``      causal GQA attention of a ``PagedBatch``'s new tokens over its pages

The paged calls take CUDA tensors.  Of the others, inputs may be CUDA tensors, or CPU tensors (ideally pinned): then they are
copied to ``device``, the call runs there, and the results come back to the CPU.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# TAM_LIBRARY=debug loads the debug-checks build (pass-2 stores checked against their
# extents; see tam.h, TAM_ERR_OVERFLOW) instead of the release library
LIB_PATH = os.path.join(_HERE, "libtam_debug.so" if os.environ.get("TAM_LIBRARY") == "debug"
                        else "libtam.so")

TAM_OK, TAM_ERR_INVALID_ARG, TAM_ERR_UNSUPPORTED, TAM_ERR_WORKSPACE = 0, 1, 2, 3
TAM_ERR_CUDA, TAM_ERR_TIMEOUT, TAM_ERR_OVERFLOW, TAM_ERR_PAGE = 4, 5, 6, 7
TAM_BF16, TAM_F32, TAM_E4M3 = 0, 1, 2

EXPORTED = (
    "tam_kv_cache_write", "tam_kv_cache_read", "tam_paged_attention_workspace",
    "tam_paged_gqa_attention",
    "tam_version", "tam_status_string", "tam_mass_oracle_workspace", "tam_mass_workspace_min",
    "tam_mass_oracle_prefill", "tam_attention_lse_workspace", "tam_attention_lse",
    "tam_mass_select_workspace", "tam_mass_select", "tam_mass_select_noalloc",
    "tam_indexer_workspace", "tam_indexer_workspace_min", "tam_indexer_topk",
    "tam_distill_kl_workspace", "tam_distill_kl_workspace_min", "tam_distill_kl",
    "tam_support_mass_curve", "tam_sparse_attention_workspace", "tam_sparse_support_attention",
    "tam_dense_workspace", "tam_dense_gqa_prefill", "tam_kernel_launches", "tam_check_status",
    "tam_mass_oracle_workspace_varlen", "tam_mass_oracle_prefill_varlen",
    "tam_dense_gqa_prefill_varlen", "tam_indexer_workspace_varlen", "tam_indexer_topk_varlen",
    "tam_sparse_support_attention_varlen", "tam_mass_fallback_rows", "tam_indexer_fallback_rows",
)


class TamError(RuntimeError):
    def __init__(self, code: int, where: str, detail=None):
        self.code = code
        self.detail = detail
        msg = f"{where}: {status_string(code)} ({code})"
        if detail is not None:
            msg += f" detail={list(detail)}"
        super().__init__(msg)


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    """Load libtam.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m top_attention_mass_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        i64, i32, sz, p = ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        L.tam_version.restype = i32
        L.tam_status_string.restype = ctypes.c_char_p
        L.tam_status_string.argtypes = [i32]
        L.tam_mass_oracle_workspace.restype = sz
        L.tam_mass_oracle_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32]
        L.tam_mass_workspace_min.restype = sz
        L.tam_mass_workspace_min.argtypes = [i64, i32, i32, i32, i32, i32, i32]
        L.tam_mass_oracle_prefill.restype = i32
        L.tam_mass_oracle_prefill.argtypes = [i64, i32, i32, i32, i32, p, p, p, i32, i32, p, p, p,
                                              p, p, p, sz, p]
        L.tam_attention_lse_workspace.restype = sz
        L.tam_attention_lse_workspace.argtypes = [i64, i32, i32, i32, i32]
        L.tam_attention_lse.restype = i32
        L.tam_attention_lse.argtypes = [i64, i32, i32, i32, i32, p, p, p, p, sz, p]
        L.tam_mass_select_workspace.restype = sz
        L.tam_mass_select_workspace.argtypes = [i64, i32, i32, i32, i32, i32, i32]
        L.tam_mass_select.restype = i32
        L.tam_mass_select.argtypes = [i64, i32, i32, i32, i32, p, p, p, i32, i32, p, p, p, p, sz,
                                      p]
        L.tam_mass_select_noalloc.restype = i32
        L.tam_mass_select_noalloc.argtypes = [i64, i32, i32, i32, i32, p, p, p, i32, i32, p, p, p,
                                              p]
        L.tam_indexer_workspace.restype = sz
        L.tam_indexer_workspace.argtypes = [i64, i32, i32, i32, i32]
        L.tam_indexer_workspace_min.restype = sz
        L.tam_indexer_workspace_min.argtypes = [i64, i32, i32, i32, i32]
        L.tam_indexer_topk.restype = i32
        L.tam_indexer_topk.argtypes = [i64, i32, i32, p, p, i32, i32, p, p, p, p, sz, p]
        L.tam_distill_kl_workspace.restype = sz
        L.tam_distill_kl_workspace.argtypes = [i64, i32, i32, i32, i32, i32]
        L.tam_distill_kl_workspace_min.restype = sz
        L.tam_distill_kl_workspace_min.argtypes = [i64, i32, i32, i32, i32, i32]
        L.tam_distill_kl.restype = i32
        L.tam_distill_kl.argtypes = [i64, i32, i32, i32, i32, p, p, p, i32, p, p, p, p, sz, p]
        L.tam_support_mass_curve.restype = i32
        L.tam_support_mass_curve.argtypes = [i64, i32, p, p, p, i32, p, p]
        L.tam_sparse_attention_workspace.restype = sz
        L.tam_sparse_attention_workspace.argtypes = [i64, i32, i32, i32, i32]
        L.tam_sparse_support_attention.restype = i32
        L.tam_sparse_support_attention.argtypes = [i64, i32, i32, i32, i32, p, p, p, p, p, i32,
                                                   i32, p, p, p, sz, p]
        L.tam_dense_workspace.restype = sz
        L.tam_dense_workspace.argtypes = [i64, i32, i32, i32, i32]
        L.tam_dense_gqa_prefill.restype = i32
        L.tam_dense_gqa_prefill.argtypes = [i64, i32, i32, i32, i32, p, p, p, p, p, p, sz, p]
        L.tam_mass_oracle_workspace_varlen.restype = sz
        L.tam_mass_oracle_workspace_varlen.argtypes = [i32, p, i32, i32, i32, i32, i32, i32]
        L.tam_mass_oracle_prefill_varlen.restype = i32
        L.tam_mass_oracle_prefill_varlen.argtypes = [i32, p, i32, i32, i32, i32, p, p, p, i32, i32,
                                                     p, p, p, p, p, p, sz, p]
        L.tam_dense_gqa_prefill_varlen.restype = i32
        L.tam_dense_gqa_prefill_varlen.argtypes = [i32, p, i32, i32, i32, i32, p, p, p, p, p, p,
                                                   sz, p]
        L.tam_indexer_workspace_varlen.restype = sz
        L.tam_indexer_workspace_varlen.argtypes = [i32, p, i32, i32, i32, i32]
        L.tam_indexer_topk_varlen.restype = i32
        L.tam_indexer_topk_varlen.argtypes = [i32, p, i32, i32, p, p, i32, i32, p, p, p, p, sz, p]
        L.tam_sparse_support_attention_varlen.restype = i32
        L.tam_sparse_support_attention_varlen.argtypes = [i32, p, i32, i32, i32, i32, p, p, p, p, p,
                                                          i32, i32, p, p, p, sz, p]
        L.tam_mass_fallback_rows.restype = i64
        L.tam_mass_fallback_rows.argtypes = [i64, i32, i32, i32, i32, i32, p, p]
        L.tam_indexer_fallback_rows.restype = i64
        L.tam_indexer_fallback_rows.argtypes = [i64, i32, i32, i32, p, p]
        L.tam_kv_cache_write.restype = i32
        L.tam_kv_cache_write.argtypes = [i64, i32, p, p, p, p, p, sz, p]
        L.tam_kv_cache_read.restype = i32
        L.tam_kv_cache_read.argtypes = [i64, i32, p, p, p, p, p, sz, p]
        L.tam_paged_attention_workspace.restype = sz
        L.tam_paged_attention_workspace.argtypes = [i64, i32, i32, p, p]
        L.tam_paged_gqa_attention.restype = i32
        L.tam_paged_gqa_attention.argtypes = [i64, i32, i32, p, p, p, p, p, p, sz, p]
        L.tam_kernel_launches.restype = ctypes.c_uint64
        L.tam_check_status.restype = i32
        L.tam_check_status.argtypes = [p, p, p]
        _lib = L
        return _lib


def status_string(code: int) -> str:
    try:
        return lib().tam_status_string(int(code)).decode()
    except Exception:
        return "status"


def version() -> int:
    return int(lib().tam_version())


def kernel_launches() -> int:
    """Kernels this library has launched in this process (all entry points)."""
    return int(lib().tam_kernel_launches())


def mass_fallback_rows(q, k, budget_k: int, workspace, stream=None) -> int:
    """Rows of the last per-query mass selection in `workspace` (a Workspace or the
    uint8 tensor a call used) that went to the fallback path; -1 if it does not stream."""
    N, Hq, Hkv, d = _shape(q, k)
    t = workspace.get(256) if isinstance(workspace, Workspace) else workspace
    return int(lib().tam_mass_fallback_rows(N, Hq, Hkv, d, _dtype_code(q), budget_k, _ptr(t),
                                            _stream(t.device, stream)))


def indexer_fallback_rows(q_idx, budget_k: int, workspace, stream=None) -> int:
    """As mass_fallback_rows, for the last per-query indexer selection."""
    N, dx = q_idx.shape
    t = workspace.get(256) if isinstance(workspace, Workspace) else workspace
    return int(lib().tam_indexer_fallback_rows(N, dx, _dtype_code(q_idx), budget_k, _ptr(t),
                                               _stream(t.device, stream)))


# ------------------------------------------------------------------ marshalling helpers

def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TAM_BF16
    if t.dtype == torch.float32:
        return TAM_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


class Workspace:
    """A reusable device workspace (uint8 tensor) that grows on demand.

    A call that gets no workspace uses one default workspace per device (the paged calls one
    per device, stream and thread, the last 16 of them).  Calls are
    ordered on their stream, so that is safe for one stream at a time; calls that run
    concurrently on several streams need one Workspace each (the status block and the
    scratch would otherwise be shared), and so do captured graphs that are replayed at the
    same time."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf: Optional[torch.Tensor] = None
        self.captured = False     # a captured paged call holds the address of buf
        self._kept = []           # buffers outgrown since, still held by such a call

    def get(self, nbytes: int) -> torch.Tensor:
        nbytes = max(int(nbytes), 256)
        if self.buf is None or self.buf.numel() < nbytes:
            if self.captured:
                self._kept.append(self.buf)
                self.captured = False
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        return self.buf


_default_ws = {}


def _workspace(device: torch.device, nbytes: int, ws: Optional[Workspace]) -> torch.Tensor:
    if ws is None:
        key = (device.type, device.index)
        ws = _default_ws.get(key)
        if ws is None:
            ws = _default_ws[key] = Workspace(device)
    return ws.get(nbytes)


def _raise(rc: int, where: str):
    if rc != TAM_OK:
        raise TamError(rc, where)


def check_status(workspace: torch.Tensor, stream=None):
    """Wait for the stream and raise if the last call on this workspace flagged an error."""
    detail = (ctypes.c_int32 * 8)()
    rc = lib().tam_check_status(_ptr(workspace), _stream(workspace.device, stream), detail)
    if rc != TAM_OK:
        raise TamError(rc, "device status", list(detail))


def _to_device(ts, device):
    """Move CPU inputs to `device` (non-blocking from pinned memory); CUDA inputs pass through."""
    out, host = [], False
    for t in ts:
        if t is None:
            out.append(None)
        elif t.is_cuda:
            out.append(t.contiguous())
        else:
            host = True
            out.append(t.contiguous().to(device, non_blocking=t.is_pinned()))
    return out, host


def _dev_of(t: torch.Tensor, device) -> torch.device:
    if t.is_cuda:
        return t.device
    return torch.device(device or "cuda")


def _shape(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q is [N, Hq, d] and k, v are [N, Hkv, d]")
    N, Hq, d = q.shape
    if k.shape[0] != N or k.shape[2] != d or k.dtype != q.dtype:
        raise ValueError("k must be [N, Hkv, d] with q's N, d and dtype")
    return N, Hq, k.shape[1], d


# ------------------------------------------------------------------ entry points

@dataclass
class Support:
    idx: torch.Tensor             # [n_sel, k] int32 ascending, -1 padded
    length: torch.Tensor          # [n_sel] int32
    value: torch.Tensor           # [n_sel, k] fp32: mass (oracle) or score (indexer)
    lse: Optional[torch.Tensor] = None    # [Hq, N] fp32
    out: Optional[torch.Tensor] = None    # [N, Hq, d]


def mass_oracle_prefill(q, k, v=None, budget_k: int = 1, block_q: int = 1, *,
                        compute_out: bool = True, return_lse: bool = True,
                        workspace: Optional[Workspace] = None, stream=None, check: bool = True,
                        device=None, workspace_bytes: Optional[int] = None) -> Support:
    """Attention-mass top-k oracle (passes 1-3) for one causal GQA prefill layer.

    workspace_bytes: pass this many workspace bytes instead of the preferred size
    (at least tam_mass_workspace_min; a smaller workspace only means more chunks)."""
    dev = _dev_of(q, device)
    (q, k, v), host = _to_device([q, k, v], dev)
    N, Hq, Hkv, d = _shape(q, k)
    if compute_out and v is None:
        raise ValueError("v is needed for the recomputed output")
    dt = _dtype_code(q)
    n_sel = N if block_q == 1 else -(-N // block_q)
    sup_idx = torch.empty(n_sel, budget_k, dtype=torch.int32, device=dev)
    sup_len = torch.empty(n_sel, dtype=torch.int32, device=dev)
    sup_mass = torch.empty(n_sel, budget_k, dtype=torch.float32, device=dev)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=dev) if return_lse else None
    out = torch.empty_like(q) if compute_out else None
    L = lib()
    nbytes = L.tam_mass_oracle_workspace(N, Hq, Hkv, d, dt, budget_k, block_q)
    if nbytes == 0:
        _raise(L.tam_mass_oracle_prefill(N, Hq, Hkv, d, dt, None, None, None, budget_k, block_q,
                                         None, None, None, None, None, None, 0, None),
               "mass_oracle_prefill")
    if workspace_bytes is not None:
        nbytes = int(workspace_bytes)
    ws = _workspace(dev, nbytes, workspace)
    rc = L.tam_mass_oracle_prefill(N, Hq, Hkv, d, dt, _ptr(q), _ptr(k), _ptr(v), budget_k, block_q,
                                   _ptr(sup_idx), _ptr(sup_len), _ptr(sup_mass), _ptr(lse),
                                   _ptr(out), _ptr(ws), min(ws.numel(), nbytes),
                                   _stream(dev, stream))
    _raise(rc, "mass_oracle_prefill")
    if check:
        check_status(ws, stream)
    res = Support(sup_idx, sup_len, sup_mass, lse, out)
    if host:
        res = Support(*[None if t is None else t.cpu() for t in
                        (res.idx, res.length, res.value, res.lse, res.out)])
    return res


def attention_lse(q, k, *, workspace: Optional[Workspace] = None, stream=None,
                  check: bool = True) -> torch.Tensor:
    """Pass 1: per-head log-sum-exp of the causal scores, [Hq, N] fp32."""
    dev = q.device
    N, Hq, Hkv, d = _shape(q, k)
    dt = _dtype_code(q)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.tam_attention_lse_workspace(N, Hq, Hkv, d, dt)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_attention_lse(N, Hq, Hkv, d, dt, _ptr(q.contiguous()), _ptr(k.contiguous()),
                             _ptr(lse), _ptr(ws), ws.numel(), _stream(dev, stream))
    _raise(rc, "attention_lse")
    if check:
        check_status(ws, stream)
    return lse


def mass_select(q, k, lse, budget_k: int, block_q: int = 1, *,
                workspace: Optional[Workspace] = None, stream=None, check: bool = True,
                workspace_bytes: Optional[int] = None) -> Support:
    """Pass 2: head-averaged mass and its top-k support, given pass 1's lse [Hq, N].

    workspace_bytes: as in mass_oracle_prefill."""
    dev = q.device
    N, Hq, Hkv, d = _shape(q, k)
    dt = _dtype_code(q)
    if lse.shape != (Hq, N) or lse.dtype != torch.float32:
        raise ValueError("lse must be [Hq, N] fp32")
    n_sel = N if block_q == 1 else -(-N // block_q)
    sup_idx = torch.empty(n_sel, budget_k, dtype=torch.int32, device=dev)
    sup_len = torch.empty(n_sel, dtype=torch.int32, device=dev)
    sup_mass = torch.empty(n_sel, budget_k, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.tam_mass_select_workspace(N, Hq, Hkv, d, dt, budget_k, block_q)
    if workspace_bytes is not None and nbytes:
        nbytes = int(workspace_bytes)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_mass_select(N, Hq, Hkv, d, dt, _ptr(q.contiguous()), _ptr(k.contiguous()),
                           _ptr(lse.contiguous()), budget_k, block_q, _ptr(sup_idx), _ptr(sup_len),
                           _ptr(sup_mass), _ptr(ws), min(ws.numel(), nbytes) if nbytes else 0,
                           _stream(dev, stream))
    _raise(rc, "mass_select")
    if check:
        check_status(ws, stream)
    return Support(sup_idx, sup_len, sup_mass)


def indexer_topk(q_idx, k_idx, budget_k: int, block_q: int = 1, *,
                 workspace: Optional[Workspace] = None, stream=None, check: bool = True,
                 device=None, workspace_bytes: Optional[int] = None) -> Support:
    """Head-collapsed indexer support: top-k of q_idx . k_idx per query (block_q = 1), or
    per block of block_q queries the top-k of the block's summed per-query softmax of
    those scores (block_q > 1; values are the block sums).

    workspace_bytes: at least tam_indexer_workspace_min (more chunks below the
    preferred size)."""
    dev = _dev_of(q_idx, device)
    (q_idx, k_idx), host = _to_device([q_idx, k_idx], dev)
    N, dx = q_idx.shape
    if k_idx.shape != q_idx.shape or k_idx.dtype != q_idx.dtype:
        raise ValueError("q_idx and k_idx must both be [N, d_idx] of one dtype")
    dt = _dtype_code(q_idx)
    n_sel = N if block_q == 1 else -(-N // block_q)
    sup_idx = torch.empty(n_sel, budget_k, dtype=torch.int32, device=dev)
    sup_len = torch.empty(n_sel, dtype=torch.int32, device=dev)
    sup_score = torch.empty(n_sel, budget_k, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.tam_indexer_workspace(N, dx, dt, budget_k, block_q)
    if workspace_bytes is not None and nbytes:
        nbytes = int(workspace_bytes)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_indexer_topk(N, dx, dt, _ptr(q_idx), _ptr(k_idx), budget_k, block_q,
                            _ptr(sup_idx), _ptr(sup_len), _ptr(sup_score), _ptr(ws),
                            min(ws.numel(), nbytes) if nbytes else 0, _stream(dev, stream))
    _raise(rc, "indexer_topk")
    if check:
        check_status(ws, stream)
    res = Support(sup_idx, sup_len, sup_score)
    if host:
        res = Support(res.idx.cpu(), res.length.cpu(), res.value.cpu())
    return res


def distill_kl(q, k, lse, q_idx, k_idx, *, workspace: Optional[Workspace] = None, stream=None,
               check: bool = True, workspace_bytes: Optional[int] = None) -> torch.Tensor:
    """The indexer's distillation target per query: KL(P_i || softmax(q_idx_i . k_idx)),
    P_i the head-averaged mass of pass 2 (given pass 1's lse [Hq, N]).  Returns [N] fp32."""
    dev = q.device
    N, Hq, Hkv, d = _shape(q, k)
    dt = _dtype_code(q)
    if lse.shape != (Hq, N) or lse.dtype != torch.float32:
        raise ValueError("lse must be [Hq, N] fp32")
    if q_idx.shape != k_idx.shape or q_idx.shape[0] != N or q_idx.dtype != q.dtype:
        raise ValueError("q_idx and k_idx must be [N, d_idx] in q's dtype")
    dx = q_idx.shape[1]
    kl = torch.empty(N, dtype=torch.float32, device=dev)
    L = lib()
    nbytes = L.tam_distill_kl_workspace(N, Hq, Hkv, d, dt, dx)
    if workspace_bytes is not None and nbytes:
        nbytes = int(workspace_bytes)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_distill_kl(N, Hq, Hkv, d, dt, _ptr(q.contiguous()), _ptr(k.contiguous()),
                          _ptr(lse.contiguous()), dx, _ptr(q_idx.contiguous()),
                          _ptr(k_idx.contiguous()), _ptr(kl), _ptr(ws),
                          min(ws.numel(), nbytes) if nbytes else 0, _stream(dev, stream))
    _raise(rc, "distill_kl")
    if check:
        check_status(ws, stream)
    return kl


def support_mass_curve(sup_val, sup_len, budgets, *, stream=None) -> torch.Tensor:
    """Budget sweep: [rows, len(budgets)] fp32, the sum of the k largest values of each
    support row for every budget k (rows of a top-kmax support, e.g. Support.value)."""
    dev = sup_val.device
    if sup_val.dim() != 2 or sup_val.dtype != torch.float32 or sup_len.dtype != torch.int32:
        raise TypeError("sup_val [rows, kmax] fp32 and sup_len [rows] int32")
    rows, kmax = sup_val.shape
    ks = (ctypes.c_int32 * len(budgets))(*[int(b) for b in budgets])
    out = torch.empty(rows, len(budgets), dtype=torch.float32, device=dev)
    rc = lib().tam_support_mass_curve(rows, kmax, _ptr(sup_val.contiguous()),
                                      _ptr(sup_len.contiguous()), ks, len(budgets), _ptr(out),
                                      _stream(dev, stream))
    _raise(rc, "support_mass_curve")
    return out


def sparse_support_attention(q, k, v, sup_idx, sup_len, block_q: int = 1, *,
                             return_lse: bool = False, workspace: Optional[Workspace] = None,
                             stream=None, check: bool = True, device=None):
    """Pass 3: attention recomputed on a given support. Returns out (and lse)."""
    dev = _dev_of(q, device)
    (q, k, v, sup_idx, sup_len), host = _to_device([q, k, v, sup_idx, sup_len], dev)
    N, Hq, Hkv, d = _shape(q, k)
    dt = _dtype_code(q)
    if sup_idx.dtype != torch.int32 or sup_len.dtype != torch.int32:
        raise TypeError("sup_idx and sup_len are int32")
    kmax = sup_idx.shape[1]
    out = torch.empty_like(q)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=dev) if return_lse else None
    L = lib()
    nbytes = L.tam_sparse_attention_workspace(N, Hq, Hkv, d, dt)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_sparse_support_attention(N, Hq, Hkv, d, dt, _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(sup_idx), _ptr(sup_len), kmax, block_q, _ptr(out),
                                        _ptr(lse), _ptr(ws), ws.numel(), _stream(dev, stream))
    _raise(rc, "sparse_support_attention")
    if check:
        check_status(ws, stream)
    if host:
        out = out.cpu()
        lse = None if lse is None else lse.cpu()
    return (out, lse) if return_lse else out


def dense_gqa_prefill(q, k, v, *, return_lse: bool = False,
                      workspace: Optional[Workspace] = None, stream=None, check: bool = True,
                      device=None):
    """Dense causal GQA attention. Returns out (and lse)."""
    dev = _dev_of(q, device)
    (q, k, v), host = _to_device([q, k, v], dev)
    N, Hq, Hkv, d = _shape(q, k)
    dt = _dtype_code(q)
    out = torch.empty_like(q)
    lse = torch.empty(Hq, N, dtype=torch.float32, device=dev) if return_lse else None
    L = lib()
    nbytes = L.tam_dense_workspace(N, Hq, Hkv, d, dt)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_dense_gqa_prefill(N, Hq, Hkv, d, dt, _ptr(q), _ptr(k), _ptr(v), _ptr(out),
                                 _ptr(lse), _ptr(ws), ws.numel(), _stream(dev, stream))
    _raise(rc, "dense_gqa_prefill")
    if check:
        check_status(ws, stream)
    if host:
        out = out.cpu()
        lse = None if lse is None else lse.cpu()
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ packed batches

def _cu_host(cu_seqlens) -> torch.Tensor:
    """cu_seqlens as a contiguous host int64 tensor (the library reads it on the host)."""
    cu = torch.as_tensor(cu_seqlens, dtype=torch.int64, device="cpu").contiguous()
    if cu.dim() != 1 or cu.numel() < 2:
        raise ValueError("cu_seqlens is [n_seq + 1] int64")
    return cu


def selection_offsets(cu_seqlens, block_q: int = 1) -> torch.Tensor:
    """First selection row of every sequence of a packed batch ([n_seq + 1] int64)."""
    cu = _cu_host(cu_seqlens)
    n = cu[1:] - cu[:-1]
    n_sel = n if block_q == 1 else (n + block_q - 1) // block_q
    return torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(n_sel, 0)])


def lse_block(lse: torch.Tensor, cu_seqlens, s: int) -> torch.Tensor:
    """The [Hq, N_s] lse block of sequence s inside a packed varlen lse."""
    cu = _cu_host(cu_seqlens)
    t0, t1 = int(cu[s]), int(cu[s + 1])
    Hq = lse.numel() // int(cu[-1]) if int(cu[-1]) else 0
    return lse[Hq * t0:Hq * t1].view(Hq, t1 - t0)


def mass_oracle_prefill_varlen(q, k, v, cu_seqlens, budget_k: int, block_q: int = 1, *,
                               compute_out: bool = True, return_lse: bool = True,
                               workspace: Optional[Workspace] = None, stream=None,
                               check: bool = True, device=None) -> Support:
    """mass_oracle_prefill over a packed batch: q [T, Hq, d], k/v [T, Hkv, d], sequence s
    owning tokens [cu_seqlens[s], cu_seqlens[s+1]).  Support rows are packed in sequence
    order (see ``selection_offsets``), key indices are positions within the sequence,
    and ``lse`` is flat (one [Hq, N_s] block per sequence, see ``lse_block``)."""
    cu = _cu_host(cu_seqlens)
    n_seq = cu.numel() - 1
    dev = _dev_of(q, device)
    (q, k, v), host = _to_device([q, k, v], dev)
    T, Hq, Hkv, d = _shape(q, k)
    if int(cu[-1]) != T:
        raise ValueError("cu_seqlens[-1] must equal the packed token count")
    if compute_out and v is None:
        raise ValueError("v is needed for the recomputed output")
    dt = _dtype_code(q)
    n_sel = int(selection_offsets(cu, block_q)[-1])
    sup_idx = torch.empty(n_sel, budget_k, dtype=torch.int32, device=dev)
    sup_len = torch.empty(n_sel, dtype=torch.int32, device=dev)
    sup_mass = torch.empty(n_sel, budget_k, dtype=torch.float32, device=dev)
    lse = torch.empty(Hq * T, dtype=torch.float32, device=dev) if return_lse else None
    out = torch.empty_like(q) if compute_out else None
    L = lib()
    cu_p = ctypes.c_void_p(cu.data_ptr())
    nbytes = L.tam_mass_oracle_workspace_varlen(n_seq, cu_p, Hq, Hkv, d, dt, budget_k, block_q)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_mass_oracle_prefill_varlen(n_seq, cu_p, Hq, Hkv, d, dt, _ptr(q), _ptr(k), _ptr(v),
                                          budget_k, block_q, _ptr(sup_idx), _ptr(sup_len),
                                          _ptr(sup_mass), _ptr(lse), _ptr(out), _ptr(ws),
                                          ws.numel() if nbytes else 0, _stream(dev, stream))
    _raise(rc, "mass_oracle_prefill_varlen")
    if check:
        check_status(ws, stream)
    res = Support(sup_idx, sup_len, sup_mass, lse, out)
    if host:
        res = Support(*[None if t is None else t.cpu() for t in
                        (res.idx, res.length, res.value, res.lse, res.out)])
    return res


def dense_gqa_prefill_varlen(q, k, v, cu_seqlens, *, return_lse: bool = False,
                             workspace: Optional[Workspace] = None, stream=None,
                             check: bool = True, device=None):
    """dense_gqa_prefill over a packed batch (layout as mass_oracle_prefill_varlen)."""
    cu = _cu_host(cu_seqlens)
    n_seq = cu.numel() - 1
    dev = _dev_of(q, device)
    (q, k, v), host = _to_device([q, k, v], dev)
    T, Hq, Hkv, d = _shape(q, k)
    if int(cu[-1]) != T:
        raise ValueError("cu_seqlens[-1] must equal the packed token count")
    dt = _dtype_code(q)
    out = torch.empty_like(q)
    lse = torch.empty(Hq * T, dtype=torch.float32, device=dev) if return_lse else None
    L = lib()
    ws = _workspace(dev, 256, workspace)
    rc = L.tam_dense_gqa_prefill_varlen(n_seq, ctypes.c_void_p(cu.data_ptr()), Hq, Hkv, d, dt,
                                        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(ws),
                                        ws.numel(), _stream(dev, stream))
    _raise(rc, "dense_gqa_prefill_varlen")
    if check:
        check_status(ws, stream)
    if host:
        out = out.cpu()
        lse = None if lse is None else lse.cpu()
    return (out, lse) if return_lse else out


def indexer_topk_varlen(q_idx, k_idx, cu_seqlens, budget_k: int, block_q: int = 1, *,
                        workspace: Optional[Workspace] = None, stream=None, check: bool = True,
                        device=None) -> Support:
    """indexer_topk over a packed batch: q_idx, k_idx [T, d_idx]; support rows packed in
    sequence order (see ``selection_offsets``), positions local to each sequence."""
    cu = _cu_host(cu_seqlens)
    n_seq = cu.numel() - 1
    dev = _dev_of(q_idx, device)
    (q_idx, k_idx), host = _to_device([q_idx, k_idx], dev)
    if q_idx.dim() != 2 or k_idx.shape != q_idx.shape or k_idx.dtype != q_idx.dtype:
        raise ValueError("q_idx and k_idx are [T, d_idx] of one dtype")
    T, dx = q_idx.shape
    if int(cu[-1]) != T:
        raise ValueError("cu_seqlens[-1] must equal the packed token count")
    dt = _dtype_code(q_idx)
    n_sel = int(selection_offsets(cu, block_q)[-1])
    sup_idx = torch.empty(n_sel, budget_k, dtype=torch.int32, device=dev)
    sup_len = torch.empty(n_sel, dtype=torch.int32, device=dev)
    sup_score = torch.empty(n_sel, budget_k, dtype=torch.float32, device=dev)
    L = lib()
    cu_p = ctypes.c_void_p(cu.data_ptr())
    nbytes = L.tam_indexer_workspace_varlen(n_seq, cu_p, dx, dt, budget_k, block_q)
    ws = _workspace(dev, max(nbytes, 256), workspace)
    rc = L.tam_indexer_topk_varlen(n_seq, cu_p, dx, dt, _ptr(q_idx), _ptr(k_idx), budget_k,
                                   block_q, _ptr(sup_idx), _ptr(sup_len), _ptr(sup_score),
                                   _ptr(ws), ws.numel() if nbytes else 0, _stream(dev, stream))
    _raise(rc, "indexer_topk_varlen")
    if check:
        check_status(ws, stream)
    res = Support(sup_idx, sup_len, sup_score)
    if host:
        res = Support(res.idx.cpu(), res.length.cpu(), res.value.cpu())
    return res


def sparse_support_attention_varlen(q, k, v, sup_idx, sup_len, cu_seqlens, block_q: int = 1, *,
                                    return_lse: bool = False,
                                    workspace: Optional[Workspace] = None, stream=None,
                                    check: bool = True, device=None):
    """sparse_support_attention over a packed batch; support rows as the varlen selection
    calls lay them out.  Returns out [T, Hq, d] (and the flat per-sequence lse blocks)."""
    cu = _cu_host(cu_seqlens)
    n_seq = cu.numel() - 1
    dev = _dev_of(q, device)
    (q, k, v, sup_idx, sup_len), host = _to_device([q, k, v, sup_idx, sup_len], dev)
    T, Hq, Hkv, d = _shape(q, k)
    if int(cu[-1]) != T:
        raise ValueError("cu_seqlens[-1] must equal the packed token count")
    if sup_idx.dtype != torch.int32 or sup_len.dtype != torch.int32:
        raise TypeError("sup_idx and sup_len are int32")
    dt = _dtype_code(q)
    out = torch.empty_like(q)
    lse = torch.empty(Hq * T, dtype=torch.float32, device=dev) if return_lse else None
    L = lib()
    ws = _workspace(dev, 256, workspace)
    rc = L.tam_sparse_support_attention_varlen(n_seq, ctypes.c_void_p(cu.data_ptr()), Hq, Hkv, d,
                                               dt, _ptr(q), _ptr(k), _ptr(v), _ptr(sup_idx),
                                               _ptr(sup_len), sup_idx.shape[1], block_q, _ptr(out),
                                               _ptr(lse), _ptr(ws), ws.numel(),
                                               _stream(dev, stream))
    _raise(rc, "sparse_support_attention_varlen")
    if check:
        check_status(ws, stream)
    if host:
        out = out.cpu()
        lse = None if lse is None else lse.cpu()
    return (out, lse) if return_lse else out


# ------------------------------------------------------------------ paged KV cache

class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("n_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class _PagedBatchStruct(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("cu_rows", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("n_seq", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("max_rows", ctypes.c_int32)]


_CACHE_DTYPES = {torch.bfloat16: TAM_BF16, torch.float32: TAM_F32,
                 torch.float8_e4m3fn: TAM_E4M3}


class PagedKVCache:
    """The K and V pages of one layer: k_pages, v_pages [n_pages, page_size, Hkv, d] CUDA
    tensors of bf16, fp32 or float8_e4m3fn, with the same strides and a contiguous head dim
    (views of a larger tensor are fine: strides are at least d and multiples of 16 bytes).
    e4m3 pages come with k_scale, v_scale [n_pages, Hkv, page_size], contiguous,
    float8_e8m0fnu or uint8: the power-of-two scale of every token and KV head (written by
    ``kv_cache_write``).  page_size is 16, 32, 64, 128 or 256; d is 64, 128 or 256.

    The tensors are the caller's and are used in place."""

    def __init__(self, k_pages, v_pages, k_scale=None, v_scale=None):
        if k_pages.dim() != 4 or not k_pages.is_cuda:
            raise ValueError("k_pages and v_pages are [n_pages, page_size, Hkv, d] CUDA tensors")
        if k_pages.dtype not in _CACHE_DTYPES:
            raise TypeError(f"unsupported cache dtype {k_pages.dtype} (bf16, fp32 or "
                            "float8_e4m3fn)")
        if (v_pages.shape != k_pages.shape or v_pages.stride() != k_pages.stride()
                or v_pages.dtype != k_pages.dtype or v_pages.device != k_pages.device):
            raise ValueError("v_pages must have k_pages' shape, strides, dtype and device")
        n_pages, page_size, Hkv, d = k_pages.shape
        if d > 1 and k_pages.stride(3) != 1:
            raise ValueError("the head dim of the pages must be contiguous")
        code = _CACHE_DTYPES[k_pages.dtype]
        if code == TAM_E4M3:
            for t in (k_scale, v_scale):
                if (t is None or t.dtype not in (torch.float8_e8m0fnu, torch.uint8)
                        or t.shape != (n_pages, Hkv, page_size) or not t.is_contiguous()
                        or t.device != k_pages.device):
                    raise ValueError("e4m3 pages need k_scale and v_scale [n_pages, Hkv, "
                                     "page_size], contiguous float8_e8m0fnu or uint8 on their "
                                     "device")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("only e4m3 pages have scales")
        self.k_pages, self.v_pages, self.k_scale, self.v_scale = k_pages, v_pages, k_scale, v_scale
        self.n_pages, self.page_size, self.Hkv, self.d = n_pages, page_size, Hkv, d
        self.dtype, self.device = k_pages.dtype, k_pages.device
        # a dimension of one entry has no meaning for its stride: give it a valid one
        stride = [k_pages.stride(x) if k_pages.shape[x] > 1 else 0 for x in range(3)]
        whole = max(d, *[s * k_pages.shape[x] for x, s in enumerate(stride)])
        stride = [s if k_pages.shape[x] > 1 else whole for x, s in enumerate(stride)]
        self._struct = _KvCacheStruct(
            k_pages.data_ptr(), v_pages.data_ptr(),
            k_scale.data_ptr() if code == TAM_E4M3 else None,
            v_scale.data_ptr() if code == TAM_E4M3 else None,
            n_pages, *stride, page_size, Hkv, d, code)
        self._ref = ctypes.addressof(self._struct)
        self._code = code

    @classmethod
    def empty(cls, n_pages: int, page_size: int, Hkv: int, d: int, dtype=torch.bfloat16,
              device="cuda") -> "PagedKVCache":
        """A cache of newly allocated, uninitialised pages."""
        shape = (n_pages, page_size, Hkv, d)
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != torch.float8_e4m3fn:
            return cls(k, v)
        ks, vs = (torch.empty(n_pages, Hkv, page_size, dtype=torch.uint8, device=device)
                  .view(torch.float8_e8m0fnu) for _ in range(2))
        return cls(k, v, ks, vs)

    def _tensors(self):
        return (self.k_pages, self.v_pages, self.k_scale, self.v_scale)


class PagedBatch:
    """The sequences of a paged call: page_table [n_seq, max_pages] int32, cu_rows [n_seq + 1]
    int32 (sequence s owns the packed rows [cu_rows[s], cu_rows[s+1]), its newest tokens) and
    kv_len [n_seq] int32 (its tokens in the cache, the new ones among them).

    Contiguous int32 CUDA tensors are used in place: a captured call reads what they hold when
    it is replayed.  Lists and host tensors are copied to the device.  max_rows is a bound on
    the new tokens of any sequence (1 for a decoding step): it picks the attention kernel, and
    is taken from cu_rows where that comes from the host."""

    def __init__(self, page_table, cu_rows, kv_len, *, max_rows: Optional[int] = None,
                 device=None):
        dev = next((t.device for t in (page_table, cu_rows, kv_len)
                    if isinstance(t, torch.Tensor) and t.is_cuda), torch.device(device or "cuda"))
        host = not (isinstance(cu_rows, torch.Tensor) and cu_rows.is_cuda)
        self.n_rows = None                      # rows of the batch, where the host knows them
        if host:
            cu = _cu_host(cu_rows)
            n = cu[1:] - cu[:-1]
            if int(cu[0]) != 0 or int(n.min()) < 0:
                raise ValueError("cu_rows starts at 0 and does not decrease")
            self.n_rows = int(cu[-1])
            if max_rows is None:
                max_rows = max(int(n.max()), 1)

        def on_device(t, name, dim):
            t = torch.as_tensor(t)
            if t.dtype.is_floating_point or t.dtype == torch.bool or t.dim() != dim:
                raise ValueError(f"{name} is a {dim}-dimensional int32 tensor")
            if (t.dtype != torch.int32 and not t.is_cuda and t.numel()
                    and not -2 ** 31 <= int(t.min()) <= int(t.max()) < 2 ** 31):
                raise ValueError(f"{name} does not fit int32")
            return t.to(device=dev, dtype=torch.int32).contiguous()

        self.page_table = on_device(page_table, "page_table", 2)
        self.cu_rows = on_device(cu_rows, "cu_rows", 1)
        self.kv_len = on_device(kv_len, "kv_len", 1)
        n_seq, max_pages = self.page_table.shape
        if self.cu_rows.shape != (n_seq + 1,) or self.kv_len.shape != (n_seq,):
            raise ValueError("cu_rows is [n_seq + 1] and kv_len [n_seq] for a page_table of "
                             "[n_seq, max_pages]")
        if max_rows is not None and max_rows < 1:
            raise ValueError("max_rows is at least 1")
        self.device = self.page_table.device
        self._struct = _PagedBatchStruct(
            self.page_table.data_ptr(), self.cu_rows.data_ptr(), self.kv_len.data_ptr(), n_seq,
            max_pages, max_rows or 0)
        self._ref = ctypes.addressof(self._struct)
        self._ws_bytes = {}                     # workspace sizes by the host values they go by

    def _tensors(self):
        return (self.page_table, self.cu_rows, self.kv_len)


# the current stream's handle, without making a Stream object where torch offers that (2 us)
_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)

# default workspaces of the paged calls: one per device, stream and thread (two threads' calls
# take turns on a stream launch by launch, not call by call)
_paged_ws = threading.local()
_PAGED_WS_KEPT = 16                             # of a thread, for programs that make streams as they go


def _paged_call(cache, batch, tensors, workspace, stream, check, body):
    """Runs body(stream handle, get_ws) on the cache's device and `stream`; get_ws(nbytes) is
    the call's workspace.  Returns body's result after the status check, if any."""
    dev = cache.device
    if batch.device != dev:
        raise ValueError("the cache and the batch must be on one CUDA device")
    for t in tensors:
        if t is not None and t.device != dev:
            raise ValueError("the rows must be on the cache's CUDA device")
    if stream is not None and stream.device != dev:
        raise ValueError("the stream must be of the cache's CUDA device")
    if workspace is not None:
        at = workspace.device if workspace.buf is None else workspace.buf.device
        if at.type != "cuda" or at.index not in (None, dev.index):
            raise ValueError("the workspace must be on the cache's CUDA device")
    if torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return _paged_call(cache, batch, tensors, workspace, stream, check, body)
    handle = _stream_handle(dev.index)
    if stream is not None and stream.cuda_stream != handle:
        # the call runs on `stream`: its allocations belong there, and what it reads must
        # outlive it
        with torch.cuda.stream(stream):
            if not torch.cuda.is_current_stream_capturing():
                for t in (*tensors, *cache._tensors(), *batch._tensors()):
                    if t is not None:
                        t.record_stream(stream)
                if workspace is not None and workspace.buf is not None:
                    workspace.buf.record_stream(stream)
            return _paged_call(cache, batch, tensors, workspace, None, check, body)
    capturing = torch.cuda.is_current_stream_capturing()
    if capturing:
        if check or workspace is None:
            raise ValueError("a captured call needs check=False and a workspace of its graph's "
                             "own")
    elif workspace is None:
        mine = _paged_ws.__dict__
        workspace = mine.get((dev.index, handle))
        if workspace is None:
            if len(mine) >= _PAGED_WS_KEPT:
                # the oldest: its memory goes back to its own stream's pool, behind its last call
                del mine[next(iter(mine))]
            workspace = mine[dev.index, handle] = Workspace(dev)

    def get_ws(nbytes):
        buf = workspace.buf
        if buf is not None and buf.numel() >= nbytes and not capturing:
            return buf
        if capturing:
            if buf is None or buf.numel() < max(nbytes, 256):
                raise ValueError(f"the workspace of a captured call needs {nbytes} bytes before "
                                 "the capture: run the call once outside it, or "
                                 "workspace.get(bytes)")
            workspace.captured = True
        elif buf is not None:
            buf.record_stream(torch.cuda.current_stream(dev))   # outgrown, perhaps still in use
        return workspace.get(nbytes)

    res, ws = body(handle, get_ws)
    if check:
        check_status(ws)
    return res


def _packed_rows(cache, t, name):
    if t.dim() != 3 or t.shape[1] != cache.Hkv or t.shape[2] != cache.d:
        raise ValueError(f"{name} is [T, Hkv, d] with the cache's Hkv and d")
    return t


def kv_cache_write(cache: PagedKVCache, batch: PagedBatch, k, v, *,
                   workspace: Optional[Workspace] = None, stream=None, check: bool = True):
    """Write the new tokens' rows k, v [T, Hkv, d] to their pages: as they are into a bf16 or
    fp32 cache of their type, quantised (one power-of-two scale per token and KV head, values
    rounded to e4m3) into an e4m3 cache."""
    _packed_rows(cache, k, "k")
    if v.shape != k.shape or v.dtype != k.dtype:
        raise ValueError("v must have k's shape and dtype")
    dt = _dtype_code(k)

    def body(handle, get_ws):
        kc, vc = k.contiguous(), v.contiguous()
        ws = get_ws(256)
        _raise(lib().tam_kv_cache_write(kc.shape[0], dt, kc.data_ptr(), vc.data_ptr(), cache._ref,
                                        batch._ref, ws.data_ptr(), ws.numel(), handle),
               "kv_cache_write")
        return None, ws

    return _paged_call(cache, batch, (k, v), workspace, stream, check, body)


def kv_cache_read(cache: PagedKVCache, batch: PagedBatch, n_rows: Optional[int] = None, *,
                  dtype=None, out=None, workspace: Optional[Workspace] = None, stream=None,
                  check: bool = True):
    """Read the batch's rows (the newest cu_rows[s+1] - cu_rows[s] tokens of every sequence)
    back out of the pages.  Returns k, v [T, Hkv, d], T = n_rows (the batch's own count where
    the host knows it), in `dtype`: the cache's, or bf16 (default) or fp32 for e4m3.
    out: a (k, v) pair to fill instead; rows behind the last sequence keep what they hold."""
    if out is not None:
        ko, vo = (_packed_rows(cache, t, "out") for t in out)
        if ko.shape != vo.shape or ko.dtype != vo.dtype or not (ko.is_contiguous()
                                                                and vo.is_contiguous()):
            raise ValueError("out is a pair of contiguous tensors of one shape and dtype")
        if (n_rows is not None and n_rows != ko.shape[0]) or (dtype is not None
                                                              and dtype != ko.dtype):
            raise ValueError("n_rows and dtype are out's own")
        T, dtype, tensors = ko.shape[0], ko.dtype, (ko, vo)
    else:
        T = batch.n_rows if n_rows is None else int(n_rows)
        if T is None:
            raise ValueError("n_rows is needed: cu_rows lives on the device")
        if T < 0:
            raise ValueError("n_rows is not negative")
        if dtype is None:
            dtype = torch.bfloat16 if cache._code == TAM_E4M3 else cache.dtype
        tensors = ()
    dt = _CACHE_DTYPES.get(dtype, TAM_E4M3)
    if dt == TAM_E4M3:
        raise TypeError(f"unsupported dtype {dtype} (bf16 or fp32)")

    def body(handle, get_ws):
        if out is not None:
            k, v = ko, vo
        else:
            k, v = (torch.empty(T, cache.Hkv, cache.d, dtype=dtype, device=cache.device)
                    for _ in range(2))
        ws = get_ws(256)
        _raise(lib().tam_kv_cache_read(T, dt, k.data_ptr(), v.data_ptr(), cache._ref, batch._ref,
                                       ws.data_ptr(), ws.numel(), handle), "kv_cache_read")
        return (k, v), ws

    return _paged_call(cache, batch, tensors, workspace, stream, check, body)


def paged_attention_workspace(n_rows: int, Hq: int, dtype, cache: PagedKVCache,
                              batch: PagedBatch) -> int:
    """Workspace bytes of paged_gqa_attention for q [n_rows, Hq, d] of `dtype` (0 for
    arguments it rejects)."""
    dt = {torch.bfloat16: TAM_BF16, torch.float32: TAM_F32}.get(dtype, -1)
    return int(lib().tam_paged_attention_workspace(n_rows, Hq, dt, cache._ref, batch._ref))


def paged_gqa_attention(q, cache: PagedKVCache, batch: PagedBatch, *, return_lse: bool = False,
                        out=None, workspace: Optional[Workspace] = None, stream=None,
                        check: bool = True):
    """Causal GQA attention of the batch's new tokens q [T, Hq, d] over their sequences' pages
    (write the new tokens' K and V first).  q is bf16 over a bf16 or e4m3 cache, fp32 over an
    fp32 or e4m3 cache.  Returns out [T, Hq, d] (and the flat per-sequence lse blocks of the
    _varlen calls).  out: a tensor to fill instead; rows behind the last sequence keep what
    they hold."""
    if q.dim() != 3 or q.shape[2] != cache.d:
        raise ValueError("q is [T, Hq, d] with the cache's d")
    if out is not None and (out.shape != q.shape or out.dtype != q.dtype
                            or not out.is_contiguous()):
        raise ValueError("out must be contiguous, with q's shape and dtype")
    dt = _dtype_code(q)
    T, Hq, _ = q.shape

    def body(handle, get_ws):
        qc = q.contiguous()
        o = torch.empty_like(qc) if out is None else out
        lse = torch.empty(Hq * T, dtype=torch.float32, device=cache.device) if return_lse else None
        L = lib()
        key = (T, Hq, dt, cache.Hkv, cache.d, cache._code)
        nbytes = batch._ws_bytes.get(key)
        if nbytes is None:
            nbytes = L.tam_paged_attention_workspace(T, Hq, dt, cache._ref, batch._ref)
            if nbytes:
                batch._ws_bytes[key] = nbytes
        ws = get_ws(nbytes)
        _raise(L.tam_paged_gqa_attention(T, Hq, dt, qc.data_ptr(), cache._ref, batch._ref,
                                         o.data_ptr(), None if lse is None else lse.data_ptr(),
                                         ws.data_ptr(), ws.numel() if nbytes else 0, handle),
               "paged_gqa_attention")
        return ((o, lse) if return_lse else o), ws

    return _paged_call(cache, batch, (q, out), workspace, stream, check, body)
