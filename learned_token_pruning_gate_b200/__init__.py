"""TokenGate gated-prefill hot path for B200 (sm_100a).

Thin Python binding over ``libtokengate.so`` (C ABI in ``include/tokengate.h``).
This module only marshals arguments: torch tensors supply device memory and the
current CUDA stream, every step runs in the library's kernels.  There is no
fallback: if the library is missing or a call fails, an exception is raised.

The four calls follow the method's forward pass (TokenGate abstract page;
news write-ups, "how it works"):

    gate_score -> topk_select -> compact_gather -> gated_attention

``gated_prefill`` chains them for one prompt batch.  Decoding from what a prefill
leaves goes through ``paged_attention``, the ``cache_*`` calls, ``gated_delta_step``
and ``beam_select`` (``pipeline.PagedCache`` and ``pipeline.GatedDecoder`` put them
together).
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import os

import numpy as np
import torch

__all__ = [
    "TG_BF16", "TG_FP32", "ALGO_AUTO", "ALGO_SIMT", "ALGO_TCGEN05", "TokenGateError",
    "library", "kept_offsets", "gate_score", "topk_select", "compact_gather", "gated_attention",
    "gated_prefill", "device_status", "EXPORTED_SYMBOLS", "attention_workspace_bytes",
    "attention_kernel", "topk_select_multi", "random_select", "gated_attention_backward",
    "attention_backward_workspace_bytes", "rmsnorm", "qkv_rope_emit", "swiglu", "gated_delta_scan",
    "topk_workspace_bytes", "topk_workspace", "delta_scan_workspace_bytes",
    "paged_attention", "paged_attention_workspace", "cache_update", "cache_compact",
    "cache_copy_pages", "cache_append", "gated_delta_step", "beam_select", "beam_select_workspace",
]

TG_BF16, TG_FP32 = 0, 1
ALGO_AUTO, ALGO_SIMT, ALGO_TCGEN05 = 0, 1, 2
MAX_BATCH = 128
MAX_GATHER_TENSORS = 8

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtokengate.so")

EXPORTED_SYMBOLS = (
    "tg_status_string", "tg_last_error_message", "tg_version", "tg_device_status",
    "tg_kept_offsets", "tg_gate_score", "tg_topk_select", "tg_compact_gather",
    "tg_gated_attention", "tg_attention_workspace_bytes", "tg_attention_kernel",
    "tg_gated_attention_noalloc", "tg_topk_select_multi", "tg_random_select",
    "tg_gated_attention_backward", "tg_attention_backward_workspace_bytes", "tg_rmsnorm",
    "tg_qkv_rope_emit", "tg_swiglu", "tg_gated_delta_scan", "tg_last_device_error",
    "tg_topk_workspace_bytes", "tg_gate_score_hist", "tg_topk_select_ws",
    "tg_gated_delta_scan_chunked", "tg_delta_scan_workspace_bytes", "tg_topk_select_multi_ws",
    "tg_paged_attention", "tg_paged_attention_workspace_bytes", "tg_cache_update",
    "tg_cache_compact", "tg_cache_copy_pages", "tg_cache_append", "tg_gated_delta_step",
    "tg_beam_select", "tg_beam_select_workspace_bytes",
)
MAX_BUDGETS = 8
MAX_SEQS = 1024
MAX_BEAMS = 32
PAGE_SIZES = (16, 32, 64, 128)
ATTN_KERNELS = {0: "attn_simt_kernel", 1: "attn_tc_kernel", 2: "attn_tc_kernel (key-range split)",
                3: "attn_pair_kernel"}


class TokenGateError(RuntimeError):
    """A libtokengate call returned an error status."""

    def __init__(self, fn, status, message):
        super().__init__(f"{fn}: {status}: {message}")
        self.status = status


class GatherTensor(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p),
                ("row_elems", ctypes.c_int32), ("rope_heads", ctypes.c_int32)]


class PagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64),
                ("layers", ctypes.c_int32)]


CacheUpdate = collections.namedtuple("CacheUpdate", "table lens refs start copy_src copy_dst")
CacheCompact = collections.namedtuple("CacheCompact",
                                      "table refs page_map copy_src copy_dst counts")

_lib = None
_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_i32p = ctypes.POINTER(ctypes.c_int32)


def library():
    """Load libtokengate.so (built by ``python -m learned_token_pruning_gate_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m learned_token_pruning_gate_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    L.tg_status_string.restype = ctypes.c_char_p
    L.tg_status_string.argtypes = [ctypes.c_int]
    L.tg_last_error_message.restype = ctypes.c_char_p
    L.tg_version.restype = ctypes.c_char_p
    L.tg_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_uint32)]
    L.tg_last_device_error.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
    L.tg_kept_offsets.argtypes = [_i32, _i32p, _i32p, _i32p, _i32p, _i32p]
    L.tg_gate_score.argtypes = [_vp, ctypes.c_int, _i64, _i32, _vp, _vp, _i32, _vp, _f32, _vp,
                                _i32, _vp]
    L.tg_topk_select.argtypes = [_vp, _i32, _i32p, _i32p, _i32p, _i32p, _vp, _vp, _vp]
    L.tg_topk_workspace_bytes.argtypes = [_i32, _i64]
    L.tg_gate_score_hist.argtypes = [_vp, ctypes.c_int, _i64, _i32, _vp, _vp, _i32, _vp, _f32,
                                     _vp, _i32, _i32p, _i32p, _i32p, _vp, ctypes.c_size_t, _i32,
                                     _vp]
    L.tg_topk_select_ws.argtypes = [_vp, _i32, _i32p, _i32p, _i32p, _i32p, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp]
    L.tg_topk_select_multi.argtypes = [_vp, _i32, _i32p, _i32p, _i32p, _i32, _i32p,
                                       ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp]
    L.tg_topk_select_multi_ws.argtypes = [_vp, _i32, _i32p, _i32p, _i32p, _i32, _i32p,
                                          ctypes.POINTER(_vp), ctypes.POINTER(_vp), _vp,
                                          ctypes.c_size_t, _vp]
    L.tg_random_select.argtypes = [_vp, _i32, _i32p, _i32p, _i32p, _i32p, _vp, _vp, _vp]
    L.tg_compact_gather.argtypes = [_vp, _i64, _i32, _i32p, _i32p, _i32p, _i32p, ctypes.c_int,
                                    ctypes.POINTER(GatherTensor), _i32, _i32, ctypes.c_double,
                                    _vp, _vp, _vp]
    L.tg_gated_attention.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i32, _i32p, _i32, _i32, _i32,
                                     _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _i32, _vp]
    L.tg_attention_workspace_bytes.argtypes = [ctypes.c_int, _i32, _i32p, _i32, _i32, _i32, _i32,
                                               ctypes.POINTER(ctypes.c_size_t)]
    L.tg_attention_kernel.argtypes = [ctypes.c_int, _i32, _i32p, _i32, _i32, _i32, _i32, _i32,
                                      ctypes.POINTER(ctypes.c_int32)]
    L.tg_gated_attention_noalloc.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i32, _i32p, _i32, _i32,
                                             _i32, _vp, _vp, _vp, _vp, _vp, _i32, _vp]
    L.tg_gated_attention_backward.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i32, _i32p, _i32, _i32,
                                              _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _vp, ctypes.c_size_t, _i32, _vp]
    L.tg_attention_backward_workspace_bytes.argtypes = [_i32, _i32p, _i32,
                                                        ctypes.POINTER(ctypes.c_size_t)]
    L.tg_rmsnorm.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i64, _i32, _f32, _vp]
    L.tg_qkv_rope_emit.argtypes = [_vp, ctypes.c_int, _i32, _i32p, _i32p, _vp, _i32, _i32, _i32,
                                   _vp, _vp, _f32, ctypes.c_double, _vp, _vp, _vp, _vp]
    L.tg_swiglu.argtypes = [_vp, _vp, ctypes.c_int, _i64, _i32, _vp]
    L.tg_gated_delta_scan.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _i32p, _i32, _i32,
                                      _f32, _vp, _vp, _vp]
    L.tg_gated_delta_scan_chunked.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _i32p,
                                              _i32, _i32, _f32, _vp, _vp, _vp, ctypes.c_size_t,
                                              _vp]
    L.tg_delta_scan_workspace_bytes.argtypes = [_i32, _i32p, _i32, _i32,
                                                ctypes.POINTER(ctypes.c_size_t)]
    sz, szp = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
    L.tg_paged_attention.argtypes = [_vp, _vp, _vp, ctypes.c_int] + [_i32] * 6 + [
        _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, sz, _vp]
    L.tg_paged_attention_workspace_bytes.argtypes = [ctypes.c_int, _i32, _i32, _i32, _i32, szp]
    L.tg_cache_update.argtypes = [_vp, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _i32] + [_vp] * 8
    L.tg_cache_compact.argtypes = [_vp, _vp, _i32, _vp, _i32, _i32, _i32] + [_vp] * 7
    L.tg_cache_copy_pages.argtypes = [ctypes.POINTER(PagePool), _i32, _i32, _vp, _vp, _i32, _vp,
                                      _vp]
    L.tg_cache_append.argtypes = [_vp, _vp, _vp, ctypes.c_int, _i64, _i32, _vp, _vp, _i32, _i32,
                                  _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp]
    L.tg_gated_delta_step.argtypes = [_vp, _vp, _vp, ctypes.c_int, _vp, _vp, _i32, _i32, _i32,
                                      _f32, _vp, _i32, _vp, _vp, _vp, _vp]
    L.tg_beam_select.argtypes = [_vp, ctypes.c_int, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp,
                                 _vp, sz, _vp]
    L.tg_beam_select_workspace_bytes.argtypes = [_i32, _i32, _i32, _i32, szp]
    for name in EXPORTED_SYMBOLS:
        if name not in ("tg_status_string", "tg_last_error_message", "tg_version",
                        "tg_topk_workspace_bytes"):
            getattr(L, name).restype = ctypes.c_int
    L.tg_topk_workspace_bytes.restype = ctypes.c_size_t
    _lib = L
    return L


def _check(fn, status):
    if status != 0:
        L = library()
        raise TokenGateError(fn, L.tg_status_string(status).decode(),
                             L.tg_last_error_message().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _host_i32(a):
    arr = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return arr, arr.ctypes.data_as(_i32p)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return TG_BF16
    if t.dtype == torch.float32:
        return TG_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libtokengate operates on CUDA tensors only")


def _expect(name, t, shape, dtype, device):
    """A caller-passed tensor must match what the call reads or writes exactly:
    the kernels take raw pointers and trust the sizes derived from the other
    arguments, so a smaller buffer would be read or written past its end."""
    if t is None or (t.shape == shape and t.dtype is dtype and t.device == device
                     and t.is_contiguous()):
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def device_status(stream=None):
    """Synchronise and return (and clear) the device status bits (0 = no failure)."""
    bits = ctypes.c_uint32(0)
    st = stream if stream is not None else _stream()
    rc = library().tg_device_status(st, ctypes.byref(bits))
    if rc not in (0, 7):
        _check("tg_device_status", rc)
    return bits.value


def kept_offsets(cu_seqlens, doc_begin, doc_end, budget) -> np.ndarray:
    """Host-side kept-row offsets cu_kept [B+1] (validates the prompt batch)."""
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    k, k_p = _host_i32(budget)
    out = np.zeros(len(s) + 1, np.int32)
    _check("tg_kept_offsets", library().tg_kept_offsets(len(s), cu_p, s_p, e_p, k_p,
                                                        out.ctypes.data_as(_i32p)))
    return out


def topk_workspace_bytes(batch, total_tokens=0):
    """Bytes of the top-K workspace (first-pass histograms) for `batch` prompts."""
    return int(library().tg_topk_workspace_bytes(int(batch), int(total_tokens)))


def topk_workspace(batch, device=None):
    """A zeroed top-K workspace for `batch` prompts (uint8 device tensor)."""
    return torch.zeros(topk_workspace_bytes(batch), dtype=torch.uint8, device=device or "cuda")


def gate_score(h, W1, b1, w2, b2, out=None, algo=ALGO_AUTO, topk_ws=None, cu_seqlens=None,
               doc_begin=None, doc_end=None):
    """z = w2 . GELU(W1 h + b1) + b2 for every row of h [n, d].

    With ``topk_ws`` (a zeroed top-K workspace) and the prompt spans, the gate
    also counts the selection's first radix pass into it (tg_gate_score_hist),
    for a following ``topk_select(..., workspace=topk_ws)``."""
    n, d = h.shape
    dg = W1.shape[0]
    if W1.shape[1] != d or W1.dtype != h.dtype:
        raise ValueError("W1 must be [d_hidden, d_model] with h's dtype")
    _expect("h", h, (n, d), h.dtype, h.device)
    _expect("W1", W1, (dg, d), h.dtype, h.device)
    _expect("b1", b1, (dg,), torch.float32, h.device)
    _expect("w2", w2, (dg,), torch.float32, h.device)
    _expect("out", out, (n,), torch.float32, h.device)
    _need_cuda(h, W1, b1, w2)
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=h.device)
    if topk_ws is None:
        _check("tg_gate_score", library().tg_gate_score(
            _ptr(h), _dtype_code(h), n, d, _ptr(W1), _ptr(b1), dg, _ptr(w2), float(b2),
            _ptr(out), algo, _stream(h.device)))
        return out
    if topk_ws.dtype != torch.uint8 or not topk_ws.is_contiguous() or topk_ws.device != h.device:
        raise ValueError("topk_ws must be a contiguous uint8 tensor on h's device")
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    _check("tg_gate_score_hist", library().tg_gate_score_hist(
        _ptr(h), _dtype_code(h), n, d, _ptr(W1), _ptr(b1), dg, _ptr(w2), float(b2), _ptr(out),
        len(s), cu_p, s_p, e_p, _ptr(topk_ws), topk_ws.numel(), algo, _stream(h.device)))
    return out


def topk_select(z, cu_seqlens, doc_begin, doc_end, budget, kept_idx=None, cu_kept=None,
                workspace=None):
    """Per-prompt top-K of the document span (question kept).

    ``workspace``: a top-K workspace, possibly holding the gate's first-pass
    histograms of these scores (tg_topk_select_ws); left zeroed.
    Returns (kept_idx [M] int32 device, cu_kept [B+1] int32 device, cu_kept_host).
    """
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    k, k_p = _host_i32(budget)
    host = kept_offsets(cu, s, e, k)
    M = int(host[-1])
    _expect("z", z, (int(cu[-1]),), torch.float32, z.device)
    _expect("kept_idx", kept_idx, (M,), torch.int32, z.device)
    _expect("cu_kept", cu_kept, (len(s) + 1,), torch.int32, z.device)
    if workspace is not None and (workspace.dtype != torch.uint8 or
                                  not workspace.is_contiguous() or workspace.device != z.device):
        raise ValueError("workspace must be a contiguous uint8 tensor on z's device")
    _need_cuda(z)
    if kept_idx is None:
        kept_idx = torch.empty(max(M, 1), dtype=torch.int32, device=z.device)[:M]
    if cu_kept is None:
        cu_kept = torch.empty(len(s) + 1, dtype=torch.int32, device=z.device)
    if workspace is None:
        _check("tg_topk_select", library().tg_topk_select(
            _ptr(z), len(s), cu_p, s_p, e_p, k_p, _ptr(kept_idx), _ptr(cu_kept),
            _stream(z.device)))
    else:
        _check("tg_topk_select_ws", library().tg_topk_select_ws(
            _ptr(z), len(s), cu_p, s_p, e_p, k_p, _ptr(kept_idx), _ptr(cu_kept), _ptr(workspace),
            workspace.numel(), _stream(z.device)))
    return kept_idx, cu_kept, host


def topk_select_multi(z, cu_seqlens, doc_begin, doc_end, budgets, workspace=None):
    """Top-K for a budget sweep from one score vector: budgets is a list of
    per-prompt budget lists (at most MAX_BUDGETS).  One launch.  With
    ``workspace`` (a top-K workspace the gate counted these scores into, see
    gate_score) every budget takes its first radix pass from that one histogram.

    Returns a list of (kept_idx [M_q] device, cu_kept [B+1] device, cu_kept_host).
    """
    _need_cuda(z)
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    _expect("z", z, (int(cu[-1]),), torch.float32, z.device)
    ks = np.ascontiguousarray(np.asarray(budgets, dtype=np.int32).reshape(len(budgets), len(s)))
    outs, kept_ptrs, cu_ptrs = [], (_vp * len(ks))(), (_vp * len(ks))()
    for q, k in enumerate(ks):
        host = kept_offsets(cu, s, e, k)
        M = int(host[-1])
        kept = torch.empty(max(M, 1), dtype=torch.int32, device=z.device)[:M]
        cuk = torch.empty(len(s) + 1, dtype=torch.int32, device=z.device)
        kept_ptrs[q], cu_ptrs[q] = kept.data_ptr() if M else None, cuk.data_ptr()
        outs.append((kept, cuk, host))
    if workspace is None:
        _check("tg_topk_select_multi", library().tg_topk_select_multi(
            _ptr(z), len(s), cu_p, s_p, e_p, len(ks), ks.ctypes.data_as(_i32p), kept_ptrs,
            cu_ptrs, _stream(z.device)))
        return outs
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.device != z.device:
        raise ValueError("workspace must be a contiguous uint8 tensor on z's device")
    _check("tg_topk_select_multi_ws", library().tg_topk_select_multi_ws(
        _ptr(z), len(s), cu_p, s_p, e_p, len(ks), ks.ctypes.data_as(_i32p), kept_ptrs, cu_ptrs,
        _ptr(workspace), workspace.numel(), _stream(z.device)))
    return outs


def random_select(keys, cu_seqlens, doc_begin, doc_end, budget):
    """Random-K selection from caller-drawn uint32 keys (a device tensor of
    torch.int32 holding the key bits, one per token): the K document tokens with
    the largest keys, question kept.  Returns (kept_idx, cu_kept, cu_kept_host)."""
    _need_cuda(keys)
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    k, k_p = _host_i32(budget)
    host = kept_offsets(cu, s, e, k)
    M = int(host[-1])
    _expect("keys", keys, (int(cu[-1]),), torch.int32, keys.device)
    kept_idx = torch.empty(max(M, 1), dtype=torch.int32, device=keys.device)[:M]
    cu_kept = torch.empty(len(s) + 1, dtype=torch.int32, device=keys.device)
    _check("tg_random_select", library().tg_random_select(
        _ptr(keys), len(s), cu_p, s_p, e_p, k_p, _ptr(kept_idx), _ptr(cu_kept),
        _stream(keys.device)))
    return kept_idx, cu_kept, host


def compact_gather(kept_idx, cu_seqlens, doc_begin, doc_end, budget, tensors, rope_heads=None,
                   head_dim=0, rope_theta=1e6, z=None, logsig_out=None, outs=None):
    """Gather kept rows of each tensor in ``tensors`` (RoPE where rope_heads[i] > 0).

    Returns (list of compacted tensors, logsig [M] fp32 or None).
    """
    if len(tensors) > MAX_GATHER_TENSORS:
        raise ValueError("too many tensors")
    cu, cu_p = _host_i32(cu_seqlens)
    s, s_p = _host_i32(doc_begin)
    e, e_p = _host_i32(doc_end)
    k, k_p = _host_i32(budget)
    M = kept_idx.shape[0]
    dtypes = {t.dtype for t in tensors}
    if len(dtypes) > 1:
        raise ValueError("all gathered tensors must share one dtype")
    dcode = _dtype_code(tensors[0]) if tensors else TG_BF16
    rope_heads = rope_heads or [0] * len(tensors)
    dev0 = tensors[0].device if tensors else kept_idx.device
    _expect("kept_idx", kept_idx, (M,), torch.int32, dev0)
    N = int(cu[-1])
    for i, t in enumerate(tensors):
        _expect(f"tensors[{i}]", t, (N,) + tuple(t.shape[1:]), tensors[0].dtype, dev0)
    if z is not None:
        _expect("z", z, (N,), torch.float32, dev0)
    if outs is None:
        outs = [torch.empty((M,) + tuple(t.shape[1:]), dtype=t.dtype, device=t.device)
                for t in tensors]
    if len(outs) != len(tensors):
        raise ValueError("one output per gathered tensor")
    for i, (t, o) in enumerate(zip(tensors, outs)):
        _expect(f"outs[{i}]", o, (M,) + tuple(t.shape[1:]), t.dtype, dev0)
    if logsig_out is not None:
        _expect("logsig_out", logsig_out, (M,), torch.float32, dev0)
    _need_cuda(kept_idx, z, *tensors)
    arr = (GatherTensor * max(len(tensors), 1))()
    for i, (src, dst) in enumerate(zip(tensors, outs)):
        if not src.is_contiguous() or not dst.is_contiguous():
            raise ValueError("gather tensors must be contiguous")
        arr[i].src = src.data_ptr()
        arr[i].dst = dst.data_ptr()
        arr[i].row_elems = src[0].numel() if src.shape[0] > 0 else int(np.prod(src.shape[1:]))
        arr[i].rope_heads = int(rope_heads[i])
    if z is not None and logsig_out is None:
        logsig_out = torch.empty(M, dtype=torch.float32, device=z.device)
    dev = (tensors[0].device if tensors else z.device)
    _check("tg_compact_gather", library().tg_compact_gather(
        _ptr(kept_idx), M, len(s), cu_p, s_p, e_p, k_p, dcode, arr, len(tensors), head_dim,
        float(rope_theta), _ptr(z), _ptr(logsig_out), _stream(dev)))
    return outs, logsig_out


def _attention_operands(q, k, v, logsig, gain, temp):
    """q [M, Hq, d], k and v [M, Hkv, d] of one dtype on one device, contiguous;
    logsig [M], gain and temp [Hq] fp32.  The kernels read k and v with q's
    element size and row count, so any mismatch would read past their end."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [rows, heads, head_dim]")
    M, Hq, dh = q.shape
    Hkv = k.shape[1]
    if Hkv <= 0 or Hq % Hkv != 0:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} kv heads")
    _expect("q", q, (M, Hq, dh), q.dtype, q.device)
    _expect("k", k, (M, Hkv, dh), q.dtype, q.device)
    _expect("v", v, (M, Hkv, dh), q.dtype, q.device)
    _expect("logsig", logsig, (M,), torch.float32, q.device)
    _expect("gain", gain, (Hq,), torch.float32, q.device)
    _expect("temp", temp, (Hq,), torch.float32, q.device)


def attention_workspace_bytes(cu_kept_host, n_q_heads, n_kv_heads, head_dim, dtype="bf16",
                              algo=ALGO_AUTO):
    """Workspace bytes tg_gated_attention may use for this batch on the current device."""
    cu, cu_p = _host_i32(cu_kept_host)
    code = 0 if dtype in ("bf16", torch.bfloat16) else 1
    out = ctypes.c_size_t(0)
    _check("tg_attention_workspace_bytes", library().tg_attention_workspace_bytes(
        code, len(cu) - 1, cu_p, n_q_heads, n_kv_heads, head_dim, algo, ctypes.byref(out)))
    return int(out.value)


def attention_kernel(cu_kept_host, n_q_heads, n_kv_heads, head_dim, dtype="bf16",
                     algo=ALGO_AUTO, with_workspace=True):
    """Name of the attention kernel tg_gated_attention launches for this batch."""
    cu, cu_p = _host_i32(cu_kept_host)
    code = 0 if dtype in ("bf16", torch.bfloat16) else 1
    out = ctypes.c_int32(-1)
    _check("tg_attention_kernel", library().tg_attention_kernel(
        code, len(cu) - 1, cu_p, n_q_heads, n_kv_heads, head_dim, algo, int(with_workspace),
        ctypes.byref(out)))
    return ATTN_KERNELS[out.value]


def gated_attention(q, k, v, cu_kept_host, logsig=None, gain=None, temp=None, out=None,
                    lse=None, algo=ALGO_AUTO, want_lse=False, workspace="auto"):
    """Token-gated causal GQA attention over packed kept rows.

    q [M, Hq, d], k/v [M, Hkv, d]; cu_kept_host [B+1] host offsets.
    workspace: "auto" (allocate what the call can use), None (no split), or a
    uint8 device tensor.  Returns (out [M, Hq, d], lse [Hq, M] or None).
    """
    _attention_operands(q, k, v, logsig, gain, temp)
    M, Hq, dh = q.shape
    Hkv = k.shape[1]
    cu, cu_p = _host_i32(cu_kept_host)
    if int(cu[-1]) != M:
        raise ValueError(f"cu_kept_host ends at {int(cu[-1])}, q has {M} rows")
    _expect("out", out, (M, Hq, dh), q.dtype, q.device)
    _expect("lse", lse, (Hq, M), torch.float32, q.device)
    if workspace is not None and not isinstance(workspace, str):
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
                workspace.device != q.device:
            raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    _need_cuda(q, k, v, logsig, gain, temp)
    if out is None:
        out = torch.empty_like(q)
    if want_lse and lse is None:
        lse = torch.empty((Hq, M), dtype=torch.float32, device=q.device)
    if isinstance(workspace, str):
        nbytes = attention_workspace_bytes(cu, Hq, Hkv, dh, q.dtype, algo)
        workspace = (torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None)
    ws_bytes = 0 if workspace is None else workspace.numel()
    _check("tg_gated_attention", library().tg_gated_attention(
        _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), len(cu) - 1, cu_p, Hq, Hkv, dh, _ptr(logsig),
        _ptr(gain), _ptr(temp), _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes, algo,
        _stream(q.device)))
    return out, lse


def attention_backward_workspace_bytes(cu_kept_host, n_q_heads):
    """Device scratch bytes gated_attention_backward needs for this batch."""
    cu, cu_p = _host_i32(cu_kept_host)
    out = ctypes.c_size_t(0)
    _check("tg_attention_backward_workspace_bytes", library().tg_attention_backward_workspace_bytes(
        len(cu) - 1, cu_p, n_q_heads, ctypes.byref(out)))
    return int(out.value)


def gated_attention_backward(q, k, v, cu_kept_host, logsig, gain, temp, out, lse, dout,
                             algo=ALGO_AUTO, workspace=None):
    """Gradient of a loss through gated_attention with respect to the log-gates
    (and the kept rows' gate scores), the gains and the temperatures.

    dout = dL/dout [M, Hq, d]; out, lse = the forward's outputs (lse [Hq, M]).
    Returns (d_logsig [M], d_z_kept [M], d_gain [Hq], d_temp [Hq]), fp32 device.
    """
    _attention_operands(q, k, v, logsig, gain, temp)
    M, Hq, dh = q.shape
    Hkv = k.shape[1]
    if logsig is None or lse is None:
        raise ValueError("the backward needs the log-gates and the forward's lse")
    _expect("out", out, (M, Hq, dh), q.dtype, q.device)
    _expect("dout", dout, (M, Hq, dh), q.dtype, q.device)
    _expect("lse", lse, (Hq, M), torch.float32, q.device)
    cu, cu_p = _host_i32(cu_kept_host)
    if int(cu[-1]) != M:
        raise ValueError(f"cu_kept_host ends at {int(cu[-1])}, q has {M} rows")
    if workspace is not None and (workspace.dtype != torch.uint8 or
                                  not workspace.is_contiguous() or workspace.device != q.device):
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    _need_cuda(q, k, v, logsig, gain, temp, out, lse, dout)
    if workspace is None:
        workspace = torch.empty(attention_backward_workspace_bytes(cu, Hq), dtype=torch.uint8,
                                device=q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    d_l, d_z = torch.empty(M, **f32), torch.empty(M, **f32)
    d_g, d_t = torch.empty(Hq, **f32), torch.empty(Hq, **f32)
    _check("tg_gated_attention_backward", library().tg_gated_attention_backward(
        _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), len(cu) - 1, cu_p, Hq, Hkv, dh, _ptr(logsig),
        _ptr(gain), _ptr(temp), _ptr(out), _ptr(lse), _ptr(dout), _ptr(d_l), _ptr(d_z), _ptr(d_g),
        _ptr(d_t), _ptr(workspace), workspace.numel(), algo, _stream(q.device)))
    return d_l, d_z, d_g, d_t


def rmsnorm(x, weight, eps=1e-6, out=None):
    """x / sqrt(mean(x^2) + eps) * weight over the last axis of x [rows, dim]."""
    rows, dim = x.shape
    _expect("x", x, (rows, dim), x.dtype, x.device)
    _expect("weight", weight, (dim,), x.dtype, x.device)
    _expect("out", out, (rows, dim), x.dtype, x.device)
    _need_cuda(x, weight)
    if out is None:
        out = torch.empty_like(x)
    _check("tg_rmsnorm", library().tg_rmsnorm(_ptr(x), _ptr(weight), _ptr(out), _dtype_code(x),
                                              rows, dim, eps, _stream(x.device)))
    return out


def qkv_rope_emit(qkv, cu_seqlens, cu_kept_host, kept_idx, n_q_heads, n_kv_heads, head_dim,
                  q_norm_w, k_norm_w, eps=1e-6, rope_theta=1e6, q_out=None, k_out=None,
                  v_out=None):
    """Split a fused QKV projection [M, (Hq + 2 Hkv) d] into q (per-head RMSNorm,
    RoPE), k (same; the layer's KV-cache slot) and v.  Returns (q, k, v)."""
    M = qkv.shape[0]
    cu, cu_p = _host_i32(cu_seqlens)
    ck, ck_p = _host_i32(cu_kept_host)
    if int(ck[-1]) != M:
        raise ValueError(f"cu_kept_host ends at {int(ck[-1])}, qkv has {M} rows")
    _expect("qkv", qkv, (M, (n_q_heads + 2 * n_kv_heads) * head_dim), qkv.dtype, qkv.device)
    _expect("kept_idx", kept_idx, (M,), torch.int32, qkv.device)
    _expect("q_norm_w", q_norm_w, (head_dim,), qkv.dtype, qkv.device)
    _expect("k_norm_w", k_norm_w, (head_dim,), qkv.dtype, qkv.device)
    _expect("q_out", q_out, (M, n_q_heads, head_dim), qkv.dtype, qkv.device)
    _expect("k_out", k_out, (M, n_kv_heads, head_dim), qkv.dtype, qkv.device)
    _expect("v_out", v_out, (M, n_kv_heads, head_dim), qkv.dtype, qkv.device)
    _need_cuda(qkv, kept_idx, q_norm_w, k_norm_w)
    mk = lambda h: torch.empty((M, h, head_dim), dtype=qkv.dtype, device=qkv.device)  # noqa: E731
    q_out = mk(n_q_heads) if q_out is None else q_out
    k_out = mk(n_kv_heads) if k_out is None else k_out
    v_out = mk(n_kv_heads) if v_out is None else v_out
    _check("tg_qkv_rope_emit", library().tg_qkv_rope_emit(
        _ptr(qkv), _dtype_code(qkv), len(cu) - 1, cu_p, ck_p, _ptr(kept_idx), n_q_heads, n_kv_heads,
        head_dim, _ptr(q_norm_w), _ptr(k_norm_w), eps, float(rope_theta), _ptr(q_out), _ptr(k_out),
        _ptr(v_out), _stream(qkv.device)))
    return q_out, k_out, v_out


def swiglu(gate_up, out=None):
    """SiLU(gate) * up of a fused [rows, 2 inter] projection."""
    rows, two = gate_up.shape
    if two % 2:
        raise ValueError("gate_up must hold the gate and up halves side by side")
    _expect("gate_up", gate_up, (rows, two), gate_up.dtype, gate_up.device)
    _expect("out", out, (rows, two // 2), gate_up.dtype, gate_up.device)
    _need_cuda(gate_up)
    if out is None:
        out = torch.empty((rows, two // 2), dtype=gate_up.dtype, device=gate_up.device)
    _check("tg_swiglu", library().tg_swiglu(_ptr(gate_up), _ptr(out), _dtype_code(gate_up), rows,
                                            two // 2, _stream(gate_up.device)))
    return out


def delta_scan_workspace_bytes(cu_kept_host, n_heads, head_dim):
    """Device scratch bytes the chunked delta-rule scan needs for this batch."""
    ck, ck_p = _host_i32(cu_kept_host)
    out = ctypes.c_size_t(0)
    _check("tg_delta_scan_workspace_bytes", library().tg_delta_scan_workspace_bytes(
        len(ck) - 1, ck_p, int(n_heads), int(head_dim), ctypes.byref(out)))
    return int(out.value)


def gated_delta_scan(q, k, v, cu_kept_host, log_alpha, beta, eps=1e-6, out=None, state=None,
                     want_state=True, algo="chunked", workspace=None):
    """Gated delta rule over each prompt's kept rows (a Gated DeltaNet layer above the
    gate): q, k, v [M, H, d] (d 64 or 128), log_alpha, beta [M, H] fp32.  Returns
    (o [M, H, d], state [B, H, d, d] fp32 or None).

    algo: "chunked" (tg_gated_delta_scan_chunked: parallel within chunks of 64
    rows; ``workspace`` a uint8 device tensor of delta_scan_workspace_bytes, or
    None to allocate one) or "recurrent" (tg_gated_delta_scan: row by row)."""
    if algo not in ("chunked", "recurrent"):
        raise ValueError(f"algo {algo!r}: 'chunked' or 'recurrent'")
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape:
        raise ValueError(f"q, k, v must share one [M, H, d] shape: {tuple(q.shape)}, "
                         f"{tuple(k.shape)}, {tuple(v.shape)}")
    M, H, d = q.shape
    if tuple(log_alpha.shape) != (M, H) or tuple(beta.shape) != (M, H):
        raise ValueError(f"log_alpha and beta must be [M, H] = {(M, H)}")
    if log_alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise ValueError("log_alpha and beta must be float32")
    for name, t in (("q", q), ("k", k), ("v", v)):
        _expect(name, t, (M, H, d), q.dtype, q.device)
    _expect("log_alpha", log_alpha, (M, H), torch.float32, q.device)
    _expect("beta", beta, (M, H), torch.float32, q.device)
    ck, ck_p = _host_i32(cu_kept_host)
    if int(ck[-1]) != M:
        raise ValueError(f"cu_kept_host ends at {int(ck[-1])}, q has {M} rows")
    B = len(ck) - 1
    _expect("out", out, (M, H, d), q.dtype, q.device)
    _expect("state", state, (B, H, d, d), torch.float32, q.device)
    _need_cuda(q, k, v, log_alpha, beta)
    if out is None:
        out = torch.empty_like(v)
    if state is None and want_state:
        state = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
    if algo == "recurrent":
        _check("tg_gated_delta_scan", library().tg_gated_delta_scan(
            _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(log_alpha), _ptr(beta), B, ck_p, H, d,
            float(eps), _ptr(out), _ptr(state) if state is not None else None,
            _stream(q.device)))
        return out, state
    if workspace is None:
        nbytes = delta_scan_workspace_bytes(ck, H, d)
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or \
            workspace.device != q.device:
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    _check("tg_gated_delta_scan_chunked", library().tg_gated_delta_scan_chunked(
        _ptr(q), _ptr(k), _ptr(v), _dtype_code(q), _ptr(log_alpha), _ptr(beta), B, ck_p, H, d,
        float(eps), _ptr(out), _ptr(state) if state is not None else None, _ptr(workspace),
        workspace.numel(), _stream(q.device)))
    return out, state


def gated_prefill(h, q, k, v, W1, b1, w2, b2, gain, temp, cu_seqlens, doc_begin, doc_end,
                  budget, rope_theta=1e6, algo=ALGO_AUTO, want_lse=False):
    """One gated layer: score (with the selection's first radix pass), select,
    compact, attend.  Returns a dict of device tensors."""
    B = len(np.asarray(doc_begin))
    ws = topk_workspace(B, device=h.device) if B > 0 else None
    z = gate_score(h, W1, b1, w2, b2, algo=algo, topk_ws=ws, cu_seqlens=cu_seqlens,
                   doc_begin=doc_begin, doc_end=doc_end)
    kept_idx, cu_kept, cu_kept_host = topk_select(z, cu_seqlens, doc_begin, doc_end, budget,
                                                  workspace=ws)
    Hq, dh = q.shape[1], q.shape[2]
    (h_c, q_c, k_c, v_c), logsig = compact_gather(
        kept_idx, cu_seqlens, doc_begin, doc_end, budget, [h, q, k, v],
        rope_heads=[0, Hq, k.shape[1], 0], head_dim=dh, rope_theta=rope_theta, z=z)
    o, lse = gated_attention(q_c, k_c, v_c, cu_kept_host, logsig, gain, temp, algo=algo,
                             want_lse=want_lse)
    return dict(z=z, kept_idx=kept_idx, cu_kept=cu_kept, cu_kept_host=cu_kept_host, h=h_c, q=q_c,
                k=k_c, v=v_c, logsig=logsig, out=o, lse=lse)


# ---- decoding ----------------------------------------------------------------------------------
#
# A decoding step is a few microseconds on the GPU, so its calls look their operands over in one
# expression (_fits) and go through the checks that name a mismatch (_expect) only when it fails.


def _fits(t, shape, dtype, index):
    """What _expect asks of a tensor, on CUDA device `index`."""
    return (t.shape == shape and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous())


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(index):
    """Makes CUDA device `index` current for a call; nothing to do when it is already."""
    if torch._C._cuda_getDevice() == index:  # (a tensor lives there: CUDA is initialised)
        return _SAME_DEVICE
    return torch.cuda.device(index)


_SAME_DEVICE = contextlib.nullcontext()


def _raw_stream(index):
    """The current stream's handle, without the Stream object that _stream makes (2 us)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _workspace(workspace, index):
    if not (workspace.dtype is torch.uint8 and workspace.get_device() == index
            and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on the operands' device")


def _expect_pools(k_pages, v_pages, logsig_pages):
    """(n_pages, n_kv_heads, page_size, head_dim) of one layer's pages."""
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be [n_pages, n_kv_heads, page_size, head_dim]")
    P, Hkv, page, d = k_pages.shape
    _expect("k_pages", k_pages, (P, Hkv, page, d), k_pages.dtype, k_pages.device)
    _expect("v_pages", v_pages, (P, Hkv, page, d), k_pages.dtype, k_pages.device)
    _expect("logsig_pages", logsig_pages, (P, page), torch.float32, k_pages.device)


def _expect_table(table, lens, device):
    if table.dim() != 2:
        raise ValueError("table must be [batch, max_pages]")
    _expect("table", table, table.shape, torch.int32, device)
    _expect("lens", lens, (table.shape[0],), torch.int32, device)


def paged_attention_workspace(batch, n_q_heads, n_kv_heads, head_dim, dtype=torch.bfloat16,
                              device=None):
    """A workspace for paged_attention of this shape (uint8 device tensor): with it a sequence's
    keys are split over several SMs.  Calls on it must not overlap on the GPU."""
    device = torch.device(device or "cuda")
    out = ctypes.c_size_t(0)
    with torch.cuda.device(device):
        _check("tg_paged_attention_workspace_bytes", library().tg_paged_attention_workspace_bytes(
            TG_BF16 if dtype in ("bf16", torch.bfloat16) else TG_FP32, batch, n_q_heads,
            n_kv_heads, head_dim, ctypes.byref(out)))
        return torch.empty(int(out.value), dtype=torch.uint8, device=device)


def _expect_paged_attention(q, k_pages, v_pages, table, lens, logsig_pages, gain, temp, out, lse):
    if q.dim() != 3:
        raise ValueError("q must be [batch, heads, head_dim]")
    B, Hq, dh = q.shape
    _expect("q", q, (B, Hq, dh), q.dtype, q.device)
    _expect_pools(k_pages, v_pages, logsig_pages)
    Hkv = k_pages.shape[1]
    if k_pages.shape[3] != dh or k_pages.dtype != q.dtype or k_pages.device != q.device:
        raise ValueError(f"k_pages: {tuple(k_pages.shape)} {k_pages.dtype} on {k_pages.device} "
                         f"for q {tuple(q.shape)} {q.dtype} on {q.device}")
    if Hkv <= 0 or Hq % Hkv != 0:
        raise ValueError(f"{Hq} query heads are not a multiple of {Hkv} kv heads")
    _expect_table(table, lens, q.device)
    if table.shape[0] != B:
        raise ValueError(f"table: {table.shape[0]} sequences, q has {B}")
    _expect("gain", gain, (Hq,), torch.float32, q.device)
    _expect("temp", temp, (Hq,), torch.float32, q.device)
    _expect("out", out, (B, Hq, dh), q.dtype, q.device)
    _expect("lse", lse, (Hq, B), torch.float32, q.device)
    _need_cuda(q)


def paged_attention(q, k_pages, v_pages, table, lens, logsig_pages=None, gain=None, temp=None,
                    out=None, lse=None, want_lse=False, workspace="auto"):
    """Token-gated attention of one new token per sequence over a paged cache.

    q [B, Hq, d]; k_pages, v_pages [P, Hkv, page, d]; table [B, max_pages] and lens [B] int32 on
    the device; logsig_pages [P, page] or None (no bias); gain (None: 1), temp (None: 1) [Hq].
    workspace: "auto" (allocate one), None (no split), or paged_attention_workspace(...), which a
    decoding loop keeps.  Returns (out [B, Hq, d], lse [Hq, B] or None)."""
    dt, i, f32, i32 = q.dtype, q.get_device(), torch.float32, torch.int32
    if q.dim() != 3 or k_pages.dim() != 4 or table.dim() != 2:
        _expect_paged_attention(q, k_pages, v_pages, table, lens, logsig_pages, gain, temp, out,
                                lse)
    B, Hq, dh = q.shape
    P, Hkv, page, d = pool = k_pages.shape
    max_pages = table.shape[1]
    if workspace is not None and not isinstance(workspace, str):
        _workspace(workspace, i)
    if not (i >= 0 and d == dh and Hkv > 0 and Hq % Hkv == 0 and q.is_contiguous()
            and _fits(k_pages, pool, dt, i) and _fits(v_pages, pool, dt, i)
            and _fits(table, (B, max_pages), i32, i) and _fits(lens, (B,), i32, i)
            and (logsig_pages is None or _fits(logsig_pages, (P, page), f32, i))
            and (gain is None or _fits(gain, (Hq,), f32, i))
            and (temp is None or _fits(temp, (Hq,), f32, i))
            and (out is None or _fits(out, (B, Hq, dh), dt, i))
            and (lse is None or _fits(lse, (Hq, B), f32, i))):
        _expect_paged_attention(q, k_pages, v_pages, table, lens, logsig_pages, gain, temp, out,
                                lse)
    with _on(i):
        one = torch.ones(Hq, device=q.device) if gain is None or temp is None else None
        gain = one if gain is None else gain
        temp = one if temp is None else temp
        out = torch.empty_like(q) if out is None else out
        if want_lse and lse is None:
            lse = gain.new_empty((Hq, B))
        if isinstance(workspace, str):
            workspace = paged_attention_workspace(B, Hq, Hkv, dh, dt, q.device)
        # a workspace of no bytes has no address: the call needs none of it
        ws_bytes = 0 if workspace is None else workspace.numel()
        _check("tg_paged_attention", library().tg_paged_attention(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _dtype_code(q), B, Hq, Hkv, dh,
            P, page, table.data_ptr(), max_pages, lens.data_ptr(), _addr(logsig_pages),
            gain.data_ptr(), temp.data_ptr(), out.data_ptr(), _addr(lse),
            workspace.data_ptr() if ws_bytes else None, ws_bytes, _raw_stream(i)))
    return out, lse


def _expect_cache_update(table, lens, refs, parent, cu_new, table_out, lens_out, refs_out, start,
                         copy_src, copy_dst):
    dev = table.device
    _expect_table(table, lens, dev)
    B, mp = table.shape
    Bo = B if parent is None else parent.shape[0]
    _expect("refs", refs, (refs.shape[0],), torch.int32, dev)
    _expect("parent", parent, (Bo,), torch.int32, dev)
    _expect("cu_new", cu_new, (Bo + 1,), torch.int32, dev)
    _expect("table_out", table_out, (Bo, mp), torch.int32, dev)
    _expect("refs_out", refs_out, refs.shape, torch.int32, dev)
    for name, t in (("lens_out", lens_out), ("start", start), ("copy_src", copy_src),
                    ("copy_dst", copy_dst)):
        _expect(name, t, (Bo,), torch.int32, dev)
    _need_cuda(table)


def cache_update(table, lens, refs, page_size, parent=None, cu_new=None, table_out=None,
                 lens_out=None, refs_out=None, start=None, copy_src=None, copy_dst=None):
    """One step of a paged cache's tables: sequence i takes the pages of sequence parent[i] (-1:
    none; parent None: its own) and grows by cu_new[i + 1] - cu_new[i] tokens.

    table [B, max_pages], lens [B], refs [P], parent [B'], cu_new [B' + 1]: int32 on the device.
    Outputs that are not given are allocated (a new table is -1 behind its sequences' pages);
    refs_out may be refs, and without parents table_out and lens_out may be table and lens.
    Returns a CacheUpdate: table, lens, refs, start [B'] (position of the first new token, -1
    where the sequence did not grow), and copy_src, copy_dst [B'], the page copies for
    cache_copy_pages that have to run before anything is appended."""
    i, i32 = table.get_device(), torch.int32
    if table.dim() != 2:
        _expect_table(table, lens, table.device)
    B, mp = table.shape
    P = refs.shape[0]
    Bo = B if parent is None else parent.shape[0]
    small = (lens_out, start, copy_src, copy_dst)
    given = [t for t in small if t is not None]
    if not (i >= 0 and _fits(table, (B, mp), i32, i) and _fits(lens, (B,), i32, i)
            and _fits(refs, (P,), i32, i) and (parent is None or _fits(parent, (Bo,), i32, i))
            and (cu_new is None or _fits(cu_new, (Bo + 1,), i32, i))
            and (table_out is None or _fits(table_out, (Bo, mp), i32, i))
            and (refs_out is None or _fits(refs_out, (P,), i32, i))
            and all([_fits(t, (Bo,), i32, i) for t in given])):
        _expect_cache_update(table, lens, refs, parent, cu_new, table_out, lens_out, refs_out,
                             start, copy_src, copy_dst)
    with _on(i):
        if table_out is None:
            table_out = table.new_full((Bo, mp), -1)
        refs_out = torch.empty_like(refs) if refs_out is None else refs_out
        if len(given) < 4:  # one allocation for those that are not given
            fresh = table.new_empty((4, Bo)).unbind()
            small = fresh if not given else [f if t is None else t for f, t in zip(fresh, small)]
        lens_out, start, copy_src, copy_dst = small
        _check("tg_cache_update", library().tg_cache_update(
            table.data_ptr(), lens.data_ptr(), B, refs.data_ptr(), P, page_size, mp,
            # (an empty list of parents has no address; null would mean that there is none)
            _addr(parent) if Bo else lens.data_ptr(), Bo, _addr(cu_new), table_out.data_ptr(),
            lens_out.data_ptr(), refs_out.data_ptr(), start.data_ptr(), copy_src.data_ptr(),
            copy_dst.data_ptr(), _raw_stream(i)))
    return CacheUpdate(table_out, lens_out, refs_out, start, copy_src, copy_dst)


def _expect_cache_compact(table, lens, refs, table_out, refs_out):
    dev = table.device
    _expect_table(table, lens, dev)
    _expect("refs", refs, (refs.shape[0],), torch.int32, dev)
    _expect("table_out", table_out, table.shape, torch.int32, dev)
    _expect("refs_out", refs_out, refs.shape, torch.int32, dev)
    _need_cuda(table)


def cache_compact(table, lens, refs, page_size, table_out=None, refs_out=None):
    """Renumbers the live pages (refs > 0) of a pool into its lowest page numbers.

    Returns a CacheCompact: table, refs (renumbered; table_out and refs_out may be table and
    refs), page_map [P] (a live page's new number, -1 for free ones), copy_src and copy_dst [P]
    (the moves, -1 behind them) and counts [2] = live pages, moves.  The moves are made by
    cache_copy_pages(pools, copy_src, copy_dst, counts[1:])."""
    i, i32 = table.get_device(), torch.int32
    shape, P = table.shape, refs.shape[0]
    if not (i >= 0 and len(shape) == 2 and _fits(table, shape, i32, i)
            and _fits(lens, shape[:1], i32, i) and _fits(refs, (P,), i32, i)
            and (table_out is None or _fits(table_out, shape, i32, i))
            and (refs_out is None or _fits(refs_out, (P,), i32, i))):
        _expect_cache_compact(table, lens, refs, table_out, refs_out)
    with _on(i):
        if table_out is None:
            table_out = table.new_full(shape, -1)
        refs_out = torch.empty_like(refs) if refs_out is None else refs_out
        page_map, src, dst = table.new_empty((3, P)).unbind()
        counts = table.new_empty(2)
        _check("tg_cache_compact", library().tg_cache_compact(
            table.data_ptr(), lens.data_ptr(), shape[0], refs.data_ptr(), P, page_size, shape[1],
            table_out.data_ptr(), refs_out.data_ptr(), page_map.data_ptr(), src.data_ptr(),
            dst.data_ptr(), counts.data_ptr(), _raw_stream(i)))
    return CacheCompact(table_out, refs_out, page_map, src, dst, counts)


def cache_copy_pages(pools, copy_src, copy_dst, count=None):
    """Copies page copy_src[i] to page copy_dst[i] in every layer of every pool [layers, P, ...];
    pairs with a negative number are skipped.  count: device int32 [1], how many pairs to look at
    (None: all).  No page may be a destination twice, nor both a source and a destination."""
    if len(pools) > MAX_GATHER_TENSORS:
        raise ValueError("too many pools")
    n, i, i32 = copy_src.shape[0], copy_src.get_device(), torch.int32
    if not (i >= 0 and _fits(copy_src, (n,), i32, i) and _fits(copy_dst, (n,), i32, i)
            and (count is None or _fits(count, (1,), i32, i))):
        _expect("copy_src", copy_src, (n,), i32, copy_src.device)
        _expect("copy_dst", copy_dst, (n,), i32, copy_src.device)
        _expect("count", count, (1,), i32, copy_src.device)
    P = None
    arr = (PagePool * max(len(pools), 1))()
    for t, a in zip(pools, arr):
        shape = t.shape
        P = shape[1] if P is None and len(shape) > 1 else P
        if len(shape) < 3 or shape[1] != P or t.get_device() != i or not t.is_contiguous():
            raise ValueError(f"pools: {tuple(shape)} on {t.device}, expected contiguous "
                             f"[layers, {P}, ...] on {copy_src.device}")
        a.base = t.data_ptr()
        a.layers = shape[0]
        a.page_bytes = t.nbytes // (shape[0] * P) if t.nbytes else 16
    _need_cuda(copy_src)
    if not pools:
        return
    with _on(i):
        _check("tg_cache_copy_pages", library().tg_cache_copy_pages(
            arr, len(pools), P, copy_src.data_ptr(), copy_dst.data_ptr(), n, _addr(count),
            _raw_stream(i)))


def _expect_cache_append(k, v, cu_new, start, table, k_pages, v_pages, logsig, logsig_pages):
    _expect_pools(k_pages, v_pages, logsig_pages)
    dev, rows = k_pages.device, k.shape[0]
    _, Hkv, _, d = k_pages.shape
    _expect("k", k, (rows, Hkv, d), k_pages.dtype, dev)
    _expect("v", v, (rows, Hkv, d), k_pages.dtype, dev)
    _expect("logsig", logsig, (rows,), torch.float32, dev)
    _expect_table(table, None, dev)
    B = table.shape[0]
    _expect("cu_new", cu_new, (B + 1,), torch.int32, dev)
    _expect("start", start, (B,), torch.int32, dev)
    _need_cuda(k)


def cache_append(k, v, cu_new, start, table, k_pages, v_pages, logsig=None, logsig_pages=None):
    """Writes rows of k, v [rows, Hkv, d] (and log-gates [rows]; None: 0) into their sequences'
    pages: row i of sequence b (cu_new[b] <= i < cu_new[b + 1]) becomes token
    start[b] + i - cu_new[b]; start[b] < 0 skips the sequence.  cu_new [B + 1], start [B],
    table [B, max_pages]: int32 on the device."""
    if logsig is not None and logsig_pages is None:
        raise ValueError("logsig without logsig_pages")
    i, i32, f32, dt = k.get_device(), torch.int32, torch.float32, k.dtype
    rows, pool, shape = k.shape[0], k_pages.shape, table.shape
    if not (i >= 0 and len(pool) == 4 and len(shape) == 2 and _fits(k_pages, pool, dt, i)
            and _fits(v_pages, pool, dt, i) and _fits(k, (rows, pool[1], pool[3]), dt, i)
            and _fits(v, k.shape, dt, i) and _fits(table, shape, i32, i)
            and _fits(cu_new, (shape[0] + 1,), i32, i) and _fits(start, shape[:1], i32, i)
            and (logsig is None or _fits(logsig, (rows,), f32, i))
            and (logsig_pages is None or _fits(logsig_pages, pool[::2], f32, i))):
        _expect_cache_append(k, v, cu_new, start, table, k_pages, v_pages, logsig, logsig_pages)
    with _on(i):
        _check("tg_cache_append", library().tg_cache_append(
            k.data_ptr(), v.data_ptr(), _addr(logsig), _dtype_code(k), rows, shape[0],
            cu_new.data_ptr(), start.data_ptr(), pool[1], pool[3], pool[0], pool[2],
            table.data_ptr(), shape[1], k_pages.data_ptr(), v_pages.data_ptr(),
            _addr(logsig_pages), _raw_stream(i)))


def _expect_delta_step(q, k, v, log_alpha, beta, state, parent, out, state_out):
    if q.dim() != 3 or state.dim() != 4:
        raise ValueError("q must be [batch, heads, head_dim], state [n, heads, head_dim, head_dim]")
    B, H, d = q.shape
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        _expect(name, t, (B, H, d), q.dtype, dev)
    _expect("log_alpha", log_alpha, (B, H), torch.float32, dev)
    _expect("beta", beta, (B, H), torch.float32, dev)
    _expect("state", state, (state.shape[0], H, d, d), torch.float32, dev)
    _expect("parent", parent, (B,), torch.int32, dev)
    _expect("state_out", state_out, (B, H, d, d), torch.float32, dev)
    if parent is None and state.shape[0] < B:
        raise ValueError(f"state: {state.shape[0]} states for {B} sequences")
    _need_cuda(q)


def gated_delta_step(q, k, v, log_alpha, beta, state, parent=None, eps=1e-6, out=None,
                     state_out=None):
    """One token of the gated delta rule per sequence, from the state that gated_delta_scan or the
    last step left: q, k, v [B, H, d], log_alpha, beta [B, H] fp32, state [S, H, d, d] fp32.

    parent [B] int32 on the device: sequence b starts from state[parent[b]] (-1: from zero), the
    reordering of a beam search; state_out may then not be state.  Without parents sequence b
    starts from state[b], and state_out=state updates in place.
    Returns (out [B, H, d], state_out [B, H, d, d])."""
    i, f32, dt = q.get_device(), torch.float32, q.dtype
    if q.dim() != 3 or state.dim() != 4:
        _expect_delta_step(q, k, v, log_alpha, beta, state, parent, out, state_out)
    B, H, d = shape = q.shape
    S = state.shape[0]
    if not (i >= 0 and q.is_contiguous() and _fits(k, shape, dt, i) and _fits(v, shape, dt, i)
            and _fits(log_alpha, (B, H), f32, i) and _fits(beta, (B, H), f32, i)
            and _fits(state, (S, H, d, d), f32, i)
            and (parent is None or _fits(parent, (B,), torch.int32, i))
            and (out is None or _fits(out, shape, dt, i))
            and (state_out is None or _fits(state_out, (B, H, d, d), f32, i))
            and (parent is not None or S >= B)):
        _expect_delta_step(q, k, v, log_alpha, beta, state, parent, out, state_out)
    with _on(i):
        out = torch.empty_like(q) if out is None else out
        if state_out is None:
            state_out = beta.new_empty((B, H, d, d))
        _check("tg_gated_delta_step", library().tg_gated_delta_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), log_alpha.data_ptr(),
            beta.data_ptr(), B, H, d, eps, state.data_ptr(), S,
            _addr(parent), state_out.data_ptr(), out.data_ptr(), _raw_stream(i)))
    return out, state_out


def beam_select_workspace(n_groups, beams, vocab, n_out, device=None):
    """A workspace for beam_select of this shape (uint8 device tensor)."""
    out = ctypes.c_size_t(0)
    _check("tg_beam_select_workspace_bytes", library().tg_beam_select_workspace_bytes(
        n_groups, beams, vocab, n_out, ctypes.byref(out)))
    return torch.empty(int(out.value), dtype=torch.uint8, device=device or "cuda")


def beam_select(logits, scores, n_out=None, workspace=None):
    """The n_out (None: as many as beams) best continuations of each group of beams: logits
    [groups * beams, vocab], scores [groups, beams] fp32 (a beam's score so far; -inf: no beam).

    Returns (scores [groups, n_out] fp32 in order, parent [groups, n_out] int32 row of logits,
    token [groups, n_out] int32); places without a candidate hold -inf, -1, -1.  parent is what
    cache_update and gated_delta_step take.  workspace: beam_select_workspace(...) or None."""
    if logits.dim() != 2 or scores.dim() != 2:
        raise ValueError("logits must be [groups * beams, vocab], scores [groups, beams]")
    G, beams = scores.shape
    V = logits.shape[1]
    i, dev = logits.get_device(), logits.device
    if workspace is not None:
        _workspace(workspace, i)
    if not (i >= 0 and _fits(logits, (G * beams, V), logits.dtype, i)
            and _fits(scores, (G, beams), torch.float32, i)):
        _expect("logits", logits, (G * beams, V), logits.dtype, dev)
        _expect("scores", scores, (G, beams), torch.float32, dev)
        _need_cuda(logits)
    n_out = beams if n_out is None else n_out
    with _on(i):
        if workspace is None:
            workspace = beam_select_workspace(G, beams, V, n_out, dev)
        best, parent, token = scores.new_empty((3, G, n_out), dtype=torch.int32).unbind()
        best = best.view(torch.float32)
        _check("tg_beam_select", library().tg_beam_select(
            logits.data_ptr(), _dtype_code(logits), scores.data_ptr(), G, beams, V, n_out,
            best.data_ptr(), parent.data_ptr(), token.data_ptr(), workspace.data_ptr(),
            workspace.numel(), _raw_stream(i)))
    return best, parent, token
