"""Python binding of liblidx.so, the GB300 lightning-indexer library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI (``include/lidx.h``).  PyTorch supplies device
memory and the current stream.  There is no CPU fallback: if the library has
not been built, or no sm_103 device is present, calls raise.

Functions carry the C names:

  lidx_indexer_fwd          V4 forward: causal mask + per-row top-k
  lidx_indexer_fwd_ranges   V4 forward over explicit per-row [ks, ke) ranges
  lidx_indexer_logits       V4 logits only, causal or explicit [ks, ke) ranges
  lidx_extract_topk_scores  gather of logits at indices
  lidx_topk_rows            per-row top-k of given logits
  lidx_indexer_scores_v41   V4.1 bf16-rounded scores under a visibility mask
  lidx_indexer_topk_v41     V4.1 scores and their per-row top-k
  lidx_indexer_bwd          backward through the selected entries
  lidx_indexer_bwd_ranges   the same over explicit per-row ranges
  lidx_indexer_fwd_noalloc  fused forward with the library's own scratch
  lidx_rope_freqs           rotary frequencies in fixed point, scaled for long contexts
  lidx_rope, lidx_rope_bwd  rotary positions of queries and keys, and their gradient
  lidx_cache_append         new keys and values into a paged 8-bit cache
  lidx_cache_attn           attention over that cache, at every key or at selected ones
  lidx_workspace_bytes, lidx_cache_attn_workspace_bytes, lidx_device_status,
  lidx_status_string, lidx_set_wait_limit_ns, lidx_debug_stall_producer

Calls run on the current stream, or on ``stream``.  There the caller makes the stream wait for the inputs,
and the reader of the outputs for the stream; what a call allocates itself is the stream's own memory.
"""

from __future__ import annotations

import ctypes as C
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblidx.so")

LIDX_OK = 0
STATUS = {0: "LIDX_OK", 1: "LIDX_ERR_NULL", 2: "LIDX_ERR_SHAPE", 3: "LIDX_ERR_ALIGN",
          4: "LIDX_ERR_UNSUPPORTED", 5: "LIDX_ERR_WORKSPACE", 6: "LIDX_ERR_CUDA",
          7: "LIDX_ERR_DEVICE_TIMEOUT", 8: "LIDX_ERR_NO_DEVICE"}
OP_INDEXER_FWD, OP_INDEXER_BWD, OP_SCORES_V41, OP_TOPK_V41 = 0, 1, 2, 3
ACT = {"relu": 0, "identity": 1}
ROPE_SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
ROPE_LAYOUT = {"interleaved": 0, "half": 1}

# every symbol include/lidx.h declares
EXPORTS = ("lidx_indexer_fwd", "lidx_indexer_fwd_ranges", "lidx_indexer_logits",
           "lidx_extract_topk_scores", "lidx_topk_rows", "lidx_indexer_scores_v41",
           "lidx_indexer_topk_v41", "lidx_indexer_bwd", "lidx_indexer_bwd_ranges",
           "lidx_workspace_bytes", "lidx_device_status", "lidx_status_string", "lidx_version",
           "lidx_indexer_fwd_noalloc", "lidx_noalloc_scratch_bytes", "lidx_set_wait_limit_ns",
           "lidx_debug_stall_producer", "lidx_rope_freqs", "lidx_rope", "lidx_cache_append",
           "lidx_cache_attn", "lidx_cache_attn_workspace_bytes")


class _RopeTensor(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("xs", C.c_int64 * 3), ("ys", C.c_int64 * 3),
                ("H", C.c_int)]


class LidxError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        msg = lib().lidx_status_string(status).decode() if _lib is not None else ""
        super().__init__(f"{call} returned {STATUS.get(status, status)}: {msg}")


_lib = None
_lock = threading.Lock()


def lib() -> C.CDLL:
    """The loaded library.  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m sparse_attention_top_tcgen05_gb300.build`")
            L = C.CDLL(LIB_PATH)
            P, i64, i32, sz = C.c_void_p, C.c_int64, C.c_int, C.c_size_t
            L.lidx_indexer_fwd.argtypes = [P, P, P, i64, i64, i64, i32, i32, i32, i32, i32,
                                           P, P, P, P, P, sz, P]
            L.lidx_indexer_fwd_ranges.argtypes = [P, P, P, i64, i64, i64, i32, i32, P, P, i32, i32,
                                                  P, P, P, P, P, sz, P]
            L.lidx_indexer_topk_v41.argtypes = [P, P, P, P, i64, i64, i64, i32, i32, i32, i32, P, P,
                                                P, P, sz, P]
            L.lidx_indexer_bwd_ranges.argtypes = [P, P, P, P, P, i64, i64, i64, i32, i32, P, P, i32,
                                                  i32, i32, P, P, P, P, sz, P]
            L.lidx_set_wait_limit_ns.argtypes = [C.c_uint64]
            L.lidx_set_wait_limit_ns.restype = C.c_uint64
            L.lidx_debug_stall_producer.argtypes = [i32]
            L.lidx_debug_stall_producer.restype = i32
            L.lidx_indexer_logits.argtypes = [P, P, P, i64, i64, i64, i32, i32, i32, P, P, i32,
                                              i32, P, P]
            L.lidx_extract_topk_scores.argtypes = [P, P, i64, i64, i64, i32, P, P]
            L.lidx_topk_rows.argtypes = [P, i64, i64, i64, i32, P, P, i32, P, P, P]
            L.lidx_indexer_scores_v41.argtypes = [P, P, P, P, i64, i64, i64, i32, i32, i32, P,
                                                  P, sz, P]
            L.lidx_indexer_bwd.argtypes = [P, P, P, P, P, i64, i64, i64, i32, i32, i32, i32, i32,
                                           i32, P, P, P, P, sz, P]
            L.lidx_indexer_fwd_noalloc.argtypes = [P, P, P, i64, i64, i64, i32, i32, i32, i32, i32,
                                                   P, P, P]
            L.lidx_indexer_fwd_noalloc.restype = i32
            L.lidx_noalloc_scratch_bytes.restype = sz
            L.lidx_workspace_bytes.argtypes = [i32, i64, i64, i64, i32, i32, i32, i32]
            L.lidx_workspace_bytes.restype = sz
            L.lidx_device_status.argtypes = [P]
            L.lidx_status_string.argtypes = [i32]
            L.lidx_status_string.restype = C.c_char_p
            L.lidx_version.restype = i32
            f32, f64 = C.c_float, C.c_double
            L.lidx_rope_freqs.argtypes = [i32, f64, i32, f64, f64, f64, f64, P]
            L.lidx_rope.argtypes = [P, i32, P, P, P, i64, i64, i32, i32, i32, i32, i32, f32, i32, P]
            L.lidx_cache_append.argtypes = [P, P, P, P, P, P, P, i64, i64, i32, i32, i32, i64, i64,
                                            P, P, P, P, P]
            L.lidx_cache_attn.argtypes = [P, P, P, P, P, P, P, P, P, P, i64, i64, i32, i32, i32, i32,
                                          i64, i64, i32, i32, f32, P, P, P, sz, P]
            L.lidx_cache_attn_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i32]
            L.lidx_cache_attn_workspace_bytes.restype = sz
            for name in ("lidx_rope_freqs", "lidx_rope", "lidx_cache_append", "lidx_cache_attn",
                         "lidx_indexer_fwd", "lidx_indexer_fwd_ranges", "lidx_indexer_logits",
                         "lidx_extract_topk_scores", "lidx_topk_rows", "lidx_indexer_scores_v41",
                         "lidx_indexer_topk_v41", "lidx_indexer_bwd", "lidx_indexer_bwd_ranges",
                         "lidx_device_status"):
                getattr(L, name).restype = i32
            _lib = L
    return _lib


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return C.c_void_p(s.cuda_stream)


def _on(stream, device):
    """The context in which `stream`'s own memory is allocated."""
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    return torch.cuda.stream(stream)


def _new(shape, dtype, device, stream):
    """An output that the call allocates.  It is the stream's on which the kernels run: a block of another stream's pool
    may still be in use there.  The caller reads it on the current stream, so it is held for that one, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _scratch(nbytes, device, stream):
    """Scratch that the call drops while its kernels may still run: of their stream's pool, which hands it out behind them."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with _on(stream, device):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _nbytes(workspace):
    """Size of a workspace, a caller's own as it is: the library refuses one that is too small."""
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _need(t, name, dtype, dim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dims, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check(rc, call):
    if rc != LIDX_OK:
        raise LidxError(rc, call)


def lidx_workspace_bytes(op, B, S, Skv, H, D, topk=0, logits_materialised=False) -> int:
    return int(lib().lidx_workspace_bytes(op, B, S, Skv, H, D, topk, int(bool(logits_materialised))))


def lidx_status_string(status: int) -> str:
    return lib().lidx_status_string(int(status)).decode()


def lidx_device_status(stream=None) -> int:
    return int(lib().lidx_device_status(_stream(stream)))


def _fwd_common(q, k, w, topk, topk_indices, materialise_logits, out, workspace, stream):
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    S, B, H, D = q.shape
    Skv = k.shape[0]
    if k.shape[1] != B or k.shape[2] != D or tuple(w.shape) != (S, B, H):
        raise ValueError("q/k/w shapes disagree")
    if topk_indices is not None:
        _need(topk_indices, "topk_indices", torch.int32, 3)
    dev = q.device
    if out is None:
        idx = _new((B, S, topk), torch.int32, dev, stream)
        sc = _new((B, S, topk), torch.float32, dev, stream)
        lg = _new((B, S, Skv), torch.float32, dev, stream) if materialise_logits else None
    else:
        idx, sc, lg = out
    ws_bytes = lidx_workspace_bytes(OP_INDEXER_FWD, B, S, Skv, H, D, topk, lg is not None)
    if workspace is None and ws_bytes:
        workspace = _scratch(ws_bytes, dev, stream)
    return (S, B, H, D, Skv), idx, sc, lg, workspace


def lidx_indexer_fwd(q, k, w, compress_ratio, topk, act="relu", topk_indices=None,
                     materialise_logits=False, stream=None, out=None, workspace=None):
    """V4 forward.  q [S,B,H,D] bf16, k [Skv,B,D] bf16, w [S,B,H] fp32.

    Returns (indices [B,S,topk] int32, scores [B,S,topk] fp32, logits or None).
    ``out`` may hold preallocated (indices, scores, logits) tensors.
    """
    (S, B, H, D, Skv), idx, sc, lg, workspace = _fwd_common(
        q, k, w, topk, topk_indices, materialise_logits, out, workspace, stream)
    rc = lib().lidx_indexer_fwd(_ptr(q), _ptr(k), _ptr(w), B, S, Skv, H, D, compress_ratio, topk,
                                ACT[act], _ptr(topk_indices), _ptr(lg), _ptr(idx), _ptr(sc),
                                _ptr(workspace), _nbytes(workspace),
                                _stream(stream))
    _check(rc, "lidx_indexer_fwd")
    return idx, sc, lg


def lidx_indexer_fwd_ranges(q, k, w, ks, ke, topk, act="relu", topk_indices=None,
                            materialise_logits=False, stream=None, out=None, workspace=None):
    """V4 forward where row (b,s) sees keys [ks[s], ke[s]) (int32 [S] CUDA tensors)."""
    _need(ks, "ks", torch.int32, 1)
    _need(ke, "ke", torch.int32, 1)
    (S, B, H, D, Skv), idx, sc, lg, workspace = _fwd_common(
        q, k, w, topk, topk_indices, materialise_logits, out, workspace, stream)
    if ks.shape[0] != S or ke.shape[0] != S:
        raise ValueError("ks/ke must have S entries")
    rc = lib().lidx_indexer_fwd_ranges(_ptr(q), _ptr(k), _ptr(w), B, S, Skv, H, D, _ptr(ks), _ptr(ke),
                                       topk, ACT[act], _ptr(topk_indices), _ptr(lg), _ptr(idx),
                                       _ptr(sc), _ptr(workspace),
                                       _nbytes(workspace), _stream(stream))
    _check(rc, "lidx_indexer_fwd_ranges")
    return idx, sc, lg


def lidx_indexer_fwd_noalloc(q, k, w, compress_ratio, topk, act="relu", stream=None, out=None):
    """The fused V4 forward using the library's own scratch array instead of a
    workspace, for callers that cannot allocate device memory.  Outputs may be
    passed in ``out`` = (indices, scores) so that the call allocates nothing."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    S, B, H, D = q.shape
    Skv = k.shape[0]
    if out is None:
        idx = _new((B, S, topk), torch.int32, q.device, stream)
        sc = _new((B, S, topk), torch.float32, q.device, stream)
    else:
        idx, sc = out
    rc = lib().lidx_indexer_fwd_noalloc(_ptr(q), _ptr(k), _ptr(w), B, S, Skv, H, D, compress_ratio,
                                        topk, ACT[act], _ptr(idx), _ptr(sc), _stream(stream))
    _check(rc, "lidx_indexer_fwd_noalloc")
    return idx, sc


def lidx_indexer_logits(q, k, w, compress_ratio=1, ks=None, ke=None, clean=True, act="relu",
                        stream=None, out=None):
    """Logits [B,S,Skv] fp32 over causal ranges or explicit per-row [ks, ke)."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    S, B, H, D = q.shape
    Skv = k.shape[0]
    if ks is not None:
        _need(ks, "ks", torch.int32, 1)
        _need(ke, "ke", torch.int32, 1)
    lg = _new((B, S, Skv), torch.float32, q.device, stream) if out is None else out
    rc = lib().lidx_indexer_logits(_ptr(q), _ptr(k), _ptr(w), B, S, Skv, H, D, compress_ratio,
                                   _ptr(ks), _ptr(ke), int(bool(clean)), ACT[act], _ptr(lg),
                                   _stream(stream))
    _check(rc, "lidx_indexer_logits")
    return lg


def lidx_extract_topk_scores(logits, idx, stream=None):
    _need(logits, "logits", torch.float32, 3)
    _need(idx, "idx", torch.int32, 3)
    B, S, Skv = logits.shape
    topk = idx.shape[2]
    out = _new((B, S, topk), torch.float32, logits.device, stream)
    rc = lib().lidx_extract_topk_scores(_ptr(logits), _ptr(idx), B, S, Skv, topk, _ptr(out),
                                        _stream(stream))
    _check(rc, "lidx_extract_topk_scores")
    return out


def lidx_topk_rows(logits, topk, compress_ratio=1, ks=None, ke=None, stream=None, out=None):
    """Top-k of each row of logits [B,S,Skv] (or [rows, Skv] with S = rows).

    Visible range per query s: causal from compress_ratio, or [ks[s], ke[s]).
    Returns (indices [..., topk] int32, scores [..., topk] fp32).
    """
    if logits.dim() == 3:
        B, S, Skv = logits.shape
    else:
        _need(logits, "logits", torch.float32, 2)
        B, (S, Skv) = 1, logits.shape
    if logits.dtype != torch.float32 or not logits.is_cuda or not logits.is_contiguous():
        raise ValueError("logits must be a contiguous CUDA float32 tensor")
    if ks is not None:
        _need(ks, "ks", torch.int32, 1)
        _need(ke, "ke", torch.int32, 1)
    shape = tuple(logits.shape[:-1]) + (topk,)
    if out is None:
        idx = _new(shape, torch.int32, logits.device, stream)
        sc = _new(shape, torch.float32, logits.device, stream)
    else:
        idx, sc = out
    rc = lib().lidx_topk_rows(_ptr(logits), B * S, S, Skv, compress_ratio, _ptr(ks), _ptr(ke), topk,
                              _ptr(idx), _ptr(sc), _stream(stream))
    _check(rc, "lidx_topk_rows")
    return idx, sc


def lidx_indexer_scores_v41(q, k, w, allowed, act="relu", stream=None, out=None, workspace=None):
    """V4.1 scores bf16 [B,S,Skv].  q [B,S,H,D], k [B,Skv,D], w [B,S,H] bf16,
    allowed [B,S,Skv] bool."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.bfloat16, 3)
    if allowed.dtype not in (torch.bool, torch.uint8):
        raise TypeError("allowed must be bool or uint8")
    if not (allowed.is_cuda and allowed.is_contiguous() and allowed.dim() == 3):
        raise ValueError("allowed must be a contiguous CUDA [B,S,Skv] tensor")
    B, S, H, D = q.shape
    Skv = k.shape[1]
    res = _new((B, S, Skv), torch.bfloat16, q.device, stream) if out is None else out
    ws_bytes = lidx_workspace_bytes(OP_SCORES_V41, B, S, Skv, H, D)
    if workspace is None and ws_bytes:
        workspace = _scratch(ws_bytes, q.device, stream)
    rc = lib().lidx_indexer_scores_v41(_ptr(q), _ptr(k), _ptr(w), _ptr(allowed), B, S, Skv, H, D,
                                       ACT[act], _ptr(res), _ptr(workspace),
                                       _nbytes(workspace), _stream(stream))
    _check(rc, "lidx_indexer_scores_v41")
    return res


def lidx_indexer_topk_v41(q, k, w, allowed, topk, act="relu", keep_scores=True, stream=None,
                          out=None, workspace=None):
    """V4.1 scores and their per-row top-k.  Returns (scores bf16 [B,S,Skv] or
    None, indices int32 [B,S,topk], top-k scores bf16 [B,S,topk])."""
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.bfloat16, 3)
    if allowed.dtype not in (torch.bool, torch.uint8):
        raise TypeError("allowed must be bool or uint8")
    if not (allowed.is_cuda and allowed.is_contiguous() and allowed.dim() == 3):
        raise ValueError("allowed must be a contiguous CUDA [B,S,Skv] tensor")
    B, S, H, D = q.shape
    Skv = k.shape[1]
    dev = q.device
    if out is None:
        res = _new((B, S, Skv), torch.bfloat16, dev, stream) if keep_scores else None
        idx = _new((B, S, topk), torch.int32, dev, stream)
        tsc = _new((B, S, topk), torch.bfloat16, dev, stream)
    else:
        res, idx, tsc = out
    ws_bytes = lidx_workspace_bytes(OP_TOPK_V41, B, S, Skv, H, D, topk, res is not None)
    if workspace is None and ws_bytes:
        workspace = _scratch(ws_bytes, dev, stream)
    rc = lib().lidx_indexer_topk_v41(_ptr(q), _ptr(k), _ptr(w), _ptr(allowed), B, S, Skv, H, D,
                                     ACT[act], topk, _ptr(res), _ptr(idx), _ptr(tsc), _ptr(workspace),
                                     _nbytes(workspace), _stream(stream))
    _check(rc, "lidx_indexer_topk_v41")
    return res, idx, tsc


def lidx_set_wait_limit_ns(ns: int) -> int:
    """Limit of every in-kernel pipeline wait (0: the 2 s default); returns the previous."""
    return int(lib().lidx_set_wait_limit_ns(int(ns)))


def lidx_debug_stall_producer(on: bool) -> int:
    """Test switch: the scoring kernel's producer loads nothing, so its waits run out."""
    return int(lib().lidx_debug_stall_producer(int(bool(on))))


def _bwd_common(q, k, w, idx, grad, grad_dtype, out, workspace, stream):
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 3)
    _need(w, "w", torch.float32, 3)
    _need(idx, "idx", torch.int32, 3)
    _need(grad, "grad", torch.float32, 3)
    S, B, H, D = q.shape
    Skv = k.shape[0]
    topk = idx.shape[2]
    dev = q.device
    gdt = {torch.float32: 0, torch.bfloat16: 1}[grad_dtype]
    if out is None:
        dq = _new((S, B, H, D), grad_dtype, dev, stream)
        dk = _new((Skv, B, D), grad_dtype, dev, stream)
        dw = _new((S, B, H), torch.float32, dev, stream)
    else:
        dq, dk, dw = out
    ws_bytes = lidx_workspace_bytes(OP_INDEXER_BWD, B, S, Skv, H, D, topk)
    if workspace is None and ws_bytes:
        workspace = _scratch(ws_bytes, dev, stream)
    return (S, B, H, D, Skv, topk, gdt), dq, dk, dw, workspace


def lidx_indexer_bwd_ranges(q, k, w, idx, grad, ks, ke, act="relu", grad_dtype=torch.float32,
                            stream=None, out=None, workspace=None):
    """Backward where row (b,s) sees keys [ks[s], ke[s]); dk is this call's partial sum."""
    _need(ks, "ks", torch.int32, 1)
    _need(ke, "ke", torch.int32, 1)
    (S, B, H, D, Skv, topk, gdt), dq, dk, dw, workspace = _bwd_common(
        q, k, w, idx, grad, grad_dtype, out, workspace, stream)
    rc = lib().lidx_indexer_bwd_ranges(_ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(grad), B, S, Skv, H,
                                       D, _ptr(ks), _ptr(ke), topk, ACT[act], gdt, _ptr(dq), _ptr(dk),
                                       _ptr(dw), _ptr(workspace),
                                       _nbytes(workspace), _stream(stream))
    _check(rc, "lidx_indexer_bwd_ranges")
    return dq, dk, dw


def lidx_indexer_bwd(q, k, w, idx, grad, compress_ratio, act="relu", grad_dtype=torch.float32,
                     stream=None, out=None, workspace=None):
    """Gradients (dq [S,B,H,D], dk [Skv,B,D] in grad_dtype (fp32 or bf16), dw [S,B,H] fp32)."""
    (S, B, H, D, Skv, topk, gdt), dq, dk, dw, workspace = _bwd_common(
        q, k, w, idx, grad, grad_dtype, out, workspace, stream)
    rc = lib().lidx_indexer_bwd(_ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(grad), B, S, Skv, H, D,
                                compress_ratio, topk, ACT[act], gdt, _ptr(dq), _ptr(dk), _ptr(dw),
                                _ptr(workspace), _nbytes(workspace),
                                _stream(stream))
    _check(rc, "lidx_indexer_bwd")
    return dq, dk, dw


# The calls below are made once for each layer of each token: their checks read each attribute once, arrays
# of sizes go to C as packed bytes, and the stream is the raw handle.
_Tensor, _bf16, _f32, _i32, _i64, _f8 = (torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.int64,
                                          torch.float8_e4m3fn)
_I2, _I3, _ROPE_TENSOR = struct.Struct("2q").pack, struct.Struct("3q").pack, struct.Struct("PP6qi4x").pack


def _strided(t, name, dtype, dev=None):
    """Checks a 4-dimensional CUDA tensor of any strides that is contiguous in its last dimension; returns its
    shape, the strides of the leading dimensions (0 where the size is 1: never stepped over) and its device."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 4:
        raise ValueError(f"{name} must have 4 dims, got {tuple(shape)}")
    a, b, c, d = t.stride()
    if d != 1 and shape[3] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    at = t.get_device()
    if dev is not None and at != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    return shape, (a if shape[0] > 1 else 0, b if shape[1] > 1 else 0, c if shape[2] > 1 else 0), at


def _dense(t, name, dtype, shape, dev):
    """Checks a contiguous CUDA tensor on device dev; None in `shape` is any size.  Returns its shape."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        s = t.shape
        if s == shape or (len(s) == len(shape) and all(m is None or n == m for n, m in zip(s, shape))):
            return s
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape} (None: any)")


def _raw_stream(stream, dev):
    if torch._C._cuda_getDevice() != dev:  # launches go to the current device
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def lidx_rope_freqs(rot_dim, theta=10000.0, scaling=None, factor=1.0, original_len=4096, beta_fast=32.0,
                    beta_slow=1.0, device="cuda") -> torch.Tensor:
    """Rotary frequencies int64 [rot_dim/2]: turns per position in 0.64 fixed point (the bits of
    unsigned integers).  scaling: None, "linear", "ntk" or "yarn" (its ramp is linear in the turns that a pair
    makes within original_len, beta_slow to beta_fast, not in the pair's index).  Any other set of
    frequencies w, in radians per position, is round(w / (2 pi) * 2**64) as int64."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALING)}")
    out = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.int64)
    rc = lib().lidx_rope_freqs(int(rot_dim), theta, ROPE_SCALING[scaling], factor, original_len, beta_fast,
                               beta_slow, _ptr(out))
    _check(rc, "lidx_rope_freqs")
    return out.to(device)


def _rope(x, pos, freqs, x2, layout, rot_off, mscale, inverse, stream, out, call):
    dtype = x.dtype if isinstance(x, _Tensor) else _bf16
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"x must be float32 or bfloat16, got {dtype}")
    shape, xs, dev = _strided(x, "x", dtype)
    T0, T1, H, D = shape
    if x2 is not None:
        shape2, xs2, _ = _strided(x2, "x2", dtype, dev)
        if shape2[0] != T0 or shape2[1] != T1 or shape2[3] != D:
            raise ValueError("x and x2 shapes disagree")
    if not isinstance(pos, _Tensor) or pos.dtype is not _i32 or not pos.is_cuda:
        raise TypeError("pos must be an int32 CUDA tensor")
    if pos.shape != (T0, T1):
        pos = pos.expand(T0, T1)  # repeated positions have stride 0
    if pos.get_device() != dev:
        raise ValueError(f"pos is on {pos.device}, not on cuda:{dev}")
    p0, p1 = pos.stride()
    pairs = _dense(freqs, "freqs", _i64, (None,), dev)[0]
    if layout not in ROPE_LAYOUT:
        raise ValueError(f"layout must be one of {list(ROPE_LAYOUT)}")
    if out is None:
        at = x.device
        y = torch.empty_like(x) if stream is None and x.is_contiguous() else _new(shape, dtype, at, stream)
        arr = _ROPE_TENSOR(x.data_ptr(), y.data_ptr(), *xs, T1 * H * D, H * D, D, H)
        if x2 is not None:
            H2 = shape2[2]
            y2 = _new(shape2, dtype, at, stream)
            arr += _ROPE_TENSOR(x2.data_ptr(), y2.data_ptr(), *xs2, T1 * H2 * D, H2 * D, D, H2)
    else:
        y, y2 = (out, None) if x2 is None else out
        sy, ys, _ = _strided(y, "out", dtype, dev)
        if sy != shape:
            raise ValueError("out has another shape than x")
        arr = _ROPE_TENSOR(x.data_ptr(), y.data_ptr(), *xs, *ys, H)
        if x2 is not None:
            sy, ys, _ = _strided(y2, "out", dtype, dev)
            if sy != shape2:
                raise ValueError("out has another shape than x2")
            arr += _ROPE_TENSOR(x2.data_ptr(), y2.data_ptr(), *xs2, *ys, shape2[2])
    rc = (_lib or lib()).lidx_rope(arr, 1 if x2 is None else 2, pos.data_ptr(), _I2(p0 if T0 > 1 else 0, p1 if T1 > 1 else 0),
                                   freqs.data_ptr(), T0, T1, D, 2 * pairs, rot_off, ROPE_LAYOUT[layout], inverse, mscale,
                                   1 if dtype is _bf16 else 0, _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, call)
    return y if x2 is None else (y, y2)


def lidx_rope(x, pos, freqs, x2=None, layout="interleaved", rot_off=0, mscale=1.0, stream=None, out=None):
    """Rotary positions of x [T0,T1,H,D] (fp32 or bf16, any strides of the leading dimensions) and, in
    the same launch, of x2 [T0,T1,H2,D].  pos: int32, broadcast to [T0,T1]; freqs: lidx_rope_freqs's,
    the rotated dims are [rot_off, rot_off + 2*len(freqs)).  Returns y, or (y, y2).  ``out`` may be the
    inputs themselves (in place)."""
    return _rope(x, pos, freqs, x2, layout, rot_off, mscale, 0, stream, out, "lidx_rope")


def lidx_rope_bwd(g, pos, freqs, x2=None, layout="interleaved", rot_off=0, mscale=1.0, stream=None, out=None):
    """Gradient of lidx_rope's x (and x2) from the gradients g (and x2) of its outputs: the inverse turn."""
    return _rope(g, pos, freqs, x2, layout, rot_off, mscale, 1, stream, out, "lidx_rope_bwd")


def _cache(k_cache, v_cache, k_scale, v_scale, block_table, B, Hkv, D, dev):
    shape = _dense(k_cache, "k_cache", _f8, (None, Hkv, None, D), dev)
    pages, Hkv, page, _ = shape
    _dense(v_cache, "v_cache", _f8, shape, dev)
    _dense(k_scale, "k_scale", _f32, (pages, Hkv), dev)
    _dense(v_scale, "v_scale", _f32, (pages, Hkv), dev)
    return pages, Hkv, page, _dense(block_table, "block_table", _i32, (B, None), dev)[1]


def lidx_cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, start, count=None, stream=None):
    """Writes k, v [B,S,Hkv,D] bf16 behind the start[b] tokens that each sequence's pages hold, in
    8 bits with a power-of-two scale for each page and head.  k_cache, v_cache [P,Hkv,page,D]
    float8_e4m3fn and k_scale, v_scale [P,Hkv] fp32 are updated in place; block_table int32
    [B,max_pages]; count int32 [B] or None: new tokens of each sequence.  Infinities and NaN are stored as
    NaN and change no scale."""
    shape, ks, dev = _strided(k, "k", _bf16)
    shape_v, vs, _ = _strided(v, "v", _bf16, dev)
    if shape_v != shape:
        raise ValueError("k and v shapes disagree")
    B, S, Hkv, D = shape
    pages, _, page, MP = _cache(k_cache, v_cache, k_scale, v_scale, block_table, B, Hkv, D, dev)
    _dense(start, "start", _i32, (B,), dev)
    if count is not None:
        _dense(count, "count", _i32, (B,), dev)
    rc = (_lib or lib()).lidx_cache_append(
        k.data_ptr(), v.data_ptr(), _I3(*ks), _I3(*vs), block_table.data_ptr(), start.data_ptr(),
        None if count is None else count.data_ptr(), B, S, Hkv, D, page, MP, pages, k_cache.data_ptr(),
        v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_cache_append")


def lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk=0) -> int:
    return int(lib().lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk))


def lidx_cache_attn(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_len, q_pos=None, compress_ratio=1,
                    topk_indices=None, softmax_scale=None, want_lse=False, stream=None, out=None,
                    workspace=None):
    """Attention of q [B,S,Hq,D] bf16 over a cache written by lidx_cache_append (scales 2^-80 .. 2^100).

    kv_len int32 [B]: keys of each sequence.  q_pos int32 [B] or None: with it, row (b,s) sees keys
    below (q_pos[b]+s+1)//compress_ratio only.  topk_indices int32 [B,S,topk] or None: the row sees
    only the listed keys (lidx_indexer_fwd's indices).  softmax_scale defaults to D**-0.5.
    A row whose query or a key it sees is not finite is NaN, with its log-sum-exp; for NaN values see lidx.h.
    Returns (out [B,S,Hq,D] bf16, lse [B,S,Hq] fp32 or None); ``out`` may hold preallocated ones."""
    shape, qs, dev = _strided(q, "q", _bf16)
    B, S, Hq, D = shape
    pages, Hkv, page, MP = _cache(k_cache, v_cache, k_scale, v_scale, block_table, B, None, D, dev)
    _dense(kv_len, "kv_len", _i32, (B,), dev)
    if q_pos is not None:
        _dense(q_pos, "q_pos", _i32, (B,), dev)
    topk = 0 if topk_indices is None else _dense(topk_indices, "topk_indices", _i32, (B, S, None), dev)[2]
    if out is None:
        o = torch.empty_like(q) if stream is None and q.is_contiguous() else _new(shape, _bf16, q.device, stream)
        lse = _new(shape[:3], _f32, q.device, stream) if want_lse else None
    else:
        o, lse = out
        _dense(o, "out", _bf16, shape, dev)
        if lse is not None:
            _dense(lse, "lse", _f32, shape[:3], dev)
        elif want_lse:
            lse = _new(shape[:3], _f32, q.device, stream)
    L = _lib or lib()
    if workspace is None:
        ws_bytes = L.lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk)
        workspace = _scratch(ws_bytes, q.device, stream)
    else:
        ws_bytes = _dense(workspace, "workspace", torch.uint8, (None,), dev)[0]
    rc = L.lidx_cache_attn(
        q.data_ptr(), _I3(*qs), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        block_table.data_ptr(), kv_len.data_ptr(), None if q_pos is None else q_pos.data_ptr(),
        None if topk_indices is None else topk_indices.data_ptr(), B, S, Hq, Hkv, D, page, MP, pages, compress_ratio,
        topk, D ** -0.5 if softmax_scale is None else softmax_scale, o.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), ws_bytes, _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_cache_attn")
    return o, lse
