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
  lidx_rope_axis_map        the axis of each pair where positions have several (time, height, width)
  lidx_norm_rope, lidx_norm_rope_bwd  norms of each head with the rotary positions in one pass, and their gradients
  lidx_cache_append         new keys and values into a paged 8-bit cache
  lidx_rope_cache_append    the same with the norm and the rotary positions of the keys on the way
  lidx_cache_attn           attention over that cache, at every key or at selected ones
  lidx_cache4_append, lidx_cache4_to_8  a paged cache of 4-bit numbers, and the same as an 8-bit one
  lidx_cache4_attn          attention over the 4-bit cache
  lidx_workspace_bytes, lidx_cache_attn_workspace_bytes, lidx_cache4_attn_workspace_bytes, lidx_device_status,
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
           "lidx_cache_attn", "lidx_cache_attn_workspace_bytes", "lidx_rope_axes", "lidx_norm_rope",
           "lidx_norm_rope_bwd", "lidx_norm_rope_bwd_workspace_bytes", "lidx_rope_cache_append",
           "lidx_cache4_append", "lidx_cache4_to_8", "lidx_cache4_attn",
           "lidx_cache4_attn_workspace_bytes")


class _RopeTensor(C.Structure):
    _fields_ = [("x", C.c_void_p), ("y", C.c_void_p), ("xs", C.c_int64 * 3), ("ys", C.c_int64 * 3),
                ("H", C.c_int)]


class _RopeTurn(C.Structure):
    _fields_ = [("pos", C.c_void_p), ("ps", C.c_int64 * 3), ("freqs", C.c_void_p), ("axis", C.c_void_p),
                ("axes", C.c_int), ("rot_dim", C.c_int), ("rot_off", C.c_int), ("layout", C.c_int), ("mscale", C.c_float)]


class _NormTensor(C.Structure):
    _fields_ = [("x", C.c_void_p), ("g", C.c_void_p), ("y", C.c_void_p), ("xs", C.c_int64 * 3), ("gs", C.c_int64 * 3),
                ("ys", C.c_int64 * 3), ("w", C.c_void_p), ("dw", C.c_void_p), ("H", C.c_int)]


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
            L.lidx_rope_axes.argtypes = [P, i32, P, i64, i64, i32, i32, i32, P]
            L.lidx_norm_rope.argtypes = [P, i32, P, f32, i64, i64, i32, i32, i32, P]
            L.lidx_norm_rope_bwd.argtypes = [P, i32, P, f32, i64, i64, i32, i32, i32, P, sz, P]
            L.lidx_rope_cache_append.argtypes = [P, P, P, P, P, P, i32, f32, P, P, P, i64, i64, i32, i32, i32, i64, i64,
                                                 P, P, P, P, P]
            L.lidx_cache4_append.argtypes = [P, P, P, P, P, P, i32, f32, P, P, P, i64, i64, i32, i32, i32, i64, i64,
                                             P, P, P, P, P, P, P]
            L.lidx_cache4_attn.argtypes = [P, P, P, P, P, P, P, P, P, P, P, P, i64, i64, i32, i32, i32, i32,
                                           i64, i64, i32, i32, f32, P, P, P, sz, P]
            L.lidx_cache4_attn_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i32, i64, i32]
            L.lidx_cache4_attn_workspace_bytes.restype = sz
            L.lidx_cache4_to_8.argtypes = [P, P, P, P, i32, i32, i32, i64, P, P, P]
            L.lidx_norm_rope_bwd_workspace_bytes.argtypes = [i32]
            L.lidx_norm_rope_bwd_workspace_bytes.restype = sz
            for name in ("lidx_rope_freqs", "lidx_rope", "lidx_cache_append", "lidx_cache_attn",
                         "lidx_rope_axes", "lidx_norm_rope", "lidx_norm_rope_bwd", "lidx_rope_cache_append",
                         "lidx_cache4_append", "lidx_cache4_to_8", "lidx_cache4_attn",
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
_ROPE_TURN, _NORM_TENSOR, _u8 = struct.Struct("P3qPP4if4x").pack, struct.Struct("PPP9qPPi4x").pack, torch.uint8


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
        if s == shape:
            return s
        if len(s) == len(shape):
            for n, m in zip(s, shape):
                if m is not None and n != m:
                    break
            else:
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


def lidx_rope_axis_map(sections, interleaved=False, device="cuda") -> torch.Tensor:
    """Axis of each rotated pair, uint8 [sum(sections)]: sections[a] pairs of axis a, one section after the other or, with
    interleaved, in turns for as long as each axis has pairs left."""
    left = [int(n) for n in sections]
    if not left or min(left) < 0 or sum(left) < 1 or len(left) > 255:
        raise ValueError("sections must be 1 to 255 numbers of pairs")
    if interleaved:
        ids = [a for i in range(max(left)) for a, n in enumerate(left) if i < n]
    else:
        ids = [a for a, n in enumerate(left) for _ in range(n)]
    return torch.tensor(ids, dtype=_u8).to(device)


def _turn(pos, freqs, layout, rot_off, mscale, axes, T0, T1, dev, own_pos=False):
    """The packed lidx_rope_turn of a rotation.  own_pos: pos may be None, for the call's own positions."""
    if pos is None and own_pos:
        pairs = _dense(freqs, "freqs", _i64, (None,), dev)[0]
        if axes is not None:
            raise ValueError("axes needs pos, with the positions on each axis")
        at = pa = p0 = p1 = axis = 0
        A = 1
    else:
        if not isinstance(pos, _Tensor) or pos.dtype is not _i32 or not pos.is_cuda:
            raise TypeError("pos must be an int32 CUDA tensor")
        if pos.get_device() != dev:
            raise ValueError(f"pos is on {pos.device}, not on cuda:{dev}")
        pairs = _dense(freqs, "freqs", _i64, (None,), dev)[0]
        if axes is None:
            A, axis = 1, 0
            if pos.shape != (T0, T1):
                pos = pos.expand(T0, T1)  # repeated positions have stride 0
            p0, p1 = pos.stride()
            pa = 0
        else:
            _dense(axes, "axes", _u8, (pairs,), dev)
            if pos.dim() < 1:
                raise ValueError("pos must have the axes as its first dim")
            A, axis = pos.shape[0], axes.data_ptr()
            if not 1 <= A <= 255:
                raise ValueError(f"pos has {A} axes: 1 to 255 are supported")
            if pos.shape != (A, T0, T1):
                pos = pos.view(A, *(1,) * (3 - pos.dim()), *pos.shape[1:]).expand(A, T0, T1)
            pa, p0, p1 = pos.stride()
        at = pos.data_ptr()
    if layout not in ROPE_LAYOUT:
        raise ValueError(f"layout must be one of {list(ROPE_LAYOUT)}")
    try:
        return _ROPE_TURN(at, pa, p0 if T0 > 1 else 0, p1 if T1 > 1 else 0, freqs.data_ptr(), axis, A, 2 * pairs, rot_off,
                          ROPE_LAYOUT[layout], mscale)
    except struct.error:
        raise ValueError(f"rot_off must be a 32-bit integer and mscale a number, got {rot_off} and {mscale}") from None


def _rope(x, pos, freqs, x2, layout, rot_off, mscale, inverse, stream, out, axes, call):
    dtype = x.dtype if isinstance(x, _Tensor) else _bf16
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"x must be float32 or bfloat16, got {dtype}")
    shape, xs, dev = _strided(x, "x", dtype)
    T0, T1, H, D = shape
    if x2 is not None:
        shape2, xs2, _ = _strided(x2, "x2", dtype, dev)
        if shape2[0] != T0 or shape2[1] != T1 or shape2[3] != D:
            raise ValueError("x and x2 shapes disagree")
    turn = _turn(pos, freqs, layout, rot_off, mscale, axes, T0, T1, dev)
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
    rc = (_lib or lib()).lidx_rope_axes(arr, 1 if x2 is None else 2, turn, T0, T1, D, inverse, 1 if dtype is _bf16 else 0,
                                        _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, call)
    return y if x2 is None else (y, y2)


def lidx_rope(x, pos, freqs, x2=None, layout="interleaved", rot_off=0, mscale=1.0, stream=None, out=None, axes=None):
    """Rotary positions of x [T0,T1,H,D] (fp32 or bf16, any strides of the leading dimensions) and, in
    the same launch, of x2 [T0,T1,H2,D].  pos: int32, broadcast to [T0,T1]; freqs: lidx_rope_freqs's,
    the rotated dims are [rot_off, rot_off + 2*len(freqs)).  Returns y, or (y, y2).  ``out`` may be the
    inputs themselves (in place).
    axes (lidx_rope_axis_map's, uint8 [len(freqs)]): positions on several axes, pos int32 [A, ...] with [...] broadcast to
    [T0,T1]; pair i turns by pos[axes[i]] (ids of A and more count as A - 1)."""
    return _rope(x, pos, freqs, x2, layout, rot_off, mscale, 0, stream, out, axes, "lidx_rope")


def lidx_rope_bwd(g, pos, freqs, x2=None, layout="interleaved", rot_off=0, mscale=1.0, stream=None, out=None, axes=None):
    """Gradient of lidx_rope's x (and x2) from the gradients g (and x2) of its outputs: the inverse turn."""
    return _rope(g, pos, freqs, x2, layout, rot_off, mscale, 1, stream, out, axes, "lidx_rope_bwd")


def _fresh(x, shape, dtype, stream):
    """An output of x's shape and type, contiguous."""
    return torch.empty_like(x) if stream is None and x.is_contiguous() else _new(shape, dtype, x.device, stream)


def _norm_side(x, weight, g, y, dw, name, dtype, w_dtype, dev, bwd, stream):
    """Checks of one tensor of a norm, its weight, gradient and outputs, which it makes where they are None; returns its
    shape, device, what goes to C and the outputs."""
    shape, (a, b, c), dev = _strided(x, "x" + name, dtype, dev)
    H, D = shape[2], shape[3]
    if weight is not None:
        _dense(weight, "weight" + name, w_dtype, (D,), dev)
    if y is None:
        y = _fresh(x, shape, dtype, stream)
        ya, yb, yc = shape[1] * H * D, H * D, D
    else:
        sy, (ya, yb, yc), _ = _strided(y, "out", dtype, dev)
        if sy != shape:
            raise ValueError(f"out has another shape than x{name}")
    if bwd:
        if dw is not None:
            _dense(dw, "out", _f32, (D,), dev)
        elif weight is not None:
            dw = _new((D,), _f32, x.device, stream)
    ga = gb = gc = gp = 0
    if bwd:
        sg, (ga, gb, gc), _ = _strided(g, "g" + name, dtype, dev)
        if sg != shape:
            raise ValueError(f"g{name} has another shape than x{name}")
        gp = g.data_ptr()
    return shape, dev, _NORM_TENSOR(x.data_ptr(), gp, y.data_ptr(), a, b, c, ga, gb, gc, ya, yb, yc,
                                    0 if weight is None else weight.data_ptr(), 0 if dw is None else dw.data_ptr(), H), y, dw


def _norm_rope(x, weight, pos, freqs, g, x2, weight2, g2, eps, layout, rot_off, mscale, axes, stream, out, workspace, bwd):
    dtype = x.dtype if isinstance(x, _Tensor) else _bf16
    if dtype is not _bf16 and dtype is not _f32:
        raise TypeError(f"x must be float32 or bfloat16, got {dtype}")
    w_dtype = weight.dtype if isinstance(weight, _Tensor) else weight2.dtype if isinstance(weight2, _Tensor) else _f32
    if w_dtype is not _bf16 and w_dtype is not _f32:
        raise TypeError(f"weight must be float32 or bfloat16, got {w_dtype}")
    if bwd and (g is None or (x2 is None) != (g2 is None)):
        raise TypeError("each of x and x2 needs the gradient of its output")
    if x2 is None and weight2 is not None:
        raise TypeError("weight2 needs x2")
    if out is None:
        o = (None,) * 4
    elif not bwd and x2 is None:
        o = (out, None)
    else:
        o, n = tuple(out), (1 if x2 is None else 2) * (2 if bwd else 1)
        if len(o) != n:
            raise ValueError(f"out has {len(o)} tensors, not {n}")
        o = o if bwd else (o[0], None, o[1], None)
    shape, dev, arr, y, dw = _norm_side(x, weight, g, o[0], o[1], "", dtype, w_dtype, None, bwd, stream)
    T0, T1, _, D = shape
    if x2 is not None:
        s2, _, arr2, y2, dw2 = _norm_side(x2, weight2, g2, o[2], o[3], "2", dtype, w_dtype, dev, bwd, stream)
        if s2[0] != T0 or s2[1] != T1 or s2[3] != D:
            raise ValueError("x and x2 shapes disagree")
        arr += arr2
    turn = _turn(pos, freqs, layout, rot_off, mscale, axes, T0, T1, dev)
    L, nt, dt, wdt = _lib or lib(), 1 if x2 is None else 2, 1 if dtype is _bf16 else 0, 1 if w_dtype is _bf16 else 0
    if bwd:
        if workspace is None:
            ws_bytes = L.lidx_norm_rope_bwd_workspace_bytes(D)
            workspace = _scratch(ws_bytes, x.device, stream)
        else:
            ws_bytes = _dense(workspace, "workspace", _u8, (None,), dev)[0]
        rc = L.lidx_norm_rope_bwd(arr, nt, turn, eps, T0, T1, D, dt, wdt, workspace.data_ptr(), ws_bytes,
                                  _raw_stream(stream, dev))
        if rc:
            raise LidxError(rc, "lidx_norm_rope_bwd")
        return (y, dw) if x2 is None else (y, dw, y2, dw2)
    rc = L.lidx_norm_rope(arr, nt, turn, eps, T0, T1, D, dt, wdt, _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_norm_rope")
    return y if x2 is None else (y, y2)


def lidx_norm_rope(x, weight, pos, freqs, x2=None, weight2=None, eps=1e-6, layout="interleaved", rot_off=0, mscale=1.0,
                   axes=None, stream=None, out=None):
    """Root-mean-square norm of each head of x [T0,T1,H,D] over its D dims, times weight [D] (fp32 or bf16; None: ones), and
    its rotary positions as lidx_rope's, in one pass; in the same launch those of x2 with weight2 (queries and keys).
    Computed in fp32 and rounded once.  Returns y, or (y, y2).  ``out`` may be the inputs themselves."""
    return _norm_rope(x, weight, pos, freqs, None, x2, weight2, None, eps, layout, rot_off, mscale, axes, stream, out, None,
                      False)


def lidx_norm_rope_bwd(g, x, weight, pos, freqs, g2=None, x2=None, weight2=None, eps=1e-6, layout="interleaved", rot_off=0,
                       mscale=1.0, axes=None, stream=None, out=None, workspace=None):
    """Gradients of lidx_norm_rope from its inputs and the gradients g (and g2) of its outputs: (dx, dw) or (dx, dw, dx2,
    dw2).  dw, the sum over all rows, is fp32 [D] (None where the weight is).  ``out`` has a tensor, or None, for each of
    them; dx may be g or x itself."""
    return _norm_rope(x, weight, pos, freqs, g, x2, weight2, g2, eps, layout, rot_off, mscale, axes, stream, out, workspace,
                      True)


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


def _append_args(k, v, freqs, pos, weight, layout, rot_off, mscale, axes, start, count):
    """Checks of the new tokens, of their norm and rotation, and what goes to C of them before the table."""
    shape, ks, dev = _strided(k, "k", _bf16)
    shape_v, vs, _ = _strided(v, "v", _bf16, dev)
    if shape_v != shape:
        raise ValueError("k and v shapes disagree")
    B, S, Hkv, D = shape
    turn = None
    if freqs is not None:
        turn = _turn(pos, freqs, layout, rot_off, mscale, axes, B, S, dev, True)
    elif pos is not None or axes is not None:
        raise ValueError("pos and axes need freqs")
    wdt = 0
    if weight is not None:
        if not isinstance(weight, _Tensor) or (weight.dtype is not _f32 and weight.dtype is not _bf16):
            raise TypeError("weight must be a float32 or bfloat16 tensor")
        _dense(weight, "weight", weight.dtype, (D,), dev)
        wdt = 1 if weight.dtype is _bf16 else 0
    _dense(start, "start", _i32, (B,), dev)
    if count is not None:
        _dense(count, "count", _i32, (B,), dev)
    return shape, dev, (k.data_ptr(), v.data_ptr(), _I3(*ks), _I3(*vs), turn,
                        None if weight is None else weight.data_ptr(), wdt)


def lidx_rope_cache_append(k, v, freqs, k_cache, v_cache, k_scale, v_scale, block_table, start, count=None, pos=None,
                           weight=None, eps=1e-6, layout="interleaved", rot_off=0, mscale=1.0, axes=None, stream=None):
    """lidx_cache_append with the norm (weight [D] fp32 or bf16; None: no norm) and the rotary positions of the keys on the
    way, as lidx_norm_rope's and lidx_rope's, in fp32: keys are rounded once, to the cache's numbers.  pos: int32, broadcast
    to [B,S] (with axes [A, ...]); None: token i of sequence b is at start[b] + i."""
    (B, S, Hkv, D), dev, args = _append_args(k, v, freqs, pos, weight, layout, rot_off, mscale, axes, start, count)
    if freqs is None:
        raise TypeError("freqs must be lidx_rope_freqs's tensor")
    pages, _, page, MP = _cache(k_cache, v_cache, k_scale, v_scale, block_table, B, Hkv, D, dev)
    rc = (_lib or lib()).lidx_rope_cache_append(
        *args, eps, block_table.data_ptr(), start.data_ptr(), None if count is None else count.data_ptr(), B, S, Hkv, D,
        page, MP, pages, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_rope_cache_append")


def _cache4(k_cache, v_cache, k_exps, v_exps, Hkv, D, dev):
    shape = _dense(k_cache, "k_cache", _u8, (None, Hkv, None, None if D is None else D // 2), dev)
    _dense(v_cache, "v_cache", _u8, shape, dev)
    _dense(k_exps, "k_exps", _i32, shape[:3], dev)
    _dense(v_exps, "v_exps", _i32, shape[:3], dev)
    return shape


def lidx_cache4_append(k, v, k_cache, v_cache, k_exps, v_exps, k_scale, v_scale, block_table, start, count=None, freqs=None,
                       pos=None, weight=None, eps=1e-6, layout="interleaved", rot_off=0, mscale=1.0, axes=None, stream=None):
    """Writes k, v [B,S,Hkv,D] bf16 behind the start[b] tokens that each sequence's pages hold, in 4 bits, with the norm
    (weight) and the rotary positions (freqs) of the keys on the way as in lidx_rope_cache_append; both may be left out.

    k_cache, v_cache uint8 [P,Hkv,page,D/2] (two codes a byte), k_exps, v_exps int32 [P,Hkv,page] (an exponent of four bits
    for each 16 dims) and k_scale, v_scale fp32 [P,Hkv] are updated in place: a slot holds code * 2^exponent * scale, the
    codes being 0 .5 1 1.5 2 3 4 6 and their negatives.  A group of 16 dims with an infinity or a NaN reads as NaN."""
    (B, S, Hkv, D), dev, args = _append_args(k, v, freqs, pos, weight, layout, rot_off, mscale, axes, start, count)
    pages, _, page, _ = _cache4(k_cache, v_cache, k_exps, v_exps, Hkv, D, dev)
    _dense(k_scale, "k_scale", _f32, (pages, Hkv), dev)
    _dense(v_scale, "v_scale", _f32, (pages, Hkv), dev)
    MP = _dense(block_table, "block_table", _i32, (B, None), dev)[1]
    rc = (_lib or lib()).lidx_cache4_append(
        *args, eps, block_table.data_ptr(), start.data_ptr(), None if count is None else count.data_ptr(), B, S, Hkv, D,
        page, MP, pages, k_cache.data_ptr(), v_cache.data_ptr(), k_exps.data_ptr(), v_exps.data_ptr(), k_scale.data_ptr(),
        v_scale.data_ptr(), _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_cache4_append")


def lidx_cache4_to_8(k_cache, v_cache, k_exps, v_exps, stream=None, out=None):
    """A 4-bit cache as an 8-bit one: (k8, v8) float8_e4m3fn [P,Hkv,page,D] that hold code * 2^exponent / 32 exactly, NaN
    where a group reads as NaN.  With scales of 32 times the 4-bit cache's they are the same cache for lidx_cache_attn."""
    dev = k_cache.get_device() if isinstance(k_cache, _Tensor) else 0
    pages, Hkv, page, half = _cache4(k_cache, v_cache, k_exps, v_exps, None, None, dev)
    shape = (pages, Hkv, page, 2 * half)
    if out is None:
        k8, v8 = _new(shape, _f8, k_cache.device, stream), _new(shape, _f8, k_cache.device, stream)
    else:
        k8, v8 = out
        _dense(k8, "out", _f8, shape, dev)
        _dense(v8, "out", _f8, shape, dev)
    rc = (_lib or lib()).lidx_cache4_to_8(k_cache.data_ptr(), v_cache.data_ptr(), k_exps.data_ptr(), v_exps.data_ptr(), Hkv,
                                          2 * half, page, pages, k8.data_ptr(), v8.data_ptr(), _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_cache4_to_8")
    return k8, v8


def lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk=0) -> int:
    return int(lib().lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk))


def lidx_cache4_attn_workspace_bytes(B, S, Hq, Hkv, D, page, max_pages, topk=0) -> int:
    return int(lib().lidx_cache4_attn_workspace_bytes(B, S, Hq, Hkv, D, page, max_pages, topk))


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
    pages, Hkv, page, MP = _cache(k_cache, v_cache, k_scale, v_scale, block_table, shape[0], None, shape[3], dev)
    return _cache_attn(False, q, shape, qs, dev, (k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                                                  v_scale.data_ptr(), block_table.data_ptr()),
                       Hkv, page, MP, pages, kv_len, q_pos, compress_ratio, topk_indices, softmax_scale, want_lse, stream, out,
                       workspace)


def lidx_cache4_attn(q, k_cache, v_cache, k_exps, v_exps, k_scale, v_scale, block_table, kv_len, q_pos=None,
                     compress_ratio=1, topk_indices=None, softmax_scale=None, want_lse=False, stream=None, out=None,
                     workspace=None):
    """lidx_cache_attn over a cache written by lidx_cache4_append (codes, exponents and scales; value scales 2^-85 .. 2^95)."""
    shape, qs, dev = _strided(q, "q", _bf16)
    pages, Hkv, page, _ = _cache4(k_cache, v_cache, k_exps, v_exps, None, shape[3], dev)
    _dense(k_scale, "k_scale", _f32, (pages, Hkv), dev)
    _dense(v_scale, "v_scale", _f32, (pages, Hkv), dev)
    MP = _dense(block_table, "block_table", _i32, (shape[0], None), dev)[1]
    return _cache_attn(True, q, shape, qs, dev, (k_cache.data_ptr(), v_cache.data_ptr(), k_exps.data_ptr(), v_exps.data_ptr(),
                                                 k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr()),
                       Hkv, page, MP, pages, kv_len, q_pos, compress_ratio, topk_indices, softmax_scale, want_lse, stream, out,
                       workspace)


def _cache_attn(four, q, shape, qs, dev, cache, Hkv, page, MP, pages, kv_len, q_pos, compress_ratio, topk_indices,
                softmax_scale, want_lse, stream, out, workspace):
    """The calls of both caches from their checked queries; cache: the addresses of the cache's parts and of its table."""
    B, S, Hq, D = shape
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
        if four:
            ws_bytes = L.lidx_cache4_attn_workspace_bytes(B, S, Hq, Hkv, D, page, MP, topk)
        else:
            ws_bytes = L.lidx_cache_attn_workspace_bytes(B, S, Hq, Hkv, D, topk)
        workspace = _scratch(ws_bytes, q.device, stream)
    else:
        ws_bytes = _dense(workspace, "workspace", torch.uint8, (None,), dev)[0]
    rc = (L.lidx_cache4_attn if four else L.lidx_cache_attn)(
        q.data_ptr(), _I3(*qs), *cache, kv_len.data_ptr(), None if q_pos is None else q_pos.data_ptr(),
        None if topk_indices is None else topk_indices.data_ptr(), B, S, Hq, Hkv, D, page, MP, pages, compress_ratio,
        topk, D ** -0.5 if softmax_scale is None else softmax_scale, o.data_ptr(), None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), ws_bytes, _raw_stream(stream, dev))
    if rc:
        raise LidxError(rc, "lidx_cache4_attn" if four else "lidx_cache_attn")
    return o, lse
