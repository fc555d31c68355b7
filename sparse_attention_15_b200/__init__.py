"""Python binding of libdsa, the B200 DSA hot path (see include/dsa.h for the contract).

Argument marshalling only: every function here reads sizes off torch tensors, allocates
outputs and workspaces (device memory plumbing) when the caller gives none, passes raw device
pointers and the CUDA stream (the current one, or the caller's `stream`) to the C entry point of
the same name, and raises DSAError on a non-OK status.  All compute runs in the library's CUDA kernels; there is no
fallback -- if libdsa.so is missing, importing a function raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = [
    "DSAError", "lib", "dsa_index_scores", "dsa_index_scores_collapsed", "dsa_hadamard_rotate",
    "dsa_topk", "dsa_index_topk", "dsa_index_topk_workspace_bytes",
    "dsa_sparse_attn", "dsa_sparse_attn_sinks", "dsa_sparse_attn_workspace_bytes",
    "dsa_sparse_attn_algo", "dsa_forward",
    "dsa_forward_workspace_bytes",
    "dsa_window_attn", "Cache", "dsa_cache_pages", "dsa_cache_row_bytes", "dsa_cache_append",
    "dsa_cache_read", "dsa_cache_attn", "dsa_cache_sparse_attn", "dsa_sparse_attn_noalloc",
    "dsa_device_status", "dsa_version",
    "dsa_test_arm_wait_timeout", "dsa_test_topk_bucket_floor", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdsa.so")

DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2}  # e4m3: indexer inputs
RELU = {"none": 0, "post_sum": 1, "per_head": 2}
GATE = {"off": 0, "sigmoid": 1, "silu": 2}
ATTN_ALGO = {"auto": 0, "gather": 1, "masked_tile": 2}
INDEXER = {"per_head": 0, "collapsed": 1, "fused": 2}
ATTN_FORM = {"expanded": 0, "latent": 1}
CACHE_FORMAT = {"bf16": 0, "e2m1": 1}
ROPE = {"off": 0, "interleaved": 1, "half": 2}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "CUDA error", 4: "timeout",
          5: "internal"}


class DSAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libdsa status {status} ({STATUS.get(status, '?')}): {message}")
        self.status = status


class ForwardArgs(ctypes.Structure):
    """Mirror of dsa_forward_args (include/dsa.h)."""
    _fields_ = [
        ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("S", ctypes.c_int), ("T", ctypes.c_int),
        ("HI", ctypes.c_int), ("DI", ctypes.c_int), ("index_scale", ctypes.c_float),
        ("relu", ctypes.c_int), ("K", ctypes.c_int), ("H", ctypes.c_int), ("DQK", ctypes.c_int),
        ("DV", ctypes.c_int), ("sm_scale", ctypes.c_float), ("gate_mode", ctypes.c_int),
        ("attn_algo", ctypes.c_int),
        ("q_idx", ctypes.c_void_p), ("k_idx", ctypes.c_void_p), ("w", ctypes.c_void_p),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("out", ctypes.c_void_p), ("scores_out", ctypes.c_void_p),
        ("idx_out", ctypes.c_void_p), ("events", ctypes.c_void_p), ("indexer", ctypes.c_int),
        ("index_dtype", ctypes.c_int), ("sink_k", ctypes.c_void_p), ("sink_v", ctypes.c_void_p),
        ("nsink", ctypes.c_int), ("attn_form", ctypes.c_int),
        ("topk_fallback_out", ctypes.c_void_p),
    ]


class CacheArgs(ctypes.Structure):
    """Mirror of dsa_cache (include/dsa.h)."""
    _fields_ = [
        ("format", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
        ("max_pages", ctypes.c_int), ("HKV", ctypes.c_int), ("DQK", ctypes.c_int),
        ("DV", ctypes.c_int), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
        ("pages", ctypes.c_void_p), ("table", ctypes.c_void_p),
    ]


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_INT_MAX = 2 ** 31 - 1
_F = ctypes.c_float
_Z = ctypes.c_size_t

_SIGNATURES = {
    "dsa_index_scores": (_I, [_I, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _P, _P]),
    "dsa_index_scores_collapsed_workspace_bytes": (_Z, [_I, _I, _I]),
    "dsa_index_scores_collapsed": (_I, [_I, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _P, _P, _Z,
                                        _P]),
    "dsa_hadamard_rotate": (_I, [_I, _P, ctypes.c_longlong, _I, _P, _P]),
    "dsa_topk": (_I, [_P, _I, _I, _I, _I, _P, _P]),
    "dsa_index_topk_workspace_bytes": (_Z, [_I, _I, _I, _I]),
    "dsa_index_topk": (_I, [_I, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _P, _P, _Z, _P,
                            _P]),
    "dsa_sparse_attn_workspace_bytes": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "dsa_sparse_attn_algo": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "dsa_sparse_attn": (_I, [_I, _P, _P, _P, _P, _I, _P, _I, _F, _I, _I, _I, _I, _I, _I, _I, _P,
                             _P, _Z, _P]),
    "dsa_sparse_attn_sinks_workspace_bytes": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "dsa_sparse_attn_sinks": (_I, [_I, _P, _P, _P, _P, _I, _P, _P, _I, _P, _I, _F, _I, _I, _I,
                                   _I, _I, _I, _I, _P, _P, _Z, _P]),
    "dsa_sparse_attn_latent_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "dsa_sparse_attn_latent": (_I, [_I, _P, _P, _P, _I, _P, _I, _P, _I, _F, _I, _I, _I, _I, _I,
                                    _I, _P, _P, _Z, _P]),
    "dsa_forward_workspace_bytes": (_Z, [ctypes.POINTER(ForwardArgs)]),
    "dsa_forward_min_workspace_bytes": (_Z, [ctypes.POINTER(ForwardArgs)]),
    "dsa_forward": (_I, [ctypes.POINTER(ForwardArgs), _P, _Z, _P]),
    "dsa_window_attn": (_I, [_I, _P, _P, _P, _P, _I, _F, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                             _P, _P]),
    "dsa_window_attn_sinks": (_I, [_I, _P, _P, _P, _P, _P, _I, _P, _I, _F, _I, _I, _I, _I, _I,
                                   _I, _I, _I, _I, _P, _P]),
    "dsa_window_attn_first": (_I, [_I, _P, _P, _P, _I, _P, _I, _F, _I, _I, _I, _I, _I, _I, _I,
                                   _I, _I, _P, _P]),
    "dsa_cache_row_bytes": (_Z, [_I, _I, _I, _I]),
    "dsa_cache_append": (_I, [ctypes.POINTER(CacheArgs), _P, _P, _P, _I, _I, _P, _I, _I, _I, _P,
                              _P, _P, _P]),
    "dsa_cache_read": (_I, [ctypes.POINTER(CacheArgs), _P, _I, _I, _P, _P, _P]),
    "dsa_cache_attn_workspace_bytes": (_Z, [ctypes.POINTER(CacheArgs), _I, _I, _I, _I, _I]),
    "dsa_cache_attn": (_I, [ctypes.POINTER(CacheArgs), _P, _P, _I, _I, _P, _I, _F, _I, _I, _I, _P,
                            _P, _Z, _P]),
    "dsa_cache_sparse_attn_workspace_bytes": (_Z, [ctypes.POINTER(CacheArgs), _I, _I, _I, _I]),
    "dsa_cache_sparse_attn": (_I, [ctypes.POINTER(CacheArgs), _P, _P, _P, _I, _P, _I, _F, _I, _I,
                                   _I, _P, _P, _Z, _P]),
    "dsa_sparse_attn_noalloc_max_scratch_bytes": (_Z, []),
    "dsa_sparse_attn_noalloc": (_I, [_I, _P, _P, _P, _P, _I, _P, _I, _F, _I, _I, _I, _I, _I, _I,
                                     _P, _P]),
    "dsa_status_string": (ctypes.c_char_p, [_I]),
    "dsa_last_error": (ctypes.c_char_p, []),
    "dsa_device_status": (_I, [_I]),
    "dsa_version": (ctypes.c_char_p, []),
    "dsa_test_arm_wait_timeout": (_I, []),
    "dsa_test_topk_bucket_floor": (ctypes.c_float, [ctypes.c_uint]),
}


def lib() -> ctypes.CDLL:
    """The loaded libdsa.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m sparse_attention_15_b200.build`"
                " (there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def _check(status: int):
    if status != 0:
        raise DSAError(status, lib().dsa_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _own(shape, dtype, device, stream, returned=True):
    """A tensor that a call allocates for itself, from the pool of the stream it runs on.  (The pool
    of another stream may hand out a block whose last use is still queued there.)  One that the
    caller gets is kept from reuse until the current stream, too, is done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _int(x):
    """An argument as a C int: past its range the end of the range (ctypes would wrap it), which the
    library refuses, or takes as a window or a number of keys that covers every key."""
    x = int(x)
    return x if -_INT_MAX <= x <= _INT_MAX else _INT_MAX if x > 0 else -_INT_MAX - 1


def _cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libdsa takes contiguous CUDA tensors")


def _dev(*ts):
    """A call's tensors: contiguous, and on the current device, where its kernels run."""
    _cuda(*ts)
    current = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.get_device() != current:
            raise ValueError(f"a tensor is on {t.device}, which is not the current device")


def _fits(name, t, shape, dtype):
    """An argument that the library reads or writes as a contiguous `shape` of `dtype`: at least as
    many elements (a larger buffer of the caller's is fine)."""
    if t is not None and (t.dtype != dtype or t.numel() < math.prod(shape)):
        raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype}: expected {tuple(shape)} {dtype}")


def _dtype_code(t):
    try:
        return DTYPE[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def dsa_version() -> str:
    return lib().dsa_version().decode()


def dsa_device_status(reset: bool = True) -> int:
    """Reads (and clears) the device status word; raises DSAError on a recorded fault."""
    st = lib().dsa_device_status(1 if reset else 0)
    _check(st)
    return st


def dsa_test_arm_wait_timeout() -> None:
    """Testing aid: the next gather-attention launch runs one bounded wait out on purpose
    (it records DSA_ERR_TIMEOUT; its output is undefined).  One-shot."""
    _check(lib().dsa_test_arm_wait_timeout())


def dsa_test_topk_bucket_floor(b: int) -> float:
    """Testing aid: the top-k's float bound of 12-bit key bucket b (host code)."""
    return float(lib().dsa_test_topk_bucket_floor(b))


def dsa_index_scores(q_idx, k_idx, w, scale, relu="none", scores=None, stream=None):
    """scores[b,s,t] = scale * sum_h w[b,s,h] (q_idx[b,s,h,:] . k_idx[b,t,:]), -inf if t > s+T-S."""
    _dev(q_idx, k_idx, w, scores)
    B, S, HI, DI = q_idx.shape
    T = k_idx.shape[1]
    if scores is None:
        scores = _own((B, S, T), torch.float32, q_idx.device, stream)
    _check(lib().dsa_index_scores(_dtype_code(q_idx), _ptr(q_idx), _ptr(k_idx), _ptr(w),
                                  float(scale), RELU[relu], B, S, T, HI, DI, _ptr(scores),
                                  _stream(stream)))
    return scores


def dsa_index_scores_collapsed(q_idx, k_idx, w, scale, relu="none", scores=None, ws=None,
                               stream=None):
    """The same scores as dsa_index_scores from the head-collapsed query
    sum_h w[b,s,h] q_idx[b,s,h,:] (bf16, no per-head ReLU; see include/dsa.h)."""
    _dev(q_idx, k_idx, w, scores, ws)
    B, S, HI, DI = q_idx.shape
    T = k_idx.shape[1]
    if scores is None:
        scores = _own((B, S, T), torch.float32, q_idx.device, stream)
    nbytes = int(lib().dsa_index_scores_collapsed_workspace_bytes(B, S, DI))
    ws = _workspace(nbytes, q_idx.device, ws, stream)
    _check(lib().dsa_index_scores_collapsed(_dtype_code(q_idx), _ptr(q_idx), _ptr(k_idx), _ptr(w),
                                            float(scale), RELU[relu], B, S, T, HI, DI,
                                            _ptr(scores), _ptr(ws), nbytes, _stream(stream)))
    return scores


def dsa_hadamard_rotate(x, out=None, stream=None):
    """x @ H / sqrt(d) over the last dimension (d in {64, 128}; float32 or bf16); out may be x."""
    _dev(x, out)
    d = x.shape[-1]
    if out is None:
        out = _own(x.shape, x.dtype, x.device, stream)
    _check(lib().dsa_hadamard_rotate(_dtype_code(x), _ptr(x), x.numel() // d, d, _ptr(out),
                                     _stream(stream)))
    return out


def dsa_topk(scores, K, idx=None, stream=None):
    """int32 [B,S,K]: the kept keys of each query in ascending order, -1 padded."""
    _dev(scores, idx)
    B, S, T = scores.shape
    if idx is None:
        idx = _own((B, S, K), torch.int32, scores.device, stream)
    _check(lib().dsa_topk(_ptr(scores), B, S, T, _int(K), _ptr(idx), _stream(stream)))
    return idx



def dsa_index_topk_workspace_bytes(B, S, T, K) -> int:
    return int(lib().dsa_index_topk_workspace_bytes(B, S, T, _int(K)))


def dsa_index_topk(q_idx, k_idx, w, scale, K, relu="none", idx=None, ws=None,
                   fallback_out=None, stream=None):
    """Fused indexer -> top-k: the indices dsa_index_scores + dsa_topk give, without the
    score matrix (candidates filtered inside the indexer).  fallback_out: optional int32
    device tensor of one element, set to 1 when the full-score fallback ran."""
    _dev(q_idx, k_idx, w, idx, ws, fallback_out)
    B, S, HI, DI = q_idx.shape
    T = k_idx.shape[1]
    k_eff = min(int(K), T)
    if idx is None:
        idx = _own((B, S, k_eff), torch.int32, q_idx.device, stream)
    nbytes = dsa_index_topk_workspace_bytes(B, S, T, K)
    ws = _workspace(nbytes, q_idx.device, ws, stream)
    _check(lib().dsa_index_topk(_dtype_code(q_idx), _ptr(q_idx), _ptr(k_idx), _ptr(w),
                                float(scale), RELU[relu], B, S, T, HI, DI, _int(K), _ptr(idx),
                                _ptr(ws), nbytes, _ptr(fallback_out), _stream(stream)))
    return idx

def dsa_sparse_attn_workspace_bytes(dtype, B, S, T, H, DQK, DV, K, algo="auto") -> int:
    code = dtype if isinstance(dtype, int) else DTYPE[dtype]
    return int(lib().dsa_sparse_attn_workspace_bytes(code, B, S, T, H, DQK, DV, K,
                                                     ATTN_ALGO[algo]))


def dsa_sparse_attn_algo(dtype, B, S, T, H, DQK, DV, K, algo="auto") -> str:
    """The algorithm ("gather" / "masked_tile") a request resolves to for this shape."""
    code = dtype if isinstance(dtype, int) else DTYPE[dtype]
    r = int(lib().dsa_sparse_attn_algo(code, B, S, T, H, DQK, DV, K, ATTN_ALGO[algo]))
    return {v: k for k, v in ATTN_ALGO.items()}[r]


def _workspace(nbytes, device, ws, stream):
    if nbytes == 0:
        return ws
    if ws is None or ws.numel() < nbytes:
        ws = _own(nbytes, torch.uint8, device, stream, returned=False)
    return ws


def dsa_sparse_attn(q, k, v, idx, gate=None, gate_mode=None, sm_scale=0.0, algo="auto",
                    out=None, ws=None, stream=None):
    """Attention of each query over its selected keys (idx), with the optional gate.
    algo: "auto", "gather" or "masked_tile"."""
    _dev(q, k, v, idx, gate, out, ws)
    B, S, H, DQK = q.shape
    T, DV = k.shape[1], v.shape[-1]
    K = idx.shape[-1]
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    if out is None:
        out = _own((B, S, H, DV), q.dtype, q.device, stream)
    nbytes = dsa_sparse_attn_workspace_bytes(_dtype_code(q), B, S, T, H, DQK, DV, K, algo)
    ws = _workspace(nbytes, q.device, ws, stream)
    _check(lib().dsa_sparse_attn(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), K,
                                 _ptr(gate), gm, float(sm_scale), B, S, T, H, DQK, DV,
                                 ATTN_ALGO[algo], _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def dsa_sparse_attn_sinks(q, k, v, idx, sink_k, sink_v, gate=None, gate_mode=None,
                          sm_scale=0.0, algo="auto", out=None, ws=None, stream=None):
    """dsa_sparse_attn with attention sinks: sink_k [NS,H,DQK], sink_v [NS,H,DV] (NS <= 128)
    join every query's softmax unmasked."""
    _dev(q, k, v, idx, sink_k, sink_v, gate, out, ws)
    B, S, H, DQK = q.shape
    T, DV = k.shape[1], v.shape[-1]
    K = idx.shape[-1]
    NS = sink_k.shape[0]
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    if out is None:
        out = _own((B, S, H, DV), q.dtype, q.device, stream)
    nbytes = int(lib().dsa_sparse_attn_sinks_workspace_bytes(_dtype_code(q), B, S, T, H, DQK, DV,
                                                             K, NS, ATTN_ALGO[algo]))
    ws = _workspace(nbytes, q.device, ws, stream)
    _check(lib().dsa_sparse_attn_sinks(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), K,
                                       _ptr(sink_k), _ptr(sink_v), NS, _ptr(gate), gm,
                                       float(sm_scale), B, S, T, H, DQK, DV, ATTN_ALGO[algo],
                                       _ptr(out), _ptr(ws), nbytes, _stream(stream)))
    return out


def dsa_sparse_attn_noalloc(q, k, v, idx, gate=None, gate_mode=None, sm_scale=0.0, out=None,
                            stream=None):
    """dsa_sparse_attn (gather form) with no workspace: the split-key partials live in the
    library's fixed device array (see include/dsa.h).  Allocates nothing but ``out`` when
    the caller gives none."""
    _dev(q, k, v, idx, gate, out)
    B, S, H, DQK = q.shape
    T, DV = k.shape[1], v.shape[-1]
    K = idx.shape[-1]
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    if out is None:
        out = _own((B, S, H, DV), q.dtype, q.device, stream)
    _check(lib().dsa_sparse_attn_noalloc(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), K,
                                         _ptr(gate), gm, float(sm_scale), B, S, T, H, DQK, DV,
                                         _ptr(out), _stream(stream)))
    return out


def dsa_sparse_attn_latent(q, kv, idx, dv=512, sink_kv=None, gate=None, gate_mode=None,
                           sm_scale=0.0, out=None, ws=None, stream=None):
    """Sparse attention over a shared latent cache (MQA form): q [B,S,H,DQK], kv [B,T,DQK]
    (keys = whole rows, values = their first ``dv`` dims), idx [B,S,K]; optional latent sink
    rows sink_kv [NS,DQK] (NS <= 128).  bf16, DQK 576, dv 512, H <= 128."""
    _dev(q, kv, idx, sink_kv, gate, out, ws)
    B, S, H, DQK = q.shape
    T = kv.shape[1]
    K = idx.shape[-1]
    NS = 0 if sink_kv is None else int(sink_kv.shape[0])
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    if out is None:
        out = _own((B, S, H, dv), q.dtype, q.device, stream)
    nbytes = int(lib().dsa_sparse_attn_latent_workspace_bytes(B, S, H, K, NS))
    ws = _workspace(nbytes, q.device, ws, stream)
    _check(lib().dsa_sparse_attn_latent(_dtype_code(q), _ptr(q), _ptr(kv), _ptr(idx), K,
                                        _ptr(sink_kv), NS, _ptr(gate), gm, float(sm_scale), B, S,
                                        T, H, DQK, int(dv), _ptr(out), _ptr(ws), nbytes,
                                        _stream(stream)))
    return out


def _forward_args(q_idx, k_idx, w, index_scale, K, q, k, v, gate, gate_mode, relu, sm_scale,
                  attn_algo, out, scores_out, idx_out, indexer="per_head", sink_k=None,
                  sink_v=None, attn_form="expanded", dv=512, topk_fallback_out=None):
    B, S, HI, DI = q_idx.shape
    T = k_idx.shape[1]
    H, DQK = q.shape[2], q.shape[3]
    DV = int(dv) if attn_form == "latent" else v.shape[-1]
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    a = ForwardArgs(
        dtype=_dtype_code(q), B=B, S=S, T=T, HI=HI, DI=DI, index_scale=float(index_scale),
        relu=RELU[relu], K=_int(K), H=H, DQK=DQK, DV=DV, sm_scale=float(sm_scale), gate_mode=gm,
        attn_algo=ATTN_ALGO[attn_algo], q_idx=q_idx.data_ptr(), k_idx=k_idx.data_ptr(),
        w=w.data_ptr(), q=q.data_ptr(), k=k.data_ptr(), v=None if v is None else v.data_ptr(),
        gate=None if gate is None else gate.data_ptr(), out=out.data_ptr(),
        scores_out=None if scores_out is None else scores_out.data_ptr(),
        idx_out=None if idx_out is None else idx_out.data_ptr(), indexer=INDEXER[indexer],
        index_dtype=1 if q_idx.dtype == torch.float8_e4m3fn else 0,
        sink_k=None if sink_k is None else sink_k.data_ptr(),
        sink_v=None if sink_v is None else sink_v.data_ptr(),
        nsink=0 if sink_k is None else int(sink_k.shape[0]), attn_form=ATTN_FORM[attn_form],
        topk_fallback_out=None if topk_fallback_out is None else topk_fallback_out.data_ptr())
    return a


def dsa_forward_workspace_bytes(args: ForwardArgs, minimum: bool = False) -> int:
    f = lib().dsa_forward_min_workspace_bytes if minimum else lib().dsa_forward_workspace_bytes
    return int(f(ctypes.byref(args)))


def dsa_forward(q_idx, k_idx, w, index_scale, K, q, k, v, gate=None, gate_mode=None,
                relu="none", sm_scale=0.0, attn_algo="auto", out=None, scores_out=None,
                idx_out=None, ws=None, ws_bytes=None, stream=None, events=None,
                indexer="per_head", sink_k=None, sink_v=None, attn_form="expanded", dv=512,
                topk_fallback_out=None):
    """The whole DSA step (indexer -> top-k -> sparse attention -> gate).
    indexer: "per_head" (the pages' per-head work), "collapsed" (see
    dsa_index_scores_collapsed) or "fused" (see dsa_index_topk; topk_fallback_out, an
    optional int32 device tensor of one element, receives whether its fallback ran).  attn_form "latent": k is the latent cache [B,T,DQK]
    (values = its first ``dv`` dims), v is None, sink_k holds latent sink rows [NS,DQK].

    Returns (out, idx); idx is idx_out if given, else a view of the workspace copy.
    ``ws_bytes`` limits the workspace handed to the library (row blocking below the
    full size)."""
    _dev(q_idx, k_idx, w, q, k, v, gate, out, scores_out, idx_out, ws, sink_k, sink_v,
         topk_fallback_out)
    B, S = q_idx.shape[:2]
    T = k_idx.shape[1]
    if out is None:
        DV = int(dv) if attn_form == "latent" else v.shape[-1]
        out = _own((B, S, q.shape[2], DV), q.dtype, q.device, stream)
    k_eff = min(int(K), T)
    if idx_out is None:
        idx_out = _own((B, S, k_eff), torch.int32, q.device, stream)
    a = _forward_args(q_idx, k_idx, w, index_scale, K, q, k, v, gate, gate_mode, relu, sm_scale,
                      attn_algo, out, scores_out, idx_out, indexer, sink_k, sink_v, attn_form,
                      dv, topk_fallback_out)
    ev_arr = None
    if events is not None:  # 4 torch.cuda.Event, recorded by the library at stage boundaries
        for e in events:
            if e.cuda_event == 0:
                e.record()  # torch creates the CUDA event on first use
        ev_arr = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
        a.events = ctypes.cast(ev_arr, ctypes.c_void_p).value
    nbytes = dsa_forward_workspace_bytes(a) if ws_bytes is None else int(ws_bytes)
    ws = _workspace(nbytes, q.device, ws, stream)
    _check(lib().dsa_forward(ctypes.byref(a), _ptr(ws), nbytes, _stream(stream)))
    return out, idx_out


def dsa_window_attn(q, k, v, window, gate=None, gate_mode=None, sm_scale=0.0, algo="auto",
                    out=None, stream=None, sink_k=None, sink_v=None, n_first=0):
    """Sliding-window causal attention with grouped KV heads (window keys incl. self);
    optional attention sinks sink_k [NS,HKV,DQK], sink_v [NS,HKV,DV] (NS <= 128), or the
    sequence's first n_first tokens (<= 128) staying visible."""
    _dev(q, k, v, gate, out, sink_k, sink_v)
    window, n_first = _int(window), _int(n_first)
    if n_first and sink_k is not None:
        raise ValueError("sink_k / sink_v and n_first are alternatives")
    B, S, H, DQK = q.shape
    T, HKV, DV = k.shape[1], k.shape[2], v.shape[-1]
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    if k.shape[1:] != (T, HKV, DQK) or v.shape[1:] != (T, HKV, DV):
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not go with q {tuple(q.shape)}"
                         " or with each other")
    if (sink_k is None) != (sink_v is None):
        raise ValueError("sink_k and sink_v go together")
    NS = 0 if sink_k is None else sink_k.shape[0]
    for name, t, shape in (("k", k, (B, T, HKV, DQK)), ("v", v, (B, T, HKV, DV)),
                           ("gate", gate, (B, S, H)), ("out", out, (B, S, H, DV)),
                           ("sink_k", sink_k, (NS, HKV, DQK)), ("sink_v", sink_v, (NS, HKV, DV))):
        _fits(name, t, shape, q.dtype)
    if out is None:
        out = _own((B, S, H, DV), q.dtype, q.device, stream)
    if n_first:
        _check(lib().dsa_window_attn_first(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v),
                                           n_first, _ptr(gate), gm, float(sm_scale), window, B,
                                           S, T, H, HKV, DQK, DV,
                                           ATTN_ALGO[algo], _ptr(out), _stream(stream)))
    elif sink_k is None:
        _check(lib().dsa_window_attn(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v), _ptr(gate), gm,
                                     float(sm_scale), window, B, S, T, H, HKV, DQK, DV,
                                     ATTN_ALGO[algo], _ptr(out), _stream(stream)))
    else:
        _check(lib().dsa_window_attn_sinks(_dtype_code(q), _ptr(q), _ptr(k), _ptr(v),
                                           _ptr(sink_k), _ptr(sink_v), NS,
                                           _ptr(gate), gm, float(sm_scale), window, B, S,
                                           T, H, HKV, DQK, DV, ATTN_ALGO[algo], _ptr(out),
                                           _stream(stream)))
    return out


# --------------------------------------------------------------------------- paged cache
def dsa_cache_row_bytes(fmt, kv_heads, dqk, dv) -> int:
    """Bytes of one token's row; fmt "bf16" or "e2m1" (4 bits)."""
    return int(lib().dsa_cache_row_bytes(CACHE_FORMAT[fmt], _int(kv_heads), _int(dqk), _int(dv)))


def dsa_cache_pages(fmt, n_pages, page_size, kv_heads, dqk, dv, device="cuda"):
    """Zeroed pages [n_pages, page_size, row]: bf16, or uint8 for the 4-bit format."""
    row = dsa_cache_row_bytes(fmt, kv_heads, dqk, dv)
    if row == 0:
        raise ValueError(f"no cache row for {fmt} kv_heads={kv_heads} dqk={dqk} dv={dv}")
    if fmt == "bf16":
        return torch.zeros((n_pages, page_size, row // 2), dtype=torch.bfloat16, device=device)
    return torch.zeros((n_pages, page_size, row), dtype=torch.uint8, device=device)


class Cache:
    """A paged key/value cache (include/dsa.h, section 5): pages [n_pages, page_size, row] (bf16
    rows, or uint8 rows held in 4 bits) and the page table [B, max_pages] int32.  Holds the
    tensors; the page table may be filled in place as sequences grow.  What it describes is fixed:
    other tensors, or these resized, take a new Cache."""

    def __init__(self, pages, table, kv_heads, dqk, dv, k_scale=1.0, v_scale=1.0):
        _cuda(pages, table)
        fmt = {torch.bfloat16: "bf16", torch.uint8: "e2m1"}.get(pages.dtype)
        if fmt is None:
            raise ValueError("pages are bf16, or uint8 for the 4-bit format")
        if table.dtype != torch.int32 or table.dim() != 2:
            raise ValueError("table is int32 [B, max_pages]")
        row = dsa_cache_row_bytes(fmt, kv_heads, dqk, dv)
        if pages.dim() != 3 or row == 0 or pages.shape[2] * pages.element_size() != row:
            raise ValueError(f"pages are [n_pages, page_size, row] with rows of {row} bytes for "
                             f"{fmt} kv_heads={kv_heads} dqk={dqk} dv={dv}")
        if table.device != pages.device:
            raise ValueError("pages and table are on different devices")
        self.pages, self.table, self.device = pages, table, pages.device
        self.kv_heads, self.dqk, self.dv = int(kv_heads), int(dqk), int(dv)
        self.args = CacheArgs(format=CACHE_FORMAT[fmt], n_pages=_int(pages.shape[0]),
                              page_size=_int(pages.shape[1]), max_pages=_int(table.shape[1]),
                              HKV=self.kv_heads, DQK=self.dqk, DV=self.dv,
                              k_scale=float(k_scale), v_scale=float(v_scale),
                              pages=pages.data_ptr(), table=table.data_ptr())
        self.ref = ctypes.byref(self.args)
        self._bf16 = torch.empty(0, dtype=torch.bfloat16, device=self.device)  # outputs' kind
        self._workspaces = {}  # workspace bytes by the sizes of a call
        self._pages_at, self._table_at = pages.data_ptr(), table.data_ptr()
        self._B, self._entries = table.shape[0], table.numel()
        self._device_index = self.device.index
        self._fixed = frozenset(self.__dict__)

    def __setattr__(self, name, value):
        # (the library reads its own copy, `args`: a new table here would not reach it)
        if name in self.__dict__.get("_fixed", ()):
            raise AttributeError(f"a Cache is not changed ({name}): make a new one")
        object.__setattr__(self, name, value)

    def _rows(self, pos):
        """(B, S) of a call with positions pos, which must suit the table and the current device."""
        shape, table = pos.shape, self.table
        if len(shape) != 2 or shape[0] != self._B:
            raise ValueError(f"pos is [B, S] with B = {self._B} (the table's rows)")
        if self.pages.data_ptr() != self._pages_at or table.data_ptr() != self._table_at or \
                table.numel() != self._entries:
            raise ValueError("the cache's tensors were moved or resized: make a new Cache")
        if self._device_index != torch.cuda.current_device():
            raise ValueError(f"the cache is on {self.device}, which is not the current device")
        self._takes("pos", pos, shape, torch.int32)
        return shape

    def _output(self, shape, stream):
        """A call's bf16 output (new_empty is the cheaper call, by 1 us)."""
        return self._bf16.new_empty(shape) if stream is None else \
            _own(shape, torch.bfloat16, self.device, stream)

    def _takes(self, name, t, shape, dtype=torch.bfloat16):
        """A call's tensor: contiguous, of this shape and type, on the cache's device; its address
        (None: not given)."""
        if t is None:
            return None
        if t.shape != shape or t.dtype != dtype or t.device != self.device or \
                not t.is_contiguous():
            raise ValueError(f"{name} is {tuple(t.shape)} {t.dtype} on {t.device}: expected a "
                             f"contiguous {tuple(shape)} {dtype} on {self.device}")
        return t.data_ptr()


def _raw_stream(stream, device):
    # (the handle alone: building a Stream object takes 2 us, a tenth of a decode call)
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def dsa_cache_append(cache, pos, k, v, rope="off", inv_freq=None, q=None, q_out=None, k_out=None,
                     stream=None):
    """Appends the tokens k [B,S,HKV,DQK], v [B,S,HKV,DV] at pos [B,S] (int32; negative: padding) to
    the cache, the last 2*len(inv_freq) dims of each key head rotated by pos * inv_freq (rope
    "interleaved": pairs (2j, 2j+1), or "half": pairs (j, j + len)), and rotates the same tokens'
    queries q [B,S,H,DQK] into q_out (may be q).  k_out, if given, receives the rotated keys (may be
    k).  Returns (rotated queries or None, k_out); with rope "off" q comes back as it is."""
    B, S = cache._rows(pos)
    takes = cache._takes
    ks = (B, S, cache.kv_heads, cache.dqk)
    kp, vp = takes("k", k, ks), takes("v", v, (B, S, cache.kv_heads, cache.dv))
    ko = takes("k_out", k_out, ks)
    H, qp, qo, fp, rot = cache.kv_heads, None, None, None, 0
    if rope == "off":
        if q_out is not None:
            raise ValueError("q_out goes with a rotation")
        q_out = q
    else:
        if inv_freq is None:
            raise ValueError("a rotation needs inv_freq")
        fp, rot = takes("inv_freq", inv_freq, (inv_freq.numel(),), torch.float32), inv_freq.numel()
        if q is not None:
            H = q.shape[2] if q.dim() == 4 else 0
            qs = (B, S, H, cache.dqk)
            qp = takes("q", q, qs)
            if q_out is None:
                q_out = cache._output(qs, stream)
            qo = takes("q_out", q_out, qs)
        elif q_out is not None:
            raise ValueError("q_out goes with q")
    _check(lib().dsa_cache_append(cache.ref, pos.data_ptr(), kp, vp, ROPE[rope], 2 * rot, fp, B, S,
                                  H, qp, qo, ko, _raw_stream(stream, cache.device)))
    return q_out, k_out


def dsa_cache_read(cache, pos, k=None, v=None, stream=None):
    """The tokens at pos [B,S] as the cache holds them: (k [B,S,HKV,DQK], v [B,S,HKV,DV]) in bf16,
    zeros where it has no row."""
    B, S = cache._rows(pos)
    ks, vs = (B, S, cache.kv_heads, cache.dqk), (B, S, cache.kv_heads, cache.dv)
    if k is None:
        k = cache._output(ks, stream)
    if v is None:
        v = cache._output(vs, stream)
    _check(lib().dsa_cache_read(cache.ref, pos.data_ptr(), B, S, cache._takes("k", k, ks),
                                cache._takes("v", v, vs), _raw_stream(stream, cache.device)))
    return k, v


def _cache_attn(q, cache, pos, idx, window, n_first, gate, gate_mode, sm_scale, out, ws, stream):
    B, S = cache._rows(pos)
    takes = cache._takes
    H = q.shape[2] if q.dim() == 4 else 0
    gm = GATE[gate_mode or ("sigmoid" if gate is not None else "off")]
    qp = takes("q", q, (B, S, H, cache.dqk))
    gp = takes("gate", gate, (B, S, H))
    if out is None:
        out = cache._output((B, S, H, cache.dv), stream)
        op = out.data_ptr()
    else:
        op = takes("out", out, (B, S, H, cache.dv))
    L, c = lib(), cache.ref
    window, n_first = _int(window), _int(n_first)
    K = None if idx is None else idx.shape[-1]
    ip = takes("idx", idx, (B, S, K), torch.int32)
    sizes = (B, S, H, K, window, n_first)  # (K None: the window form, which no K stands for)
    nbytes = cache._workspaces.get(sizes)
    if nbytes is None:
        nbytes = int(L.dsa_cache_attn_workspace_bytes(c, B, S, H, window, n_first)
                     if idx is None else L.dsa_cache_sparse_attn_workspace_bytes(c, B, S, H, K))
        cache._workspaces[sizes] = nbytes
    wp = None
    if nbytes:
        if ws is None:
            ws = _own(nbytes, torch.uint8, cache.device, stream, returned=False)
        elif not ws.is_contiguous() or ws.device != cache.device or \
                ws.numel() * ws.element_size() < nbytes:
            raise ValueError(f"ws is a contiguous tensor of at least {nbytes} bytes on "
                             f"{cache.device}")
        wp = ws.data_ptr()
    st = _raw_stream(stream, cache.device)
    if idx is None:
        _check(L.dsa_cache_attn(c, qp, pos.data_ptr(), window, n_first, gp, gm, float(sm_scale), B, S,
                                H, op, wp, nbytes, st))
    else:
        _check(L.dsa_cache_sparse_attn(c, qp, pos.data_ptr(), ip, K, gp, gm, float(sm_scale), B, S,
                                       H, op, wp, nbytes, st))
    return out


def dsa_cache_attn(q, cache, pos, window=0, n_first=0, gate=None, gate_mode=None, sm_scale=0.0,
                   out=None, ws=None, stream=None):
    """Attention of the tokens q [B,S,H,DQK] at pos [B,S] over the cache: every key t <= pos
    (window 0), or t > pos - window together with t < n_first.  From 64 tokens of a sequence on,
    dsa_cache_read of what they see and dsa_window_attn are faster."""
    return _cache_attn(q, cache, pos, None, window, n_first, gate, gate_mode, sm_scale, out, ws,
                       stream)


def dsa_cache_sparse_attn(q, cache, pos, idx, gate=None, gate_mode=None, sm_scale=0.0, out=None,
                          ws=None, stream=None):
    """Attention of the tokens q [B,S,H,DQK] at pos [B,S] over the selected keys idx [B,S,K] of the
    cache (int32, -1 padded, as dsa_topk and dsa_index_topk give them; those take one length for a
    batch, so sequences of different lengths are indexed one by one)."""
    return _cache_attn(q, cache, pos, idx, 0, 0, gate, gate_mode, sm_scale, out, ws, stream)
