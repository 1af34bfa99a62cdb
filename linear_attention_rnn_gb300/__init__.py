"""GB300 (sm_103a) chunked Gated DeltaNet -- Python binding of libgdn.

Beside the chunked rule (chunk_fwd, chunk_bwd, the layer and the segment calls) there
are the operators that a stack with other mixers and a decoding loop need:
delta_step, one token per row of the gated delta rule; decay_fwd, decay_bwd and
decay_step, linear attention with a decay for each head; attn_fwd and attn_bwd,
causal softmax attention with grouped heads, over packed sequences or caches.  Around
softmax attention: rope_fwd and rope_bwd, norms of query and key heads with the position
rotation; for serving from a paged cache rope_append, which writes the turned keys into
its pages, attn_paged, attn_paged_weights and cache_evict.

Thin marshalling over the C ABI in include/gdn.h: shape/dtype checks,
allocation of outputs and workspace with torch, and the ctypes call on the
current CUDA stream.  Every step of the computation runs in the library's
kernels; there is no fallback path.  If libgdn.so has not been built, the
first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional, Tuple

import torch

from . import inputs  # noqa: F401  (seeded input generator)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libgdn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "gdn.h")

GDN_OK = 0
STATUS = {0: "GDN_OK", -1: "GDN_ERR_ARG", -2: "GDN_ERR_SHAPE", -3: "GDN_ERR_WORKSPACE",
          -4: "GDN_ERR_CUDA", -5: "GDN_ERR_TIMEOUT", -6: "GDN_ERR_UNSUPPORTED"}

_lib = None
_several_devices = True  # whether operands can be on different ones; lib() finds out


class GDNError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = lib().gdn_strerror(code).decode() if _lib is not None else str(code)
        super().__init__(f"{where}: {STATUS.get(code, code)} ({msg})")
        self.code = code


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libgdn.so in-tree (nvcc, sm_103a)."""
    this = globals()["build"]
    from .build import build as _build
    globals()["build"] = this  # (importing the submodule of that name replaces it)
    return _build(force=force, verbose=verbose)


def header_functions():
    """Names of the functions include/gdn.h declares."""
    txt = open(HEADER).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(gdn_[a-z_0-9]+)\s*\(", txt)))


def lib():
    global _lib, _several_devices
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libgdn.so is not built ({LIB_PATH}); run linear_attention_rnn_gb300.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.gdn_strerror.argtypes = [I]
        L.gdn_strerror.restype = ctypes.c_char_p
        L.gdn_default_segments.argtypes = [I, I, I, I]
        L.gdn_default_segments.restype = I
        for name in ("gdn_fwd_workspace_bytes", "gdn_bwd_workspace_bytes"):
            f = getattr(L, name)
            f.argtypes = [I] * 8
            f.restype = Z
        L.gdn_chunk_fwd.argtypes = [P] * 8 + [I] * 8 + [P, Z, P]
        L.gdn_chunk_fwd.restype = I
        L.gdn_chunk_bwd.argtypes = [P] * 14 + [I] * 8 + [P, Z, P]
        L.gdn_chunk_bwd.restype = I
        L.gdn_chunk_fwd_timed.argtypes = [P] * 8 + [I] * 8 + [P, Z, P, P, I]
        L.gdn_chunk_fwd_timed.restype = I
        L.gdn_chunk_bwd_timed.argtypes = [P] * 14 + [I] * 8 + [P, Z, P, P, I]
        L.gdn_chunk_bwd_timed.restype = I
        L.gdn_saved_bytes.argtypes = [I] * 8
        L.gdn_saved_bytes.restype = Z
        L.gdn_chunk_fwd_ex.argtypes = [P] * 8 + [I] * 8 + [P, Z, P, Z, P, P, I]
        L.gdn_chunk_fwd_ex.restype = I
        L.gdn_chunk_bwd_ex.argtypes = [P] * 14 + [I] * 8 + [P, Z, P, Z, P, P, I]
        L.gdn_chunk_bwd_ex.restype = I
        L.gdn_affine_compose.argtypes = [P] * 4 + [I] * 4 + [P]
        L.gdn_affine_compose.restype = I
        L.gdn_debug_ut.argtypes = [P] * 8 + [I] * 7 + [P]
        L.gdn_debug_ut.restype = I
        L.gdn_workspace_status.argtypes = [P, P]
        L.gdn_workspace_status.restype = I
        L.gdn_layer_workspace_bytes.argtypes = [I] * 9
        L.gdn_layer_workspace_bytes.restype = Z
        L.gdn_layer_fwd.argtypes = [P] * 10 + [I] * 8 + [P, Z, P]
        L.gdn_layer_fwd.restype = I
        L.gdn_layer_bwd.argtypes = [P] * 17 + [I] * 8 + [P, Z, P]
        L.gdn_layer_bwd.restype = I
        L.gdn_segment_fold.argtypes = [P] * 6 + [I] * 8 + [P, Z, P]
        L.gdn_segment_fold.restype = I
        L.gdn_chunk_fwd_noalloc.argtypes = [P] * 8 + [I] * 7 + [P]
        L.gdn_chunk_fwd_noalloc.restype = I
        L.gdn_noalloc_status.argtypes = [P]
        L.gdn_noalloc_status.restype = I
        LL = ctypes.c_longlong
        L.gdn_delta_step.argtypes = [P] * 8 + [I] * 6 + [LL] * 3 + [P]
        L.gdn_delta_step.restype = I
        L.gdn_decay_step.argtypes = [P] * 7 + [I] * 6 + [LL] * 3 + [P]
        L.gdn_decay_step.restype = I
        L.gdn_decay_workspace_bytes.argtypes = [I] * 8
        L.gdn_decay_workspace_bytes.restype = Z
        L.gdn_decay_fwd.argtypes = [P] * 8 + [I] * 7 + [LL] * 3 + [P, Z, P]
        L.gdn_decay_fwd.restype = I
        L.gdn_decay_bwd.argtypes = [P] * 12 + [I] * 7 + [LL] * 3 + [P, Z, P]
        L.gdn_decay_bwd.restype = I
        L.gdn_attn_workspace_bytes.argtypes = [I] * 8
        L.gdn_attn_workspace_bytes.restype = Z
        L.gdn_attn_fwd.argtypes = [P] * 8 + [I] * 7 + [ctypes.c_float] + [LL] * 3 + [P, Z, P]
        L.gdn_attn_fwd.restype = I
        L.gdn_attn_bwd.argtypes = [P] * 11 + [I] * 6 + [ctypes.c_float] + [LL] * 3 + [P, Z, P]
        L.gdn_attn_bwd.restype = I
        F = ctypes.c_float
        L.gdn_rope_fwd.argtypes = [P] * 9 + [I] * 7 + [F] + [LL] * 4 + [P]
        L.gdn_rope_fwd.restype = I
        L.gdn_rope_workspace_bytes.argtypes = [I] * 4
        L.gdn_rope_workspace_bytes.restype = Z
        L.gdn_rope_bwd.argtypes = [P] * 13 + [I] * 7 + [F] + [LL] * 6 + [P, Z, P]
        L.gdn_rope_bwd.restype = I
        L.gdn_rope_append.argtypes = [P] * 12 + [I] * 9 + [F] + [LL] * 4 + [P] * 3
        L.gdn_rope_append.restype = I
        L.gdn_attn_paged_workspace_bytes.argtypes = [I] * 8
        L.gdn_attn_paged_workspace_bytes.restype = Z
        L.gdn_attn_paged.argtypes = [P] * 8 + [I] * 10 + [F, LL, P, P, LL, P, Z, P]
        L.gdn_attn_paged.restype = I
        L.gdn_attn_paged_weights.argtypes = [P] * 7 + [I] * 10 + [F, LL, P, LL, P, Z, P]
        L.gdn_attn_paged_weights.restype = I
        L.gdn_cache_evict_workspace_bytes.argtypes = [I] * 4
        L.gdn_cache_evict_workspace_bytes.restype = Z
        L.gdn_cache_evict.argtypes = [P] * 7 + [I] * 9 + [P, P, LL, LL, P, Z, P]
        L.gdn_cache_evict.restype = I
        L.gdn_selftest_wait_timeout.argtypes = [ctypes.c_longlong, P, P]
        L.gdn_selftest_wait_timeout.restype = I
        _several_devices = torch.cuda.device_count() > 1
        _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    """The raw handle of the device's current stream (without the Stream object
    that torch.cuda.current_stream builds, 2 us of a single-token call)."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check(t, name, dtype, shape=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dims(q, k, v, g, beta):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, D]")
    B, T, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    _check(q, "q", torch.bfloat16, (B, T, Hk, dk))
    _check(k, "k", torch.bfloat16)
    _check(v, "v", torch.bfloat16, (B, T, Hv, dv))
    _check(g, "g", torch.float32, (B, T, Hv))
    _check(beta, "beta", torch.float32, (B, T, Hv))
    return B, T, Hk, Hv, dk, dv


def default_segments(B: int, T: int, Hv: int, chunk: int = 128) -> int:
    return int(lib().gdn_default_segments(B, T, Hv, chunk))


def fwd_workspace_bytes(B, T, Hk, Hv, dk=128, dv=128, chunk=128, n_segments=0) -> int:
    return int(lib().gdn_fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, n_segments))


def bwd_workspace_bytes(B, T, Hk, Hv, dk=128, dv=128, chunk=128, n_segments=0) -> int:
    return int(lib().gdn_bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, n_segments))


def saved_bytes(B, T, Hk, Hv, dk=128, dv=128, chunk=128, n_segments=0) -> int:
    """Bytes of the buffer in which a forward keeps w, u, P and T (and, with
    segments, the segments' entering states) for its backward."""
    return int(lib().gdn_saved_bytes(B, T, Hk, Hv, dk, dv, chunk, n_segments))


def _events(events):
    """ctypes array of raw cudaEvent_t handles of torch.cuda.Event objects
    (each must have been recorded once, so that it exists)."""
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    return arr, len(events)


def _workspace(nbytes, device, ws):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        return ws
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


def chunk_fwd(q, k, v, g, beta, h0=None, *, chunk: int = 128, n_segments: int = 0,
              want_hT: bool = True, o=None, hT=None, workspace=None, events=None, saved=None
              ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Forward of the chunked gated delta rule.  Returns (o, hT).
    events: optional torch.cuda.Event list recorded after each kernel launch.
    saved: optional uint8 CUDA buffer of saved_bytes(...) bytes in which the
    forward keeps w, u, P and T for chunk_bwd(..., saved=the same buffer)."""
    B, T, Hk, Hv, dk, dv = _dims(q, k, v, g, beta)
    dev = q.device
    _check(h0, "h0", torch.float32, (B, Hv, dk, dv))
    if o is None:
        o = torch.empty((B, T, Hv, dv), dtype=torch.bfloat16, device=dev)
    _check(o, "o", torch.bfloat16, (B, T, Hv, dv))
    if want_hT and hT is None:
        hT = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev)
    nbytes = fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, n_segments)
    ws = _workspace(nbytes, dev, workspace)
    if saved is not None:
        ev = _events(events) if events else (None, 0)
        rc = lib().gdn_chunk_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                    _ptr(o), _ptr(hT), B, T, Hk, Hv, dk, dv, chunk, n_segments,
                                    _ptr(saved), saved.numel() * saved.element_size(), _ptr(ws),
                                    ws.numel(), _stream(dev), *ev)
        if rc != GDN_OK:
            raise GDNError(rc, "gdn_chunk_fwd_ex")
        return o, hT
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(o), _ptr(hT), B, T,
            Hk, Hv, dk, dv, chunk, n_segments, _ptr(ws), ws.numel(), _stream(dev)]
    if events:
        rc = lib().gdn_chunk_fwd_timed(*args, *_events(events))
    else:
        rc = lib().gdn_chunk_fwd(*args)
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_chunk_fwd")
    return o, hT


def chunk_bwd(q, k, v, g, beta, h0, dO, dhT=None, *, chunk: int = 128, n_segments: int = 0,
              want_dh0: bool = True, out=None, workspace=None, events=None, saved=None):
    """Backward of the chunked gated delta rule.
    Returns (dq, dk, dv, dg, dbeta, dh0).
    out: optional (dq, dk, dv, dg, dbeta, dh0) tensors to write (dh0 may be
    None), e.g. views of one buffer that leaves the device in one copy.
    events: optional torch.cuda.Event list recorded after each kernel launch."""
    B, T, Hk, Hv, dk, dv = _dims(q, k, v, g, beta)
    dev = q.device
    _check(h0, "h0", torch.float32, (B, Hv, dk, dv))
    _check(dO, "dO", torch.bfloat16, (B, T, Hv, dv))
    _check(dhT, "dhT", torch.float32, (B, Hv, dk, dv))
    if out is not None:
        dq, dk_, dv_, dg, db, dh0 = out
        _check(dq, "dq", torch.bfloat16, tuple(q.shape))
        _check(dk_, "dk", torch.bfloat16, tuple(k.shape))
        _check(dv_, "dv", torch.bfloat16, tuple(v.shape))
        _check(dg, "dg", torch.float32, tuple(g.shape))
        _check(db, "dbeta", torch.float32, tuple(beta.shape))
        _check(dh0, "dh0", torch.float32, (B, Hv, dk, dv))
    else:
        dq = torch.empty_like(q)
        dk_ = torch.empty_like(k)
        dv_ = torch.empty_like(v)
        dg = torch.empty_like(g)
        db = torch.empty_like(beta)
        dh0 = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    nbytes = bwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, n_segments)
    ws = _workspace(nbytes, dev, workspace)
    if saved is not None:  # w, u, P, T kept by chunk_fwd(..., saved=saved) on these inputs
        ev = _events(events) if events else (None, 0)
        rc = lib().gdn_chunk_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0),
                                    _ptr(dO), _ptr(dhT), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg),
                                    _ptr(db), _ptr(dh0), B, T, Hk, Hv, dk, dv, chunk, n_segments,
                                    _ptr(saved), saved.numel() * saved.element_size(), _ptr(ws),
                                    ws.numel(), _stream(dev), *ev)
        if rc != GDN_OK:
            raise GDNError(rc, "gdn_chunk_bwd_ex")
        return dq, dk_, dv_, dg, db, dh0
    args = [_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(h0), _ptr(dO), _ptr(dhT),
            _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dg), _ptr(db), _ptr(dh0), B, T, Hk, Hv, dk, dv,
            chunk, n_segments, _ptr(ws), ws.numel(), _stream(dev)]
    if events:
        rc = lib().gdn_chunk_bwd_timed(*args, *_events(events))
    else:
        rc = lib().gdn_chunk_bwd(*args)
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_chunk_bwd")
    return dq, dk_, dv_, dg, db, dh0


def layer_workspace_bytes(backward, B, T, Hk, Hv, dk=128, dv=128, chunk=128, n_segments=0) -> int:
    return int(lib().gdn_layer_workspace_bytes(int(backward), B, T, Hk, Hv, dk, dv, chunk,
                                               n_segments))


def layer_fwd(q, k, v, a, b, z=None, h0=None, *, chunk: int = 128, n_segments: int = 0,
              keep_o: bool = True, want_hT: bool = True, workspace=None):
    """Layer forward: q, k raw (normalised inside), a, b gate logits
    (g = -softplus(a), beta = sigmoid(b)), optional output gate z.
    Returns (y, o, hT): o is the ungated output (None unless keep_o and z)."""
    B, T, Hk, Hv, dk, dv = _dims(q, k, v, a, b)
    dev = q.device
    _check(z, "z", torch.bfloat16, (B, T, Hv, dv))
    _check(h0, "h0", torch.float32, (B, Hv, dk, dv))
    y = torch.empty((B, T, Hv, dv), dtype=torch.bfloat16, device=dev)
    o = torch.empty_like(y) if (keep_o and z is not None) else None
    hT = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev) if want_hT else None
    ws = _workspace(layer_workspace_bytes(0, B, T, Hk, Hv, dk, dv, chunk, n_segments), dev,
                    workspace)
    rc = lib().gdn_layer_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(z), _ptr(h0),
                             _ptr(y), _ptr(o), _ptr(hT), B, T, Hk, Hv, dk, dv, chunk, n_segments,
                             _ptr(ws), ws.numel(), _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_layer_fwd")
    return y, o, hT


def layer_bwd(q, k, v, a, b, z, h0, o, dy, dhT=None, *, chunk: int = 128, n_segments: int = 0,
              want_dh0: bool = True, workspace=None):
    """Layer backward.  Returns (dq, dk, dv, da, db, dz, dh0) for the raw q, k
    and the gate logits; dz is None without a gate."""
    B, T, Hk, Hv, dk, dv = _dims(q, k, v, a, b)
    dev = q.device
    _check(z, "z", torch.bfloat16, (B, T, Hv, dv))
    _check(o, "o", torch.bfloat16, (B, T, Hv, dv))
    _check(dy, "dy", torch.bfloat16, (B, T, Hv, dv))
    _check(h0, "h0", torch.float32, (B, Hv, dk, dv))
    _check(dhT, "dhT", torch.float32, (B, Hv, dk, dv))
    dq, dk_, dv_ = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    da, db = torch.empty_like(a), torch.empty_like(b)
    dz = torch.empty_like(z) if z is not None else None
    dh0 = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    ws = _workspace(layer_workspace_bytes(1, B, T, Hk, Hv, dk, dv, chunk, n_segments), dev,
                    workspace)
    rc = lib().gdn_layer_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(z), _ptr(h0),
                             _ptr(o), _ptr(dy), _ptr(dhT), _ptr(dq), _ptr(dk_), _ptr(dv_),
                             _ptr(da), _ptr(db), _ptr(dz), _ptr(dh0), B, T, Hk, Hv, dk, dv, chunk,
                             n_segments, _ptr(ws), ws.numel(), _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_layer_bwd")
    return dq, dk_, dv_, da, db, dz, dh0


def affine_compose(A: torch.Tensor, Bm: torch.Tensor):
    """Inclusive prefix of affine maps along dim 1: A [batch, n, dk, dk],
    B [batch, n, dk, dv] (fp32)."""
    batch, n, dk, _ = A.shape
    dv = Bm.shape[3]
    _check(A, "A", torch.float32, (batch, n, dk, dk))
    _check(Bm, "B", torch.float32, (batch, n, dk, dv))
    Ao = torch.empty_like(A)
    Bo = torch.empty_like(Bm)
    rc = lib().gdn_affine_compose(_ptr(A), _ptr(Bm), _ptr(Ao), _ptr(Bo), batch, n, dk, dv,
                                  _stream(A.device))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_affine_compose")
    return Ao, Bo


def segment_fold(k, v, g, beta, n_segments: int = 1, *, chunk: int = 128, want_A: bool = True,
                 workspace=None):
    """Per-segment affine maps (A_s, B_s) of the inter-chunk recurrence:
    A [B, Hv, S, dk, dk] (None if want_A is False) and B [B, Hv, S, dk, dv],
    fp32, with the state leaving segment s equal to A_s h_in + B_s."""
    B, T, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    _check(k, "k", torch.bfloat16)
    _check(v, "v", torch.bfloat16, (B, T, Hv, dv))
    _check(g, "g", torch.float32, (B, T, Hv))
    _check(beta, "beta", torch.float32, (B, T, Hv))
    dev = k.device
    A = (torch.empty((B, Hv, n_segments, dk, dk), dtype=torch.float32, device=dev)
         if want_A else None)
    Bm = torch.empty((B, Hv, n_segments, dk, dv), dtype=torch.float32, device=dev)
    nbytes = fwd_workspace_bytes(B, T, Hk, Hv, dk, dv, chunk, 1)
    ws = _workspace(nbytes, dev, workspace)
    rc = lib().gdn_segment_fold(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(A), _ptr(Bm), B, T,
                                Hk, Hv, dk, dv, chunk, n_segments, _ptr(ws), ws.numel(),
                                _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_segment_fold")
    return A, Bm


def _check_rows(t, name, H, d, n=None):
    """bf16 rows [.., H, d] whose heads and columns are contiguous; the tokens may
    be further apart (a part of a wider buffer).  Returns the elements between
    tokens."""
    if t.dtype is torch.bfloat16 and t.is_cuda and t.is_contiguous() and t.shape == (n, H, d):
        return H * d  # (the usual case, at a third of what the checks below take)
    if t.dtype is torch.bfloat16 and t.is_cuda and t.dim() == 3 and t.shape == (n, H, d) and H > 1 < n:
        st = t.stride()  # (a part of a wider buffer, likewise)
        if st[2] == 1 and st[1] == d and st[0] >= H * d and not st[0] % 8:
            return st[0]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() < 3 or tuple(t.shape[-2:]) != (H, d) or (n is not None and t.numel() != n * H * d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"{'' if n is None else str(n) + ' '}rows of ({H}, {d})")
    if t.numel() == 0:
        return H * d
    if t.stride(-1) != 1 or (H > 1 and t.stride(-2) != d):
        raise ValueError(f"{name} must have contiguous heads and columns")
    # the row dimensions as one: each is the next one's whole extent
    shape, strides = [], []
    for n_i, s_i in zip(t.shape[:-2], t.stride()[:-2]):
        if n_i > 1:
            shape.append(n_i)
            strides.append(s_i)
    for i in range(len(shape) - 1):
        if strides[i] != shape[i + 1] * strides[i + 1]:
            raise ValueError(f"{name} must have rows a constant stride apart")
    stride = strides[-1] if strides else H * d
    if stride < H * d or stride % 8:
        raise ValueError(f"{name} must have rows at least {H * d} elements apart, by a multiple of 8")
    return stride


def _check_devices(q, *operands):
    """All operands on q's device, which is the current one (a kernel is launched there).
    For machines with several devices; with one it would only take time."""
    for t in operands:
        if t is not None and t.device != q.device:
            raise ValueError(f"operands are on {q.device} and {t.device}")
    if torch.cuda.current_device() != q.device.index:
        raise ValueError(f"operands are on {q.device}, which is not the current device")


def _current_device() -> int:
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -1


@functools.lru_cache(maxsize=512)
def _planned_bytes(name, device, *sizes) -> int:
    """A workspace's size by the library's plan, which counts the current device's SMs."""
    return int(getattr(lib(), name)(*sizes))


_STATUS_BYTES = 256  # a workspace that holds the status word alone may be left out


def _scratch(nbytes, device, ws):
    """(pointer, bytes) of the caller's workspace, or of one allocated here."""
    if ws is None:
        if nbytes <= _STATUS_BYTES:
            return None, 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    elif not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError("workspace must be a contiguous CUDA tensor")
    elif ws.numel() * ws.element_size() < nbytes:
        raise ValueError("workspace too small")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _step(name, q, k, v, gates, state, slots, o):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [R, H, D]")
    R, Hk, dk = k.shape
    _, Hv, dv = v.shape
    sq = _check_rows(q, "q", Hk, dk, R)
    sk = _check_rows(k, "k", Hk, dk, R)
    sv = _check_rows(v, "v", Hv, dv, R)
    if state.dim() != 4:
        raise ValueError("state must be [slots, Hv, d_k, d_v]")
    n = state.shape[0]
    _check(state, "state", torch.float32, (n, Hv, dk, dv))
    if slots is not None:
        _check(slots, "slots", torch.int32, (R,))
    elif n < R:
        raise ValueError(f"{R} rows need as many states, got {n}")
    if o is None:
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
    else:
        _check(o, "o", torch.bfloat16, (R, Hv, dv))
    if _several_devices:
        _check_devices(q, k, v, state, slots, o)
    rc = name(q.data_ptr(), k.data_ptr(), v.data_ptr(), *gates,
              state.data_ptr(), _ptr(slots), o.data_ptr(), R, n, Hk, Hv, dk, dv, sq, sk, sv,
              torch._C._cuda_getCurrentRawStream(q.device.index))
    if rc != GDN_OK:
        raise GDNError(rc, name.__name__)
    return o


def delta_step(q, k, v, g, beta, state, slots=None, *, o=None) -> torch.Tensor:
    """One token per row of the gated delta rule: q, k [R, Hk, 128], v [R, Hv, 128]
    (bf16), g, beta [R, Hv]; state [n, Hv, 128, 128] (fp32) is updated in place.
    slots: int32 [R], the state of each row (None: row r's state is r); a
    negative slot is a padded row, whose output is zero.  Returns o [R, Hv, 128]."""
    rows = v.shape[:2]
    _check(g, "g", torch.float32, rows)
    _check(beta, "beta", torch.float32, rows)
    if _several_devices:
        _check_devices(q, g, beta)
    return _step(lib().gdn_delta_step, q, k, v, (g.data_ptr(), beta.data_ptr()), state, slots, o)


def decay_step(q, k, v, decay, state, slots=None, *, o=None) -> torch.Tensor:
    """One token per row of linear attention with a decay for each head (decay
    [Hv], the log-decays); otherwise as delta_step."""
    _check(decay, "decay", torch.float32, v.shape[1:2])
    if _several_devices:
        _check_devices(q, decay)
    return _step(lib().gdn_decay_step, q, k, v, (decay.data_ptr(),), state, slots, o)


def decay_workspace_bytes(backward, n_seqs, total, max_seqlen, Hk, Hv, dk=128, dv=128) -> int:
    return _planned_bytes("gdn_decay_workspace_bytes", _current_device(), int(backward), n_seqs,
                          total, max_seqlen, Hk, Hv, dk, dv)


def _decay_dims(q, k, v, decay, cu_seqlens, max_seqlen):
    """Packed [total, H, D] with cu_seqlens, or [B, T, H, D] without."""
    if cu_seqlens is not None:
        if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
            raise ValueError("q, k, v must be [total, H, D] with cu_seqlens")
        _check(cu_seqlens, "cu_seqlens", torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must hold the sequences' starts and the total")
        n, total = cu_seqlens.numel() - 1, k.shape[0]
        longest = total if max_seqlen is None else int(max_seqlen)
    else:
        if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
            raise ValueError("q, k, v must be [B, T, H, D] without cu_seqlens")
        n, longest = k.shape[:2]
        total = n * longest
    Hk, dk = k.shape[-2:]
    Hv, dv = v.shape[-2:]
    if q.shape != k.shape or v.shape[:-2] != k.shape[:-2]:
        raise ValueError(f"q, k, v have shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    strides = [_check_rows(q, "q", Hk, dk, total), _check_rows(k, "k", Hk, dk, total),
               _check_rows(v, "v", Hv, dv, total)]
    _check(decay, "decay", torch.float32, (Hv,))
    return n, total, longest, Hk, Hv, dk, dv, strides


def decay_fwd(q, k, v, decay, h0=None, *, cu_seqlens=None, max_seqlen=None, want_hT: bool = True,
              o=None, hT=None, workspace=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Linear attention with a decay for each head (decay [Hv], the log-decays,
    <= 0): S_t = exp(decay) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.  q, k, v are
    [B, T, H, 128], or with cu_seqlens (int32, on the device) packed sequences
    [total, H, 128]; max_seqlen then bounds the longest one (it only steers how
    the work is split).  h0 [n, Hv, 128, 128].  hT may be h0 itself, the states then
    being replaced; otherwise outputs must not overlap inputs.  Returns (o, hT)."""
    n, total, longest, Hk, Hv, dk, dv, strides = _decay_dims(q, k, v, decay, cu_seqlens, max_seqlen)
    dev = q.device
    _check(h0, "h0", torch.float32, (n, Hv, dk, dv))
    if o is None:
        o = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check(o, "o", torch.bfloat16, v.shape)
    if hT is not None:
        _check(hT, "hT", torch.float32, (n, Hv, dk, dv))
    elif want_hT:
        hT = torch.empty((n, Hv, dk, dv), dtype=torch.float32, device=dev)
    if _several_devices:
        _check_devices(q, k, v, decay, h0, cu_seqlens, o, hT, workspace)
    wp, wn, ws = _scratch(_planned_bytes("gdn_decay_workspace_bytes", dev.index, 0, n, total, longest,
                                         Hk, Hv, dk, dv), dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_decay_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(h0), _ptr(cu_seqlens),
                             _ptr(o), _ptr(hT), n, total, longest, Hk, Hv, dk, dv, *strides,
                             wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_decay_fwd")
    return o, hT


def decay_bwd(q, k, v, decay, h0, dO, dhT=None, *, cu_seqlens=None, max_seqlen=None,
              want_dh0: bool = True, workspace=None):
    """Backward of decay_fwd.  Returns (dq, dk, dv, dh0); dq and dk are summed over
    the value heads that share a key head."""
    n, total, longest, Hk, Hv, dk, dv, strides = _decay_dims(q, k, v, decay, cu_seqlens, max_seqlen)
    dev = q.device
    _check(h0, "h0", torch.float32, (n, Hv, dk, dv))
    _check(dO, "dO", torch.bfloat16, tuple(v.shape))
    _check(dhT, "dhT", torch.float32, (n, Hv, dk, dv))
    dq = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    dk_ = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    dv_ = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    dh0 = torch.empty((n, Hv, dk, dv), dtype=torch.float32, device=dev) if want_dh0 else None
    if _several_devices:
        _check_devices(q, k, v, decay, h0, dO, dhT, cu_seqlens, workspace)
    wp, wn, ws = _scratch(_planned_bytes("gdn_decay_workspace_bytes", dev.index, 1, n, total, longest,
                                         Hk, Hv, dk, dv), dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_decay_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(decay), _ptr(h0), _ptr(dO), _ptr(dhT),
                             _ptr(cu_seqlens), _ptr(dq), _ptr(dk_), _ptr(dv_), _ptr(dh0), n, total,
                             longest, Hk, Hv, dk, dv, *strides, wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_decay_bwd")
    return dq, dk_, dv_, dh0


def attn_workspace_bytes(backward, n_seqs, total_q, total_k, max_k, Hq, Hk, d=128) -> int:
    return _planned_bytes("gdn_attn_workspace_bytes", _current_device(), int(backward), n_seqs,
                          total_q, total_k, max_k, Hq, Hk, d)


def _attn_dims(q, k, v, cu_q, cu_k, scale):
    """Packed [total, H, D] with cu_q and cu_k, or [B, T, H, D] without."""
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k go together")
    dims = 4 if cu_q is None else 3
    if q.dim() != dims or k.dim() != dims or v.dim() != dims:
        raise ValueError("q, k, v must be [B, T, H, D], or [total, H, D] with cu_q and cu_k")
    if cu_q is not None:
        for name, t in (("cu_q", cu_q), ("cu_k", cu_k)):
            _check(t, name, torch.int32)
        if cu_q.dim() != 1 or cu_q.numel() < 1 or cu_q.shape != cu_k.shape:
            raise ValueError("cu_q and cu_k must hold as many starts and the total")
        n, total_q, total_k = cu_q.numel() - 1, q.shape[0], k.shape[0]
    else:
        if q.shape[0] != k.shape[0]:
            raise ValueError(f"q has {q.shape[0]} sequences, k {k.shape[0]}")
        n, total_q, total_k = q.shape[0], q.shape[0] * q.shape[1], k.shape[0] * k.shape[1]
    Hq, d = q.shape[-2:]
    Hk = k.shape[-2]
    if v.shape != k.shape or k.shape[-1] != d:
        raise ValueError(f"q, k, v have shapes {tuple(q.shape)}, {tuple(k.shape)}, {tuple(v.shape)}")
    strides = [_check_rows(q, "q", Hq, d, total_q), _check_rows(k, "k", Hk, d, total_k),
               _check_rows(v, "v", Hk, d, total_k)]
    return n, total_q, total_k, Hq, Hk, d, d ** -0.5 if scale is None else float(scale), strides


def attn_fwd(q, k, v, *, cu_q=None, cu_k=None, k_len=None, max_q=None, max_k=None, scale=None,
             want_lse: bool = True, o=None, lse=None, workspace=None
             ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Causal softmax attention with grouped heads: q [total_q, Hq, 128], k, v
    [total_k, Hk, 128] hold packed sequences that start at cu_q and cu_k (int32,
    on the device), or are [B, T, H, 128] without them.  The last query of a
    sequence sees all of its keys, each one before it one key fewer; k_len
    (int32) gives the used rows of caches with a fixed capacity.  max_k bounds the
    keys of a sequence and steers how they are split over the SMs (packed keys without
    it are split as if one sequence had all of them); max_q is accepted beside it and
    changes nothing.  scale defaults to 1 / sqrt(128).  Returns (o, lse), lse [.., Hq]
    in fp32."""
    n, total_q, total_k, Hq, Hk, d, scale, strides = _attn_dims(q, k, v, cu_q, cu_k, scale)
    dev = q.device
    _check(k_len, "k_len", torch.int32, (n,))
    longest = int(max_k) if max_k is not None else (k.shape[1] if cu_k is None else total_k)
    if o is None:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _check(lse, "lse", torch.float32, q.shape[:-1])
    elif want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    if _several_devices:
        _check_devices(q, k, v, cu_q, cu_k, k_len, o, lse, workspace)
    wp, wn, ws = _scratch(_planned_bytes("gdn_attn_workspace_bytes", dev.index, 0, n, total_q, total_k,
                                         longest, Hq, Hk, d), dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(k_len), _ptr(o),
                            _ptr(lse), n, total_q, total_k, longest, Hq, Hk, d, scale, *strides,
                            wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_attn_fwd")
    return o, lse


def attn_bwd(q, k, v, o, lse, dO, *, cu_q=None, cu_k=None, max_q=None, max_k=None, scale=None,
             workspace=None):
    """Backward of attn_fwd (without k_len).  Returns (dq, dk, dv); dk and dv are
    summed over the query heads that share a key head.  max_q and max_k are accepted
    as there and change nothing."""
    n, total_q, total_k, Hq, Hk, d, scale, strides = _attn_dims(q, k, v, cu_q, cu_k, scale)
    dev = q.device
    _check(o, "o", torch.bfloat16, tuple(q.shape))
    _check(dO, "dO", torch.bfloat16, tuple(q.shape))
    _check(lse, "lse", torch.float32, tuple(q.shape[:-1]))
    dq = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    dk = torch.empty(k.shape, dtype=torch.bfloat16, device=dev)
    dv = torch.empty(v.shape, dtype=torch.bfloat16, device=dev)
    if _several_devices:
        _check_devices(q, k, v, o, lse, dO, cu_q, cu_k, workspace)
    wp, wn, ws = _scratch(_planned_bytes("gdn_attn_workspace_bytes", dev.index, 1, n, total_q, total_k, 0,
                                         Hq, Hk, d), dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(cu_q),
                            _ptr(cu_k), _ptr(dq), _ptr(dk), _ptr(dv), n, total_q, total_k, Hq, Hk, d,
                            scale, *strides, wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_attn_bwd")
    return dq, dk, dv


def _scratch_all(nbytes, device, ws):
    """As _scratch, for workspaces without a status word: none is made where none is needed."""
    if ws is None and nbytes:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return _scratch(nbytes, device, ws)


# ---- heads' norms and rotation, and the paged cache that they feed -----------------------
class _PageStrides(ctypes.Structure):
    _fields_ = [("page", ctypes.c_longlong), ("row", ctypes.c_longlong), ("head", ctypes.c_longlong)]


@functools.lru_cache(maxsize=256)
def _page_layout(shape, strides):
    """The C struct of a cache's strides (a dimension of one element has any)."""
    st = [max(shape[3], 8) if n <= 1 else s for n, s in zip(shape[:3], strides[:3])]
    return _PageStrides(st[0], st[1], st[2])


def _check_pages(t, name, Hk=None, like=None, d=None):
    """A cache [pages, page_size, Hk, d] in bf16 whose rows of d values are contiguous and
    lie multiples of 8 elements apart; returns its strides as the C struct."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 4 or (Hk is not None and t.shape[2] != Hk):
        raise ValueError(f"{name} must be [pages, page_size, {'Hk' if Hk is None else Hk}, d], got {tuple(t.shape)}")
    if like is not None and t.shape != like.shape:
        raise ValueError(f"k_pages and v_pages have shapes {tuple(like.shape)} and {tuple(t.shape)}")
    if d is not None and t.shape[3] != d:
        raise ValueError(f"{name} has heads of {t.shape[3]}, expected {d}")
    d = t.shape[3]
    strides = t.stride()
    if t.numel():
        if strides[3] != 1:
            raise ValueError(f"{name} must have contiguous rows")
        for n, s in zip(t.shape[:3], strides[:3]):
            if n > 1 and (s < d or s % 8):
                raise ValueError(f"{name} must have rows at least {d} elements apart, by multiples of 8")
        return _page_layout(t.shape, strides)
    return _page_layout(t.shape, (d, d, d, 1))


def _check_table(t, name, n):
    """int32 [n, pages] whose rows are contiguous; returns (pages, entries between rows)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype is not torch.int32:
        raise ValueError(f"{name} must be {torch.int32}, got {t.dtype}")
    if t.dim() != 2 or t.shape[0] != n:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected ({n}, pages)")
    m = t.shape[1]
    if t.numel() and ((m > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < m)):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return m, (t.stride(0) if t.numel() and n > 1 else m)


@functools.lru_cache(maxsize=64)
def _pair_axes(pair_axis, n_pairs):
    if len(pair_axis) != n_pairs or not all(0 <= a < 256 for a in pair_axis):
        raise ValueError(f"pair_axis must name an axis for each of the {n_pairs} pairs")
    return bytes(pair_axis)


def _rope_dims(q, k, positions, inv_freq, q_weight, k_weight, pair_axis):
    """Rows [n, H, d] or [B, T, H, d]; returns the sizes and the row strides of q and k."""
    qs, ks = q.shape, k.shape
    rows = qs[:-2]
    if len(qs) < 3 or rows != ks[:-2] or qs[-1] != ks[-1]:
        raise ValueError(f"q and k must be [.., H, d] with equal rows, got {tuple(qs)} and {tuple(ks)}")
    Hq, d = qs[-2:]
    Hk = ks[-2]
    n = qs[0] if len(qs) == 3 else rows.numel()
    sq, sk = _check_rows(q, "q", Hq, d, n), _check_rows(k, "k", Hk, d, n)
    if q_weight is not None:
        _check(q_weight, "q_weight", torch.float32, (d,))
    if k_weight is not None:
        _check(k_weight, "k_weight", torch.float32, (d,))
    axes, pairs, table = 1, 0, None
    if inv_freq is not None:
        _check(inv_freq, "inv_freq", torch.float32)
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must hold a frequency for each pair")
        pairs = inv_freq.shape[0]
        if positions is None:
            raise ValueError("inv_freq needs positions")
        _check(positions, "positions", torch.int32)
        if positions.shape != rows:
            if positions.dim() != len(rows) + 1 or positions.shape[1:] != rows or positions.shape[0] < 1:
                raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {tuple(rows)} "
                                 f"or an axis more in front")
            axes = positions.shape[0]
    if pair_axis is not None:
        table = _pair_axes(pair_axis if pair_axis.__class__ is tuple else tuple(int(x) for x in pair_axis), pairs)
    return n, Hq, Hk, d, axes, pairs, table, sq, sk


def _rows_out(t, name, like, n, H, d):
    """An output's rows: contiguous ones made here, or the caller's (a part of a wider buffer)."""
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format), H * d
    if t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    return t, _check_rows(t, name, H, d, n)


def rope_fwd(q, k, positions, inv_freq, *, q_weight=None, k_weight=None, eps: float = 1e-6, pair_axis=None,
             interleaved: bool = False, q_out=None, k_out=None):
    """Norms of query and key heads with the position rotation in the same pass: every head
    x of q [.., Hq, 128] and k [.., Hk, 128] becomes x w / sqrt(mean(x^2) + eps) (without
    its weight, fp32 [128], it stays x), then each of its first P pairs turns by
    positions[pair_axis[j]] * inv_freq[j].  inv_freq: fp32 [P], P a multiple of 8 up to 64
    (None: no rotation); positions: int32, the rows' shape, or [axes, ..] with pair_axis, a
    sequence of P axis numbers (time, height, width).  Pair j is (j, j + P), or
    (2j, 2j + 1) if interleaved.  q_out and k_out may be q and k.  Returns (q_out, k_out)."""
    n, Hq, Hk, d, axes, pairs, table, sq, sk = _rope_dims(q, k, positions, inv_freq, q_weight, k_weight, pair_axis)
    q_out, so = _rows_out(q_out, "q_out", q, n, Hq, d)
    k_out, sko = _rows_out(k_out, "k_out", k, n, Hk, d)
    if _several_devices:
        _check_devices(q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    rc = lib().gdn_rope_fwd(q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
                            _ptr(inv_freq), table, q_out.data_ptr(), k_out.data_ptr(), n, Hq, Hk, d, axes, pairs,
                            interleaved, eps, sq, sk, so, sko, _stream(q.device))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_rope_fwd")
    return q_out, k_out


def rope_workspace_bytes(n, Hq, Hk, d=128) -> int:
    return _planned_bytes("gdn_rope_workspace_bytes", _current_device(), n, Hq, Hk, d)


def rope_bwd(q, k, positions, inv_freq, dq_out, dk_out, *, q_weight=None, k_weight=None, eps: float = 1e-6,
             pair_axis=None, interleaved: bool = False, dq=None, dk=None, workspace=None):
    """Backward of rope_fwd: q and k are its inputs, dq_out and dk_out the cotangents of its
    outputs (dq may be dq_out, dk may be dk_out).  Returns (dq, dk, dq_weight, dk_weight), the
    last two in fp32 (None without the weight)."""
    n, Hq, Hk, d, axes, pairs, table, sq, sk = _rope_dims(q, k, positions, inv_freq, q_weight, k_weight, pair_axis)
    if dq_out.shape != q.shape or dk_out.shape != k.shape:
        raise ValueError(f"dq_out and dk_out have shapes {tuple(dq_out.shape)} and {tuple(dk_out.shape)}, expected "
                         f"{tuple(q.shape)} and {tuple(k.shape)}")
    sg, sgk = _check_rows(dq_out, "dq_out", Hq, d, n), _check_rows(dk_out, "dk_out", Hk, d, n)
    dq, so = _rows_out(dq, "dq", q, n, Hq, d)
    dk, sko = _rows_out(dk, "dk", k, n, Hk, d)
    dev = q.device
    dqw = torch.empty(d, dtype=torch.float32, device=dev) if q_weight is not None else None
    dkw = torch.empty(d, dtype=torch.float32, device=dev) if k_weight is not None else None
    if _several_devices:
        _check_devices(q, k, positions, inv_freq, q_weight, k_weight, dq_out, dk_out, dq, dk, workspace)
    need = 0 if dqw is None and dkw is None else _planned_bytes("gdn_rope_workspace_bytes", dev.index, n, Hq, Hk, d)
    wp, wn, ws = _scratch_all(need, dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_rope_bwd(q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
                            _ptr(inv_freq), table, dq_out.data_ptr(), dk_out.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                            _ptr(dqw), _ptr(dkw), n, Hq, Hk, d, axes, pairs, interleaved, eps, sq, sk, sg, sgk, so, sko,
                            wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_rope_bwd")
    return dq, dk, dqw, dkw


def rope_append(q, k, v, positions, inv_freq, k_pages, v_pages, slots, *, q_weight=None, k_weight=None,
                eps: float = 1e-6, pair_axis=None, interleaved: bool = False, q_out=None) -> torch.Tensor:
    """rope_fwd of new tokens whose keys, and values v [.., Hk, 128] as they are, go into a
    cache: k_pages and v_pages [pages, page_size, Hk, 128] (any strides that are multiples of
    8; page_size a multiple of 16).  slots: int32, the rows' shape; token t goes to page
    slots[t] // page_size, row slots[t] % page_size, and nowhere if that is outside the cache (a
    padded token).  Returns q_out."""
    n, Hq, Hk, d, axes, pairs, table, sq, sk = _rope_dims(q, k, positions, inv_freq, q_weight, k_weight, pair_axis)
    if v.shape != k.shape:
        raise ValueError(f"k and v have shapes {tuple(k.shape)} and {tuple(v.shape)}")
    sv = _check_rows(v, "v", Hk, d, n)
    ks = _check_pages(k_pages, "k_pages", Hk, d=d)
    vs = _check_pages(v_pages, "v_pages", Hk, k_pages)
    _check(slots, "slots", torch.int32, q.shape[:-2])
    q_out, so = _rows_out(q_out, "q_out", q, n, Hq, d)
    if _several_devices:
        _check_devices(q, k, v, positions, inv_freq, q_weight, k_weight, k_pages, v_pages, slots, q_out)
    rc = lib().gdn_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(q_weight), _ptr(k_weight),
                               _ptr(positions), _ptr(inv_freq), table, q_out.data_ptr(), k_pages.data_ptr(),
                               v_pages.data_ptr(), slots.data_ptr(), n, k_pages.shape[0], k_pages.shape[1], Hq, Hk, d,
                               axes, pairs, interleaved, eps, sq, sk, sv, so, ctypes.byref(ks), ctypes.byref(vs),
                               _stream(q.device))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_rope_append")
    return q_out


def _paged_dims(q, k_pages, page_table, k_len, cu_q, max_k, scale):
    """New tokens packed [total, H, D] with cu_q, or [B, T, H, D] without, over pages."""
    if q.dim() != (4 if cu_q is None else 3):
        raise ValueError("q must be [B, T, H, D], or [total, H, D] with cu_q")
    if cu_q is not None:
        _check(cu_q, "cu_q", torch.int32)
        if cu_q.dim() != 1 or cu_q.numel() < 1:
            raise ValueError("cu_q must hold the sequences' starts and the total")
        n, total = cu_q.numel() - 1, q.shape[0]
    else:
        n, total = q.shape[0], q.shape[0] * q.shape[1]
    Hq, d = q.shape[-2:]
    sq = _check_rows(q, "q", Hq, d, total)
    ks = _check_pages(k_pages, "k_pages", d=d)
    P, page, Hk = k_pages.shape[:3]
    pages, st = _check_table(page_table, "page_table", n)
    _check(k_len, "k_len", torch.int32, (n,))
    if k_len is None:
        raise ValueError("k_len must give the used rows of every sequence")
    longest = pages * page if max_k is None else int(max_k)
    return n, total, longest, P, page, pages, Hq, Hk, d, d ** -0.5 if scale is None else float(scale), sq, ks, st


def attn_paged_workspace_bytes(n_seqs, total_q, max_rows, max_q, max_k, Hq, Hk, d=128) -> int:
    return _planned_bytes("gdn_attn_paged_workspace_bytes", _current_device(), n_seqs, total_q, max_rows, max_q, max_k,
                          Hq, Hk, d)


def attn_paged(q, k_pages, v_pages, page_table, k_len, *, cu_q=None, max_q=None, max_k=None, scale=None,
               want_lse: bool = True, o=None, lse=None, workspace=None
               ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """attn_fwd of new tokens over a paged cache: q [total_q, Hq, 128] with cu_q, or [B, T, Hq,
    128]; k_pages, v_pages [pages, page_size, Hk, 128] as for rope_append; page_table int32
    [n, ..], the pages of each sequence (an entry outside the cache is an absent page, whose
    keys nobody sees); k_len int32 [n], their used rows, the new tokens' own among them.  max_q
    and max_k bound a sequence's new tokens and its keys; they steer what is started, not what is
    computed.  Returns (o, lse)."""
    n, total, longest, P, page, pages, Hq, Hk, d, scale, sq, ks, st = _paged_dims(q, k_pages, page_table, k_len, cu_q,
                                                                                  max_k, scale)
    vs = _check_pages(v_pages, "v_pages", Hk, k_pages)
    dev = q.device
    if o is None:
        o = torch.empty(q.shape, dtype=torch.bfloat16, device=dev)
    else:
        _check(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _check(lse, "lse", torch.float32, q.shape[:-1])
    elif want_lse:
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=dev)
    if _several_devices:
        _check_devices(q, k_pages, v_pages, page_table, k_len, cu_q, o, lse, workspace)
    most = q.shape[1] if cu_q is None else 0 if max_q is None else int(max_q)
    wp, wn, ws = _scratch_all(_planned_bytes("gdn_attn_paged_workspace_bytes", dev.index, n, total, pages * page, most,
                                             longest, Hq, Hk, d), dev, workspace)  # (ws: kept alive over the call)
    rc = lib().gdn_attn_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), page_table.data_ptr(),
                              k_len.data_ptr(), _ptr(cu_q), o.data_ptr(), _ptr(lse), n, total, most, longest, P, page,
                              pages, Hq, Hk, d, scale, sq, ctypes.byref(ks), ctypes.byref(vs), st, wp, wn, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_attn_paged")
    return o, lse


def attn_paged_weights(q, k_pages, lse, page_table, k_len, weights, *, cu_q=None, max_q=None, max_k=None, scale=None,
                       workspace=None) -> torch.Tensor:
    """Adds to weights [pages, Hk, page_size] (fp32) the attention weight that each cached key
    receives from the queries of an attn_paged call (its q, pages, table and lengths, and its
    lse), summed over them and over the query heads of each key head.  Returns weights."""
    n, total, longest, P, page, pages, Hq, Hk, d, scale, sq, ks, st = _paged_dims(q, k_pages, page_table, k_len, cu_q,
                                                                                  max_k, scale)
    _check(lse, "lse", torch.float32, q.shape[:-1])
    _check(weights, "weights", torch.float32, (P, Hk, page))
    if _several_devices:
        _check_devices(q, k_pages, lse, page_table, k_len, weights, cu_q, workspace)
    most = q.shape[1] if cu_q is None else 0 if max_q is None else int(max_q)
    wp, wn, ws = _scratch(_STATUS_BYTES, q.device, workspace)
    rc = lib().gdn_attn_paged_weights(q.data_ptr(), k_pages.data_ptr(), lse.data_ptr(), page_table.data_ptr(),
                                      k_len.data_ptr(), _ptr(cu_q), weights.data_ptr(), n, total, most, longest, P, page,
                                      pages, Hq, Hk, d, scale, sq, ctypes.byref(ks), st, wp, wn, _stream(q.device))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_attn_paged_weights")
    return weights


def cache_evict_workspace_bytes(n_seqs, max_rows, budget, Hk) -> int:
    return int(lib().gdn_cache_evict_workspace_bytes(n_seqs, max_rows, budget, Hk))


def cache_evict(k_pages, v_pages, weights, page_table, k_len, budget: int, *, recent: int = 0, to_table=None,
                new_len=None, workspace=None) -> torch.Tensor:
    """Drops the lightest keys of a paged cache: of each sequence and key head the last `recent`
    keys stay and of the others those with the largest weights [pages, Hk, page_size] (ties: the
    lowest index), `budget` in all.  What stays moves in its order, with its values and weights, to
    the first rows of the pages that to_table [n, ..] lists (None, or page_table itself: the
    sequence's own, in place; no page may occur twice then).  Other target pages may not occur twice
    either, nor hold a key of the call: a copy of page_table is such a target, whose rows would be
    written while others still read them; leave to_table out instead.
    Returns the new lengths, int32 [n] (new_len, if given; it must not overlap k_len)."""
    ks = _check_pages(k_pages, "k_pages")
    P, page, Hk, d = k_pages.shape
    vs = _check_pages(v_pages, "v_pages", Hk, k_pages)
    _check(weights, "weights", torch.float32, (P, Hk, page))
    if k_len.dim() != 1:
        raise ValueError("k_len must give the used rows of every sequence")
    n = k_len.shape[0]
    _check(k_len, "k_len", torch.int32)
    pages, st = _check_table(page_table, "page_table", n)
    budget, recent = min(int(budget), 2 ** 31 - 1), min(int(recent), 2 ** 31 - 1)
    to_pages, sto = _check_table(to_table, "to_table", n) if to_table is not None else (0, 0)
    if new_len is None:
        new_len = torch.empty(n, dtype=torch.int32, device=k_len.device)
    else:
        _check(new_len, "new_len", torch.int32, (n,))
    if _several_devices:
        _check_devices(k_pages, v_pages, weights, page_table, k_len, to_table, new_len, workspace)
    wp, wn, ws = _scratch_all(cache_evict_workspace_bytes(n, pages * page, budget, Hk), k_len.device, workspace)
    rc = lib().gdn_cache_evict(k_pages.data_ptr(), v_pages.data_ptr(), weights.data_ptr(), page_table.data_ptr(),
                               _ptr(to_table), k_len.data_ptr(), new_len.data_ptr(), n, P, page, pages, to_pages, Hk, d,
                               budget, recent, ctypes.byref(ks), ctypes.byref(vs), st, sto, wp, wn,
                               _stream(k_len.device))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_cache_evict")
    return new_len


def debug_ut(k, v, g, beta, chunk: int = 128, tiles: bool = False):
    """Per-chunk S, T (fp32) and w, u (bf16), each [B, Hv, N, chunk, .].

    The library exports 128-row tiles; with chunk = 64 each holds two chunks
    (S and T block diagonal).  tiles=True returns those tiles as exported,
    [B, Hv, ceil(T / 128), 128, .]."""
    B, T, Hk, dk = k.shape
    Hv, dv = v.shape[2], v.shape[3]
    _check(k, "k", torch.bfloat16)
    _check(v, "v", torch.bfloat16, (B, T, Hv, dv))
    _check(g, "g", torch.float32, (B, T, Hv))
    _check(beta, "beta", torch.float32, (B, T, Hv))
    NT = (T + 127) // 128
    dev = k.device
    S = torch.empty((B, Hv, NT, 128, 128), dtype=torch.float32, device=dev)
    Tm = torch.empty_like(S)
    w = torch.empty((B, Hv, NT, 128, dk), dtype=torch.bfloat16, device=dev)
    u = torch.empty((B, Hv, NT, 128, dv), dtype=torch.bfloat16, device=dev)
    rc = lib().gdn_debug_ut(_ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S), _ptr(Tm), _ptr(w),
                            _ptr(u), B, T, Hk, Hv, dk, dv, chunk, _stream(dev))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_debug_ut")
    if tiles or chunk == 128:
        return S, Tm, w, u
    N = (T + chunk - 1) // chunk  # chunk 64: the diagonal blocks and row halves of the tiles

    def diag(x):
        x6 = x.view(B, Hv, NT, 2, 64, 2, 64)
        return torch.stack([x6[:, :, :, 0, :, 0, :], x6[:, :, :, 1, :, 1, :]], 3).reshape(
            B, Hv, 2 * NT, 64, 64)[:, :, :N]

    def rows(x):
        return x.reshape(B, Hv, 2 * NT, 64, x.shape[-1])[:, :, :N]

    return diag(S), diag(Tm), rows(w), rows(u)


def workspace_status(ws: torch.Tensor) -> int:
    """Status code (GDN_OK or GDN_ERR_TIMEOUT) of the bounded in-kernel waits of
    the last forward/backward call that used workspace `ws`.  Synchronises the
    current stream."""
    return lib().gdn_workspace_status(_ptr(ws), _stream(ws.device))


def selftest_wait_timeout(limit_ns: int, status: torch.Tensor) -> int:
    """Runs one block whose bounded wait can never complete and must give up
    after limit_ns; returns the library's status code (GDN_ERR_TIMEOUT = -5 is
    the expected outcome).  status: a one-element int32 CUDA tensor."""
    _check(status, "status", torch.int32, (1,))
    return lib().gdn_selftest_wait_timeout(int(limit_ns), _ptr(status), _stream(status.device))


__all__ = ["build", "lib", "chunk_fwd", "chunk_bwd", "layer_fwd", "layer_bwd",
           "layer_workspace_bytes", "saved_bytes", "affine_compose", "segment_fold", "debug_ut",
           "fwd_workspace_bytes", "bwd_workspace_bytes", "default_segments", "GDNError",
           "header_functions", "delta_step", "decay_step", "decay_fwd", "decay_bwd",
           "decay_workspace_bytes", "attn_fwd", "attn_bwd", "attn_workspace_bytes", "rope_fwd", "rope_bwd",
           "rope_workspace_bytes", "rope_append", "attn_paged", "attn_paged_workspace_bytes", "attn_paged_weights", "cache_evict",
           "cache_evict_workspace_bytes", "workspace_status", "selftest_wait_timeout"]
