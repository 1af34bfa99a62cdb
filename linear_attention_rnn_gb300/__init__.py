"""GB300 (sm_103a) chunked Gated DeltaNet -- Python binding of libgdn.

Beside the chunked rule (chunk_fwd, chunk_bwd, the layer and the segment calls) there
are the operators that a stack with other mixers and a decoding loop need:
delta_step, one token per row of the gated delta rule; decay_fwd, decay_bwd and
decay_step, linear attention with a decay for each head; attn_fwd and attn_bwd,
causal softmax attention with grouped heads, over packed sequences or caches.

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
           "decay_workspace_bytes", "attn_fwd", "attn_bwd", "attn_workspace_bytes", "workspace_status", "selftest_wait_timeout"]
