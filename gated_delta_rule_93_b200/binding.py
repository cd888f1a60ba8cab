"""Thin Python binding of ``libgdr.so`` (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this
module checks tensor devices, dtypes, shapes and contiguity, then passes
raw device pointers and the current CUDA stream through ctypes.  There is no
CPU fallback: if the library is missing, or a tensor is not on a CUDA
device, the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")
_lib = None
_lock = threading.Lock()

GDR_OK, GDR_ERR_INVALID_ARG, GDR_ERR_UNSUPPORTED, GDR_ERR_WORKSPACE, GDR_ERR_CUDA, \
    GDR_ERR_TIMEOUT, GDR_ERR_RANGE, GDR_ERR_SLOT = range(8)
GDR_F32, GDR_BF16 = 0, 1
GDR_GATE_SCALAR, GDR_GATE_PER_CHANNEL = 0, 1
GDR_ACTS = {"none": 0, "silu": 1, "sigmoid": 2}
SLOT_ZERO, SLOT_SKIP = -1, -2  # values of src that are not a slot

EXPORTS = (
    "gdr_chunk_fwd_workspace_bytes",
    "gdr_chunk_fwd_kernel_launches",
    "gdr_chunk_fwd",
    "gdr_chunk_fwd_segmented",
    "gdr_chunk_fwd_segmented_noalloc",
    "gdr_chunk_fwd_varlen",
    "gdr_chunk_fwd_gla",
    "gdr_chunk_fwd_prologue",
    "gdr_chunk_bwd_workspace_bytes",
    "gdr_chunk_bwd",
    "gdr_dplr_fwd",
    "gdr_step",
    "gdr_step_slots",
    "gdr_slot_map",
    "gdr_group_norm_fwd",
    "gdr_group_norm_bwd_workspace_bytes",
    "gdr_group_norm_bwd",
    "gdr_prologue_fwd",
    "gdr_prologue_bwd_workspace_bytes",
    "gdr_prologue_bwd",
    "gdr_get_device_status",
    "gdr_status_string",
    "gdr_last_error_message",
    "gdr_version",
    "gdr_testing_skip_stage_load",
)


class GdrError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{status_string(status)}: {msg}")
        self.status = status


def lib():
    """Load ``libgdr.so`` once; raise if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m gated_delta_rule_93_b200.build` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            L.gdr_chunk_fwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
            L.gdr_chunk_fwd_workspace_bytes.restype = sz
            L.gdr_chunk_fwd_kernel_launches.argtypes = [i, i, i, i, i, i, i, i]
            L.gdr_chunk_fwd_kernel_launches.restype = i
            L.gdr_chunk_fwd.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, i, i, i, i, i, i,
                                        vp, sz, vp]
            L.gdr_chunk_fwd.restype = i
            L.gdr_chunk_fwd_segmented.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, i, i, i, i,
                                                  i, i, i, vp, sz, vp]
            L.gdr_chunk_fwd_segmented.restype = i
            L.gdr_chunk_fwd_segmented_noalloc.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp,
                                                          i, i, i, i, i, i, i, vp]
            L.gdr_chunk_fwd_segmented_noalloc.restype = i
            L.gdr_chunk_fwd_varlen.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, vp, i, i, i,
                                               i, i, i, vp]
            L.gdr_chunk_fwd_varlen.restype = i
            L.gdr_chunk_fwd_gla.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, i, i, i, i, i, i,
                                            vp]
            L.gdr_chunk_fwd_gla.restype = i
            L.gdr_chunk_fwd_prologue.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, vp, i, i,
                                                 i, i, i, i, i, vp]
            L.gdr_chunk_fwd_prologue.restype = i
            L.gdr_chunk_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.gdr_chunk_bwd_workspace_bytes.restype = sz
            L.gdr_chunk_bwd.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        vp, i, i, i, i, i, vp, sz, vp]
            L.gdr_chunk_bwd.restype = i
            L.gdr_dplr_fwd.argtypes = [vp, vp, vp, vp, vp, i, vp, i, vp, vp, vp, i, i, i, i, i,
                                       vp]
            L.gdr_dplr_fwd.restype = i
            L.gdr_step.argtypes = [vp, vp, vp, i, vp, i, vp, vp, vp, i, i, i, i, vp]
            L.gdr_step.restype = i
            ll, f = ctypes.c_longlong, ctypes.c_float
            L.gdr_step_slots.argtypes = [vp, vp, vp, i, ll, ll, ll, vp, i, vp, vp, i, vp, i, ll,
                                         vp, vp, vp, vp, i, i, i, i, i, i, vp]
            L.gdr_step_slots.restype = i
            L.gdr_slot_map.argtypes = [vp, vp, vp, ll, i, i, i, i, i, vp, vp, vp, vp, vp]
            L.gdr_slot_map.restype = i
            L.gdr_group_norm_fwd.argtypes = [vp, vp, i, ll, ll, vp, vp, i, i, i, f, vp, ll, i, i,
                                             vp]
            L.gdr_group_norm_fwd.restype = i
            L.gdr_group_norm_bwd_workspace_bytes.argtypes = [ll, i, i, i, i]
            L.gdr_group_norm_bwd_workspace_bytes.restype = sz
            L.gdr_group_norm_bwd.argtypes = [vp, vp, vp, i, ll, ll, vp, vp, i, i, i, f, vp, vp, vp,
                                             vp, ll, i, i, vp, sz, vp]
            L.gdr_group_norm_bwd.restype = i
            L.gdr_prologue_fwd.argtypes = [vp, vp, i, ll, ll, vp, i, vp, vp, i, vp, vp, vp, vp, ll,
                                           i, i, i, vp]
            L.gdr_prologue_fwd.restype = i
            L.gdr_prologue_bwd_workspace_bytes.argtypes = [ll, i, i, i]
            L.gdr_prologue_bwd_workspace_bytes.restype = sz
            L.gdr_prologue_bwd.argtypes = [vp, vp, i, ll, ll, vp, i, vp, vp, i, vp, vp, vp, vp, vp,
                                           vp, vp, vp, vp, ll, i, i, i, vp, sz, vp]
            L.gdr_prologue_bwd.restype = i
            L.gdr_get_device_status.argtypes = [vp]
            L.gdr_get_device_status.restype = i
            L.gdr_status_string.argtypes = [i]
            L.gdr_status_string.restype = ctypes.c_char_p
            L.gdr_last_error_message.argtypes = []
            L.gdr_last_error_message.restype = ctypes.c_char_p
            L.gdr_version.argtypes = []
            L.gdr_version.restype = i
            L.gdr_testing_skip_stage_load.argtypes = [i]
            L.gdr_testing_skip_stage_load.restype = i
            _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().gdr_status_string(int(s)).decode()


def _check(rc):
    if rc != GDR_OK:
        raise GdrError(rc, lib().gdr_last_error_message().decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream_handle(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype=None, shape=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _in_dtype(dt):
    if dt == torch.bfloat16:
        return GDR_BF16
    if dt == torch.float32:
        return GDR_F32
    raise TypeError(f"q/k/v dtype must be bfloat16 or float32, got {dt}")


def chunk_fwd_workspace_bytes(B, T, H, dk, dv, C=64, dtype=torch.bfloat16, gate="scalar"):
    gk = GDR_GATE_PER_CHANNEL if gate == "channel" else GDR_GATE_SCALAR
    return int(lib().gdr_chunk_fwd_workspace_bytes(B, T, H, dk, dv, C, _in_dtype(dtype), gk))


def chunk_fwd_kernel_launches(B, T, H, dk, dv, C=64, dtype=torch.bfloat16, gate="scalar"):
    """Kernels one ``chunk_fwd`` call launches on the current device."""
    gk = GDR_GATE_PER_CHANNEL if gate == "channel" else GDR_GATE_SCALAR
    return int(lib().gdr_chunk_fwd_kernel_launches(B, T, H, dk, dv, C, _in_dtype(dtype), gk))


def chunk_fwd(q, k, v, g, beta, S0=None, *, output_final_state=True, o=None, S_T=None, C=64,
              workspace=None, stream=None):
    """Chunkwise forward, ``gdr_chunk_fwd``.  Returns (o, S_T or None).

    q, k [B,T,H,dk]; v [B,T,H,dv] (bf16 or fp32, one dtype); g [B,T,H] (scalar
    gate) or [B,T,H,dk] (per-channel gate) fp32 log alpha; beta [B,T,H] fp32;
    S0 [B,H,dv,dk] fp32 or None.
    """
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    with torch.cuda.device(dev):
        # the segment rule depends on the SM count of q's device, which the
        # library reads from the current device
        ws = chunk_fwd_workspace_bytes(B, T, H, dk, dv, C, dt, "channel" if gk else "scalar")
        if ws and workspace is None:
            workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        rc = lib().gdr_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk,
                                 _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, C,
                                 _ptr(workspace), workspace.numel() if workspace is not None
                                 else 0, _stream_handle(stream))
    _check(rc)
    return o, S_T


def step(q, k, v, g, beta, S, *, o=None, stream=None):
    """One decode step, ``gdr_step``: S [N,H,dv,dk] fp32 is updated in place.

    q, k [N,H,dk]; v [N,H,dv]; g [N,H] or [N,H,dk]; beta [N,H].  Returns o.
    """
    _need(q, "q")
    dev = q.device
    N, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (N, H, dk), dev)
    _need(v, "v", dt, (N, H, dv), dev)
    if g.dim() == 3:
        _need(g, "g", torch.float32, (N, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (N, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (N, H), dev)
    _need(S, "S", torch.float32, (N, H, dv, dk), dev)
    if o is None:
        o = torch.empty((N, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (N, H, dv), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_step(_ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk, _ptr(beta),
                            _ptr(S), _ptr(o), N, H, dk, dv, _stream_handle(stream))
    _check(rc)
    return o


def testing_skip_stage_load(chunk):
    """Test-only: the next tensor-core chunked forward on this thread skips the
    input load of `chunk`, so its bounded waits time out (see gdr_testing.h)."""
    _check(lib().gdr_testing_skip_stage_load(int(chunk)))


def device_status(stream=None):
    """Synchronise and read/clear the library's device status word (0 = OK)."""
    return int(lib().gdr_get_device_status(_stream_handle(stream)))


def chunk_fwd_segmented(q, k, v, g, beta, S0=None, *, segments, workspace,
                        output_final_state=True, o=None, S_T=None, C=64, stream=None):
    """``gdr_chunk_fwd_segmented``: the chunked forward as ``segments`` segments
    per sequence in the caller's ``workspace`` (a uint8 CUDA tensor of at least
    3*B*segments*H*dv*dk*4 bytes).  Returns (o, S_T or None)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if not isinstance(workspace, torch.Tensor) or workspace.device != dev:
        raise ValueError("workspace must be a tensor on the inputs' device")
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_fwd_segmented(
            _ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk, _ptr(beta), _ptr(S0),
            _ptr(o), _ptr(S_T), B, T, H, dk, dv, C, int(segments), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream_handle(stream))
    _check(rc)
    return o, S_T


# Bytes of the scratch array built into the library (GDR_NOALLOC_SCRATCH_BYTES).
NOALLOC_SCRATCH_BYTES = 24 * 1024 * 1024


def chunk_fwd_segmented_noalloc(q, k, v, g, beta, S0=None, *, segments, o, S_T=None, C=64,
                                stream=None):
    """``gdr_chunk_fwd_segmented_noalloc``: the segment path with its scratch in
    the library's fixed array, for callers that cannot allocate device memory
    while they run the mixer.  The caller passes every output (``o``, and
    ``S_T`` or None); nothing is allocated here or in the library.  Calls
    that overlap on the GPU race on the shared array.  Returns (o, S_T)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_fwd_segmented_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk, _ptr(beta), _ptr(S0),
            _ptr(o), _ptr(S_T), B, T, H, dk, dv, C, int(segments), _stream_handle(stream))
    _check(rc)
    return o, S_T


def chunk_fwd_varlen(q, k, v, g, beta, cu_seqlens, S0=None, *, output_final_state=True, o=None,
                     S_T=None, C=64, stream=None):
    """``gdr_chunk_fwd_varlen``: N packed sequences of different lengths.

    q, k [total, H, dk]; v [total, H, dv] (bf16); g [total, H] or
    [total, H, dk] fp32; beta [total, H] fp32; cu_seqlens int32 CUDA tensor
    [N + 1] (sequence i = tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1);
    S0 [N, H, dv, dk] fp32 or None.  Returns (o [total, H, dv], S_T or None).
    """
    _need(q, "q")
    dev = q.device
    total, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (total, H, dk), dev)
    _need(v, "v", dt, (total, H, dv), dev)
    if g.dim() == 3:
        _need(g, "g", torch.float32, (total, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (total, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (total, H), dev)
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dtype != torch.int32 or \
            cu_seqlens.device != dev or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 tensor [N + 1] on the inputs' device")
    N = cu_seqlens.numel() - 1
    if S0 is not None:
        _need(S0, "S0", torch.float32, (N, H, dv, dk), dev)
    if o is None:
        o = torch.empty((total, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (total, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((N, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (N, H, dv, dk), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_fwd_varlen(
            _ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk, _ptr(beta), _ptr(cu_seqlens),
            _ptr(S0), _ptr(o), _ptr(S_T), N, total, H, dk, dv, C, _stream_handle(stream))
    _check(rc)
    return o, S_T


def chunk_fwd_gla(q, k, v, g, S0=None, *, output_final_state=True, o=None, S_T=None, C=64,
                  stream=None):
    """``gdr_chunk_fwd_gla``: gated linear attention, S_t = S_{t-1} Diag(alpha_t)
    + v_t k_t^T, o_t = S_t q_t (no beta).  q, k [B,T,H,dk]; v [B,T,H,dv] (bf16);
    g [B,T,H] or [B,T,H,dk] fp32 log alpha; S0 [B,H,dv,dk] fp32 or None.
    Returns (o, S_T or None)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_fwd_gla(_ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk,
                                     _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv, C,
                                     _stream_handle(stream))
    _check(rc)
    return o, S_T


def chunk_fwd_prologue(q, k, v, a, b, gate_scale, S0=None, *, norm_q=True, norm_k=True,
                       output_final_state=True, o=None, S_T=None, C=64, stream=None):
    """``gdr_chunk_fwd_prologue``: the chunked forward from raw projections.

    q, k [B,T,H,dk] (raw; bf16 or fp32); v [B,T,H,dv]; a [B,T,H] (scalar
    gate) or [B,T,H,dk] (per-channel gate) and b [B,T,H] fp32 gate and beta
    logits; gate_scale [H] fp32.  In the kernel: q, k L2-normalised (per the
    flags), beta = sigmoid(b), g = -gate_scale[h] softplus(a).
    Returns (o, S_T or None)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if a.dim() == 4:
        _need(a, "a", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(a, "a", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    _need(b, "b", torch.float32, (B, T, H), dev)
    _need(gate_scale, "gate_scale", torch.float32, (H,), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    flags = (1 if norm_q else 0) | (2 if norm_k else 0)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_fwd_prologue(_ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(a),
                                          gk, _ptr(gate_scale), _ptr(b), _ptr(S0),
                                          _ptr(o), _ptr(S_T), B, T, H, dk, dv, C, flags,
                                          _stream_handle(stream))
    _check(rc)
    return o, S_T


def chunk_bwd_workspace_bytes(B, T, H, dk, dv, dtype=torch.bfloat16, gate="scalar"):
    """Workspace ``chunk_bwd`` needs for this shape, input dtype and gate kind."""
    gk = GDR_GATE_PER_CHANNEL if gate == "channel" else GDR_GATE_SCALAR
    return int(lib().gdr_chunk_bwd_workspace_bytes(B, T, H, dk, dv, _in_dtype(dtype), gk))


def chunk_bwd(q, k, v, g, beta, dout, S0=None, dS_T=None, *, want_dS0=True, workspace=None,
              out=None, stream=None):
    """``gdr_chunk_bwd``: gradients of the chunked forward.

    Inputs as ``chunk_fwd``; dout [B,T,H,dv] fp32; dS_T [B,H,dv,dk] fp32 or
    None.  Returns dict dq, dk, dv, dg, dbeta, dS0 (fp32; dS0 None unless
    want_dS0)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(dout, "dout", torch.float32, (B, T, H, dv), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if dS_T is not None:
        _need(dS_T, "dS_T", torch.float32, (B, H, dv, dk), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    if out is None:  # (or the caller's preallocated dict of the same tensors)
        out = dict(dq=torch.empty((B, T, H, dk), **f32), dk=torch.empty((B, T, H, dk), **f32),
                   dv=torch.empty((B, T, H, dv), **f32), dg=torch.empty(tuple(g.shape), **f32),
                   dbeta=torch.empty((B, T, H), **f32),
                   dS0=torch.empty((B, H, dv, dk), **f32) if want_dS0 else None)
    for name, shape in (("dq", (B, T, H, dk)), ("dk", (B, T, H, dk)), ("dv", (B, T, H, dv)),
                        ("dg", tuple(g.shape)), ("dbeta", (B, T, H))):
        _need(out[name], name, torch.float32, shape, dev)
    if out.get("dS0") is not None:
        _need(out["dS0"], "dS0", torch.float32, (B, H, dv, dk), dev)
    ws = chunk_bwd_workspace_bytes(B, T, H, dk, dv, dt, "channel" if gk else "scalar")
    if workspace is None and ws:
        workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _in_dtype(dt), _ptr(g), gk,
                                 _ptr(beta), _ptr(S0), _ptr(dout), _ptr(dS_T), _ptr(out["dq"]),
                                 _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
                                 _ptr(out["dbeta"]), _ptr(out.get("dS0")), B, T, H, dk, dv,
                                 _ptr(workspace),
                                 workspace.numel() * workspace.element_size()
                                 if workspace is not None else 0, _stream_handle(stream))
    _check(rc)
    return out


def dplr_fwd(q, k, v, a, b, g, S0=None, *, output_final_state=True, o=None, S_T=None,
             stream=None):
    """``gdr_dplr_fwd``: S_t = S_{t-1}(Diag(alpha_t) + a_t b_t^T) + v_t k_t^T,
    o_t = S_t q_t.  q, k, a, b [B,T,H,d]; v [B,T,H,d] (one dtype); g [B,T,H]
    or [B,T,H,d] fp32; S0 [B,H,d,d] fp32 or None.  Returns (o, S_T or None)."""
    _need(q, "q")
    dev = q.device
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    for t_, n_ in ((k, "k"), (a, "a"), (b, "b")):
        _need(t_, n_, dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    if g.dim() == 4:
        _need(g, "g", torch.float32, (B, T, H, dk), dev)
        gk = GDR_GATE_PER_CHANNEL
    else:
        _need(g, "g", torch.float32, (B, T, H), dev)
        gk = GDR_GATE_SCALAR
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dv, dk), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if output_final_state and S_T is None:
        S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dv, dk), dev)
    with torch.cuda.device(dev):
        rc = lib().gdr_dplr_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _in_dtype(dt),
                                _ptr(g), gk, _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv,
                                _stream_handle(stream))
    _check(rc)
    return o, S_T


# ------------------------------------------------------------------------------
# The operators around the mixer.  A decode loop calls them once per layer and
# token, so their checks cost as little as they can: `_expect` looks at a
# tensor once and leaves the wording of an error to `_need`.

def _expect(t, name, dtype, shape, device):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        _need(t, name, dtype, shape, device)


def _row_stride(t, name, dtype, shape, device):
    """Elements between the rows of ``t`` [..., H, d]: the last two dimensions
    are dense, those before them advance by one distance (a slice of a fused
    projection, for example)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device (no CPU path exists)")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.is_contiguous():
        return shape[-1] * shape[-2]
    size, stride = t.shape, t.stride()
    width, row = size[-1] * size[-2], None
    ok = (size[-1] == 1 or stride[-1] == 1) and (size[-2] == 1 or stride[-2] == size[-1])
    count = 1  # rows covered by the dimensions from the last leading one on
    for n, step in zip(reversed(size[:-2]), reversed(stride[:-2])):
        if n == 1:
            continue
        if row is None:
            row = step
        ok = ok and step == row * count
        count *= n
    if not ok or (row is not None and row < width):
        raise ValueError(f"{name} must have dense last two dimensions and rows one distance apart "
                         f"(strides {tuple(stride)} of shape {tuple(size)})")
    return width if row is None else row


def _launch(fn, device, stream, *args):
    """Call ``fn(*args, stream)`` with ``device`` current."""
    index = device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, handle)
    if rc:
        _check(rc)


def _owned_by(stream, *tensors):
    """Keep what this module allocated for a call on ``stream`` until it is done."""
    if stream is not None:
        for t in tensors:
            if t is not None and t.numel():
                t.record_stream(stream)


def _workspace(workspace, need, device, stream):
    """The caller's workspace, looked at, or a new one of ``need`` bytes."""
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        _owned_by(stream, workspace)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or \
            not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace


def step_slots(q, k, v, g, beta, pool, src, *, dst=None, cu_seqlens=None, gate_scale=None,
               norm_q=False, norm_k=False, o=None, stream=None):
    """``gdr_step_slots``: the recurrent form over a pool of state slots.  Returns o.

    q, k [total,Hk,dk]; v [total,H,dv] (bf16 or fp32, rows any distance apart;
    H a multiple of Hk); g [total,H] or [total,H,dk] and beta [total,H] fp32:
    log alpha and the write strength, or with ``gate_scale`` [H] the logits a
    and b.  pool [slots,H,dv,dk] fp32 (updated in place; slots any distance
    apart); src [R], dst [total] or None, cu_seqlens [R+1] or None (one token
    a request), all int32.  src holds a slot, SLOT_ZERO or SLOT_SKIP; without
    dst a request's last state goes back to src.  Rows of ``o`` that no request
    covers are left as they were (unset in an ``o`` allocated here).
    """
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [total, Hk, dk] tensor")
    dev, dt = q.device, q.dtype
    total, Hk, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("v must be a [total, H, dv] tensor")
    H, dv = v.shape[1:]
    qs = _row_stride(q, "q", dt, (total, Hk, dk), dev)
    ks = _row_stride(k, "k", dt, (total, Hk, dk), dev)
    vs = _row_stride(v, "v", dt, (total, H, dv), dev)
    gk = GDR_GATE_PER_CHANNEL if g.dim() == 3 else GDR_GATE_SCALAR
    f32, i32 = torch.float32, torch.int32
    _expect(g, "g", f32, (total, H, dk) if gk else (total, H), dev)
    _expect(beta, "beta", f32, (total, H), dev)
    if gate_scale is not None:
        _expect(gate_scale, "gate_scale", f32, (H,), dev)
    slots = pool.shape[0]
    if pool.is_contiguous():
        _expect(pool, "pool", f32, (slots, H, dv, dk), dev)
        slot_stride = H * dv * dk
    else:
        if pool.dim() != 4 or pool.stride()[1:] != (dv * dk, dk, 1):
            raise ValueError("the slots of pool [slots, H, dv, dk] must be dense")
        slot_stride = _row_stride(pool.flatten(2), "pool", f32, (slots, H, dv * dk), dev)
    R = src.shape[0] if src.dim() == 1 else -1
    _expect(src, "src", i32, (max(R, 0),), dev)
    if dst is not None:
        _expect(dst, "dst", i32, (total,), dev)
    if cu_seqlens is not None:
        _expect(cu_seqlens, "cu_seqlens", i32, (R + 1,), dev)
    elif R != total:
        raise ValueError(f"without cu_seqlens src must hold one slot for each of {total} tokens")
    if o is None:
        o = torch.empty((total, H, dv), dtype=dt, device=dev)
        _owned_by(stream, o)
    else:
        _expect(o, "o", dt, (total, H, dv), dev)
    _launch((_lib or lib()).gdr_step_slots, dev, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(),
            _in_dtype(dt), qs, ks, vs, g.data_ptr(), gk, beta.data_ptr(),
            None if gate_scale is None else gate_scale.data_ptr(),
            (1 if norm_q else 0) | (2 if norm_k else 0), pool.data_ptr(), slots, slot_stride,
            src.data_ptr(), None if dst is None else dst.data_ptr(),
            None if cu_seqlens is None else cu_seqlens.data_ptr(), o.data_ptr(), R, total, Hk, H,
            dk, dv)
    return o


def slot_map(lens, kept, table, slots, max_tokens, *, keep_all=True, out=None, stream=None):
    """``gdr_slot_map``: offsets and slots of a batch, from its lengths.

    lens, kept [R] and table [R,W] int32 (rows any distance apart); ``slots``
    is the size of the pool, ``max_tokens`` the room for tokens.  Returns a
    dict of int32 tensors: cu_seqlens [R+1], src [R], request and dst
    [max_tokens] (see ``step_slots``; -1 behind the last token).
    """
    if not isinstance(lens, torch.Tensor) or lens.dim() != 1:
        raise ValueError("lens must be a [R] tensor")
    if not lens.is_cuda:
        raise ValueError("lens must be on a CUDA device (no CPU path exists)")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a [R, W] tensor")
    dev, i32 = lens.device, torch.int32
    R, W = table.shape
    _expect(lens, "lens", i32, (R,), dev)
    _expect(kept, "kept", i32, (R,), dev)
    ts = W
    if table.is_contiguous():
        _expect(table, "table", i32, (R, W), dev)
    else:
        ts = _row_stride(table[:, None], "table", i32, (R, 1, W), dev)
    if out is None:
        room = max(max_tokens, 0)
        parts = torch.empty(2 * R + 1 + 2 * room, dtype=i32, device=dev)
        _owned_by(stream, parts)
        cu, src, request, dst = parts.split((R + 1, R, room, room))
        out = {"cu_seqlens": cu, "src": src, "request": request, "dst": dst}
    else:
        for name, n in (("cu_seqlens", R + 1), ("src", R), ("request", max_tokens),
                        ("dst", max_tokens)):
            _expect(out[name], name, i32, (n,), dev)
    _launch((_lib or lib()).gdr_slot_map, dev, stream, lens.data_ptr(), kept.data_ptr(),
            table.data_ptr(), ts, R, W, slots, max_tokens, 1 if keep_all else 0,
            out["cu_seqlens"].data_ptr(), out["request"].data_ptr(), out["src"].data_ptr(),
            out["dst"].data_ptr())
    return out


def _norm_args(x, z, weight, bias, act):
    """The checks both directions of the output norm share."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x must be a [..., G, D] tensor")
    dev, dt, shape = x.device, x.dtype, x.shape
    G, D = shape[-2:]
    xs = _row_stride(x, "x", dt, shape, dev)
    zs = _row_stride(z, "z", dt, shape, dev) if z is not None else 0
    per = weight if weight is not None else bias
    per_channel = per is not None and per.dim() == 2
    affine = (G, D) if per_channel else (D,)
    if weight is not None:
        _expect(weight, "weight", torch.float32, affine, dev)
    if bias is not None:
        _expect(bias, "bias", torch.float32, affine, dev)
    if act not in GDR_ACTS:
        raise ValueError(f"act must be one of {', '.join(GDR_ACTS)}, got {act!r}")
    rows = x.numel() // (G * D) if G * D else 0
    return dev, dt, shape, rows, G, D, xs, zs, 1 if per_channel else 0, affine


def group_norm_fwd(x, z=None, weight=None, bias=None, *, act="silu", center=False, eps=1e-5,
                   y=None, stream=None):
    """``gdr_group_norm_fwd``: each group (head) of each token normalised, with
    an activation.  Returns y, shaped as x.

    x [..., G, D] and the gate z (or None) bf16 or fp32, rows any distance
    apart; weight, bias fp32 [D] or [G, D] or None.  y = act(z) l or, without
    z, act(l), where l = n w + b.
    """
    dev, dt, shape, rows, G, D, xs, zs, pc, _ = _norm_args(x, z, weight, bias, act)
    if y is None:
        y = torch.empty(shape, dtype=dt, device=dev)
        _owned_by(stream, y)
    else:
        _expect(y, "y", dt, shape, dev)
    _launch((_lib or lib()).gdr_group_norm_fwd, dev, stream, x.data_ptr(),
            None if z is None else z.data_ptr(), _in_dtype(dt), xs, zs,
            None if weight is None else weight.data_ptr(),
            None if bias is None else bias.data_ptr(), pc, GDR_ACTS[act], 1 if center else 0, eps,
            y.data_ptr(), rows, G, D)
    return y


def group_norm_bwd(dy, x, z=None, weight=None, bias=None, *, act="silu", center=False, eps=1e-5,
                   workspace=None, out=None, stream=None):
    """``gdr_group_norm_bwd``: gradients of ``group_norm_fwd`` (same arguments).

    dy as x, contiguous.  Returns dict dx (fp32, what ``chunk_bwd`` takes as
    dout), dz (dtype of z), dweight, dbias (fp32); what has no input is None.
    """
    dev, dt, shape, rows, G, D, xs, zs, pc, affine = _norm_args(x, z, weight, bias, act)
    _expect(dy, "dy", dt, shape, dev)
    f32 = torch.float32
    want = {"dx": (f32, shape), "dz": (dt, shape) if z is not None else None,
            "dweight": (f32, affine) if weight is not None else None,
            "dbias": (f32, affine) if bias is not None else None}
    if out is None:
        out = {n: w and torch.empty(w[1], dtype=w[0], device=dev) for n, w in want.items()}
        _owned_by(stream, *out.values())
    else:  # (the caller's preallocated dict of the same tensors)
        for n, w in want.items():
            if w is not None:
                _expect(out[n], n, w[0], w[1], dev)
    L = _lib or lib()
    if weight is not None or bias is not None:
        need = L.gdr_group_norm_bwd_workspace_bytes(rows, G, D, _in_dtype(dt), pc)
        workspace = _workspace(workspace, need, dev, stream)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _launch(L.gdr_group_norm_bwd, dev, stream, dy.data_ptr(), x.data_ptr(), ptr(z), _in_dtype(dt),
            xs, zs, ptr(weight), ptr(bias), pc, GDR_ACTS[act], 1 if center else 0, eps,
            out["dx"].data_ptr(), ptr(out["dz"]) if z is not None else None,
            ptr(out["dweight"]) if weight is not None else None,
            ptr(out["dbias"]) if bias is not None else None, rows, G, D, ptr(workspace),
            workspace.numel() * workspace.element_size() if workspace is not None else 0)
    return out


def _prologue_args(q, k, a, b, gate_scale):
    """The checks both directions of the prologue share."""
    if not isinstance(q, torch.Tensor) or q.dim() < 3:
        raise ValueError("q must be a [..., Hk, dk] tensor")
    dev, dt, shape = q.device, q.dtype, q.shape
    lead, Hk, dk = shape[:-2], shape[-2], shape[-1]
    qs = _row_stride(q, "q", dt, shape, dev)
    ks = _row_stride(k, "k", dt, shape, dev)
    H = b.shape[-1]
    gk = GDR_GATE_PER_CHANNEL if a.dim() == q.dim() else GDR_GATE_SCALAR
    f32 = torch.float32
    _expect(a, "a", f32, (*lead, H, dk) if gk else (*lead, H), dev)
    _expect(b, "b", f32, (*lead, H), dev)
    _expect(gate_scale, "gate_scale", f32, (H,), dev)
    tokens = b.numel() // H if H else 0
    return dev, dt, shape, (*lead, H, dk), tokens, Hk, H, dk, qs, ks, gk


def prologue_fwd(q, k, a, b, gate_scale, *, norm_q=True, norm_k=True, out=None, stream=None):
    """``gdr_prologue_fwd``: raw projections to what ``chunk_fwd`` and ``chunk_bwd``
    take.  Returns (q, k, g, beta).

    q, k [..., Hk, dk] raw (bf16 or fp32, rows any distance apart); a [..., H]
    or [..., H, dk] and b [..., H] fp32 logits; gate_scale [H] fp32.  q, k come
    back normalised (per the flags) with one copy for each of the H value
    heads; g = -gate_scale softplus(a), beta = sigmoid(b).
    """
    dev, dt, _, full, tokens, Hk, H, dk, qs, ks, gk = _prologue_args(q, k, a, b, gate_scale)
    if out is None:
        new = lambda shape, dtype: torch.empty(shape, dtype=dtype, device=dev)  # noqa: E731
        out = (new(full, dt), new(full, dt), new(a.shape, torch.float32),
               new(b.shape, torch.float32))
        _owned_by(stream, *out)
    else:  # (the caller's preallocated q, k, g, beta)
        for t, n, d, s in zip(out, ("q out", "k out", "g", "beta"),
                              (dt, dt, torch.float32, torch.float32),
                              (full, full, a.shape, b.shape)):
            _expect(t, n, d, s, dev)
    qn, kn, g, beta = out
    _launch((_lib or lib()).gdr_prologue_fwd, dev, stream, q.data_ptr(), k.data_ptr(),
            _in_dtype(dt), qs, ks, a.data_ptr(), gk, b.data_ptr(), gate_scale.data_ptr(),
            (1 if norm_q else 0) | (2 if norm_k else 0), qn.data_ptr(), kn.data_ptr(),
            g.data_ptr(), beta.data_ptr(), tokens, Hk, H, dk)
    return qn, kn, g, beta


def prologue_bwd(q, k, a, b, gate_scale, dq, dk, dg, dbeta, *, norm_q=True, norm_k=True,
                 workspace=None, out=None, stream=None):
    """``gdr_prologue_bwd``: gradients of ``prologue_fwd`` (same arguments) from
    those of its outputs, as ``chunk_bwd`` returns them (fp32).

    dq, dk [..., H, dk]; dg as a; dbeta [..., H].  Returns dict dq, dk (shape
    and dtype of the raw q, k), da, db, dgate_scale (fp32).
    """
    dev, dt, shape, full, tokens, Hk, H, d, qs, ks, gk = _prologue_args(q, k, a, b, gate_scale)
    f32 = torch.float32
    _expect(dq, "dq", f32, full, dev)
    _expect(dk, "dk", f32, full, dev)
    _expect(dg, "dg", f32, a.shape, dev)
    _expect(dbeta, "dbeta", f32, b.shape, dev)
    want = {"dq": (dt, shape), "dk": (dt, shape), "da": (f32, a.shape), "db": (f32, b.shape),
            "dgate_scale": (f32, (H,))}
    if out is None:
        out = {n: torch.empty(s, dtype=t, device=dev) for n, (t, s) in want.items()}
        _owned_by(stream, *out.values())
    else:  # (the caller's preallocated dict of the same tensors)
        for n, (t, s) in want.items():
            _expect(out[n], n, t, s, dev)
    L = _lib or lib()
    workspace = _workspace(workspace, L.gdr_prologue_bwd_workspace_bytes(tokens, H, d, gk), dev,
                           stream)
    _launch(L.gdr_prologue_bwd, dev, stream, q.data_ptr(), k.data_ptr(), _in_dtype(dt), qs, ks,
            a.data_ptr(), gk, b.data_ptr(), gate_scale.data_ptr(),
            (1 if norm_q else 0) | (2 if norm_k else 0), dq.data_ptr(), dk.data_ptr(),
            dg.data_ptr(), dbeta.data_ptr(), out["dq"].data_ptr(), out["dk"].data_ptr(),
            out["da"].data_ptr(), out["db"].data_ptr(), out["dgate_scale"].data_ptr(), tokens, Hk,
            H, d, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
