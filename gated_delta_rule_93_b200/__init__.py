"""Gated delta-rule sequence mixer for NVIDIA B200 (sm_100a).

The computation lives in ``libgdr.so`` (CUDA kernels behind the C ABI in
``include/gdr.h``); ``binding`` is a ctypes front-end with the same names.
Importing this package does not load the library; the first call does.
"""
from .binding import (  # noqa: F401
    SLOT_SKIP,
    SLOT_ZERO,
    GdrError,
    chunk_bwd,
    chunk_bwd_workspace_bytes,
    chunk_fwd,
    chunk_fwd_gla,
    chunk_fwd_prologue,
    chunk_fwd_kernel_launches,
    chunk_fwd_segmented,
    chunk_fwd_varlen,
    chunk_fwd_workspace_bytes,
    dplr_fwd,
    device_status,
    group_norm_bwd,
    group_norm_fwd,
    lib,
    prologue_bwd,
    prologue_fwd,
    slot_map,
    status_string,
    step,
    step_slots,
)

__all__ = ["chunk_bwd", "chunk_bwd_workspace_bytes", "chunk_fwd", "chunk_fwd_gla", "chunk_fwd_prologue", "chunk_fwd_kernel_launches", "chunk_fwd_segmented", "chunk_fwd_varlen",
           "chunk_fwd_workspace_bytes", "dplr_fwd", "step", "device_status", "lib", "status_string",
           "GdrError", "SLOT_SKIP", "SLOT_ZERO", "group_norm_bwd", "group_norm_fwd", "prologue_bwd",
           "prologue_fwd", "slot_map", "step_slots"]
