"""Mamba-2 SSD mixer core on MI355X (gfx950): Python binding of libssd.so.

The entry points mirror the C ABI in include/ssd.h one to one:

    ssd_conv_fwd        causal depthwise conv (k=4) + SiLU, dt = softplus(dt + dt_bias)
    ssd_chunk_scan_fwd  chunked (64) SSD scan with groups, documents, states, D skip, z gate
    ssd_chunk_scan_fwd_static  the same scan with its split workspace in the library's static
                        scratch: for callers that cannot allocate device memory
    ssd_mixer_fwd       both in one call (staged, or the scan convolving the raw columns on chip)
    ssd_resume_fwd      decode tokens rescanned with the working chunk: bit-identical to the forward
    ssd_step            one decode token per sequence
    ssd_s6_scan_fwd     the Mamba-1 selective scan (per-channel diagonal state)
    ssd_chunk_scan_bwd  backward (VJP) of the scan for a zero-state prefill
    ssd_conv_bwd        backward of the conv prologue
    ssd_mixer_bwd       backward of conv + scan
    ssd_delta_scan_fwd  the gated delta rule over a sequence (chunks of 64)
    ssd_delta_step      one decode token of the gated delta rule per sequence
    ssd_delta_scan_bwd  backward (VJP) of the gated delta rule
    ssd_norm_fwd        layer or RMS norm of rows, with weight, bias and a silu gate
    ssd_norm_bwd        its backward, with the weights' reductions
    ssd_glr_scan_fwd    the gated linear recurrence (one number of state a channel)
    ssd_glr_step        one decode token of it per sequence
    ssd_glr_scan_bwd    its backward (VJP)
    ssd_add_norm_fwd    layer or RMS norm with a residual's addition and an 8-bit output with scales
    ssd_add_norm_bwd    its backward
    ssd_proj_fp8_fwd    a projection in 8-bit floating point with block scales

This module only marshals torch tensors (device pointers, row strides, the
current HIP stream) into the library; every step of the computation runs in
the HIP kernels.  There is no fallback: if libssd.so is not built, or a
tensor is not on the GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = ["load", "ssd_conv_fwd", "ssd_chunk_scan_fwd", "ssd_chunk_scan_fwd_static", "SSD_STATIC_SCRATCH_BYTES", "ssd_mixer_fwd", "ssd_resume_fwd", "ssd_step",
           "ssd_s6_scan_fwd", "ssd_chunk_scan_workspace_size", "ssd_mixer_workspace_size", "ssd_s6_workspace_size",
           "ssd_chunk_scan_bwd", "ssd_conv_bwd", "ssd_mixer_bwd", "ssd_chunk_scan_bwd_workspace_size",
           "ssd_conv_bwd_workspace_size", "ssd_mixer_bwd_workspace_size",
           "ssd_delta_scan_fwd", "ssd_delta_scan_workspace_size", "ssd_delta_scan_bwd",
           "ssd_delta_scan_bwd_workspace_size", "ssd_delta_step", "ssd_norm_fwd", "ssd_norm_bwd", "ssd_norm_bwd_workspace_size",
           "ssd_glr_scan_fwd", "ssd_glr_scan_workspace_size", "ssd_glr_step", "ssd_glr_scan_bwd",
           "ssd_glr_scan_bwd_workspace_size", "ssd_add_norm_fwd", "ssd_add_norm_bwd",
           "ssd_proj_fp8_fwd", "ssd_proj_fp8_tile_rows",
           "SSDError", "LIB_PATH", "SSD_F32", "SSD_BF16", "SSD_ACT_SILU", "SSD_ACT_NONE"]

# SSD_LIBRARY names another build of the same library (the host-sanitized one the ABI checks use)
LIB_PATH = os.environ.get("SSD_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libssd.so")

SSD_F32, SSD_BF16 = 0, 1
SSD_STATIC_SCRATCH_BYTES = 32 << 20     # include/ssd.h
SSD_ACT_SILU, SSD_ACT_NONE = 0, 1

_lib = None


class SSDError(RuntimeError):
    """A non-zero ssd_status_t; .status holds the code."""

    def __init__(self, status: int, name: str, message: str):
        super().__init__(f"{name}: {message}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libssd.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m selective_state_space_14_amd.build` "
                           "(or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    I, P, I64, SZ = ctypes.c_int, ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    lib.ssd_last_error.restype = ctypes.c_char_p
    lib.ssd_last_error.argtypes = []
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [I]
    lib.ssd_version.restype = I
    lib.ssd_version.argtypes = []
    lib.ssd_conv_fwd.restype = I
    lib.ssd_conv_fwd.argtypes = [I, I, I, I, I, I, I, I, P, I64, P, P, P, I64, P, P, P, P, I, P, I64, P, P]
    lib.ssd_chunk_scan_fwd.restype = I
    # ... z, z_row_stride, doc_ids, lengths, init_state, final_state, y, y_row_stride, workspace, bytes, stream
    lib.ssd_chunk_scan_fwd.argtypes = [I, I, I, I, I, I, I, I, P, I64, P, I64, P, I64, P, I64, I, P, P, P, P,
                                       I64, P, P, P, P, P, I64, P, SZ, P]
    lib.ssd_chunk_scan_fwd_static.restype = I
    lib.ssd_chunk_scan_fwd_static.argtypes = [I, I, I, I, I, I, I, I, P, I64, P, I64, P, I64, P, I64, I, P, P, P, P,
                                              I64, P, P, P, P, P, I64, P]
    lib.ssd_chunk_scan_workspace_size.restype = SZ
    lib.ssd_chunk_scan_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.ssd_mixer_fwd.restype = I
    lib.ssd_mixer_fwd.argtypes = [I, I, I, I, I, I, I, I, I, P, I64, P, P, P, I64, P, P, P, P, I64, P, P, P, P, P, P,
                                  I, P, I64, P, SZ, P]
    lib.ssd_mixer_workspace_size.restype = SZ
    lib.ssd_mixer_workspace_size.argtypes = [I, I, I, I, I, I, I]
    lib.ssd_resume_fwd.restype = I
    lib.ssd_resume_fwd.argtypes = [I, I, I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, I, P, P, P, P, P, P, P, P]
    lib.ssd_step.restype = I
    lib.ssd_step.argtypes = [I, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, P, I, P, P]
    lib.ssd_s6_scan_fwd.restype = I
    lib.ssd_s6_scan_fwd.argtypes = [I, I, I, I, I, P, I64, P, I64, I, P, P, P, I64, P, I64, P, P, I64, P, P, P,
                                    P, I64, P, SZ, P]
    lib.ssd_chunk_scan_bwd.restype = I
    lib.ssd_chunk_scan_bwd.argtypes = [I, I, I, I, I, I, I, I, P, I64, P, I64, P, I64, P, I64, I, P, P, P, P, I64, P,
                                       P, I64, P, I64, P, I64, P, I64, P, I64, P, P, P, P, I64, P, SZ, P]
    lib.ssd_conv_bwd.restype = I
    lib.ssd_conv_bwd.argtypes = [I, I, I, I, I, I, I, I, P, I64, P, P, P, I, P, I64, P, I64, P, P, P, SZ, P]
    lib.ssd_mixer_bwd.restype = I
    lib.ssd_mixer_bwd.argtypes = [I, I, I, I, I, I, I, I, I, P, I64, P, P, P, I64, P, P, P, P, I64, P, I, P, I64, P,
                                  I64, P, P, P, I64, P, P, P, P, I64, P, SZ, P]
    for nm in ("ssd_chunk_scan_bwd_workspace_size", "ssd_conv_bwd_workspace_size", "ssd_mixer_bwd_workspace_size"):
        getattr(lib, nm).restype = SZ
        getattr(lib, nm).argtypes = [I, I, I, I, I, I, I]
    F = ctypes.c_float
    # q, k, v, dt (softplus, bias), A, beta (sigmoid), scale, qk_norm: the shared head of the delta calls
    delta = [P, I64, P, I64, P, I64, P, I64, I, P, P, P, I64, I, F, I]
    lib.ssd_delta_scan_fwd.restype = I
    lib.ssd_delta_scan_fwd.argtypes = [I, I, I, I, I, I, I, I, *delta, P, P, P, P, P, I64, P, SZ, P]
    lib.ssd_delta_scan_bwd.restype = I
    lib.ssd_delta_scan_bwd.argtypes = [I, I, I, I, I, I, I, I, *delta, P, P, P, P, I64, P, P, I64, P, I64, P, I64, P,
                                       I64, P, I64, P, P, P, P, SZ, P]
    for nm in ("ssd_delta_scan_workspace_size", "ssd_delta_scan_bwd_workspace_size"):
        getattr(lib, nm).restype = SZ
        getattr(lib, nm).argtypes = [I, I, I, I, I, I, I]
    lib.ssd_delta_step.restype = I
    lib.ssd_delta_step.argtypes = [I, I, I, I, I, I, *delta, P, P, I64, P]
    lib.ssd_norm_fwd.restype = I
    lib.ssd_norm_fwd.argtypes = [I64, I, I, I, I, I, F, P, I64, P, P, P, I64, P, I64, P]
    lib.ssd_norm_bwd.restype = I
    lib.ssd_norm_bwd.argtypes = [I64, I, I, I, I, I, F, P, I64, P, P, P, I64, P, I64, P, I64, P, P, P, I64, P, SZ, P]
    lib.ssd_norm_bwd_workspace_size.restype = SZ
    lib.ssd_norm_bwd_workspace_size.argtypes = [I64, I, I]
    lib.ssd_s6_workspace_size.restype = SZ
    lib.ssd_s6_workspace_size.argtypes = [I, I, I, I, I]
    # x, r, i, r_bias, i_bias, A: the shared head of the recurrence's calls
    glr = [P, I64, P, I64, P, I64, P, P, P]
    lib.ssd_glr_scan_fwd.restype = I
    lib.ssd_glr_scan_fwd.argtypes = [I, I, I, I, *glr, P, P, P, P, P, P, I64, P, SZ, P]
    lib.ssd_glr_step.restype = I
    lib.ssd_glr_step.argtypes = [I, I, I, *glr, P, P, I64, P]
    lib.ssd_glr_scan_bwd.restype = I
    lib.ssd_glr_scan_bwd.argtypes = [I, I, I, I, *glr, P, P, P, P, P, I64, P, P, I64, P, I64, P, I64, P, P, P, P, P, SZ, P]
    for nm in ("ssd_glr_scan_workspace_size", "ssd_glr_scan_bwd_workspace_size"):
        getattr(lib, nm).restype = SZ
        getattr(lib, nm).argtypes = [I, I, I, I]
    lib.ssd_add_norm_fwd.restype = I
    lib.ssd_add_norm_fwd.argtypes = [I64, I, I, I, I, I, F, P, I64, P, I64, P, P, P, I64, P, I64, P, I64, P, I64, P, I64, P]
    lib.ssd_add_norm_bwd.restype = I
    lib.ssd_add_norm_bwd.argtypes = [I64, I, I, I, I, F, P, I64, P, P, P, I64, P, I64, P, I64, P, I64, P, P, P, I64, P, SZ, P]
    lib.ssd_proj_fp8_tile_rows.restype = I
    lib.ssd_proj_fp8_tile_rows.argtypes = [I, I, I, I]
    lib.ssd_proj_fp8_fwd.restype = I
    lib.ssd_proj_fp8_fwd.argtypes = [I, I, I, I, P, I64, P, I64, P, I64, P, I64, P, I64, P]
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        lib = load()
        raise SSDError(status, lib.ssd_status_string(status).decode(), lib.ssd_last_error().decode())


def _dtype_code(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float32:
        return SSD_F32
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    raise TypeError(f"{name}: dtype {t.dtype} is not supported (float32 or bfloat16; other types are refused, "
                    "not converted)")


def _ptr(t, name, dtype=None, device=True):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device and not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _rows(t, name, B, L, width):
    """Validate a [B, L, width] view with a contiguous inner dim; return its row stride."""
    if t is None:
        return 0
    if t.dim() != 3 or t.shape[0] != B or t.shape[1] != L or t.shape[2] != width:
        raise ValueError(f"{name}: expected shape [{B}, {L}, {width}], got {list(t.shape)}")
    if t.stride(2) != 1 and width > 1:
        raise ValueError(f"{name}: the innermost dimension must be contiguous")
    rs = t.stride(1)
    if B > 1 and L > 0 and t.stride(0) != L * rs:
        raise ValueError(f"{name}: batch rows must be L * row_stride elements apart")
    return rs


def _contig(t, name, shape):
    if t is None:
        return
    if list(t.shape) != list(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {list(shape)}, got {list(t.shape)}")


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def ssd_conv_fwd(xbc_raw, conv_w, *, H, P, N, G, K=4, conv_b=None, dt_raw=None, dt_bias=None, doc_ids=None,
                 conv_state_in=None, conv_state_out=None, act=SSD_ACT_SILU, xbc_out=None, dt_out=None, stream=None):
    """Causal depthwise conv + activation over xbc_raw [B, L, conv_dim] and dt = softplus(dt_raw + dt_bias).

    Returns (xbc_out [B, L, conv_dim] in xbc_raw's dtype, dt_out [B, L, H] fp32 or None)."""
    lib = load()
    B, L = xbc_raw.shape[0], xbc_raw.shape[1]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    rs_in = _rows(xbc_raw, "xbc_raw", B, L, C)
    if xbc_out is None:
        xbc_out = torch.empty((B, L, C), dtype=xbc_raw.dtype, device=xbc_raw.device)
    rs_out = _rows(xbc_out, "xbc_out", B, L, C)
    rs_dt = 0
    if dt_raw is not None:
        rs_dt = _rows(dt_raw, "dt_raw", B, L, H)
        if dt_out is None:
            dt_out = torch.empty((B, L, H), dtype=torch.float32, device=xbc_raw.device)
        _contig(dt_out, "dt_out", (B, L, H))
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    _contig(conv_state_in, "conv_state_in", (B, K - 1, C))
    _contig(conv_state_out, "conv_state_out", (B, K - 1, C))
    st = lib.ssd_conv_fwd(
        B, L, H, P, N, G, K, dtype,
        _ptr(xbc_raw, "xbc_raw"), rs_in,
        _ptr(conv_w, "conv_w", torch.float32), _ptr(conv_b, "conv_b", torch.float32),
        _ptr(dt_raw, "dt_raw", xbc_raw.dtype), rs_dt,
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(doc_ids, "doc_ids", torch.int32),
        _ptr(conv_state_in, "conv_state_in", xbc_raw.dtype), _ptr(conv_state_out, "conv_state_out", xbc_raw.dtype),
        int(act), _ptr(xbc_out, "xbc_out", xbc_raw.dtype), rs_out,
        _ptr(dt_out, "dt_out", torch.float32), _stream(stream))
    _check(st)
    return xbc_out, dt_out


def ssd_chunk_scan_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_chunk_scan_workspace_size(B, L, H, P, N, G, dtype))


def ssd_chunk_scan_fwd(x, Bm, Cm, dt, A, *, H, P, N, G, D=None, z=None, doc_ids=None, lengths=None, init_state=None,
                       final_state=None, y=None, dt_softplus=False, dt_bias=None, chunk=64, workspace=None,
                       stream=None):
    """SSD scan.  x [B,L,H*P], Bm/Cm [B,L,G*N] (same dtype), dt [B,L,H] fp32, A [H] fp32.

    Returns y [B, L, H*P] fp32 (and writes final_state if given)."""
    lib = load()
    B, L = x.shape[0], x.shape[1]
    dtype = _dtype_code(x, "x")
    rs_x = _rows(x, "x", B, L, H * P)
    rs_b = _rows(Bm, "Bm", B, L, G * N)
    rs_c = _rows(Cm, "Cm", B, L, G * N)
    rs_dt = _rows(dt, "dt", B, L, H)
    rs_z = _rows(z, "z", B, L, H * P)
    if y is None:
        y = torch.empty((B, L, H * P), dtype=torch.float32, device=x.device)
    rs_y = _rows(y, "y", B, L, H * P)
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    _contig(lengths, "lengths", (B,))
    _contig(init_state, "init_state", (B, H, P, N))
    _contig(final_state, "final_state", (B, H, P, N))
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssd_chunk_scan_fwd(
        B, L, H, P, N, G, chunk, dtype,
        _ptr(x, "x"), rs_x, _ptr(Bm, "Bm", x.dtype), rs_b, _ptr(Cm, "Cm", x.dtype), rs_c,
        _ptr(dt, "dt", torch.float32), rs_dt, int(bool(dt_softplus)), _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32),
        _ptr(z, "z", x.dtype), rs_z, _ptr(doc_ids, "doc_ids", torch.int32), _ptr(lengths, "lengths", torch.int32),
        _ptr(init_state, "init_state", torch.float32), _ptr(final_state, "final_state", torch.float32),
        _ptr(y, "y", torch.float32), rs_y, _ptr(workspace, "workspace"), ws, _stream(stream))
    _check(st)
    return y


def ssd_chunk_scan_fwd_static(x, Bm, Cm, dt, A, *, H, P, N, G, D=None, z=None, doc_ids=None, lengths=None,
                              init_state=None, final_state=None, y=None, dt_softplus=False, dt_bias=None, chunk=64,
                              stream=None):
    """ssd_chunk_scan_fwd with the split workspace taken from the library's static scratch (allocates no
    device memory itself when y is given).  Same arguments and results as ssd_chunk_scan_fwd with a workspace."""
    lib = load()
    B, L = x.shape[0], x.shape[1]
    dtype = _dtype_code(x, "x")
    rs_x = _rows(x, "x", B, L, H * P)
    rs_b = _rows(Bm, "Bm", B, L, G * N)
    rs_c = _rows(Cm, "Cm", B, L, G * N)
    rs_dt = _rows(dt, "dt", B, L, H)
    rs_z = _rows(z, "z", B, L, H * P)
    if y is None:
        y = torch.empty((B, L, H * P), dtype=torch.float32, device=x.device)
    rs_y = _rows(y, "y", B, L, H * P)
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    _contig(lengths, "lengths", (B,))
    _contig(init_state, "init_state", (B, H, P, N))
    _contig(final_state, "final_state", (B, H, P, N))
    st = lib.ssd_chunk_scan_fwd_static(
        B, L, H, P, N, G, chunk, dtype,
        _ptr(x, "x"), rs_x, _ptr(Bm, "Bm", x.dtype), rs_b, _ptr(Cm, "Cm", x.dtype), rs_c,
        _ptr(dt, "dt", torch.float32), rs_dt, int(bool(dt_softplus)), _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32),
        _ptr(z, "z", x.dtype), rs_z, _ptr(doc_ids, "doc_ids", torch.int32), _ptr(lengths, "lengths", torch.int32),
        _ptr(init_state, "init_state", torch.float32), _ptr(final_state, "final_state", torch.float32),
        _ptr(y, "y", torch.float32), rs_y, _stream(stream))
    _check(st)
    return y


def ssd_mixer_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_mixer_workspace_size(B, L, H, P, N, G, dtype))


def ssd_mixer_fwd(xbc_raw, dt_raw, conv_w, A, *, H, P, N, G, K=4, conv_b=None, dt_bias=None, D=None, z=None,
                  doc_ids=None, lengths=None, conv_state_in=None, conv_state_out=None, init_state=None, final_state=None,
                  act=SSD_ACT_SILU, y=None, chunk=64, workspace=None, stream=None):
    """Conv prologue + scan in one pass.  xbc_raw [B, L, conv_dim], dt_raw [B, L, H] (same dtype),
    conv_w [conv_dim, K] fp32, A [H] fp32; the rest as in ssd_conv_fwd / ssd_chunk_scan_fwd.

    Returns y [B, L, H*P] fp32 (and writes final_state / conv_state_out if given)."""
    lib = load()
    B, L = xbc_raw.shape[0], xbc_raw.shape[1]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    rs_in = _rows(xbc_raw, "xbc_raw", B, L, C)
    rs_dt = _rows(dt_raw, "dt_raw", B, L, H)
    rs_z = _rows(z, "z", B, L, H * P)
    if y is None:
        y = torch.empty((B, L, H * P), dtype=torch.float32, device=xbc_raw.device)
    rs_y = _rows(y, "y", B, L, H * P)
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    _contig(lengths, "lengths", (B,))
    _contig(conv_state_in, "conv_state_in", (B, K - 1, C))
    _contig(conv_state_out, "conv_state_out", (B, K - 1, C))
    _contig(init_state, "init_state", (B, H, P, N))
    _contig(final_state, "final_state", (B, H, P, N))
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssd_mixer_fwd(
        B, L, H, P, N, G, K, chunk, dtype,
        _ptr(xbc_raw, "xbc_raw"), rs_in,
        _ptr(conv_w, "conv_w", torch.float32), _ptr(conv_b, "conv_b", torch.float32),
        _ptr(dt_raw, "dt_raw", xbc_raw.dtype), rs_dt, _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32),
        _ptr(z, "z", xbc_raw.dtype), rs_z, _ptr(doc_ids, "doc_ids", torch.int32), _ptr(lengths, "lengths", torch.int32),
        _ptr(conv_state_in, "conv_state_in", xbc_raw.dtype), _ptr(conv_state_out, "conv_state_out", xbc_raw.dtype),
        _ptr(init_state, "init_state", torch.float32), _ptr(final_state, "final_state", torch.float32),
        int(act), _ptr(y, "y", torch.float32), rs_y, _ptr(workspace, "workspace"), ws, _stream(stream))
    _check(st)
    return y


def ssd_resume_fwd(xbc_raw, dt_raw, conv_w, A, conv_state, chunk_xbc, chunk_dt, chunk_state, chunk_y, *, pos,
                   H, P, N, G, K=4, z=None, chunk_z=None, conv_b=None, dt_bias=None, D=None, act=SSD_ACT_SILU, y=None,
                   stream=None):
    """Append n = xbc_raw.shape[1] tokens to the working chunk (pos tokens already in it) and return their
    y [B, n, H*P] fp32, bit-identical to the sequential forward.  xbc_raw [B, n, conv_dim], dt_raw [B, n, H],
    z [B, n, H*P] (same dtype, contiguous); conv_state [B, K-1, conv_dim], chunk_xbc [B, 64, conv_dim],
    chunk_z [B, 64, H*P] (same dtype), chunk_dt [B, 64, H], chunk_state [B, H, P, N], chunk_y [B, 64, H*P] fp32."""
    lib = load()
    B, n = xbc_raw.shape[0], xbc_raw.shape[1]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    _contig(xbc_raw, "xbc_raw", (B, n, C))
    _contig(dt_raw, "dt_raw", (B, n, H))
    _contig(z, "z", (B, n, H * P))
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(conv_state, "conv_state", (B, K - 1, C))
    _contig(chunk_xbc, "chunk_xbc", (B, 64, C))
    _contig(chunk_dt, "chunk_dt", (B, 64, H))
    _contig(chunk_z, "chunk_z", (B, 64, H * P))
    _contig(chunk_state, "chunk_state", (B, H, P, N))
    _contig(chunk_y, "chunk_y", (B, 64, H * P))
    if y is None:
        y = torch.empty((B, n, H * P), dtype=torch.float32, device=xbc_raw.device)
    _contig(y, "y", (B, n, H * P))
    st = lib.ssd_resume_fwd(
        B, H, P, N, G, K, dtype, int(pos), n,
        _ptr(xbc_raw, "xbc_raw"), _ptr(dt_raw, "dt_raw", xbc_raw.dtype), _ptr(z, "z", xbc_raw.dtype),
        _ptr(conv_w, "conv_w", torch.float32), _ptr(conv_b, "conv_b", torch.float32),
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32), int(act),
        _ptr(conv_state, "conv_state", xbc_raw.dtype), _ptr(chunk_xbc, "chunk_xbc", xbc_raw.dtype),
        _ptr(chunk_dt, "chunk_dt", torch.float32), _ptr(chunk_z, "chunk_z", xbc_raw.dtype),
        _ptr(chunk_state, "chunk_state", torch.float32), _ptr(chunk_y, "chunk_y", torch.float32),
        _ptr(y, "y", torch.float32), _stream(stream))
    _check(st)
    return y


def ssd_step(xbc_raw, dt_raw, conv_w, A, conv_state, ssm_state, *, H, P, N, G, K=4, z=None, conv_b=None,
             dt_bias=None, D=None, act=SSD_ACT_SILU, y=None, stream=None):
    """One decode token.  xbc_raw [B, conv_dim], dt_raw [B, H] (same dtype), conv_state [B, K-1, conv_dim]
    (same dtype) and ssm_state [B, H, P, N] fp32 are updated in place.  Returns y [B, H*P] fp32."""
    lib = load()
    B = xbc_raw.shape[0]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    _contig(xbc_raw, "xbc_raw", (B, C))
    _contig(dt_raw, "dt_raw", (B, H))
    _contig(z, "z", (B, H * P))
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(conv_state, "conv_state", (B, K - 1, C))
    _contig(ssm_state, "ssm_state", (B, H, P, N))
    if y is None:
        y = torch.empty((B, H * P), dtype=torch.float32, device=xbc_raw.device)
    _contig(y, "y", (B, H * P))
    st = lib.ssd_step(
        B, H, P, N, G, K, dtype,
        _ptr(xbc_raw, "xbc_raw"), _ptr(dt_raw, "dt_raw", xbc_raw.dtype), _ptr(z, "z", xbc_raw.dtype),
        _ptr(conv_w, "conv_w", torch.float32), _ptr(conv_b, "conv_b", torch.float32),
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32),
        _ptr(conv_state, "conv_state", xbc_raw.dtype), _ptr(ssm_state, "ssm_state", torch.float32), int(act),
        _ptr(y, "y", torch.float32), _stream(stream))
    _check(st)
    return y


def ssd_s6_workspace_size(B, L, D, N, dtype=SSD_BF16) -> int:
    return int(load().ssd_s6_workspace_size(B, L, D, N, dtype))


def ssd_s6_scan_fwd(x, dt, A, Bm, Cm, *, D_skip=None, z=None, doc_ids=None, init_state=None, final_state=None,
                    y=None, dt_softplus=False, dt_bias=None, workspace=None, stream=None):
    """Mamba-1 selective scan.  x, dt [B, L, D] and Bm, Cm [B, L, N] (one dtype), A [D, N] fp32.

    Returns y [B, L, D] fp32 (and writes final_state [B, D, N] if given)."""
    lib = load()
    B, L, Dn = x.shape
    N = A.shape[1] if A.dim() == 2 else 0
    dtype = _dtype_code(x, "x")
    rs_x = _rows(x, "x", B, L, Dn)
    rs_dt = _rows(dt, "dt", B, L, Dn)
    rs_b = _rows(Bm, "Bm", B, L, N)
    rs_c = _rows(Cm, "Cm", B, L, N)
    rs_z = _rows(z, "z", B, L, Dn)
    if y is None:
        y = torch.empty((B, L, Dn), dtype=torch.float32, device=x.device)
    rs_y = _rows(y, "y", B, L, Dn)
    _contig(A, "A", (Dn, N))
    _contig(D_skip, "D_skip", (Dn,))
    _contig(dt_bias, "dt_bias", (Dn,))
    _contig(doc_ids, "doc_ids", (B, L))
    _contig(init_state, "init_state", (B, Dn, N))
    _contig(final_state, "final_state", (B, Dn, N))
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssd_s6_scan_fwd(
        B, L, Dn, N, dtype,
        _ptr(x, "x"), rs_x, _ptr(dt, "dt", x.dtype), rs_dt, int(bool(dt_softplus)),
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(A, "A", torch.float32),
        _ptr(Bm, "Bm", x.dtype), rs_b, _ptr(Cm, "Cm", x.dtype), rs_c, _ptr(D_skip, "D_skip", torch.float32),
        _ptr(z, "z", x.dtype), rs_z, _ptr(doc_ids, "doc_ids", torch.int32),
        _ptr(init_state, "init_state", torch.float32), _ptr(final_state, "final_state", torch.float32),
        _ptr(y, "y", torch.float32), rs_y, _ptr(workspace, "workspace"), ws, _stream(stream))
    _check(st)
    return y


def ssd_chunk_scan_bwd_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_chunk_scan_bwd_workspace_size(B, L, H, P, N, G, dtype))


def ssd_conv_bwd_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_conv_bwd_workspace_size(B, L, H, P, N, G, dtype))


def ssd_mixer_bwd_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_mixer_bwd_workspace_size(B, L, H, P, N, G, dtype))


def _params(batch):
    """The allocator of parameter gradients: an empty batch, for which the library does nothing, leaves them zero."""
    return torch.empty if batch else torch.zeros


def _ws(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    return workspace


def ssd_chunk_scan_bwd(x, Bm, Cm, dt, A, grad_y, *, H, P, N, G, D=None, z=None, doc_ids=None, dt_softplus=False,
                       dt_bias=None, chunk=64, workspace=None, stream=None):
    """Backward of the zero-state scan.  Returns a dict of fp32 gradients: x, Bm, Cm, dt, A (and D, z, dt_bias
    where those inputs are given).  A workspace is allocated here when none is passed."""
    lib = load()
    B, L = x.shape[0], x.shape[1]
    dtype = _dtype_code(x, "x")
    dev = x.device
    rs_x = _rows(x, "x", B, L, H * P)
    rs_b = _rows(Bm, "Bm", B, L, G * N)
    rs_c = _rows(Cm, "Cm", B, L, G * N)
    rs_dt = _rows(dt, "dt", B, L, H)
    rs_z = _rows(z, "z", B, L, H * P)
    rs_gy = _rows(grad_y, "grad_y", B, L, H * P)
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"x": torch.empty(B, L, H * P, **f32), "Bm": torch.empty(B, L, G * N, **f32),
         "Cm": torch.empty(B, L, G * N, **f32), "dt": torch.empty(B, L, H, **f32), "A": _params(B)(H, **f32),
         "D": _params(B)(H, **f32) if D is not None else None,
         "z": torch.empty(B, L, H * P, **f32) if z is not None else None,
         "dt_bias": _params(B)(H, **f32) if dt_softplus else None}
    ws = _ws(workspace, ssd_chunk_scan_bwd_workspace_size(B, L, H, P, N, G, dtype), dev)
    nb = ws.numel() * ws.element_size()
    st = lib.ssd_chunk_scan_bwd(
        B, L, H, P, N, G, chunk, dtype,
        _ptr(x, "x"), rs_x, _ptr(Bm, "Bm", x.dtype), rs_b, _ptr(Cm, "Cm", x.dtype), rs_c,
        _ptr(dt, "dt", torch.float32), rs_dt, int(bool(dt_softplus)), _ptr(dt_bias, "dt_bias", torch.float32),
        _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32), _ptr(z, "z", x.dtype), rs_z,
        _ptr(doc_ids, "doc_ids", torch.int32), _ptr(grad_y, "grad_y", torch.float32), rs_gy,
        _ptr(g["x"], "dx"), H * P, _ptr(g["Bm"], "dB"), G * N, _ptr(g["Cm"], "dC"), G * N, _ptr(g["dt"], "ddt"), H,
        _ptr(g["dt_bias"], "ddt_bias"), _ptr(g["A"], "dA"), _ptr(g["D"], "dD"), _ptr(g["z"], "dz"), H * P,
        _ptr(ws, "workspace"), nb, _stream(stream))
    _check(st)
    return {k: v for k, v in g.items() if v is not None}


def ssd_conv_bwd(xbc_raw, conv_w, grad_xbc, *, H, P, N, G, K=4, conv_b=None, doc_ids=None, act=SSD_ACT_SILU,
                 workspace=None, stream=None):
    """Backward of the zero-state conv + act.  Returns a dict: raw [B, L, conv_dim], w [conv_dim, K] (and bias)."""
    lib = load()
    B, L = xbc_raw.shape[0], xbc_raw.shape[1]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    dev = xbc_raw.device
    rs_in = _rows(xbc_raw, "xbc_raw", B, L, C)
    rs_g = _rows(grad_xbc, "grad_xbc", B, L, C)
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(doc_ids, "doc_ids", (B, L))
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"raw": torch.empty(B, L, C, **f32), "w": torch.empty(C, K, **f32),
         "bias": torch.empty(C, **f32) if conv_b is not None else None}
    ws = _ws(workspace, ssd_conv_bwd_workspace_size(B, L, H, P, N, G, dtype), dev)
    st = lib.ssd_conv_bwd(
        B, L, H, P, N, G, K, dtype, _ptr(xbc_raw, "xbc_raw"), rs_in, _ptr(conv_w, "conv_w", torch.float32),
        _ptr(conv_b, "conv_b", torch.float32), _ptr(doc_ids, "doc_ids", torch.int32), int(act),
        _ptr(grad_xbc, "grad_xbc", torch.float32), rs_g, _ptr(g["raw"], "dxbc_raw"), C, _ptr(g["w"], "dconv_w"),
        _ptr(g["bias"], "dconv_b"), _ptr(ws, "workspace"), ws.numel() * ws.element_size(), _stream(stream))
    _check(st)
    return {k: v for k, v in g.items() if v is not None}


def ssd_mixer_bwd(xbc_raw, dt_raw, conv_w, A, grad_y, *, H, P, N, G, K=4, conv_b=None, dt_bias=None, D=None, z=None,
                  doc_ids=None, act=SSD_ACT_SILU, chunk=64, workspace=None, stream=None):
    """Backward of ssd_mixer_fwd for zero states.  Returns a dict of fp32 gradients: raw, w, dt_raw, A (and bias,
    dt_bias, D, z where those inputs are given)."""
    lib = load()
    B, L = xbc_raw.shape[0], xbc_raw.shape[1]
    C = H * P + 2 * G * N
    dtype = _dtype_code(xbc_raw, "xbc_raw")
    dev = xbc_raw.device
    rs_in = _rows(xbc_raw, "xbc_raw", B, L, C)
    rs_dt = _rows(dt_raw, "dt_raw", B, L, H)
    rs_z = _rows(z, "z", B, L, H * P)
    rs_gy = _rows(grad_y, "grad_y", B, L, H * P)
    _contig(conv_w, "conv_w", (C, K))
    _contig(conv_b, "conv_b", (C,))
    _contig(dt_bias, "dt_bias", (H,))
    _contig(A, "A", (H,))
    _contig(D, "D", (H,))
    _contig(doc_ids, "doc_ids", (B, L))
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"raw": torch.empty(B, L, C, **f32), "w": torch.empty(C, K, **f32),
         "bias": torch.empty(C, **f32) if conv_b is not None else None, "dt_raw": torch.empty(B, L, H, **f32),
         "dt_bias": _params(B)(H, **f32) if dt_bias is not None else None, "A": _params(B)(H, **f32),
         "D": _params(B)(H, **f32) if D is not None else None,
         "z": torch.empty(B, L, H * P, **f32) if z is not None else None}
    ws = _ws(workspace, ssd_mixer_bwd_workspace_size(B, L, H, P, N, G, dtype), dev)
    st = lib.ssd_mixer_bwd(
        B, L, H, P, N, G, K, chunk, dtype, _ptr(xbc_raw, "xbc_raw"), rs_in, _ptr(conv_w, "conv_w", torch.float32),
        _ptr(conv_b, "conv_b", torch.float32), _ptr(dt_raw, "dt_raw", xbc_raw.dtype), rs_dt,
        _ptr(dt_bias, "dt_bias", torch.float32), _ptr(A, "A", torch.float32), _ptr(D, "D", torch.float32),
        _ptr(z, "z", xbc_raw.dtype), rs_z, _ptr(doc_ids, "doc_ids", torch.int32), int(act),
        _ptr(grad_y, "grad_y", torch.float32), rs_gy, _ptr(g["raw"], "dxbc_raw"), C, _ptr(g["w"], "dconv_w"),
        _ptr(g["bias"], "dconv_b"), _ptr(g["dt_raw"], "ddt_raw"), H, _ptr(g["dt_bias"], "ddt_bias"),
        _ptr(g["A"], "dA"), _ptr(g["D"], "dD"), _ptr(g["z"], "dz"), H * P, _ptr(ws, "workspace"),
        ws.numel() * ws.element_size(), _stream(stream))
    _check(st)
    return {k: v for k, v in g.items() if v is not None}


# ---- the gated delta rule and the row norm.  These calls run on the inputs' own GPU, whichever is current.
class _Call:
    """The device and the tensor checks of one call: every tensor has to be on the first input's GPU.  A small call's
    time is the host's, so tensors that are as expected take one test."""

    __slots__ = ("dev",)

    def __init__(self, x, name):
        _ptr(x, name)
        self.dev = x.device

    def ptr(self, t, name, dtype=None):
        if t is None:
            return None
        p = _ptr(t, name, dtype)
        if t.device != self.dev:
            raise ValueError(f"{name}: on {t.device}, expected {self.dev} as the first input")
        return p

    def vec(self, t, name, dtype, shape):
        if t is None:
            return None
        if t.shape == shape and t.dtype is dtype and t.device == self.dev and t.is_contiguous():
            return t.data_ptr()
        _contig(t, name, shape)
        return self.ptr(t, name, dtype)

    def rows(self, t, name, dtype, shape):
        """(pointer, row stride) of a tensor of `shape`, its rows a uniform number of elements apart; dtype None: any."""
        if t is None:
            return None, 0
        if t.shape == shape and t.device == self.dev and (t.dtype is dtype or dtype is None):
            if t.is_contiguous():
                return t.data_ptr(), shape[-1]
            st = t.stride()
            if st[-1] == 1:                           # columns of wider rows
                if len(st) == 2 and shape[0] > 1:
                    return t.data_ptr(), st[0]
                if len(st) == 3 and shape[1] > 1 and (shape[0] == 1 or st[0] == shape[1] * st[1]):
                    return t.data_ptr(), st[1]
        p = self.ptr(t, name, dtype)
        if t.shape != shape:
            raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
        if t.is_contiguous():
            return p, shape[-1]
        if t.stride(-1) != 1 and shape[-1] > 1:
            raise ValueError(f"{name}: the innermost dimension must be contiguous")
        # the row index runs over the leading dimensions: those of more than one entry must nest
        rs, step = None, 1
        for n, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
            if n == 1:
                continue
            if rs is None:
                rs = st
            elif st != rs * step:
                raise ValueError(f"{name}: batch rows must be L * row_stride elements apart")
            step *= n
        # a single row: any stride that holds it and keeps the alignment
        return p, (-(-shape[-1] // 8) * 8 if rs is None else rs)

    def run(self, fn, args):
        """fn(*args, stream) on the tensors' device and its current stream."""
        index = self.dev.index
        stream = torch._C._cuda_getCurrentRawStream(index)
        if index == torch._C._cuda_getDevice():
            st = fn(*args, stream)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, stream)
        if st:
            _check(st)


def _on_stream(fn):
    """A call with `stream`, a torch stream or a raw handle, makes it the current one, so that what the call allocates
    (outputs, a workspace that is free again on return) belongs to the stream that uses it.  A torch stream of another
    GPU than the tensors' is refused; a raw handle, which does not tell, is taken as one of theirs."""

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        at = next((t.device for t in (*args, *kw.values()) if isinstance(t, torch.Tensor) and t.is_cuda), None)
        if at is not None and getattr(stream, "device", at) != at:
            raise ValueError(f"stream: on {stream.device}, expected {at} as the tensors")
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=at)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    call.__doc__ = (fn.__doc__ or "") + "  stream: a torch stream or a raw handle, on the tensors' GPU, to run on in place of the current one."
    return call


def _delta_head(c, lead, T, q, k, v, dt, A, beta, H, P, N, G, scale, qk_norm, dt_softplus, dt_bias, beta_sigmoid):
    """The arguments that the delta calls share; lead: the dimensions before the columns, (B, L) or (B,)."""
    qp, qs = c.rows(q, "q", T, lead + (G * N,))
    kp, ks = c.rows(k, "k", T, lead + (G * N,))
    vp, vs = c.rows(v, "v", T, lead + (H * P,))
    dp, ds = c.rows(dt, "dt", torch.float32, lead + (H,))
    bp, bs = c.rows(beta, "beta", torch.float32, lead + (H,))
    return [qp, qs, kp, ks, vp, vs, dp, ds, int(bool(dt_softplus)), c.vec(dt_bias, "dt_bias", torch.float32, (H,)),
            c.vec(A, "A", torch.float32, (H,)), bp, bs, int(bool(beta_sigmoid)),
            N ** -0.5 if scale is None else float(scale), int(bool(qk_norm))]


def ssd_delta_scan_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_delta_scan_workspace_size(B, L, H, P, N, G, dtype))


@_on_stream
def ssd_delta_scan_fwd(q, k, v, dt, A, beta, *, H, P, N, G, scale=None, qk_norm=False, dt_softplus=False, dt_bias=None,
                       beta_sigmoid=False, doc_ids=None, lengths=None, init_state=None, final_state=None, y=None,
                       chunk=64, workspace=None):
    """The gated delta rule.  q, k [B, L, G*N], v [B, L, H*P] (one dtype), dt, beta [B, L, H] fp32, A [H] fp32.
    scale: N^-0.5 if None.  Returns y [B, L, H*P] in q's dtype (and writes final_state [B, H, P, N] if given).  A
    workspace is allocated here when none is passed."""
    lib = load()
    c = _Call(q, "q")
    dtype = _dtype_code(q, "q")
    B, L, T = q.shape[0], q.shape[1], q.dtype
    head = _delta_head(c, (B, L), T, q, k, v, dt, A, beta, H, P, N, G, scale, qk_norm, dt_softplus, dt_bias, beta_sigmoid)
    if y is None:
        y = torch.empty((B, L, H * P), dtype=T, device=c.dev)
    yp, ys = c.rows(y, "y", T, (B, L, H * P))
    ws = _ws(workspace, ssd_delta_scan_workspace_size(B, L, H, P, N, G, dtype), c.dev)
    state = (B, H, P, N)
    c.run(lib.ssd_delta_scan_fwd,
          (B, L, H, P, N, G, chunk, dtype, *head, c.vec(doc_ids, "doc_ids", torch.int32, (B, L)),
           c.vec(lengths, "lengths", torch.int32, (B,)), c.vec(init_state, "init_state", torch.float32, state),
           c.vec(final_state, "final_state", torch.float32, state), yp, ys, c.ptr(ws, "workspace"),
           ws.numel() * ws.element_size()))
    return y


@_on_stream
def ssd_delta_step(q, k, v, dt, A, beta, state, *, H, P, N, G, scale=None, qk_norm=False, dt_softplus=False,
                   dt_bias=None, beta_sigmoid=False, y=None):
    """One token of the gated delta rule.  q, k [B, G*N], v [B, H*P] (one dtype), dt, beta [B, H] fp32, A [H] fp32;
    state [B, H, P, N] fp32 is updated in place.  scale: N^-0.5 if None.  Returns y [B, H*P] in q's dtype."""
    lib = load()
    c = _Call(q, "q")
    dtype = _dtype_code(q, "q")
    B, T = q.shape[0], q.dtype
    head = _delta_head(c, (B,), T, q, k, v, dt, A, beta, H, P, N, G, scale, qk_norm, dt_softplus, dt_bias, beta_sigmoid)
    if y is None:
        y = torch.empty((B, H * P), dtype=T, device=c.dev)
    yp, ys = c.rows(y, "y", T, (B, H * P))
    c.run(lib.ssd_delta_step, (B, H, P, N, G, dtype, *head, c.vec(state, "state", torch.float32, (B, H, P, N)), yp, ys))
    return y


def _norm_groups(c, shape, tensors):
    """(rows, groups, strides by name) of norm operands: the last dimension is a group; where some operand's rows are not
    a uniform distance apart, the dimension before it holds the groups of a row (the heads of a token's row)."""
    W = shape[-1]
    n = 1
    for s in shape[:-1]:
        n *= s
    try:
        return n, 1, {name: c.rows(t, name, dtype, shape) for name, (t, dtype) in tensors.items()}
    except ValueError:
        # heads side by side: else flatten() below would hand the library a copy
        if len(shape) < 3 or any(t is not None and (t.shape != shape or t.stride(-2) != W or (W > 1 and t.stride(-1) != 1))
                                 for t, _ in tensors.values()):
            raise
    g = shape[-2]
    flat = shape[:-2] + (g * W,)
    return n // g, g, {name: c.rows(None if t is None else t.flatten(-2), name, dtype, flat)
                       for name, (t, dtype) in tensors.items()}


def ssd_delta_scan_bwd_workspace_size(B, L, H, P, N, G, dtype=SSD_BF16) -> int:
    return int(load().ssd_delta_scan_bwd_workspace_size(B, L, H, P, N, G, dtype))


@_on_stream
def ssd_delta_scan_bwd(q, k, v, dt, A, beta, grad_y, *, H, P, N, G, scale=None, qk_norm=False, dt_softplus=False,
                       dt_bias=None, beta_sigmoid=False, doc_ids=None, lengths=None, init_state=None,
                       grad_final_state=None, chunk=64, workspace=None):
    """Backward of ssd_delta_scan_fwd; grad_y [B, L, H*P] in q's dtype, grad_final_state [B, H, P, N] fp32 or None.
    Returns a dict: q, k, v in q's dtype, dt, beta [B, L, H] and A [H] fp32, and where those inputs are given (dt_bias:
    where dt_softplus is) dt_bias [H] and init_state [B, H, P, N] fp32.  A workspace is allocated here when none is
    passed."""
    lib = load()
    c = _Call(q, "q")
    dtype = _dtype_code(q, "q")
    B, L, T = q.shape[0], q.shape[1], q.dtype
    head = _delta_head(c, (B, L), T, q, k, v, dt, A, beta, H, P, N, G, scale, qk_norm, dt_softplus, dt_bias, beta_sigmoid)
    gp, gs = c.rows(grad_y, "grad_y", T, (B, L, H * P))
    f32, same, state = dict(dtype=torch.float32, device=c.dev), dict(dtype=T, device=c.dev), (B, H, P, N)
    g = {"q": torch.empty(B, L, G * N, **same), "k": torch.empty(B, L, G * N, **same),
         "v": torch.empty(B, L, H * P, **same), "dt": torch.empty(B, L, H, **f32), "beta": torch.empty(B, L, H, **f32),
         "A": _params(B)(H, **f32)}
    if dt_softplus:
        g["dt_bias"] = _params(B)(H, **f32)
    if init_state is not None:
        g["init_state"] = torch.empty(state, **f32)
    ws = _ws(workspace, ssd_delta_scan_bwd_workspace_size(B, L, H, P, N, G, dtype), c.dev)
    out = lambda n: g[n].data_ptr() if n in g else None  # noqa: E731
    c.run(lib.ssd_delta_scan_bwd,
          (B, L, H, P, N, G, chunk, dtype, *head, c.vec(doc_ids, "doc_ids", torch.int32, (B, L)),
           c.vec(lengths, "lengths", torch.int32, (B,)), c.vec(init_state, "init_state", torch.float32, state), gp, gs,
           c.vec(grad_final_state, "grad_final_state", torch.float32, state), out("q"), G * N, out("k"), G * N, out("v"),
           H * P, out("dt"), H, out("beta"), H, out("A"), out("dt_bias"), out("init_state"), c.ptr(ws, "workspace"),
           ws.numel() * ws.element_size()))
    return g


@_on_stream
def ssd_norm_fwd(x, weight=None, *, bias=None, z=None, rms=False, eps=1e-5, out_dtype=None, y=None):
    """Norm of x's last dimension, times weight plus bias, times silu(z).  x [..., W] fp32 or bf16, its rows a uniform
    distance apart, or [..., heads, W] with the heads of a row side by side; weight, bias fp32 [W]; z in the output's
    dtype, which is y's, else out_dtype, else z's, else x's.  Returns y."""
    lib = load()
    c = _Call(x, "x")
    shape, W = x.shape, x.shape[-1]
    T = y.dtype if y is not None else out_dtype or (x.dtype if z is None else z.dtype)
    if y is None:
        y = torch.empty(shape, dtype=T, device=c.dev)
    if x.numel() == 0:
        return y
    R, groups, at = _norm_groups(c, shape, {"x": (x, None), "z": (z, T), "y": (y, T)})
    c.run(lib.ssd_norm_fwd, (R, groups, W, _dtype_code(x, "x"), _dtype_code(y, "y"), int(bool(rms)), float(eps), *at["x"],
                             c.vec(weight, "weight", torch.float32, (W,)), c.vec(bias, "bias", torch.float32, (W,)),
                             *at["z"], *at["y"]))
    return y


def ssd_norm_bwd_workspace_size(R, groups, W) -> int:
    return int(load().ssd_norm_bwd_workspace_size(R, groups, W))


@_on_stream
def ssd_norm_bwd(x, grad_y, weight=None, *, bias=None, z=None, rms=False, eps=1e-5, workspace=None):
    """Backward of ssd_norm_fwd; grad_y (and z) in the output's dtype.  Returns a dict: x in x's dtype, weight and
    bias fp32 [W] and z in z's dtype, where those inputs are given.  A workspace is allocated here when none is
    passed."""
    lib = load()
    c = _Call(x, "x")
    shape, W, T = x.shape, x.shape[-1], grad_y.dtype
    f32 = dict(dtype=torch.float32, device=c.dev)
    g = {"x": torch.empty(shape, dtype=x.dtype, device=c.dev)}
    if weight is not None:
        g["weight"] = torch.empty(W, **f32)
    if bias is not None:
        g["bias"] = torch.empty(W, **f32)
    if z is not None:
        g["z"] = torch.empty(shape, dtype=T, device=c.dev)
    R, groups, at = _norm_groups(c, shape, {"x": (x, None), "z": (z, T), "grad_y": (grad_y, T), "dx": (g["x"], None),
                                            "dz": (g.get("z"), T)})
    ws, nb = None, 0
    if weight is not None or bias is not None:
        ws = _ws(workspace, ssd_norm_bwd_workspace_size(R, groups, W), c.dev)
        nb = ws.numel() * ws.element_size()
    out = lambda n: g[n].data_ptr() if n in g else None  # noqa: E731
    c.run(lib.ssd_norm_bwd, (R, groups, W, _dtype_code(x, "x"), _dtype_code(grad_y, "grad_y"), int(bool(rms)), float(eps),
                             *at["x"], c.vec(weight, "weight", torch.float32, (W,)),
                             c.vec(bias, "bias", torch.float32, (W,)), *at["z"], *at["grad_y"], *at["dx"], out("weight"),
                             out("bias"), *at["dz"], c.ptr(ws, "workspace"), nb))
    return g


# ---- the gated linear recurrence
def _like(t, dtype):
    """A contiguous output of t's shape: half the host's time of a shape spelt out, and small calls' time is the host's."""
    return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)


def _new(dev, lead, width, dtype):
    """A contiguous output of another width; two dimensions with their strides, which is the faster form too."""
    if len(lead) == 1:
        return torch.empty_strided((lead[0], width), (width, 1), dtype=dtype, device=dev)
    return torch.empty(lead + (width,), dtype=dtype, device=dev)


def _glr_head(c, lead, T, D, x, r, i, A, r_bias, i_bias):
    """The arguments that the recurrence's calls share; lead: the dimensions before the channels, (B, L) or (B,)."""
    return [*c.rows(x, "x", T, lead + (D,)), *c.rows(r, "r", T, lead + (D,)), *c.rows(i, "i", T, lead + (D,)),
            c.vec(r_bias, "r_bias", torch.float32, (D,)), c.vec(i_bias, "i_bias", torch.float32, (D,)),
            c.vec(A, "A", torch.float32, (D,))]


def ssd_glr_scan_workspace_size(B, L, D, dtype=SSD_BF16) -> int:
    return int(load().ssd_glr_scan_workspace_size(B, L, D, dtype))


@_on_stream
def ssd_glr_scan_fwd(x, r, i, A, *, r_bias=None, i_bias=None, doc_ids=None, lengths=None, init_state=None,
                     final_state=None, chunk_states=None, y=None, workspace=None):
    """The gated linear recurrence h <- a h + sqrt(1 - a^2) sigmoid(i + i_bias) x, a = exp(sigmoid(r + r_bias) A).
    x, r, i [B, L, D] (one dtype), A, r_bias, i_bias [D] fp32.  Returns y [B, L, D] in x's dtype (and writes final_state
    [B, D] and chunk_states [B, ceil(L / 64), D], fp32, if given).  A workspace is allocated here when none is passed."""
    lib = load()
    c = _Call(x, "x")
    dtype, T = _dtype_code(x, "x"), x.dtype
    B, L, D = x.shape
    head = _glr_head(c, (B, L), T, D, x, r, i, A, r_bias, i_bias)
    if y is None:
        y = _like(x, T)
    yp, ys = c.rows(y, "y", T, (B, L, D))
    need = ssd_glr_scan_workspace_size(B, L, D, dtype)
    ws = _ws(workspace, need, c.dev) if need or workspace is not None else None
    c.run(lib.ssd_glr_scan_fwd,
          (B, L, D, dtype, *head, c.vec(doc_ids, "doc_ids", torch.int32, (B, L)),
           c.vec(lengths, "lengths", torch.int32, (B,)), c.vec(init_state, "init_state", torch.float32, (B, D)),
           c.vec(final_state, "final_state", torch.float32, (B, D)),
           c.vec(chunk_states, "chunk_states", torch.float32, (B, -(-L // 64), D)), yp, ys, c.ptr(ws, "workspace"),
           0 if ws is None else ws.numel() * ws.element_size()))
    return y


@_on_stream
def ssd_glr_step(x, r, i, A, state, *, r_bias=None, i_bias=None, y=None):
    """One token of the gated linear recurrence.  x, r, i [B, D] (one dtype), A, r_bias, i_bias [D] fp32; state [B, D]
    fp32 is updated in place.  Returns y [B, D] in x's dtype."""
    lib = load()
    c = _Call(x, "x")
    dtype, T = _dtype_code(x, "x"), x.dtype
    B, D = x.shape
    head = _glr_head(c, (B,), T, D, x, r, i, A, r_bias, i_bias)
    if y is None:
        y = _like(x, T)
    yp, ys = c.rows(y, "y", T, (B, D))
    c.run(lib.ssd_glr_step, (B, D, dtype, *head, c.vec(state, "state", torch.float32, (B, D)), yp, ys))
    return y


def ssd_glr_scan_bwd_workspace_size(B, L, D, dtype=SSD_BF16) -> int:
    return int(load().ssd_glr_scan_bwd_workspace_size(B, L, D, dtype))


@_on_stream
def ssd_glr_scan_bwd(x, r, i, A, grad_y, *, r_bias=None, i_bias=None, doc_ids=None, lengths=None, init_state=None,
                     grad_final_state=None, chunk_states=None, workspace=None):
    """Backward of ssd_glr_scan_fwd; grad_y [B, L, D] in x's dtype, grad_final_state [B, D] fp32 or None, chunk_states as
    the forward wrote them for these inputs (None: computed again).  Returns a dict: x, r, i in x's dtype, A [D] fp32, and
    where those inputs are given r_bias, i_bias [D] and init_state [B, D] fp32.  A workspace is allocated here when none
    is passed."""
    lib = load()
    c = _Call(x, "x")
    dtype, T = _dtype_code(x, "x"), x.dtype
    B, L, D = x.shape
    head = _glr_head(c, (B, L), T, D, x, r, i, A, r_bias, i_bias)
    gp, gs = c.rows(grad_y, "grad_y", T, (B, L, D))
    f32 = torch.float32
    g = {"x": _like(x, T), "r": _like(x, T), "i": _like(x, T)}
    for n, v in (("A", A), ("r_bias", r_bias), ("i_bias", i_bias)):
        if v is not None:
            g[n] = _like(v, f32) if B else torch.zeros(D, dtype=f32, device=c.dev)
    if init_state is not None:
        g["init_state"] = _like(init_state, f32)
    ws = _ws(workspace, ssd_glr_scan_bwd_workspace_size(B, L, D, dtype), c.dev)
    out = lambda n: g[n].data_ptr() if n in g else None  # noqa: E731
    c.run(lib.ssd_glr_scan_bwd,
          (B, L, D, dtype, *head, c.vec(doc_ids, "doc_ids", torch.int32, (B, L)),
           c.vec(lengths, "lengths", torch.int32, (B,)), c.vec(init_state, "init_state", torch.float32, (B, D)),
           c.vec(chunk_states, "chunk_states", torch.float32, (B, -(-L // 64), D)), gp, gs,
           c.vec(grad_final_state, "grad_final_state", torch.float32, (B, D)), out("x"), D, out("r"), D, out("i"), D,
           out("A"), out("r_bias"), out("i_bias"), out("init_state"), c.ptr(ws, "workspace"),
           ws.numel() * ws.element_size()))
    return g


# ---- the norm with the residual's addition and 8-bit output
def _lead_rows(shape):
    n = 1
    for s in shape[:-1]:
        n *= s
    return n


@_on_stream
def ssd_add_norm_fwd(x, residual=None, weight=None, *, bias=None, z=None, rms=False, eps=1e-5, out_dtype=None, want_y=True,
                     want_q=False, sum=None, y=None, q=None, q_scale=None):
    """Norm of x + residual, times weight plus bias, times silu(z), in the output's type and in 8 bits.  x, residual
    [..., W] fp32 or bf16, weight, bias fp32 [W], z in the output's dtype, which is y's, else out_dtype, else z's, else
    x's.  Returns a dict: "sum" in the residual's dtype where there is one, "y" unless want_y is false, and with want_q
    "q" (float8_e4m3fn) and "scale" (fp32 [..., ceil(W / 128)]).  Outputs may be given: sum (the residual itself: in
    place), y, q, q_scale."""
    lib = load()
    c = _Call(x, "x")
    shape, W = x.shape, x.shape[-1]
    T = y.dtype if y is not None else out_dtype or (x.dtype if z is None else z.dtype)
    if (want_y or y is not None) and y is None:
        y = _like(x, T)
    blocks = shape[:-1] + (-(-W // 128),)
    if want_q or q is not None or q_scale is not None:
        q = _like(x, torch.float8_e4m3fn) if q is None else q
        q_scale = _new(c.dev, shape[:-1], blocks[-1], torch.float32) if q_scale is None else q_scale
    RT = x.dtype if residual is None else residual.dtype
    if residual is not None and sum is None:
        sum = _like(x, RT)
    out = {n: t for n, t in (("sum", sum), ("y", y), ("q", q), ("scale", q_scale)) if t is not None}
    if x.numel() == 0:
        return out
    code = SSD_F32 if T == torch.float32 else SSD_BF16 if T == torch.bfloat16 else -1
    c.run(lib.ssd_add_norm_fwd,
          (_lead_rows(shape), W, _dtype_code(x, "x"), _dtype_code(x if residual is None else residual, "residual"), code,
           int(bool(rms)), float(eps), *c.rows(x, "x", None, shape), *c.rows(residual, "residual", None, shape),
           c.vec(weight, "weight", torch.float32, (W,)), c.vec(bias, "bias", torch.float32, (W,)), *c.rows(z, "z", T, shape),
           *c.rows(sum, "sum", RT, shape), *c.rows(y, "y", T, shape), *c.rows(q, "q", torch.float8_e4m3fn, shape),
           *c.rows(q_scale, "q_scale", torch.float32, blocks)))
    return out


@_on_stream
def ssd_add_norm_bwd(sum, grad_y, grad_sum=None, weight=None, *, bias=None, z=None, rms=False, eps=1e-5, workspace=None):
    """Backward of ssd_add_norm_fwd from its sum; grad_y (and z) in the output's dtype, grad_sum, what reaches the sum past
    the norm, in sum's.  Returns a dict: sum (the gradient of x and of the residual alike) in sum's dtype, weight and bias
    fp32 [W] and z in z's dtype, where those inputs are given.  A workspace is allocated here when none is passed."""
    lib = load()
    c = _Call(sum, "sum")
    shape, W, T = sum.shape, sum.shape[-1], grad_y.dtype
    R = _lead_rows(shape)
    g = {"sum": _like(sum, sum.dtype)}
    if weight is not None:
        g["weight"] = _like(weight, torch.float32)
    if bias is not None:
        g["bias"] = _like(bias, torch.float32)
    if z is not None:
        g["z"] = _like(sum, T)
    ws, nb = None, 0
    if weight is not None or bias is not None:
        ws = _ws(workspace, ssd_norm_bwd_workspace_size(R, 1, W), c.dev)
        nb = ws.numel() * ws.element_size()
    out = lambda n: g[n].data_ptr() if n in g else None  # noqa: E731
    c.run(lib.ssd_add_norm_bwd,
          (R, W, _dtype_code(sum, "sum"), _dtype_code(grad_y, "grad_y"), int(bool(rms)), float(eps),
           *c.rows(sum, "sum", None, shape), c.vec(weight, "weight", torch.float32, (W,)),
           c.vec(bias, "bias", torch.float32, (W,)), *c.rows(z, "z", T, shape), *c.rows(grad_y, "grad_y", T, shape),
           *c.rows(grad_sum, "grad_sum", sum.dtype, shape), out("sum"), W, out("weight"), out("bias"), out("z"), W,
           c.ptr(ws, "workspace"), nb))
    return g


# ---- the 8-bit projection
def ssd_proj_fp8_tile_rows(M, N, K, dtype=SSD_BF16) -> int:
    """Rows of y of a workgroup of the kernel for these sizes (16, 32, 64, 128 or 256), 0 where there is none; dtype: y's."""
    return int(load().ssd_proj_fp8_tile_rows(M, N, K, dtype))


@_on_stream
def ssd_proj_fp8_fwd(a, a_scale, w, w_scale, *, out_dtype=torch.bfloat16, y=None):
    """a times w transposed in float8_e4m3fn with a scale for every block of 128.  a [..., K] with a_scale fp32
    [..., ceil(K / 128)] (ssd_add_norm_fwd's "q" and "scale"), w [N, K] with w_scale fp32 [ceil(N / 128), ceil(K / 128)].
    Returns y [..., N] in y's dtype, else out_dtype."""
    lib = load()
    c = _Call(a, "a")
    lead, K, N = a.shape[:-1], a.shape[-1], w.shape[0]
    blocks = -(-K // 128)
    T = out_dtype if y is None else y.dtype
    if y is None:
        y = _new(c.dev, lead, N, T)
    c.run(lib.ssd_proj_fp8_fwd,
          (_lead_rows(a.shape), N, K, _dtype_code(y, "y"), *c.rows(a, "a", torch.float8_e4m3fn, a.shape),
           *c.rows(a_scale, "a_scale", torch.float32, lead + (blocks,)), *c.rows(w, "w", torch.float8_e4m3fn, (N, K)),
           *c.rows(w_scale, "w_scale", torch.float32, (-(-N // 128), blocks)), *c.rows(y, "y", T, lead + (N,))))
    return y
