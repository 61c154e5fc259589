"""Bindings of the operators around a linear-attention layer (include/gdnqat.h): linear attention
with a decay for each head, the gated norm behind it and the residual norm between blocks.

Argument checks, allocations and the call itself are in the extension csrc/layer_ext.cpp: the small calls take a
few microseconds on the GPU, less than the same checks in Python. There is no fallback. Outputs and workspaces
that are not given are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import ctypes
import importlib.util
import threading

import torch

from . import build as _build
from .gdnqat import LaArgs, _check, _state_flags, load

LA_FLAG_HEAD_DECAY = 1
_ENTRIES = ("la_chunk_fwd", "la_chunk_fwd_workspace_size", "la_chunk_bwd", "la_chunk_bwd_workspace_size",
            "gdn_upload_i32", "la_decode_step", "gated_norm_fwd", "gated_norm_bwd", "gated_norm_bwd_workspace_size", "residual_norm_fwd",
            "residual_norm_bwd", "residual_norm_bwd_workspace_size")


_lock = threading.Lock()


class _Unloaded:
    """Stands for the extension until its first use, which loads it and the library (building what is missing)."""

    def __getattr__(self, name):
        global _ext
        lib = load()
        with _lock:
            if _ext is self:
                spec = importlib.util.spec_from_file_location("gdnqat_layer", _build.build_extension())
                ext = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(ext)
                ext.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES}, _check)
                _ext = ext
        return getattr(_ext, name)


_ext = _Unloaded()


def _elsewhere(fn, t, stream, *args, **kw):
    """The call on another stream or device than the current ones: made current around it, so that its
    allocations belong to that stream too."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)


def la_chunk_workspace_bytes(q_shape, v_shape, cu_seqlens=None, *, head_decay=False, backward=False):
    """la_chunk_fwd_workspace_size (backward: la_chunk_bwd_workspace_size) for q [B,T,Hqk,dk] and v
    [B,T,Hv,dv] (shapes only; of cu_seqlens only the number of sequences matters); 0 for shapes that the calls
    refuse."""
    B, T, Hqk, dk = q_shape
    Hv, dv = v_shape[2], v_shape[3]
    cu_host, N = None, B
    if cu_seqlens is not None:
        cu_host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
        N = cu_host.numel() - 1
    at = None if cu_host is None else cu_host.data_ptr()
    a = LaArgs(None, None, None, None, None, at, at, None, None, B, T, N, Hqk, Hv, dk, dv, 1.0,
               LA_FLAG_HEAD_DECAY if head_decay else 0)
    fn = "la_chunk_bwd_workspace_size" if backward else "la_chunk_fwd_workspace_size"
    return int(getattr(load(), fn)(ctypes.byref(a)))


def la_chunk_fwd(q, k, v, g, h0=None, cu_seqlens=None, *, scale=1.0, o=None, hT=None, output_final_state=True,
                 workspace=None, stream=None):
    """Linear attention with a decay for each head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
    q, k [B,T,Hqk,dk] bf16; v [B,T,Hv,dv] bf16 (value head h reads q/k head h // (Hv // Hqk)); g
    [B,T,Hv] fp32, or [Hv] for one fixed decay per head; h0 [N,Hv,dk,dv] fp32 or None; cu_seqlens [N+1] of
    whole numbers of sequences packed on the T axis of B = 1, or None: read before the call returns, by waiting for
    the stream where it is a CUDA tensor, which a captured call therefore refuses. dk, dv in {64, 128}.
    Returns (o [B,T,Hv,dv] bf16, hT [N,Hv,dk,dv] fp32 or None)."""
    if stream is None:
        r = _ext.la_chunk_fwd(q, k, v, g, h0, cu_seqlens, scale, o, hT, output_final_state, workspace)
        if r is not NotImplemented:
            return r
    return _elsewhere(la_chunk_fwd, q, stream, q, k, v, g, h0, cu_seqlens, scale=scale, o=o, hT=hT,
                      output_final_state=output_final_state, workspace=workspace)


def la_chunk_bwd(q, k, v, g, h0=None, cu_seqlens=None, dout=None, dhT=None, *, scale=1.0, want_dh0=True,
                 workspace=None, stream=None):
    """Gradients of <o, dout> + <hT, dhT> of la_chunk_fwd with the same inputs. dout [B,T,Hv,dv] bf16;
    dhT [N,Hv,dk,dv] fp32 or None. Returns (dq, dk, dv bf16, dg fp32 of g's shape, dh0 [N,Hv,dk,dv]
    fp32 or None unless want_dh0); dq and dk are summed over the value heads that share a q/k head."""
    if stream is None:
        r = _ext.la_chunk_bwd(q, k, v, g, h0, cu_seqlens, dout, dhT, scale, want_dh0, workspace)
        if r is not NotImplemented:
            return r
    return _elsewhere(la_chunk_bwd, q, stream, q, k, v, g, h0, cu_seqlens, dout, dhT, scale=scale, want_dh0=want_dh0,
                      workspace=workspace)


def la_decode_step(q, k, v, g, state, *, state_out=None, state_qdq=True, scale=1.0, o=None, stream=None,
                   codec="e4m3"):
    """One token per sequence of la_chunk_fwd's recurrence. q, k [N,Hqk,dk] bf16; v [N,Hv,dv] bf16; g
    [N,Hv] fp32; state [N,Hv,dk,dv] fp32, updated in place unless state_out receives the new one. o is
    taken from the updated state before its QDQ (state_qdq; codec "e4m3" tiles or "int8" blocks).
    Returns o [N,Hv,dv] bf16."""
    if stream is None:
        r = _ext.la_decode_step(q, k, v, g, state, state_out, _state_flags(state_qdq, codec), scale, o)
        if r is not NotImplemented:
            return r
    return _elsewhere(la_decode_step, q, stream, q, k, v, g, state, state_out=state_out, state_qdq=state_qdq,
                      scale=scale, o=o, codec=codec)


def gated_norm_fwd(x, z, w, *, eps=1e-6, y=None, stream=None):
    """y = rms(x) w silu(z) over the last dimension, rms(x) = x / sqrt(mean(x^2) + eps): the norm behind
    a mixing core (one row per token and head) and its gate. x [..., D] bf16 or fp32; z [..., D] bf16;
    w [D] bf16 or fp32. Returns y [..., D] bf16."""
    if stream is None:
        r = _ext.gated_norm_fwd(x, z, w, eps, y)
        if r is not NotImplemented:
            return r
    return _elsewhere(gated_norm_fwd, x, stream, x, z, w, eps=eps, y=y)


def gated_norm_bwd(dy, x, z, w, *, eps=1e-6, workspace=None, stream=None):
    """Gradients of gated_norm_fwd: dy [..., D] bf16. Returns (dx of x's type, dz bf16, dw [D] fp32)."""
    if stream is None:
        r = _ext.gated_norm_bwd(dy, x, z, w, eps, workspace)
        if r is not NotImplemented:
            return r
    return _elsewhere(gated_norm_bwd, x, stream, dy, x, z, w, eps=eps, workspace=workspace)


def residual_norm_fwd(y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, h_out=None, x=None, stream=None):
    """h_out = h + alpha n, n = rms(y) w_post (w_post None: n = y); x = rms(h_out) w_pre: the norm after a
    block, its scaled residual and the norm before the next block. y [..., D] bf16 (the block's output);
    h [..., D] bf16 or fp32 (the residual stream); w_pre, w_post [D], both bf16 or both fp32. h_out may
    be h. Returns (h_out of h's type, x bf16)."""
    if stream is None:
        r = _ext.residual_norm_fwd(y, h, w_pre, w_post, alpha, eps, h_out, x)
        if r is not NotImplemented:
            return r
    return _elsewhere(residual_norm_fwd, h, stream, y, h, w_pre, w_post, alpha=alpha, eps=eps, h_out=h_out, x=x)


def residual_norm_bwd(dx, dh_out, y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, workspace=None, stream=None):
    """Gradients of residual_norm_fwd with the same y, h, w_pre, w_post. dx [..., D] bf16; dh_out [..., D] of
    h's type or None (zero). Returns (dy bf16, dh of h's type, dw_pre [D] fp32, dw_post [D] fp32 or None)."""
    if stream is None:
        r = _ext.residual_norm_bwd(y, h, w_pre, w_post, alpha, eps, dx, dh_out, workspace)
        if r is not NotImplemented:
            return r
    return _elsewhere(residual_norm_bwd, h, stream, dx, dh_out, y, h, w_pre, w_post, alpha=alpha, eps=eps,
                      workspace=workspace)
