"""Bindings of the operators around a linear-attention layer (include/gdnqat.h): linear attention
with a decay for each head, the gated norm behind it and the residual norm between blocks.

As in gdnqat.py: argument marshalling only, no fallback. Outputs and workspaces that are not given
are allocated on the stream that the call runs on. The small calls take a few microseconds on the
GPU, so the common case (current device, current stream) does nothing but check, allocate and call.
"""
from __future__ import annotations

import ctypes

import torch

from .gdnqat import LaArgs, LaGrads, _check, _state_flags, load

LA_FLAG_HEAD_DECAY = 1
_BF16, _F32 = torch.bfloat16, torch.float32
_DTYPES = {_BF16: 0, _F32: 1}
_byref = ctypes.byref
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _elsewhere(fn, t, stream, *args, **kw):
    """The call on another stream or device than the current ones: made current around it, so that its
    allocations belong to that stream too."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    with torch.cuda.device(t.device):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)


def _is(t, dtype, shape, dev, name):
    """The address of a contiguous CUDA tensor of this type, shape and device (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on device {dev}, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _code(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return code


def _workspace(given, need, device):
    if given is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return given


def _room(ws, dev):
    """Address and size of a workspace."""
    return _is(ws, torch.uint8, ws.shape, dev, "workspace"), ws.numel()


def _cu_host(cu_seqlens):
    return cu_seqlens.detach().to("cpu", torch.int32).contiguous()


def _la_args(q, k, v, g, h0, cu_seqlens, scale, dev):
    """The argument structure without its outputs, and the host and device cu_seqlens that must outlive the call."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, D]")
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    head = g.dim() == 1
    cu_host = cu_dev = None
    N = B
    if cu_seqlens is not None:
        cu_host = _cu_host(cu_seqlens)
        # from pageable memory: staged before the copy returns, without waiting for the stream
        cu_dev = (cu_seqlens if cu_seqlens.is_cuda else cu_host).to(q.device, torch.int32, non_blocking=True).contiguous()
        N = cu_host.numel() - 1
    a = LaArgs(_is(q, _BF16, q.shape, dev, "q"), _is(k, _BF16, q.shape, dev, "k"),
               _is(v, _BF16, (B, T, Hv, dv), dev, "v"), _is(g, _F32, (Hv,) if head else (B, T, Hv), dev, "g"),
               _is(h0, _F32, (N, Hv, dk, dv), dev, "h0"), None if cu_dev is None else cu_dev.data_ptr(),
               None if cu_host is None else cu_host.data_ptr(), None, None, B, T, N, Hqk, Hv, dk, dv, float(scale),
               LA_FLAG_HEAD_DECAY if head else 0)
    return a, (N, Hv, dk, dv), (cu_host, cu_dev)


def la_chunk_workspace_bytes(q_shape, v_shape, cu_seqlens=None, *, head_decay=False, backward=False):
    """la_chunk_fwd_workspace_size (backward: la_chunk_bwd_workspace_size) for q [B,T,Hqk,dk] and v
    [B,T,Hv,dv] (shapes only); 0 for shapes that the calls refuse."""
    B, T, Hqk, dk = q_shape
    Hv, dv = v_shape[2], v_shape[3]
    cu_host, N = None, B
    if cu_seqlens is not None:
        cu_host = _cu_host(cu_seqlens)
        N = cu_host.numel() - 1
    at = None if cu_host is None else cu_host.data_ptr()
    a = LaArgs(None, None, None, None, None, at, at, None, None, B, T, N, Hqk, Hv, dk, dv, 1.0,
               LA_FLAG_HEAD_DECAY if head_decay else 0)
    fn = "la_chunk_bwd_workspace_size" if backward else "la_chunk_fwd_workspace_size"
    return int(getattr(load(), fn)(_byref(a)))


def la_chunk_fwd(q, k, v, g, h0=None, cu_seqlens=None, *, scale=1.0, o=None, hT=None, output_final_state=True,
                 workspace=None, stream=None):
    """Linear attention with a decay for each head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
    q, k [B,T,Hqk,dk] bf16; v [B,T,Hv,dv] bf16 (value head h reads q/k head h // (Hv // Hqk)); g
    [B,T,Hv] fp32, or [Hv] for one fixed decay per head; h0 [N,Hv,dk,dv] fp32 or None; cu_seqlens int32
    [N+1] (CPU or CUDA) of sequences packed on the T axis of B = 1, or None. dk, dv in {64, 128}.
    Returns (o [B,T,Hv,dv] bf16, hT [N,Hv,dk,dv] fp32 or None)."""
    dev = q.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(la_chunk_fwd, q, stream, q, k, v, g, h0, cu_seqlens, scale=scale, o=o, hT=hT,
                          output_final_state=output_final_state, workspace=workspace)
    lib = load()
    a, state, _keep = _la_args(q, k, v, g, h0, cu_seqlens, scale, dev)
    if o is None:
        o = torch.empty_like(v)
    if hT is None and output_final_state:
        hT = torch.empty(state, dtype=_F32, device=q.device)
    a.o, a.hT = _is(o, _BF16, v.shape, dev, "o"), _is(hT, _F32, state, dev, "hT")
    ws = _workspace(workspace, lib.la_chunk_fwd_workspace_size(_byref(a)), q.device)
    st = lib.la_chunk_fwd(_byref(a), *_room(ws, dev), _raw_stream(dev))
    if st:
        _check("la_chunk_fwd", st)
    return o, hT


def la_chunk_bwd(q, k, v, g, h0=None, cu_seqlens=None, dout=None, dhT=None, *, scale=1.0, want_dh0=True,
                 workspace=None, stream=None):
    """Gradients of <o, dout> + <hT, dhT> of la_chunk_fwd with the same inputs. dout [B,T,Hv,dv] bf16;
    dhT [N,Hv,dk,dv] fp32 or None. Returns (dq, dk, dv bf16, dg fp32 of g's shape, dh0 [N,Hv,dk,dv]
    fp32 or None unless want_dh0); dq and dk are summed over the value heads that share a q/k head."""
    dev = q.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(la_chunk_bwd, q, stream, q, k, v, g, h0, cu_seqlens, dout, dhT, scale=scale,
                          want_dh0=want_dh0, workspace=workspace)
    lib = load()
    if dout is None:
        raise ValueError("dout is required")
    a, state, _keep = _la_args(q, k, v, g, h0, cu_seqlens, scale, dev)
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(g)
    dh0 = torch.empty(state, dtype=_F32, device=q.device) if want_dh0 else None
    gr = LaGrads(_is(dout, _BF16, v.shape, dev, "dout"), _is(dhT, _F32, state, dev, "dhT"), dq.data_ptr(), dk.data_ptr(),
                 dv.data_ptr(), dg.data_ptr(), None if dh0 is None else dh0.data_ptr())
    ws = _workspace(workspace, lib.la_chunk_bwd_workspace_size(_byref(a)), q.device)
    st = lib.la_chunk_bwd(_byref(a), _byref(gr), *_room(ws, dev), _raw_stream(dev))
    if st:
        _check("la_chunk_bwd", st)
    return dq, dk, dv, dg, dh0


def la_decode_step(q, k, v, g, state, *, state_out=None, state_qdq=True, scale=1.0, o=None, stream=None,
                   codec="e4m3"):
    """One token per sequence of la_chunk_fwd's recurrence. q, k [N,Hqk,dk] bf16; v [N,Hv,dv] bf16; g
    [N,Hv] fp32; state [N,Hv,dk,dv] fp32, updated in place unless state_out receives the new one. o is
    taken from the updated state before its QDQ (state_qdq; codec "e4m3" tiles or "int8" blocks).
    Returns o [N,Hv,dv] bf16."""
    flags = _state_flags(state_qdq, codec)
    dev = q.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(la_decode_step, q, stream, q, k, v, g, state, state_out=state_out, state_qdq=state_qdq,
                          scale=scale, o=o, codec=codec)
    lib = load()
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [N, H, D]")
    N, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    full = (N, Hv, dk, dv)
    if o is None:
        o = torch.empty_like(v)
    at = _is(state, _F32, full, dev, "state")
    st = lib.la_decode_step(_is(q, _BF16, q.shape, dev, "q"), _is(k, _BF16, q.shape, dev, "k"),
                            _is(v, _BF16, (N, Hv, dv), dev, "v"), _is(g, _F32, (N, Hv), dev, "g"), at,
                            at if state_out is None else _is(state_out, _F32, full, dev, "state_out"),
                            _is(o, _BF16, v.shape, dev, "o"), N, Hqk, Hv, dk, dv, float(scale), flags, _raw_stream(dev))
    if st:
        _check("la_decode_step", st)
    return o


def _rows(x):
    if x.dim() == 0:
        raise ValueError("the normalised tensor needs a last dimension")
    D = x.shape[-1]
    return (x.numel() // D if D else 0), D


def gated_norm_fwd(x, z, w, *, eps=1e-6, y=None, stream=None):
    """y = rms(x) w silu(z) over the last dimension, rms(x) = x / sqrt(mean(x^2) + eps): the norm behind
    a mixing core (one row per token and head) and its gate. x [..., D] bf16 or fp32; z [..., D] bf16;
    w [D] bf16 or fp32. Returns y [..., D] bf16."""
    dev = x.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(gated_norm_fwd, x, stream, x, z, w, eps=eps, y=y)
    lib = load()
    tx, tw = _code(x, "x"), _code(w, "w")
    rows, D = _rows(x)
    if y is None:
        y = torch.empty_like(z)
    st = lib.gated_norm_fwd(_is(x, x.dtype, x.shape, dev, "x"), tx, _is(z, _BF16, x.shape, dev, "z"),
                            _is(w, w.dtype, (D,), dev, "w"), tw, _is(y, _BF16, x.shape, dev, "y"), rows, D, float(eps),
                            _raw_stream(dev))
    if st:
        _check("gated_norm_fwd", st)
    return y


def gated_norm_bwd(dy, x, z, w, *, eps=1e-6, workspace=None, stream=None):
    """Gradients of gated_norm_fwd: dy [..., D] bf16. Returns (dx of x's type, dz bf16, dw [D] fp32)."""
    dev = x.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(gated_norm_bwd, x, stream, dy, x, z, w, eps=eps, workspace=workspace)
    lib = load()
    tx, tw = _code(x, "x"), _code(w, "w")
    rows, D = _rows(x)
    dx, dz = torch.empty_like(x), torch.empty_like(z)
    dw = torch.empty(D, dtype=_F32, device=x.device)
    ws = _workspace(workspace, lib.gated_norm_bwd_workspace_size(rows, D), x.device)
    st = lib.gated_norm_bwd(_is(dy, _BF16, x.shape, dev, "dy"), _is(x, x.dtype, x.shape, dev, "x"), tx,
                            _is(z, _BF16, x.shape, dev, "z"), _is(w, w.dtype, (D,), dev, "w"), tw, dx.data_ptr(),
                            dz.data_ptr(), dw.data_ptr(), rows, D, float(eps), *_room(ws, dev), _raw_stream(dev))
    if st:
        _check("gated_norm_bwd", st)
    return dx, dz, dw


def _weights(w_pre, w_post, D, dev):
    """Their type code and addresses."""
    tw = _code(w_pre, "w_pre")
    return tw, _is(w_pre, w_pre.dtype, (D,), dev, "w_pre"), _is(w_post, w_pre.dtype, (D,), dev, "w_post (as w_pre)")


def residual_norm_fwd(y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, h_out=None, x=None, stream=None):
    """h_out = h + alpha n, n = rms(y) w_post (w_post None: n = y); x = rms(h_out) w_pre: the norm after a
    block, its scaled residual and the norm before the next block. y [..., D] bf16 (the block's output);
    h [..., D] bf16 or fp32 (the residual stream); w_pre, w_post [D], both bf16 or both fp32. h_out may
    be h. Returns (h_out of h's type, x bf16)."""
    dev = h.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(residual_norm_fwd, h, stream, y, h, w_pre, w_post, alpha=alpha, eps=eps, h_out=h_out, x=x)
    lib = load()
    th = _code(h, "h")
    rows, D = _rows(h)
    tw, w1, w2 = _weights(w_pre, w_post, D, dev)
    if h_out is None:
        h_out = torch.empty_like(h)
    if x is None:
        x = torch.empty_like(y)
    st = lib.residual_norm_fwd(_is(y, _BF16, h.shape, dev, "y"), _is(h, h.dtype, h.shape, dev, "h"), th, w2, w1, tw,
                               _is(h_out, h.dtype, h.shape, dev, "h_out"), _is(x, _BF16, h.shape, dev, "x"), rows, D,
                               float(alpha), float(eps), _raw_stream(dev))
    if st:
        _check("residual_norm_fwd", st)
    return h_out, x


def residual_norm_bwd(dx, dh_out, y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, workspace=None, stream=None):
    """Gradients of residual_norm_fwd with the same y, h, w_pre, w_post. dx [..., D] bf16; dh_out [..., D] of
    h's type or None (zero). Returns (dy bf16, dh of h's type, dw_pre [D] fp32, dw_post [D] fp32 or None)."""
    dev = h.get_device()
    if stream is not None or dev != _device():
        return _elsewhere(residual_norm_bwd, h, stream, dx, dh_out, y, h, w_pre, w_post, alpha=alpha, eps=eps,
                          workspace=workspace)
    lib = load()
    th = _code(h, "h")
    rows, D = _rows(h)
    tw, w1, w2 = _weights(w_pre, w_post, D, dev)
    dy, dh = torch.empty_like(y), torch.empty_like(h)
    dw_pre = torch.empty(D, dtype=_F32, device=h.device)
    dw_post = torch.empty_like(dw_pre) if w_post is not None else None
    ws = _workspace(workspace, lib.residual_norm_bwd_workspace_size(rows, D), h.device)
    st = lib.residual_norm_bwd(_is(dx, _BF16, h.shape, dev, "dx"), _is(dh_out, h.dtype, h.shape, dev, "dh_out"),
                               _is(y, _BF16, h.shape, dev, "y"), _is(h, h.dtype, h.shape, dev, "h"), th, w2, w1, tw,
                               dy.data_ptr(), dh.data_ptr(), None if dw_post is None else dw_post.data_ptr(),
                               dw_pre.data_ptr(), rows, D, float(alpha), float(eps),
                               *_room(ws, dev), _raw_stream(dev))
    if st:
        _check("residual_norm_bwd", st)
    return dy, dh, dw_pre, dw_post
