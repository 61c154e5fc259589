"""Bindings of the operators around a linear-attention layer (include/gdnqat.h): linear attention
with a decay for each head, the gated norm behind it and the residual norm between blocks.

As in gdnqat.py: argument marshalling only, no fallback. Outputs and workspaces that are not given
are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from .gdnqat import LaArgs, LaGrads, _check, _dev, _ptr, _state_flags, load

LA_FLAG_HEAD_DECAY = 1
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


@contextlib.contextmanager
def _on(device, stream):
    """The device and the stream of a call, so that its allocations belong to that stream."""
    if device.type != "cuda":
        raise ValueError(f"tensors must be CUDA tensors, got one on {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
        else:
            with torch.cuda.stream(stream):
                yield ctypes.c_void_p(stream.cuda_stream)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _shaped(t, shape, name):
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _workspace(given, need, device):
    if given is None:
        return torch.empty(max(need, 256), dtype=torch.uint8, device=device)
    return _dev(given, torch.uint8, "workspace")


def _la_args(q, k, v, g, h0, cu_seqlens, scale):
    """The argument structure without its outputs, N, and the host and device cu_seqlens that must
    outlive the call."""
    q, k, v = (_dev(t, torch.bfloat16, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    g, h0 = _dev(g, torch.float32, "g"), _dev(h0, torch.float32, "h0")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, D]")
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    _shaped(k, q.shape, "k")
    _shaped(v, (B, T, Hv, dv), "v")
    head = g.dim() == 1
    _shaped(g, (Hv,) if head else (B, T, Hv), "g")
    _same_device(q.device, k=k, v=v, g=g, h0=h0)
    cu_host = cu_dev = None
    N = B
    if cu_seqlens is not None:
        cu_host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
        cu_dev = (cu_seqlens if cu_seqlens.is_cuda else cu_host).to(q.device, torch.int32).contiguous()
        N = cu_host.numel() - 1
    _shaped(h0, (N, Hv, dk, dv), "h0")
    a = LaArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(h0), _ptr(cu_dev), _ptr(cu_host), None, None, B, T, N, Hqk, Hv,
               dk, dv, float(scale), LA_FLAG_HEAD_DECAY if head else 0)
    return a, (cu_host, cu_dev)


def la_chunk_workspace_bytes(q_shape, v_shape, cu_seqlens=None, *, head_decay=False, backward=False):
    """la_chunk_fwd_workspace_size (backward: la_chunk_bwd_workspace_size) for q [B,T,Hqk,dk] and v
    [B,T,Hv,dv] (shapes only); 0 for shapes that the calls refuse."""
    B, T, Hqk, dk = q_shape
    Hv, dv = v_shape[2], v_shape[3]
    cu_host, N = None, B
    if cu_seqlens is not None:
        cu_host = cu_seqlens.detach().to("cpu", torch.int32).contiguous()
        N = cu_host.numel() - 1
    a = LaArgs(None, None, None, None, None, _ptr(cu_host), _ptr(cu_host), None, None, B, T, N, Hqk, Hv, dk, dv, 1.0,
               LA_FLAG_HEAD_DECAY if head_decay else 0)
    fn = "la_chunk_bwd_workspace_size" if backward else "la_chunk_fwd_workspace_size"
    return int(getattr(load(), fn)(ctypes.byref(a)))


def la_chunk_fwd(q, k, v, g, h0=None, cu_seqlens=None, *, scale=1.0, o=None, hT=None, output_final_state=True,
                 workspace=None, stream=None):
    """Linear attention with a decay for each head: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.
    q, k [B,T,Hqk,dk] bf16; v [B,T,Hv,dv] bf16 (value head h reads q/k head h // (Hv // Hqk)); g
    [B,T,Hv] fp32, or [Hv] for one fixed decay per head; h0 [N,Hv,dk,dv] fp32 or None; cu_seqlens int32
    [N+1] (CPU or CUDA) of sequences packed on the T axis of B = 1, or None. dk, dv in {64, 128}.
    Returns (o [B,T,Hv,dv] bf16, hT [N,Hv,dk,dv] fp32 or None)."""
    lib = load()
    with _on(q.device, stream) as st:
        a, _keep = _la_args(q, k, v, g, h0, cu_seqlens, scale)
        if o is None:
            o = torch.empty(v.shape, dtype=torch.bfloat16, device=q.device)
        if hT is None and output_final_state:
            hT = torch.empty((a.N, a.Hv, a.dk, a.dv), dtype=torch.float32, device=q.device)
        a.o = _ptr(_shaped(_dev(o, torch.bfloat16, "o"), v.shape, "o"))
        a.hT = _ptr(_shaped(_dev(hT, torch.float32, "hT"), (a.N, a.Hv, a.dk, a.dv), "hT"))
        _same_device(q.device, o=o, hT=hT, workspace=workspace)
        ws = _workspace(workspace, int(lib.la_chunk_fwd_workspace_size(ctypes.byref(a))), q.device)
        _check("la_chunk_fwd", lib.la_chunk_fwd(ctypes.byref(a), _ptr(ws), ws.numel(), st))
    return o, hT


def la_chunk_bwd(q, k, v, g, h0=None, cu_seqlens=None, dout=None, dhT=None, *, scale=1.0, want_dh0=True,
                 workspace=None, stream=None):
    """Gradients of <o, dout> + <hT, dhT> of la_chunk_fwd with the same inputs. dout [B,T,Hv,dv] bf16;
    dhT [N,Hv,dk,dv] fp32 or None. Returns (dq, dk, dv bf16, dg fp32 of g's shape, dh0 [N,Hv,dk,dv]
    fp32 or None unless want_dh0); dq and dk are summed over the value heads that share a q/k head."""
    lib = load()
    with _on(q.device, stream) as st:
        a, _keep = _la_args(q, k, v, g, h0, cu_seqlens, scale)
        if dout is None:
            raise ValueError("dout is required")
        state = (a.N, a.Hv, a.dk, a.dv)
        _shaped(_dev(dout, torch.bfloat16, "dout"), v.shape, "dout")
        _shaped(_dev(dhT, torch.float32, "dhT"), state, "dhT")
        _same_device(q.device, dout=dout, dhT=dhT, workspace=workspace)
        dq, dk, dv, dg = (torch.empty_like(t) for t in (q, k, v, g))
        dh0 = torch.empty(state, dtype=torch.float32, device=q.device) if want_dh0 else None
        gr = LaGrads(_ptr(dout), _ptr(dhT), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dh0))
        ws = _workspace(workspace, int(lib.la_chunk_bwd_workspace_size(ctypes.byref(a))), q.device)
        _check("la_chunk_bwd", lib.la_chunk_bwd(ctypes.byref(a), ctypes.byref(gr), _ptr(ws), ws.numel(), st))
    return dq, dk, dv, dg, dh0


def la_decode_step(q, k, v, g, state, *, state_out=None, state_qdq=True, scale=1.0, o=None, stream=None,
                   codec="e4m3"):
    """One token per sequence of la_chunk_fwd's recurrence. q, k [N,Hqk,dk] bf16; v [N,Hv,dv] bf16; g
    [N,Hv] fp32; state [N,Hv,dk,dv] fp32, updated in place unless state_out receives the new one. o is
    taken from the updated state before its QDQ (state_qdq; codec "e4m3" tiles or "int8" blocks).
    Returns o [N,Hv,dv] bf16."""
    lib = load()
    flags = _state_flags(state_qdq, codec)
    q, k, v = (_dev(t, torch.bfloat16, n) for t, n in ((q, "q"), (k, "k"), (v, "v")))
    g, state = _dev(g, torch.float32, "g"), _dev(state, torch.float32, "state")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v must be [N, H, D]")
    N, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    _shaped(k, q.shape, "k")
    _shaped(v, (N, Hv, dv), "v")
    _shaped(g, (N, Hv), "g")
    _shaped(state, (N, Hv, dk, dv), "state")
    if state_out is None:
        state_out = state
    _shaped(_dev(state_out, torch.float32, "state_out"), state.shape, "state_out")
    with _on(q.device, stream) as st:
        if o is None:
            o = torch.empty(v.shape, dtype=torch.bfloat16, device=q.device)
        _shaped(_dev(o, torch.bfloat16, "o"), v.shape, "o")
        _same_device(q.device, k=k, v=v, g=g, state=state, state_out=state_out, o=o)
        _check("la_decode_step", lib.la_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(state_out),
                                                    _ptr(o), N, Hqk, Hv, dk, dv, float(scale), flags, st))
    return o


def _typed(t, name):
    """A contiguous CUDA tensor of bf16 or fp32 and its type code (None passes)."""
    if t is None:
        return 0
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    _dev(t, t.dtype, name)
    return _DTYPES[t.dtype]


def _rows(x):
    if x.dim() == 0:
        raise ValueError("the normalised tensor needs a last dimension")
    D = x.shape[-1]
    return (x.numel() // D if D else 0), D


def gated_norm_fwd(x, z, w, *, eps=1e-6, y=None, stream=None):
    """y = rms(x) w silu(z) over the last dimension, rms(x) = x / sqrt(mean(x^2) + eps): the norm behind
    a mixing core (one row per token and head) and its gate. x [..., D] bf16 or fp32; z [..., D] bf16;
    w [D] bf16 or fp32. Returns y [..., D] bf16."""
    lib = load()
    tx, tw = _typed(x, "x"), _typed(w, "w")
    rows, D = _rows(x)
    _shaped(_dev(z, torch.bfloat16, "z"), x.shape, "z")
    _shaped(w, (D,), "w")
    with _on(x.device, stream) as st:
        if y is None:
            y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
        _shaped(_dev(y, torch.bfloat16, "y"), x.shape, "y")
        _same_device(x.device, z=z, w=w, y=y)
        _check("gated_norm_fwd", lib.gated_norm_fwd(_ptr(x), tx, _ptr(z), _ptr(w), tw, _ptr(y), rows, D, float(eps), st))
    return y


def gated_norm_bwd(dy, x, z, w, *, eps=1e-6, workspace=None, stream=None):
    """Gradients of gated_norm_fwd: dy [..., D] bf16. Returns (dx of x's type, dz bf16, dw [D] fp32)."""
    lib = load()
    tx, tw = _typed(x, "x"), _typed(w, "w")
    rows, D = _rows(x)
    _shaped(_dev(z, torch.bfloat16, "z"), x.shape, "z")
    _shaped(_dev(dy, torch.bfloat16, "dy"), x.shape, "dy")
    _shaped(w, (D,), "w")
    with _on(x.device, stream) as st:
        _same_device(x.device, dy=dy, z=z, w=w, workspace=workspace)
        dx, dz = torch.empty_like(x), torch.empty_like(z)
        dw = torch.empty(D, dtype=torch.float32, device=x.device)
        ws = _workspace(workspace, int(lib.gated_norm_bwd_workspace_size(rows, D)), x.device)
        _check("gated_norm_bwd", lib.gated_norm_bwd(_ptr(dy), _ptr(x), tx, _ptr(z), _ptr(w), tw, _ptr(dx), _ptr(dz),
                                                    _ptr(dw), rows, D, float(eps), _ptr(ws), ws.numel(), st))
    return dx, dz, dw


def _residual_inputs(y, h, w_pre, w_post):
    th, tw = _typed(h, "h"), _typed(w_pre, "w_pre")
    if w_post is not None and _typed(w_post, "w_post") != tw:
        raise ValueError(f"w_post must be {w_pre.dtype} as w_pre is, got {w_post.dtype}")
    rows, D = _rows(h)
    _shaped(_dev(y, torch.bfloat16, "y"), h.shape, "y")
    _shaped(w_pre, (D,), "w_pre")
    _shaped(w_post, (D,), "w_post")
    return rows, D, th, tw


def residual_norm_fwd(y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, h_out=None, x=None, stream=None):
    """h_out = h + alpha n, n = rms(y) w_post (w_post None: n = y); x = rms(h_out) w_pre: the norm after a
    block, its scaled residual and the norm before the next block. y [..., D] bf16 (the block's output);
    h [..., D] bf16 or fp32 (the residual stream); w_pre, w_post [D], both bf16 or both fp32. h_out may
    be h. Returns (h_out of h's type, x bf16)."""
    lib = load()
    rows, D, th, tw = _residual_inputs(y, h, w_pre, w_post)
    with _on(h.device, stream) as st:
        if h_out is None:
            h_out = torch.empty_like(h)
        if x is None:
            x = torch.empty(h.shape, dtype=torch.bfloat16, device=h.device)
        _shaped(_dev(h_out, h.dtype, "h_out"), h.shape, "h_out")
        _shaped(_dev(x, torch.bfloat16, "x"), h.shape, "x")
        _same_device(h.device, y=y, w_pre=w_pre, w_post=w_post, h_out=h_out, x=x)
        _check("residual_norm_fwd", lib.residual_norm_fwd(_ptr(y), _ptr(h), th, _ptr(w_post), _ptr(w_pre), tw,
                                                          _ptr(h_out), _ptr(x), rows, D, float(alpha), float(eps), st))
    return h_out, x


def residual_norm_bwd(dx, dh_out, y, h, w_pre, w_post=None, *, alpha=1.0, eps=1e-6, workspace=None, stream=None):
    """Gradients of residual_norm_fwd with the same y, h, w_pre, w_post. dx [..., D] bf16; dh_out [..., D] of
    h's type or None (zero). Returns (dy bf16, dh of h's type, dw_pre [D] fp32, dw_post [D] fp32 or None)."""
    lib = load()
    rows, D, th, tw = _residual_inputs(y, h, w_pre, w_post)
    _shaped(_dev(dx, torch.bfloat16, "dx"), h.shape, "dx")
    _shaped(_dev(dh_out, h.dtype, "dh_out"), h.shape, "dh_out")
    with _on(h.device, stream) as st:
        _same_device(h.device, dx=dx, dh_out=dh_out, y=y, w_pre=w_pre, w_post=w_post, workspace=workspace)
        dy, dh = torch.empty_like(y), torch.empty_like(h)
        dw_pre = torch.empty(D, dtype=torch.float32, device=h.device)
        dw_post = torch.empty_like(dw_pre) if w_post is not None else None
        ws = _workspace(workspace, int(lib.residual_norm_bwd_workspace_size(rows, D)), h.device)
        _check("residual_norm_bwd", lib.residual_norm_bwd(
            _ptr(dx), _ptr(dh_out), _ptr(y), _ptr(h), th, _ptr(w_post), _ptr(w_pre), tw, _ptr(dy), _ptr(dh),
            _ptr(dw_post), _ptr(dw_pre), rows, D, float(alpha), float(eps), _ptr(ws), ws.numel(), st))
    return dy, dh, dw_pre, dw_post
