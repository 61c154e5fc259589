"""Plain 64-bit references of the linear-attention and norm operators (CPU, elementary operations)."""
import torch

F64 = torch.float64


def qdq_e4m3(S):
    """E4M3 of [..., dk, dv] with one scale per dk rows x 64 columns."""
    x = S.unflatten(-1, (-1, 64))
    sc = x.abs().amax((-3, -1), keepdim=True) / 448
    sc = torch.where(sc == 0, torch.ones_like(sc), sc)
    r = x / sc
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6))).clamp(-6, 8) - 3)
    return (torch.round(r / step) * step * sc).flatten(-2)


def qdq_int8(S):
    x = S.unflatten(-1, (-1, 32))
    sc = x.abs().amax(-1, keepdim=True) / 127
    sc = torch.where(sc == 0, torch.ones_like(sc), sc)
    return (torch.round(x / sc) * sc).flatten(-2)


def la(q, k, v, g, h0, cu, scale, dout=None, dhT=None):
    """Token by token: o, hT and, with dout, the gradients dq, dk, dv, dg, dh0 (a dict)."""
    q, k, v, g = (t.detach().cpu().to(F64) for t in (q, k, v, g))
    B, T, Hv, dv = v.shape
    Hqk, dk = q.shape[2:]
    r = Hv // Hqk
    head = g.dim() == 1
    a = torch.exp(g.expand(B, T, Hv))
    if cu is None:
        spans = [(n, 0, T) for n in range(B)]
    else:
        c = [int(x) for x in cu]
        spans = [(0, c[n], c[n + 1]) for n in range(len(c) - 1)]
    N = len(spans)
    qe, ke = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    out = {"o": torch.zeros(B, T, Hv, dv, dtype=F64), "hT": torch.zeros(N, Hv, dk, dv, dtype=F64)}
    train = dout is not None
    if train:
        do = dout.detach().cpu().to(F64)
        dq, dkk, dvv = torch.zeros(B, T, Hv, dk, dtype=F64), torch.zeros(B, T, Hv, dk, dtype=F64), torch.zeros_like(v)
        dgg, dh0 = torch.zeros(B, T, Hv, dtype=F64), torch.zeros(N, Hv, dk, dv, dtype=F64)
    for n, (b, t0, t1) in enumerate(spans):
        S = torch.zeros(Hv, dk, dv, dtype=F64) if h0 is None else h0[n].detach().cpu().to(F64)
        states = [S]
        for t in range(t0, t1):
            S = a[b, t][:, None, None] * S + ke[b, t][:, :, None] * v[b, t][:, None, :]
            if train:
                states.append(S)
            out["o"][b, t] = scale * torch.einsum("hk,hkv->hv", qe[b, t], S)
        out["hT"][n] = S
        if not train:
            continue
        dS = torch.zeros(Hv, dk, dv, dtype=F64) if dhT is None else dhT[n].detach().cpu().to(F64)
        for t in reversed(range(t0, t1)):
            dS = dS + scale * qe[b, t][:, :, None] * do[b, t][:, None, :]
            dq[b, t] = scale * torch.einsum("hkv,hv->hk", states[t - t0 + 1], do[b, t])
            dkk[b, t] = torch.einsum("hkv,hv->hk", dS, v[b, t])
            dvv[b, t] = torch.einsum("hkv,hk->hv", dS, ke[b, t])
            dgg[b, t] = a[b, t] * (states[t - t0] * dS).sum((1, 2))
            dS = a[b, t][:, None, None] * dS
        dh0[n] = dS
    if train:
        out.update(dq=dq.unflatten(2, (Hqk, r)).sum(3), dk=dkk.unflatten(2, (Hqk, r)).sum(3), dv=dvv,
                   dg=dgg.sum((0, 1)) if head else dgg, dh0=dh0)
    return out


def decode(q, k, v, g, state, scale, codec):
    q, k, v, g, state = (t.detach().cpu().to(F64) for t in (q, k, v, g, state))
    r = v.shape[1] // q.shape[1]
    S = torch.exp(g)[..., None, None] * state + k.repeat_interleave(r, 1)[..., None] * v[:, :, None, :]
    o = scale * torch.einsum("nhk,nhkv->nhv", q.repeat_interleave(r, 1), S)
    return o, {None: lambda x: x, "e4m3": qdq_e4m3, "int8": qdq_int8}[codec](S)


def _rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm(x, z, w, eps, dy=None):
    """y, or (y, dx, dz, dw)."""
    x, z, w = (t.detach().cpu().to(F64).requires_grad_() for t in (x, z, w))
    y = _rms(x, eps) * w * z / (1 + torch.exp(-z))
    if dy is None:
        return y.detach()
    return (y.detach(), *torch.autograd.grad(y, [x, z, w], dy.detach().cpu().to(F64)))


def residual_norm(y, h, w_pre, w_post, alpha, eps, dx=None, dh_out=None):
    """(h_out, x), or (h_out, x, dy, dh, dw_pre, dw_post or None)."""
    y, h, w_pre = (t.detach().cpu().to(F64).requires_grad_() for t in (y, h, w_pre))
    wp = None if w_post is None else w_post.detach().cpu().to(F64).requires_grad_()
    h2 = h + alpha * (y if wp is None else _rms(y, eps) * wp)
    x = _rms(h2, eps) * w_pre
    if dx is None:
        return h2.detach(), x.detach()
    up = [dx.detach().cpu().to(F64), torch.zeros_like(h2) if dh_out is None else dh_out.detach().cpu().to(F64)]
    got = torch.autograd.grad([x, h2], [y, h, w_pre] + ([] if wp is None else [wp]), up)
    return (h2.detach(), x.detach(), *got, *([None] if wp is None else []))


def rel(a, b):
    """2-norm of the difference over that of the reference (0 for two empty or all-zero tensors)."""
    a, b = a.detach().cpu().to(F64), b.detach().cpu().to(F64)
    d, n = (a - b).norm().item(), b.norm().item()
    return d / n if n else (0.0 if d == 0 else float("inf"))
