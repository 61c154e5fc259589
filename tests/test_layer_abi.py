"""The C entry points of the linear-attention and norm operators, without a GPU: host-side validation returns
the documented status before a device is touched, sizes need none. The pointers are fake and never read; a call
that passes validation is made only where no GPU is present (it stops at the device check)."""
import ctypes

import pytest
import torch

import fp8_state_qat_gb300 as lib
from fp8_state_qat_gb300 import gdnqat as B

BASE, STEP = 1 << 40, 1 << 33
NO_GPU = not torch.cuda.is_available()
BF, F32 = 0, 1


@pytest.fixture(scope="module")
def so():
    return lib.load()


def at(i, off=0):
    return BASE + i * STEP + off


def la_args(**over):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), h0=None, cu_seqlens=None, cu_seqlens_host=None, o=at(4), hT=at(5),
             B=2, T=300, N=2, Hqk=2, Hv=4, dk=128, dv=64, scale=1.0, flags=0)
    a.update(over)
    return B.LaArgs(**a)


def la_grads(**over):
    a = dict(dout=at(10), dhT=at(11), dq=at(12), dk=at(13), dv=at(14), dg=at(15), dh0=at(16))
    a.update(over)
    return B.LaGrads(**a)


def fwd(so, a, ws=at(20), room=1 << 40):
    return so.la_chunk_fwd(ctypes.byref(a), ws, room, None)


def bwd(so, a, g, ws=at(20), room=1 << 40):
    return so.la_chunk_bwd(ctypes.byref(a), ctypes.byref(g), ws, room, None)


BAD_LA = [
    (dict(dk=96), B.GDN_ERR_UNSUPPORTED_SHAPE),
    (dict(dv=256), B.GDN_ERR_UNSUPPORTED_SHAPE),
    (dict(Hv=3), B.GDN_ERR_INVALID_ARG),            # not a multiple of Hqk
    (dict(Hqk=0), B.GDN_ERR_INVALID_ARG),
    (dict(N=3), B.GDN_ERR_INVALID_ARG),             # dense: N == B
    (dict(T=-1), B.GDN_ERR_INVALID_ARG),
    (dict(flags=2), B.GDN_ERR_INVALID_ARG),
    (dict(q=None), B.GDN_ERR_INVALID_ARG),
    (dict(v=at(2, 8)), B.GDN_ERR_INVALID_ARG),      # not 16-byte aligned
    (dict(g=at(3, 2)), B.GDN_ERR_INVALID_ARG),
    (dict(h0=at(6, 4)), B.GDN_ERR_INVALID_ARG),
    (dict(B=30000, N=30000, T=30000), B.GDN_ERR_INVALID_ARG),   # more tokens than 32 bits count
]


@pytest.mark.parametrize("over,want", BAD_LA)
def test_la_refusals(so, over, want):
    assert fwd(so, la_args(**over)) == want
    assert bwd(so, la_args(**over), la_grads()) == want


@pytest.mark.parametrize("over,want", [
    (dict(o=None), B.GDN_ERR_INVALID_ARG),
    (dict(o=at(2, 64)), B.GDN_ERR_INVALID_ARG),             # over v
    (dict(o=at(5, 64)), B.GDN_ERR_INVALID_ARG),             # over hT
    (dict(h0=at(5, 256)), B.GDN_ERR_INVALID_ARG),           # hT over a part of h0
    (dict(hT=at(3)), B.GDN_ERR_INVALID_ARG),                # over g
])
def test_la_forward_refusals(so, over, want):
    assert fwd(so, la_args(**over)) == want


@pytest.mark.parametrize("over", [dict(dout=None), dict(dq=None), dict(dg=None), dict(dv=at(14, 4)), dict(dk=at(1)),
                                  dict(dq=at(13, 16)), dict(dg=at(10, 64)), dict(dh0=at(11))])
def test_la_backward_refusals(so, over):
    assert bwd(so, la_args(o=None, hT=None), la_grads(**over)) == B.GDN_ERR_INVALID_ARG
    assert so.la_chunk_bwd(ctypes.byref(la_args()), None, at(20), 1 << 40, None) == B.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("cu,T", [([0, 50, 40, 300], 300), ([0, 50, 60, 299], 300), ([1, 50, 60, 300], 300)])
def test_la_packed_refusals(so, cu, T):
    host = (ctypes.c_int32 * len(cu))(*cu)
    a = la_args(B=1, N=len(cu) - 1, T=T, cu_seqlens=at(7), cu_seqlens_host=ctypes.addressof(host))
    assert fwd(so, a) == B.GDN_ERR_INVALID_ARG
    a = la_args(B=1, N=len(cu) - 1, T=T, cu_seqlens=at(7))   # no host copy
    assert fwd(so, a) == B.GDN_ERR_INVALID_ARG


def test_la_workspace(so):
    need = lib.la_chunk_workspace_bytes((2, 300, 2, 128), (2, 300, 4, 64))
    assert need == so.la_chunk_fwd_workspace_size(ctypes.byref(la_args())) > 256
    more = lib.la_chunk_workspace_bytes((2, 300, 2, 128), (2, 300, 4, 64), backward=True)
    assert more > 2 * need
    assert lib.la_chunk_workspace_bytes((2, 300, 2, 96), (2, 300, 4, 64)) == 0
    assert lib.la_chunk_workspace_bytes((1, 90, 2, 64), (1, 90, 2, 64), torch.tensor([0, 40, 90])) > 0
    assert lib.la_chunk_workspace_bytes((1, 90, 2, 64), (1, 90, 2, 64), torch.tensor([0, 40, 91])) == 0
    a = la_args()
    assert fwd(so, a, room=need - 1) == B.GDN_ERR_WORKSPACE_TOO_SMALL
    assert fwd(so, a, ws=None) == B.GDN_ERR_WORKSPACE_TOO_SMALL
    assert fwd(so, a, ws=at(20, 64)) == B.GDN_ERR_INVALID_ARG   # 256-byte alignment
    assert bwd(so, a, la_grads(), room=more - 1) == B.GDN_ERR_WORKSPACE_TOO_SMALL
    if NO_GPU:
        assert fwd(so, a, room=need) == B.GDN_ERR_UNSUPPORTED_ARCH
        assert bwd(so, a, la_grads(), room=more) == B.GDN_ERR_UNSUPPORTED_ARCH
        same = la_args(h0=at(5))                                 # hT may be h0
        assert fwd(so, same) == B.GDN_ERR_UNSUPPORTED_ARCH


def decode(so, **over):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), state=at(4), state_out=at(4), o=at(5), N=3, Hqk=2, Hv=2, dk=64, dv=256,
             scale=1.0, flags=1)
    a.update(over)
    return so.la_decode_step(*a.values(), None)


@pytest.mark.parametrize("over,want", [
    (dict(dk=32), B.GDN_ERR_UNSUPPORTED_SHAPE), (dict(dv=96), B.GDN_ERR_UNSUPPORTED_SHAPE),
    (dict(Hv=3), B.GDN_ERR_INVALID_ARG), (dict(N=-1), B.GDN_ERR_INVALID_ARG), (dict(flags=4), B.GDN_ERR_INVALID_ARG),
    (dict(k=None), B.GDN_ERR_INVALID_ARG), (dict(state=at(4, 4)), B.GDN_ERR_INVALID_ARG),
    (dict(state_out=at(4, 64)), B.GDN_ERR_INVALID_ARG), (dict(o=at(4, 32)), B.GDN_ERR_INVALID_ARG),
    (dict(N=1 << 30, Hv=2), B.GDN_ERR_INVALID_ARG),
])
def test_decode_refusals(so, over, want):
    assert decode(so, **over) == want


def gated(so, **over):
    a = dict(x=at(0), tx=F32, z=at(1), w=at(2), tw=F32, y=at(3), rows=8, D=64, eps=1e-6)
    a.update(over)
    return so.gated_norm_fwd(*a.values(), None)


@pytest.mark.parametrize("over,want", [
    (dict(tx=2), B.GDN_ERR_INVALID_ARG), (dict(tw=-1), B.GDN_ERR_INVALID_ARG), (dict(D=0), B.GDN_ERR_INVALID_ARG),
    (dict(D=8193), B.GDN_ERR_UNSUPPORTED_SHAPE), (dict(rows=-1), B.GDN_ERR_INVALID_ARG),
    (dict(eps=-1.0), B.GDN_ERR_INVALID_ARG), (dict(eps=float("nan")), B.GDN_ERR_INVALID_ARG),
    (dict(z=None), B.GDN_ERR_INVALID_ARG), (dict(x=at(0, 2)), B.GDN_ERR_INVALID_ARG), (dict(y=at(0, 64)), B.GDN_ERR_INVALID_ARG),
    (dict(y=at(1)), B.GDN_ERR_INVALID_ARG),
])
def test_gated_norm_refusals(so, over, want):
    assert gated(so, **over) == want


def test_norm_backward_refusals(so):
    def gb(**over):
        a = dict(dy=at(0), x=at(1), tx=BF, z=at(2), w=at(3), tw=F32, dx=at(4), dz=at(5), dw=at(6), rows=8, D=64, eps=1e-6,
                 ws=at(7), room=1 << 30)
        a.update(over)
        return so.gated_norm_bwd(*a.values(), None)
    assert gb(dw=None) == gb(dx=at(1)) == gb(dz=at(5, 1)) == gb(dx=at(5, 64)) == gb(dy=None) == B.GDN_ERR_INVALID_ARG
    need = so.gated_norm_bwd_workspace_size(8, 64)
    assert need > 0 and so.gated_norm_bwd_workspace_size(8, 9000) == 0
    assert gb(room=need - 1) == gb(ws=None) == B.GDN_ERR_WORKSPACE_TOO_SMALL

    def rb(**over):
        a = dict(dx=at(0), dh_out=at(1), y=at(2), h=at(3), th=F32, w_post=at(4), w_pre=at(5), tw=F32, dy=at(6), dh=at(7),
                 dw_post=at(8), dw_pre=at(9), rows=8, D=64, alpha=1.0, eps=1e-6, ws=at(10), room=1 << 30)
        a.update(over)
        return so.residual_norm_bwd(*a.values(), None)
    assert rb(dw_post=None) == rb(w_post=None) == rb(dw_pre=None) == rb(dh=at(3)) == rb(dy=at(1)) == B.GDN_ERR_INVALID_ARG
    assert rb(room=so.residual_norm_bwd_workspace_size(8, 64) - 1) == B.GDN_ERR_WORKSPACE_TOO_SMALL
    if NO_GPU:
        assert gb(room=need) == rb(dh=at(1)) == rb(dh_out=None) == rb(w_post=None, dw_post=None) == B.GDN_ERR_UNSUPPORTED_ARCH


def test_residual_norm_refusals(so):
    def rf(**over):
        a = dict(y=at(0), h=at(1), th=BF, w_post=None, w_pre=at(2), tw=F32, h_out=at(3), x=at(4), rows=8, D=64, alpha=1.0,
                 eps=1e-6)
        a.update(over)
        return so.residual_norm_fwd(*a.values(), None)
    assert rf(w_pre=None) == rf(x=at(3)) == rf(x=at(1)) == rf(h_out=at(1, 64)) == rf(th=3) == B.GDN_ERR_INVALID_ARG
    if NO_GPU:
        assert rf() == rf(h_out=at(1)) == rf(rows=0) == B.GDN_ERR_UNSUPPORTED_ARCH


def test_python_refuses_cpu_tensors(so):
    t = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        lib.gated_norm_fwd(t, t, t[0])
    with pytest.raises(TypeError, match="tensor"):
        lib.gated_norm_fwd(1, t, t[0])
    with pytest.raises(ValueError, match="codec"):
        lib.la_decode_step(t, t, t, t, t, codec="fp4")
