"""Rows of the norms that share a CTA: those past the end, and neighbours. References and tolerances as in
test_gpu_norm.py."""
import ctypes

import pytest
import torch

import layer_reference as ref
from test_gpu_norm import BF, F32, TOL_W, near, rows_of

pytestmark = pytest.mark.gpu


def residual_case(R, D, th, post, seed=0):
    y, h, dx, dh = rows_of(R, D, BF, seed + 1), rows_of(R, D, th, seed + 2, 2.0), rows_of(R, D, BF, seed + 3), rows_of(R, D, th, seed + 4)
    w1 = 1 + 0.3 * rows_of(1, D, F32, seed + 5)[0]
    w2 = 1 + 0.3 * rows_of(1, D, F32, seed + 6)[0] if post else None
    return y, h, w1, w2, dx, dh


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("D", [64, 256, 1000, 2048, 8192])
@pytest.mark.parametrize("R", [1, 3, 33])
def test_residual_norm_without_eps(gdn, R, D, post):
    """eps = 0: the rows that a CTA holds past the end are zero and have no norm, and must leave no trace."""
    y, h, w1, w2, dx, dh = residual_case(R, D, F32, post)
    want = ref.residual_norm(y, h, w1, w2, 0.5, 0.0, dx, dh)
    d = [cuda(t) for t in (y, h, w1, w2)]
    got = gdn.residual_norm_fwd(*d, alpha=0.5, eps=0.0) + gdn.residual_norm_bwd(cuda(dx), cuda(dh), *d, alpha=0.5, eps=0.0)
    for a, b, tol in zip(got, want, (None, None, None, None, TOL_W, TOL_W)):
        if b is not None:
            near(a, b, tol)


@pytest.mark.parametrize("D", [64, 256, 1000, 2048, 8192])
@pytest.mark.parametrize("R", [1, 3, 33])
def test_gated_norm_without_eps(gdn, R, D):
    x, z, dy = rows_of(R, D, F32, 1), rows_of(R, D, BF, 2), rows_of(R, D, BF, 3)
    w = 1 + 0.3 * rows_of(1, D, F32, 4)[0]
    want = ref.gated_norm(x, z, w, 0.0, dy)
    d = [cuda(t) for t in (x, z, w)]
    for a, b, tol in zip((gdn.gated_norm_fwd(*d, eps=0.0), *gdn.gated_norm_bwd(cuda(dy), *d, eps=0.0)), want,
                         (None, None, None, TOL_W)):
        near(a, b, tol)


@pytest.mark.parametrize("th", [BF, F32])
@pytest.mark.parametrize("D", [40, 64, 128, 200, 512])
def test_rows_do_not_depend_on_their_neighbours(gdn, D, th):
    """A row whose h cancels alpha n takes its sums another way; the rows beside it keep every bit of theirs."""
    R = 512
    y, h, w1, w2, dx, dh = residual_case(R, D, th, True)
    other = h.clone()
    n = ref.residual_norm(y, torch.zeros(R, D), w1, w2, 0.5, 1e-6)[0]
    other[::4] = (-n[::4]).to(th)
    a, b = (gdn.residual_norm_bwd(*(cuda(t) for t in (dx, dh, y, s, w1, w2)), alpha=0.5)[:2] for s in (h, other))
    keep = [r for r in range(R) if r % 4]
    for s, t in zip(a, b):
        assert torch.equal(s[keep], t[keep])


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("th", [BF, F32])
@pytest.mark.parametrize("D", [100, 256, 2048, 8192])
def test_gradient_of_the_stream_in_place(gdn, D, th, post):
    """dh may be dh_out (the C call; the Python one makes its outputs): the same bits as in separate buffers."""
    R = 37
    y, h, w1, w2, dx, dh = (cuda(t) for t in residual_case(R, D, th, post))
    want = gdn.residual_norm_bwd(dx, dh, y, h, w1, w2, alpha=0.5)
    lib = gdn.load()
    dy, dw1, dw2 = torch.empty_like(y), torch.empty(D, device="cuda"), torch.empty(D, device="cuda") if post else None
    n = lib.residual_norm_bwd_workspace_size(R, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    bf16, f32 = 0, 1
    status = lib.residual_norm_bwd(P(dx), P(dh), P(y), P(h), f32 if th == F32 else bf16, P(w2), P(w1), f32, P(dy), P(dh),
                                   P(dw2), P(dw1), R, D, 0.5, 1e-6, P(ws), n, torch.cuda.current_stream().cuda_stream)
    assert status == 0
    for a, b in zip((dy, dh, dw1, dw2), want):
        assert a is b is None or torch.equal(a, b)
