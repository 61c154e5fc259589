"""The gated norm and the residual norm on the GPU against 64-bit references.

Tolerances: a bf16 output is an fp32 value rounded once: bf16 has 8 significant bits, so an element
just above a power of two moves by up to 2^-8 = 3.9e-3 of itself (4e-3 with the fp32 part); an fp32 output has the error of sums of up to 8192 terms in a tree and of a few
roundings, 2e-6; a weight gradient sums up to `rows` terms of both signs in fp32, 5e-6.
"""
import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 4.0e-3, F32: 2e-6}
TOL_W = 5e-6


def rows_of(R, D, dtype, seed, scale=1.0):
    return (scale * torch.randn(R, D, generator=torch.Generator().manual_seed(seed))).to(dtype)


def near(got, want, tol=None):
    assert torch.isfinite(got.float()).all()
    e = ref.rel(got, want)
    assert e <= (tol or TOL[got.dtype]), e


SIZES = [(1, 1), (3, 7), (5, 8), (1, 64), (33, 64), (7, 65), (300, 128), (9, 129), (40, 256), (11, 257), (6, 512),
         (5, 1000), (4, 1023), (9, 1024), (3, 2048), (2, 2056), (3, 4095), (2, 8192), (2, 8191), (1000, 16)]


@pytest.mark.parametrize("R,D", SIZES)
@pytest.mark.parametrize("tx,tw", [(BF, F32), (F32, BF), (F32, F32)])
def test_gated_norm(gdn, R, D, tx, tw):
    x, z, dy = rows_of(R, D, tx, 1), rows_of(R, D, BF, 2, 2.0), rows_of(R, D, BF, 3)
    w = (1 + 0.3 * rows_of(1, D, F32, 4)[0]).to(tw)
    want = ref.gated_norm(x, z, w, 1e-6, dy)
    d = [t.cuda() for t in (x, z, w)]
    near(gdn.gated_norm_fwd(*d), want[0])
    dx, dz, dw = gdn.gated_norm_bwd(dy.cuda(), *d)
    assert dx.dtype == tx and dz.dtype == BF and dw.dtype == F32
    if D > 1:   # with one column rms is +-1 but for eps, and dx is a rounding residue
        near(dx, want[1])
    near(dz, want[2])
    near(dw, want[3], TOL_W)


@pytest.mark.parametrize("R,D", SIZES)
@pytest.mark.parametrize("th,tw,post", [(BF, F32, False), (BF, BF, True), (F32, F32, True), (F32, BF, False)])
def test_residual_norm(gdn, R, D, th, tw, post):
    y, h, dx, dh = rows_of(R, D, BF, 1), rows_of(R, D, th, 2, 2.0), rows_of(R, D, BF, 3), rows_of(R, D, th, 4)
    w1 = (1 + 0.3 * rows_of(1, D, F32, 5)[0]).to(tw)
    w2 = (1 + 0.3 * rows_of(1, D, F32, 6)[0]).to(tw) if post else None
    want = ref.residual_norm(y, h, w1, w2, 0.5, 1e-6, dx, dh)
    c = lambda t: t.cuda() if t is not None else None  # noqa: E731
    h2, x = gdn.residual_norm_fwd(c(y), c(h), c(w1), c(w2), alpha=0.5)
    near(h2, want[0])
    near(x, want[1])
    dy, dhh, d1, d2 = gdn.residual_norm_bwd(c(dx), c(dh), c(y), c(h), c(w1), c(w2), alpha=0.5)
    if D > 1 or not post:
        near(dy, want[2])
    near(dhh, want[3])
    near(d1, want[4], TOL_W)
    assert (d2 is None) == (w2 is None)
    if post:
        near(d2, want[5], TOL_W)


@pytest.mark.parametrize("D", [64, 200, 256, 300, 1000, 2048, 8192])
def test_stream_that_cancels(gdn, D):
    """Rows whose h nearly cancels alpha n, beside ordinary ones: the sums over h_out keep their accuracy."""
    R = 21
    y, dx, dh = rows_of(R, D, BF, 1), rows_of(R, D, BF, 2), rows_of(R, D, F32, 3)
    w1, w2 = (1 + 0.3 * rows_of(1, D, F32, s)[0] for s in (4, 5))
    n = ref.residual_norm(y, torch.zeros(R, D), w1, w2, 0.5, 1e-6)[0]
    h = rows_of(R, D, F32, 6)
    for r, keep in ((3, 1e-3), (4, 0.0), (11, 0.2), (20, 0.05)):
        h[r] = (-n[r] * (1 - keep)).float() + (0 if keep else 1e-2 * h[r])
    want = ref.residual_norm(y, h, w1, w2, 0.5, 1e-6, dx, dh)
    c = [t.cuda() for t in (y, h, w1, w2)]
    got = gdn.residual_norm_fwd(*c, alpha=0.5) + gdn.residual_norm_bwd(dx.cuda(), dh.cuda(), *c, alpha=0.5)
    # h_out of those rows has lost up to 10 bits of h to the cancellation itself: 2^-24 x 1000 = 6e-5 of it; it is of
    # the size of the others' rounding there, but the gradients divide by it, so they are held row by row
    for a, b in zip(got[1:4], want[1:4]):
        for r in range(R):
            e = ref.rel(a[r], b[r])
            assert e <= TOL[a.dtype] + (1e-3 if r in (3, 4) else 2e-5 if r in (11, 20) else 0), (r, e)
    near(got[0], want[0])


def test_many_rows(gdn):
    """More rows than the grid takes at once."""
    R, D = 40000, 64
    x, z, dy = rows_of(R, D, BF, 1), rows_of(R, D, BF, 2), rows_of(R, D, BF, 3)
    w = 1 + 0.3 * rows_of(1, D, F32, 4)[0]
    want = ref.gated_norm(x, z, w, 1e-6, dy)
    near(gdn.gated_norm_fwd(x.cuda(), z.cuda(), w.cuda()), want[0])
    got = gdn.gated_norm_bwd(dy.cuda(), x.cuda(), z.cuda(), w.cuda())
    for a, b, tol in zip(got, want[1:], (None, None, TOL_W)):
        near(a, b, tol)
    R, D = 3000, 1000
    y, h, dx = rows_of(R, D, BF, 1), rows_of(R, D, F32, 2), rows_of(R, D, BF, 3)
    w1, w2 = (1 + 0.3 * rows_of(1, D, F32, s)[0] for s in (5, 6))
    want = ref.residual_norm(y, h, w1, w2, 1.5, 1e-6, dx, None)
    got = gdn.residual_norm_fwd(y.cuda(), h.cuda(), w1.cuda(), w2.cuda(), alpha=1.5) + \
        gdn.residual_norm_bwd(dx.cuda(), None, y.cuda(), h.cuda(), w1.cuda(), w2.cuda(), alpha=1.5)
    for a, b, tol in zip(got, want, (None, None, None, None, TOL_W, TOL_W)):
        near(a, b, tol)


def test_unaligned_rows_and_pointers(gdn):
    """Tensors that start off a 16-byte boundary take the element-wise accesses, with the same values."""
    R, D = 10, 128
    x, z, dy = rows_of(R, D, F32, 1), rows_of(R, D, BF, 2), rows_of(R, D, BF, 3)
    w = 1 + 0.3 * rows_of(1, D, F32, 4)[0]

    def shifted(t, by):
        buf = torch.zeros(t.numel() + by, dtype=t.dtype, device="cuda")
        buf[by:] = t.cuda().flatten()
        return buf[by:].view(t.shape)
    want = ref.gated_norm(x, z, w, 1e-6, dy)
    for by in (1, 3):
        d = [shifted(t, by) for t in (x, z, w)]
        near(gdn.gated_norm_fwd(*d), want[0])
        for a, b, tol in zip(gdn.gated_norm_bwd(shifted(dy, by), *d), want[1:], (None, None, TOL_W)):
            near(a, b, tol)


def test_extreme_values(gdn):
    """Gates far out saturate without NaN; rows of zeros and of large values have finite norms."""
    D = 64
    x = torch.ones(4, D)
    x[1] = 0.0
    x[2] = 1e18
    x[3] = 1e-18
    z = torch.zeros(4, D)
    z[0, :8] = torch.tensor([-3e38, -1000, -100, -20, 20, 100, 1000, 3e38])
    w = torch.ones(D)
    y = gdn.gated_norm_fwd(x.cuda(), z.to(BF).cuda(), w.cuda()).float().cpu()
    want = ref.gated_norm(x, z.to(BF), w, 1e-6)
    assert torch.isfinite(y).all()
    assert torch.allclose(y.double(), want, rtol=2 ** -8, atol=1e-30)
    dy = torch.ones(4, D).to(BF).cuda()
    z[0, 0], z[0, 7] = -1000, 1000   # the gradient of the gate is finite wherever the gate's square is
    for t in gdn.gated_norm_bwd(dy, x.cuda(), z.to(BF).cuda(), w.cuda()):
        assert torch.isfinite(t.float()).all()


def test_rows_are_independent(gdn):
    """A row of NaN or infinities leaves the others, and no element of its own is finite by accident."""
    R, D = 37, 128
    x, z = rows_of(R, D, BF, 1), rows_of(R, D, BF, 2)
    w = 1 + 0.3 * rows_of(1, D, F32, 4)[0].cuda()
    clean = gdn.gated_norm_fwd(x.cuda(), z.cuda(), w)
    x[5, 3], x[20, 100] = float("nan"), float("inf")
    got = gdn.gated_norm_fwd(x.cuda(), z.cuda(), w)
    keep = [r for r in range(R) if r not in (5, 20)]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[5]).all()


def test_no_rows(gdn):
    x, z, w = torch.zeros(0, 64, device="cuda"), torch.zeros(0, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    assert gdn.gated_norm_fwd(x, z, w).shape == (0, 64)
    dx, dz, dw = gdn.gated_norm_bwd(z, x, z, w)
    assert dx.shape == (0, 64) and not dw.any()
    h2, xx = gdn.residual_norm_fwd(z, x, w, w)
    assert h2.shape == xx.shape == (0, 64)
    *_, d1, d2 = gdn.residual_norm_bwd(z, x, z, x, w, w)
    assert not d1.any() and not d2.any()


def test_in_place_stream(gdn):
    """The residual stream may be updated where it lies, and its gradient likewise; on any stream."""
    R, D = 50, 256
    y, h, dx, dh = rows_of(R, D, BF, 1), rows_of(R, D, F32, 2), rows_of(R, D, BF, 3), rows_of(R, D, F32, 4)
    w1 = 1 + 0.3 * rows_of(1, D, F32, 5)[0]
    d = [t.cuda() for t in (y, h, w1)]
    h2, x = gdn.residual_norm_fwd(*d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hh = d[1].clone()
    s.wait_stream(torch.cuda.current_stream())
    h3, x3 = gdn.residual_norm_fwd(d[0], hh, d[2], h_out=hh, stream=s)
    s.synchronize()
    assert h3 is hh and torch.equal(h2, hh) and torch.equal(x, x3)


def test_repeat_bit_for_bit(gdn):
    R, D = 5000, 128
    x, z, dy = rows_of(R, D, F32, 1).cuda(), rows_of(R, D, BF, 2).cuda(), rows_of(R, D, BF, 3).cuda()
    w = torch.ones(D, device="cuda")
    a, b = gdn.gated_norm_bwd(dy, x, z, w), gdn.gated_norm_bwd(dy, x, z, w)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_gradients_against_differences(gdn):
    """<y, dy> is linear in w, so its difference between two weights is dw's product with the step; x is
    stepped along dx, the fp32 h along dh. Slack: 6 standard deviations of the outputs' rounding and
    1% for the cubic term of a step of 2% of the values."""
    R, D = 200, 256
    x, z, dy = rows_of(R, D, F32, 1), rows_of(R, D, BF, 2), rows_of(R, D, BF, 3)
    w, w2 = (1 + 0.3 * rows_of(1, D, F32, s)[0] for s in (4, 5))

    def loss(x, w):
        t = gdn.gated_norm_fwd(x.cuda(), z.cuda(), w.cuda()).cpu().double() * dy.double()
        return t.sum().item(), 6 * 2 ** -9 * (t * t).sum().sqrt().item()
    dx, _, dw = (t.cpu().double() for t in gdn.gated_norm_bwd(dy.cuda(), x.cuda(), z.cuda(), w.cuda()))
    (a, na), (b, nb) = loss(x, w), loss(x, w2)
    assert abs(b - a - (dw * (w2.double() - w.double())).sum().item()) <= na + nb
    e = 0.02 * dx / dx.abs().max() * R ** 0.5
    (a, na), (b, nb) = loss((x.double() + e).float(), w), loss((x.double() - e).float(), w)
    want = 2 * (dx * e).sum().item()
    assert abs(a - b - want) <= na + nb + 0.01 * abs(want)

    yb, h, dh_out = rows_of(R, D, BF, 6), rows_of(R, D, F32, 7), rows_of(R, D, F32, 8)

    def loss2(h):
        h2, xx = gdn.residual_norm_fwd(yb.cuda(), h.cuda(), w.cuda(), w2.cuda(), alpha=0.7)
        t = xx.cpu().double() * dy.double()
        return t.sum().item() + (h2.cpu().double() * dh_out.double()).sum().item(), 6 * 2 ** -9 * (t * t).sum().sqrt().item()
    dh = gdn.residual_norm_bwd(dy.cuda(), dh_out.cuda(), yb.cuda(), h.cuda(), w.cuda(), w2.cuda(), alpha=0.7)[1].cpu().double()
    e = 0.05 * dh / dh.abs().max()
    (a, na), (b, nb) = loss2((h.double() + e).float()), loss2((h.double() - e).float())
    want = 2 * (dh * e).sum().item()
    assert abs(a - b - want) <= na + nb + 0.01 * abs(want)


def test_refusals(gdn):
    x, z, w = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="bfloat16 or"):
        gdn.gated_norm_fwd(x.half(), z, w)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.gated_norm_fwd(x[:, ::2], z[:, ::2], w[:32])
    with pytest.raises(ValueError, match="shape"):
        gdn.gated_norm_fwd(x, z, w[:32].contiguous())
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gated_norm_fwd(x.cpu(), z, w)
    with pytest.raises(ValueError, match="w_post"):
        gdn.residual_norm_fwd(z, x, w, w.to(BF))
    big = torch.ones(1, 8193, device="cuda")
    with pytest.raises(gdn.GdnError) as e:
        gdn.gated_norm_fwd(big, big.to(BF), big[0])
    assert e.value.status == 3
    with pytest.raises(gdn.GdnError) as e:
        gdn.gated_norm_bwd(z, x, z, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(gdn.GdnError) as e:
        gdn.gated_norm_fwd(x, z, w, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(gdn.GdnError) as e:
        gdn.gated_norm_fwd(z, z, w, y=z)     # y over its inputs
    assert e.value.status == 1
