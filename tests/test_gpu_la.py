"""Linear attention with a decay for each head on the GPU against the 64-bit token recurrence.

Tolerances (2-norm of the difference over that of the reference), from the roundings on the path:
* o, dq, dk, dv are bf16. Rounding to 8 significant bits moves a value by at most 2^-8 of it, in the
  root mean square over many values by at most 2^-8 / sqrt(3) = 2.3e-3; the output, the weights of the
  products inside a chunk and the state that the products across chunks read are each rounded
  once: sqrt(3) times 2.3e-3 = 3.9e-3, and 1.5 times that for short outputs, 5.9e-3. Sums over the
  value heads of a q/k head add fp32 partials.
* hT, dh0 are sums of fp32 accuracy: 24-bit products and sums of up to a few hundred terms, 1e-5.
* dg is a sum over pairs of tokens whose factors are products of fp32 accuracy, of both signs: 2e-5.
  Where the decays are strong it is a small difference, which the bound allows for by the size of
  dL/d(prefix sums) instead of dg's own.
"""
import itertools

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TOL = {"o": 5.9e-3, "dq": 5.9e-3, "dk": 5.9e-3, "dv": 5.9e-3, "hT": 1e-5, "dh0": 1e-5, "dg": 2e-5}


def inputs(B, T, Hqk, Hv, dk, dv, seed, lens=None, head=False, h0=True, g_mean=3.0):
    gen = torch.Generator().manual_seed(seed)
    cu = None
    if lens is not None:
        B, T = 1, sum(lens)
        cu = torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32)
    N = len(lens) if lens is not None else B

    def randn(*s):
        return torch.randn(*s, generator=gen)

    def unit(*s):
        x = randn(*s)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-9)).to(BF)
    x = dict(q=unit(B, T, Hqk, dk), k=unit(B, T, Hqk, dk), v=randn(B, T, Hv, dv).to(BF),
             g=torch.log(torch.sigmoid(randn(*((Hv,) if head else (B, T, Hv))) + g_mean)),
             h0=randn(N, Hv, dk, dv) * 0.1 if h0 else None, cu=cu)
    grads = dict(dout=randn(B, T, Hv, dv).to(BF), dhT=randn(N, Hv, dk, dv) * 0.1)
    return x, grads


def cuda(t):
    return t.cuda() if t is not None else None


def run_fwd(gdn, x, scale, **kw):
    return gdn.la_chunk_fwd(*(cuda(x[n]) for n in ("q", "k", "v", "g", "h0")), x["cu"], scale=scale, **kw)


def run_bwd(gdn, x, gr, scale, **kw):
    got = gdn.la_chunk_bwd(*(cuda(x[n]) for n in ("q", "k", "v", "g", "h0")), x["cu"], cuda(gr["dout"]),
                           cuda(gr["dhT"]), scale=scale, **kw)
    return dict(zip(("dq", "dk", "dv", "dg", "dh0"), got))


def check(got, want, names):
    for n in names:
        assert torch.isfinite(got[n].float()).all(), n
        assert ref.rel(got[n], want[n]) <= TOL[n], (n, ref.rel(got[n], want[n]))


def check_all(gdn, x, gr, scale):
    o, hT = run_fwd(gdn, x, scale)
    got = dict(o=o, hT=hT, **run_bwd(gdn, x, gr, scale))
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), scale, gr["dout"], gr["dhT"])
    check(got, want, [n for n in want])
    return got


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(gdn, T):
    check_all(gdn, *inputs(2, T, 2, 2, 128, 128, seed=T), 0.7)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("Hqk,Hv", [(1, 1), (2, 6), (3, 3)])
def test_heads_and_widths(gdn, dk, dv, Hqk, Hv):
    check_all(gdn, *inputs(1, 200, Hqk, Hv, dk, dv, seed=dk + dv + Hv), 1.0)


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("lens", [[1], [5, 0, 1, 130, 64, 0], [0, 0], [257, 3, 128, 127, 129, 1, 1, 40], [0, 700]])
def test_packed_sequences(gdn, lens, head):
    check_all(gdn, *inputs(1, 0, 2, 4, 64, 128, seed=sum(lens), lens=lens, head=head), 1.0)


@pytest.mark.parametrize("head", [False, True])
def test_no_initial_state_and_no_final_gradient(gdn, head):
    x, gr = inputs(2, 190, 2, 2, 64, 64, seed=3, h0=False, head=head)
    gr["dhT"] = None
    check_all(gdn, x, gr, 1.0)
    o, hT = run_fwd(gdn, x, 1.0, output_final_state=False)
    assert hT is None
    assert run_bwd(gdn, x, gr, 1.0, want_dh0=False)["dh0"] is None


def test_many_chunks_few_heads(gdn):
    """One long sequence: its chunks are split among CTAs and joined."""
    check_all(gdn, *inputs(1, 5003, 1, 1, 64, 128, seed=9), 1.0)
    check_all(gdn, *inputs(1, 0, 1, 2, 128, 128, seed=10, lens=[3100, 17, 0, 1500]), 1.0)


def test_slow_decay(gdn):
    """Memories of thousands of tokens: the state carries over many chunks."""
    check_all(gdn, *inputs(1, 2500, 1, 2, 128, 64, seed=11, g_mean=8.0), 1.0)


def test_no_decay(gdn):
    x, gr = inputs(1, 700, 1, 2, 64, 64, seed=12)
    x["g"] = torch.zeros_like(x["g"])
    check_all(gdn, x, gr, 1.0)


def _check_strong(gdn, x, gr):
    got = {**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)}
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), 1.0, gr["dout"], gr["dhT"])
    check(got, want, ["o", "hT", "dq", "dk", "dv", "dh0"])
    size = max(want["dg"].norm().item(), 1e-3 * (want["dq"] * x["q"].double()).norm().item())
    assert (got["dg"].cpu().double() - want["dg"]).norm().item() <= TOL["dg"] * size


@pytest.mark.parametrize("value", [-20.0, -60.0, -200.0, -3.0e38, -float("inf")])
def test_strong_decay_everywhere(gdn, value):
    x, gr = inputs(1, 260, 2, 2, 64, 64, seed=13)
    x["g"] = torch.full_like(x["g"], value)
    x["h0"][:, :, 0, 0] = 1.0   # dh0 and hT stay nonzero below
    got = {**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)}
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), 1.0, gr["dout"], gr["dhT"])
    check(got, want, ["o", "hT", "dq", "dk", "dv"])
    # dh0 and dg are e^value times the size of the other gradients, zero where that is zero in fp32
    assert (got["dh0"].cpu().double() - want["dh0"]).norm().item() <= TOL["dh0"] * want["dh0"].norm().item() + 1e-36
    size = want["dg"].norm().item() + 1e-7 * want["dq"].norm().item()
    assert (got["dg"].cpu().double() - want["dg"]).norm().item() <= 1e-3 * size


def test_resets_inside_a_sequence(gdn):
    """g = -inf starts the state anew; the tokens around it keep full accuracy."""
    x, gr = inputs(1, 400, 2, 2, 64, 64, seed=14)
    for t in (0, 1, 40, 127, 128, 130, 255, 300, 399):
        x["g"][:, t, 0] = -float("inf")
    x["g"][:, 17, 1] = -90.0
    x["g"][:, 200:210, 1] = -40.0
    _check_strong(gdn, x, gr)


def test_other_sequences_cannot_reach_a_sequence(gdn):
    """NaN and infinities in the other packed sequences stay there, forwards and backwards."""
    x, gr = inputs(1, 0, 1, 2, 64, 64, seed=15, lens=[70, 50, 300, 20])
    clean = {**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)}
    bad = float("nan")
    for n in ("q", "k", "v", "g"):
        x[n] = x[n].clone()
        x[n][:, 70:120] = bad
        x[n][:, 420:] = float("inf")
        bad = -bad
    gr["dout"][:, 70:120] = float("inf")
    gr["dout"][:, 420:] = bad
    got = {**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)}
    for n in ("o", "dq", "dk", "dv", "dg"):
        for a, b in ((0, 70), (120, 420)):
            assert torch.equal(got[n][:, a:b], clean[n][:, a:b]), n
    for n in ("hT", "dh0"):
        assert torch.equal(got[n][[0, 2]], clean[n][[0, 2]]), n


def test_runs_repeat_bit_for_bit(gdn):
    x, gr = inputs(1, 0, 2, 4, 128, 128, seed=16, lens=[1000, 77, 513], head=True)
    runs = [{**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)} for _ in range(3)]
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]) and torch.equal(runs[0][n], runs[2][n]), n


def test_state_carries_between_calls(gdn):
    """A prompt in two pieces: the second starts from the first's hT."""
    x, _ = inputs(2, 333, 2, 2, 128, 128, seed=17)
    o, hT = run_fwd(gdn, x, 1.0)
    first = {**{n: x[n][:, :100].contiguous() for n in ("q", "k", "v", "g")}, "h0": x["h0"], "cu": None}
    oa, ha = run_fwd(gdn, first, 1.0)
    rest = {**{n: x[n][:, 100:].contiguous() for n in ("q", "k", "v", "g")}, "h0": ha, "cu": None}
    ob, hb = run_fwd(gdn, rest, 1.0)
    assert ref.rel(torch.cat([oa, ob], 1), o.double()) <= TOL["o"]
    assert ref.rel(hb, hT.double()) <= TOL["hT"]


def test_final_state_in_place_and_given_buffers(gdn):
    x, _ = inputs(2, 150, 1, 2, 64, 64, seed=18)
    o, hT = run_fwd(gdn, x, 1.0)
    d = {n: cuda(x[n]) for n in ("q", "k", "v", "g", "h0")}
    need = gdn.la_chunk_workspace_bytes(x["q"].shape, x["v"].shape)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")   # its contents do not matter
    buf = torch.empty_like(o)
    o2, h2 = gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], o=buf, hT=d["h0"], workspace=ws)
    assert o2 is buf and h2 is d["h0"]
    assert torch.equal(o, o2) and torch.equal(hT, h2)
    gdn.gdn_check_device_status(ws)


def test_other_stream(gdn):
    x, gr = inputs(1, 500, 2, 2, 64, 64, seed=19)
    want = {**dict(zip(("o", "hT"), run_fwd(gdn, x, 1.0))), **run_bwd(gdn, x, gr, 1.0)}
    d = {n: cuda(x[n]) for n in ("q", "k", "v", "g", "h0")}
    dout, dhT = cuda(gr["dout"]), cuda(gr["dhT"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, hT = gdn.la_chunk_fwd(*d.values(), stream=s)
    got = gdn.la_chunk_bwd(*d.values(), None, dout, dhT, stream=s)
    s.synchronize()
    for a, n in zip((o, hT, *got), ("o", "hT", "dq", "dk", "dv", "dg", "dh0")):
        assert torch.equal(a, want[n]), n


def test_graph_capture(gdn):
    x, gr = inputs(1, 300, 1, 2, 64, 64, seed=20)
    d = {n: cuda(x[n]) for n in ("q", "k", "v", "g", "h0")}
    dout, dhT = cuda(gr["dout"]), cuda(gr["dhT"])
    want = gdn.la_chunk_fwd(*d.values()) + gdn.la_chunk_bwd(*d.values(), None, dout, dhT)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gdn.la_chunk_fwd(*d.values()) + gdn.la_chunk_bwd(*d.values(), None, dout, dhT)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_against_differences(gdn):
    """L = <o, dout> + <hT, dhT> is linear in each of q, k, v, h0, so a difference of the kernel's own L
    between two values is the gradient's product with the step, up to the rounding of o: at most 2^-9
    of each o, of random sign, 6 standard deviations allowed. g is stepped along dg."""
    x, gr = inputs(1, 400, 2, 2, 64, 64, seed=21)
    y, _ = inputs(1, 400, 2, 2, 64, 64, seed=22)

    def loss(**over):
        z = {**x, **over}
        o, hT = run_fwd(gdn, z, 1.0)
        o, w = o.cpu().double(), gr["dout"].double()
        noise = 6 * 2 ** -9 * ((o * w) ** 2).sum().sqrt().item()
        return (o * w).sum().item() + (hT.cpu().double() * gr["dhT"].double()).sum().item(), noise
    base, noise = loss()
    got = run_bwd(gdn, x, gr, 1.0)
    for n in ("q", "k", "v", "h0"):
        other, noise2 = loss(**{n: y[n]})
        step = (got["d" + n].cpu().double() * (y[n].double() - x[n].double()))
        slack = noise + noise2 + 6 * 2 ** -9 * (step ** 2).sum().sqrt().item()
        assert abs(other - base - step.sum().item()) <= slack, n
    dg = got["dg"].cpu().double()
    e = 0.05 * dg / dg.abs().max()
    up, n1 = loss(g=(x["g"].double() + e).float())
    down, n2 = loss(g=(x["g"].double() - e).float())
    # central difference: the cubic term is (e/|e|_inf)^2 = 0.0025 / 6 of the third derivative, under 1%
    want = 2 * (dg * e).sum().item()
    assert abs(up - down - want) <= n1 + n2 + 0.01 * abs(want)


# ---- decode ----
def decode_inputs(N, Hqk, Hv, dk, dv, seed):
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen)
    return (randn(N, Hqk, dk).to(BF), randn(N, Hqk, dk).to(BF), randn(N, Hv, dv).to(BF),
            torch.log(torch.sigmoid(randn(N, Hv) + 3)), 0.5 * randn(N, Hv, dk, dv))


@pytest.mark.parametrize("codec", [None, "e4m3", "int8"])
@pytest.mark.parametrize("N,Hqk,Hv,dk,dv", [(1, 1, 1, 64, 64), (3, 2, 4, 128, 64), (2, 5, 5, 64, 256), (7, 1, 3, 128, 128),
                                            (1, 2, 2, 128, 256)])
def test_decode(gdn, N, Hqk, Hv, dk, dv, codec):
    x = decode_inputs(N, Hqk, Hv, dk, dv, seed=N + dv)
    d = [t.cuda() for t in x]
    out = torch.empty_like(d[4])
    o = gdn.la_decode_step(*d, state_out=out, state_qdq=codec is not None, codec=codec or "e4m3", scale=0.5)
    ro, rS = ref.decode(*x, 0.5, codec)
    assert ref.rel(o, ro) <= 2 ** -9            # one rounding of an fp32 value
    assert torch.equal(d[4].cpu(), x[4])        # the input state stays
    if codec is None:
        assert ref.rel(out, rS) <= 2 ** -22     # two fp32 roundings and exp's
        return
    # bit for bit the fp32 formula on the updated state: scale = amax times the rounded 1 / 448 or 1 / 127
    plain = torch.empty_like(d[4])
    gdn.la_decode_step(*d, state_out=plain, state_qdq=False, scale=0.5)
    w, axes, top = (64, (-3, -1), 448.0) if codec == "e4m3" else (32, (-1,), 127.0)
    t = plain.unflatten(-1, (-1, w))
    sc = t.abs().amax(axes, keepdim=True) * torch.tensor(1.0 / top, device="cuda")
    code = (t / sc).to(torch.float8_e4m3fn).float() if codec == "e4m3" else torch.round(t / sc)
    assert torch.equal(out, (code * sc).flatten(-2))
    # the standalone QDQ's scale is the quotient itself, an ulp away at most
    want = gdn.fp8_tile_qdq(plain.reshape(N * Hv, dk, dv), 64)[0] if codec == "e4m3" else gdn.int8_block_qdq(plain, 32)[0]
    assert ((out.flatten() - want.flatten()).abs() <= 1e-6 * want.abs().max()).double().mean().item() >= 0.999
    # and the 64-bit definition's but for quotients next to a rounding boundary
    same = (out.cpu().double() - rS).abs() <= 1e-5 * rS.abs().max()
    assert same.double().mean().item() >= 0.999
    o2 = gdn.la_decode_step(*d, state_qdq=True, codec=codec, scale=0.5)   # in place
    assert torch.equal(d[4], out) and torch.equal(o, o2)


def test_decode_zero_state_and_reset(gdn):
    q, k, v, g, S = (t.cuda() for t in decode_inputs(2, 1, 2, 64, 64, seed=5))
    S.zero_()
    k0 = torch.zeros_like(k)
    for codec in ("e4m3", "int8"):
        out = torch.full_like(S, 7.0)
        o = gdn.la_decode_step(q, k0, v, g, S, state_out=out, codec=codec)
        assert torch.equal(out, S) and not o.any()   # an all-zero tile: scale 1, no NaN
    S = torch.randn_like(S)
    out = torch.empty_like(S)
    gdn.la_decode_step(q, k, v, torch.full_like(g, -float("inf")), S, state_out=out, state_qdq=False)
    want = k.float().repeat_interleave(2, 1)[..., None] * v.float()[:, :, None, :]
    assert torch.equal(out, want)


def test_decode_continues_a_prompt(gdn):
    x, _ = inputs(2, 130, 2, 2, 128, 128, seed=23)
    o, hT = run_fwd(gdn, x, 0.3)
    first = {**{n: x[n][:, :127].contiguous() for n in ("q", "k", "v", "g")}, "h0": x["h0"], "cu": None}
    _, S = run_fwd(gdn, first, 0.3)
    for t in range(127, 130):
        ot = gdn.la_decode_step(*(x[n][:, t].contiguous().cuda() for n in ("q", "k", "v", "g")), S, state_qdq=False,
                                scale=0.3)
        assert ref.rel(ot, o[:, t].double()) <= TOL["o"]
    assert ref.rel(S, hT.double()) <= TOL["hT"]


def test_decode_no_sequences(gdn):
    x = [t.cuda() for t in decode_inputs(0, 1, 2, 64, 64, seed=1)]
    assert gdn.la_decode_step(*x).shape == (0, 2, 64)


def test_refusals(gdn):
    x, gr = inputs(1, 64, 2, 2, 64, 64, seed=1)
    d = {n: cuda(x[n]) for n in ("q", "k", "v", "g", "h0")}
    with pytest.raises(ValueError, match="contiguous"):
        gdn.la_chunk_fwd(d["q"].transpose(1, 2), d["k"], d["v"], d["g"])
    with pytest.raises(ValueError, match="bfloat16"):
        gdn.la_chunk_fwd(d["q"].float(), d["k"], d["v"], d["g"])
    with pytest.raises(ValueError, match="CUDA"):
        gdn.la_chunk_fwd(x["q"], d["k"], d["v"], d["g"])
    with pytest.raises(ValueError, match="shape"):
        gdn.la_chunk_fwd(d["q"], d["k"][:, :32].contiguous(), d["v"], d["g"])
    with pytest.raises(ValueError, match="shape"):
        gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"][:, :, :1].contiguous())
    with pytest.raises(ValueError, match="dout"):
        gdn.la_chunk_bwd(d["q"], d["k"], d["v"], d["g"])
    with pytest.raises(gdn.GdnError) as e:
        z = torch.zeros(1, 4, 1, 96, dtype=BF, device="cuda")
        gdn.la_chunk_fwd(z, z, z, torch.zeros(1, 4, 1, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(gdn.GdnError) as e:
        gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(gdn.GdnError) as e:
        gdn.la_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu_seqlens=torch.tensor([0, 40, 30, 64]))
    assert e.value.status == 1
    with pytest.raises(ValueError, match="codec"):
        gdn.la_decode_step(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["g"][:, 0], d["h0"], codec="fp4")
