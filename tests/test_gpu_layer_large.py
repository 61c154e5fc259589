"""Tensors of more than 2^31 elements: the last rows, heads and sequences are what a call on them alone gives."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_gated_norm_rows_past_32_bits(gdn):
    R, D = (1 << 31) // 128 + 4099, 128
    x = torch.empty(R, D, dtype=BF, device="cuda").normal_()
    z = torch.empty(R, D, dtype=BF, device="cuda").normal_()
    w = torch.ones(D, device="cuda")
    y = gdn.gated_norm_fwd(x, z, w)
    tail = [t[-5000:].clone() for t in (x, z)]
    assert torch.equal(y[-5000:], gdn.gated_norm_fwd(*tail, w))
    dx, dz, _ = gdn.gated_norm_bwd(y, x, z, w)
    a, b, _ = gdn.gated_norm_bwd(y[-5000:].clone(), *tail, w)
    assert torch.equal(dx[-5000:], a) and torch.equal(dz[-5000:], b)


def test_decode_states_past_32_bits(gdn):
    N, H, dk, dv = 9000, 16, 128, 128
    state = torch.empty(N, H, dk, dv, device="cuda").normal_()
    q, k = (torch.empty(N, H, dk, dtype=BF, device="cuda").normal_() for _ in range(2))
    v = torch.empty(N, H, dv, dtype=BF, device="cuda").normal_()
    g = -torch.rand(N, H, device="cuda")
    last = [t[-3:].clone() for t in (q, k, v, g, state)]
    o = gdn.la_decode_step(q, k, v, g, state)
    assert torch.equal(o[-3:], gdn.la_decode_step(*last))
    assert torch.equal(state[-3:], last[4])


def test_linear_attention_tokens_past_32_bits(gdn):
    T, H, d, tail = 135000, 128, 128, 777
    lens = [T - tail - 130, 130, tail]
    cu = torch.tensor([0, lens[0], lens[0] + lens[1], T], dtype=torch.int32)
    assert T * H * d > 1 << 31
    q, k, v, do = (torch.empty(1, T, H, d, dtype=BF, device="cuda").normal_(std=0.3) for _ in range(4))
    g = torch.empty(1, T, H, device="cuda").uniform_(-0.2, 0)
    dhT = torch.empty(3, H, d, d, device="cuda").normal_()
    o, hT = gdn.la_chunk_fwd(q, k, v, g, None, cu)
    got = gdn.la_chunk_bwd(q, k, v, g, None, cu, do, dhT)
    one = [t[:, -tail:].clone() for t in (q, k, v, g, do)]
    o1, h1 = gdn.la_chunk_fwd(*one[:4])
    want = gdn.la_chunk_bwd(*one[:4], None, None, one[4], dhT[2:].clone())
    assert torch.equal(o[:, -tail:], o1) and torch.equal(hT[2:], h1)
    for a, b in zip(got[:4], want[:4]):
        assert torch.equal(a[:, -tail:], b)
    assert torch.equal(got[4][2:], want[4])
