"""The 8-bit codec of la_decode_step, bit for bit as include/gdnqat.h states it: scale = fl(amax fl(1 / 448)) (INT8:
fl(amax fl(1 / 127))), 1 where that is zero, and the code of fl(x / scale), all in fp32. Its scale is at most an
ulp from that of fp8_tile_qdq and int8_block_qdq, so that a state that the step has written keeps its codes there."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32 = torch.float32


def qdq(S, codec):
    x = S.unflatten(-1, (-1, 64 if codec == "e4m3" else 32))
    top = 448.0 if codec == "e4m3" else 127.0
    amax = x.abs().amax((-3, -1) if codec == "e4m3" else -1, keepdim=True)
    sc = amax * torch.tensor(np.float32(1) / np.float32(top), dtype=F32)
    sc = torch.where(sc == 0, torch.ones_like(sc), sc)
    c = x / sc
    c = c.to(torch.float8_e4m3fn).to(F32) if codec == "e4m3" else torch.round(c)
    return (c * sc).flatten(-2), sc


@pytest.mark.parametrize("codec", ["e4m3", "int8"])
@pytest.mark.parametrize("size", [1.0, 1e-20, 3e-38, 1e30])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 256)])
def test_bits(gdn, dk, dv, size, codec):
    gen = torch.Generator().manual_seed(dk + dv)
    N, H = 3, 2
    S = size * torch.randn(N, H, dk, dv, generator=gen)
    S[0, 0] = 0.0
    S[1, 1, :, 64:] = 0.0
    q, v, g = (torch.randn(N, H, dk, generator=gen).to(torch.bfloat16), torch.randn(N, H, dv, generator=gen).to(torch.bfloat16),
               torch.zeros(N, H))
    k = torch.zeros_like(q)   # with g = 0: the updated state is the state
    out = torch.empty_like(S, device="cuda")
    gdn.la_decode_step(q.cuda(), k.cuda(), v.cuda(), g.cuda(), S.cuda(), state_out=out, codec=codec)
    want, _ = qdq(S, codec)
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("codec", ["e4m3", "int8"])
def test_codes_are_those_of_the_standalone_qdq(gdn, codec):
    gen = torch.Generator().manual_seed(5)
    S = torch.randn(4, 8, 128, 128, generator=gen)
    written, sc = qdq(S, codec)
    again, scales = (gdn.fp8_tile_qdq(written.flatten(0, 1).cuda(), 64) if codec == "e4m3" else gdn.int8_block_qdq(written.cuda(), 32))
    again, scales = again.cpu().view_as(S), scales.cpu().reshape(sc.shape)
    assert ((scales - sc).abs() <= 2.0 ** -23 * sc).all()
    width = 64 if codec == "e4m3" else 32
    codes = [torch.round(t.unflatten(-1, (-1, width)).double() / s.double() * 512) for t, s in ((written, sc), (again, scales))]
    assert torch.equal(*codes)
