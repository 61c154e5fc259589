"""The workspace of the chunked linear-attention calls depends on sizes and flags only: one that was made for a packing
serves every other packing of as many tokens into as many sequences."""
import ctypes

import pytest
import torch

import fp8_state_qat_gb300 as lib
from fp8_state_qat_gb300 import gdnqat as B

T = 4096
PACKINGS = [[0, 2048, T], [0, 100, T], [0, 0, T], [0, T, T], [0, 1365, T]]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("Hqk,Hv,dk,dv", [(1, 1, 64, 64), (2, 2, 128, 128), (1, 3, 128, 64), (20, 20, 128, 64), (32, 64, 64, 128)])
def test_size(Hqk, Hv, dk, dv, backward):
    sizes = {lib.la_chunk_workspace_bytes((1, T, Hqk, dk), (1, T, Hv, dv), torch.tensor(cu), backward=backward)
             for cu in PACKINGS}
    assert len(sizes) == 1 and 0 not in sizes


@pytest.mark.parametrize("room", PACKINGS)
@pytest.mark.skipif(torch.cuda.is_available(), reason="calls with addresses that are none, up to the device check")
def test_a_workspace_of_another_packing_is_accepted(room):
    so = lib.load()
    shapes = ((1, T, 2, 128), (1, T, 2, 128))
    for cu in PACKINGS:
        host = (ctypes.c_int32 * 3)(*cu)
        at = [(1 << 40) + i * (1 << 33) for i in range(16)]
        a = B.LaArgs(*at[:4], None, at[4], ctypes.addressof(host), at[5], at[6], 1, T, 2, 2, 2, 128, 128, 1.0, 0)
        g = B.LaGrads(at[7], None, *at[8:12], None)
        n = lib.la_chunk_workspace_bytes(*shapes, torch.tensor(room))
        assert so.la_chunk_fwd(ctypes.byref(a), at[13], n, None) == B.GDN_ERR_UNSUPPORTED_ARCH
        n = lib.la_chunk_workspace_bytes(*shapes, torch.tensor(room), backward=True)
        assert so.la_chunk_bwd(ctypes.byref(a), ctypes.byref(g), at[13], n, None) == B.GDN_ERR_UNSUPPORTED_ARCH


@pytest.mark.gpu
def test_results_on_one_workspace(gdn):
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (0.2 * torch.randn(1, T, 2, 128, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(4))
    g = -torch.rand(1, T, 2, generator=gen, device="cuda")
    for backward in (False, True):
        n = gdn.la_chunk_workspace_bytes(q.shape, v.shape, torch.tensor(PACKINGS[0]), backward=backward)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        for cu in PACKINGS:
            cu = torch.tensor(cu)
            if backward:
                got, want = (gdn.la_chunk_bwd(q, k, v, g, None, cu, do, workspace=w) for w in (ws, None))
            else:
                got, want = (gdn.la_chunk_fwd(q, k, v, g, None, cu, workspace=w) for w in (ws, None))
            gdn.gdn_check_device_status(ws)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
