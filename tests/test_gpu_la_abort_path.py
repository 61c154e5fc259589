"""The bounded waits of the linear-attention kernels give up on purpose and without a fault: a test-only library
holds them with a limit of zero polls (tests/native_la). The call must come back, gdn_check_device_status must
report the timeout, and the next regular call on the same workspace must be right."""
import ctypes

import pytest
import torch

import layer_reference as ref
import native_la
from fp8_state_qat_gb300 import gdnqat as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [100, 128, 1000])
def test_waits_that_give_up(gdn, T):
    lib, tlib = gdn.load(), native_la.load()
    gen = torch.Generator().manual_seed(T)
    q, k, v = (0.1 * torch.randn(2, T, 2, 128, generator=gen).to(torch.bfloat16) for _ in range(3))
    g = -torch.rand(2, T, 2, generator=gen)
    do = torch.randn(2, T, 2, 128, generator=gen).to(torch.bfloat16)
    d = [t.cuda() for t in (q, k, v, g, do)]
    outs = [torch.zeros_like(d[0]) for _ in range(4)]
    dg, hT, dh0 = torch.zeros_like(d[3]), *(torch.zeros(2, 2, 128, 128, device="cuda") for _ in range(2))
    a = B.LaArgs(*(t.data_ptr() for t in d[:4]), None, None, None, outs[0].data_ptr(), hT.data_ptr(), 2, T, 2, 2, 2, 128, 128,
                 1.0, 0)
    gr = B.LaGrads(d[4].data_ptr(), None, *(t.data_ptr() for t in outs[1:]), dg.data_ptr(), dh0.data_ptr())
    P, SZ = ctypes.c_void_p, ctypes.c_size_t
    tlib.la_testing_fwd.argtypes = [P, P, SZ, P]
    tlib.la_testing_bwd.argtypes = [P, P, P, SZ, P]
    n = lib.la_chunk_bwd_workspace_size(ctypes.byref(a))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert tlib.la_testing_fwd(ctypes.byref(a), ws.data_ptr(), n, st) == 0
    assert lib.gdn_check_device_status(ws.data_ptr(), st) == B.GDN_ERR_DEVICE_TIMEOUT
    assert tlib.la_testing_bwd(ctypes.byref(a), ctypes.byref(gr), ws.data_ptr(), n, st) == 0
    assert lib.gdn_check_device_status(ws.data_ptr(), st) == B.GDN_ERR_DEVICE_TIMEOUT
    torch.cuda.synchronize()   # no sticky error: the kernels returned
    assert lib.la_chunk_fwd(ctypes.byref(a), ws.data_ptr(), n, st) == B.GDN_OK
    assert lib.gdn_check_device_status(ws.data_ptr(), st) == B.GDN_OK
    assert lib.la_chunk_bwd(ctypes.byref(a), ctypes.byref(gr), ws.data_ptr(), n, st) == B.GDN_OK
    assert lib.gdn_check_device_status(ws.data_ptr(), st) == B.GDN_OK
    want = ref.la(q, k, v, g, None, None, 1.0, do, None)
    for name, t in zip(("o", "dq", "dk", "dv", "dg", "hT", "dh0"), (*outs, dg, hT, dh0)):
        assert ref.rel(t, want[name]) <= (5.9e-3 if t.dtype == torch.bfloat16 else 2e-5), name
