"""gdn_upload_i32 without a GPU: its refusals come before a device is touched."""
import ctypes

import pytest
import torch

import fp8_state_qat_gb300 as lib
from fp8_state_qat_gb300 import gdnqat as B

DEVICE = 1 << 40   # never written: no call below gets past the device check


def upload(host, device, n):
    return lib.load().gdn_upload_i32(host, device, n, None)


def test_refusals():
    host = (ctypes.c_int32 * 4)(0, 1, 2, 3)
    at = ctypes.addressof(host)
    for args in ((at, DEVICE, -1), (None, DEVICE, 4), (at, None, 4), (at + 2, DEVICE, 1), (at, DEVICE + 1, 4)):
        assert upload(*args) == B.GDN_ERR_INVALID_ARG, args


@pytest.mark.skipif(torch.cuda.is_available(), reason="stops at the device check where there is no GPU")
def test_stops_at_the_device_check():
    host = (ctypes.c_int32 * 4)(0, 1, 2, 3)
    assert upload(ctypes.addressof(host), DEVICE, 4) == B.GDN_ERR_UNSUPPORTED_ARCH
    assert upload(None, None, 0) == B.GDN_ERR_UNSUPPORTED_ARCH
