"""The stream argument of the layer operators."""
import types

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_stream_of_another_device(gdn):
    """Such a stream makes its own device current, and the call would go to some other stream of the tensors'
    device, in no order with the one that was asked for. (A stand-in for the stream: it is refused unused.)"""
    x, z, w = (torch.ones(4, 64, device="cuda", dtype=t) for t in (torch.float32, torch.bfloat16, torch.float32))
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        gdn.gated_norm_fwd(x, z, w[0].contiguous(), stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = gdn.gated_norm_fwd(x, z, w[0].contiguous(), stream=s)
    s.synchronize()
    assert torch.equal(y, gdn.gated_norm_fwd(x, z, w[0].contiguous()))
