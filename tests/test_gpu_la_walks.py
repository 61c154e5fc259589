"""The backward of linear attention with few and with many walks over sequences: few run the two directions side by
side and take <S, dS> from the stored states, many take it on the backwards walk. Both have to agree with the 64-bit
recurrence, and with themselves when calls follow one another on one workspace."""
import pytest
import torch

import layer_reference as ref
from test_gpu_la import TOL, cuda, inputs, run_bwd

pytestmark = pytest.mark.gpu
FEW, MANY = [1, 130, 300], [1, 128, 129, 0, 64, 200, 5, 127] * 5   # times 2 heads, 2 value tiles: 12 and 160 walks


def off(got, want, floor=0.0):
    got, want = got.cpu().double(), want.double()
    return (got - want).norm().item() / max(want.norm().item(), floor, 1e-30)


@pytest.mark.parametrize("head", [False, True])
@pytest.mark.parametrize("lens", [FEW, MANY], ids=["few", "many"])
def test_gradients(gdn, lens, head):
    x, gr = inputs(1, 0, 2, 2, 128, 128, 3, lens=lens, head=head)
    got = run_bwd(gdn, x, gr, 0.3)
    want = ref.la(*(x[n] for n in ("q", "k", "v", "g", "h0", "cu")), 0.3, gr["dout"], gr["dhT"])
    for n in ("dq", "dk", "dv", "dh0"):
        assert off(got[n], want[n]) <= TOL[n], n
    assert off(got["dg"], want["dg"], 1e-3 * (want["dq"] * x["q"].double()).norm().item()) <= TOL["dg"]


def test_calls_in_a_row_share_no_state(gdn):
    """The workspace of one call is the next one's: neither walk may start before the call before it is over."""
    x, gr = inputs(1, 0, 2, 2, 128, 128, 4, lens=FEW)
    y, gy = inputs(1, 0, 2, 2, 128, 128, 5, lens=FEW)
    size = gdn.la_chunk_workspace_bytes(x["q"].shape, x["v"].shape, x["cu"], backward=True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    first, second = run_bwd(gdn, x, gr, 0.3), run_bwd(gdn, y, gy, 0.3)
    a = [cuda(x[n]) for n in ("q", "k", "v", "g", "h0")], cuda(gr["dout"]), cuda(gr["dhT"])
    b = [cuda(y[n]) for n in ("q", "k", "v", "g", "h0")], cuda(gy["dout"]), cuda(gy["dhT"])
    out = []
    for _ in range(20):
        for t, d, e in (a, b):
            out.append(gdn.la_chunk_bwd(*t, x["cu"], d, e, scale=0.3, workspace=ws))
    for i, got in enumerate(out):
        for n, z in zip(("dq", "dk", "dv", "dg", "dh0"), got):
            assert torch.equal(z, (first, second)[i % 2][n]), (i, n)
