"""The operators together, as examples/la_layer.py uses them: the block's gradients against autograd through a plain
form, its training, and its prompt -> decode handoff."""
import importlib.util
import os

import pytest
import torch

import layer_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "la_layer.py")
    spec = importlib.util.spec_from_file_location("la_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def plain_block(block, y, h):
    """The block in 32-bit elementary operations, token by token."""
    n = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * block.w_post
    h = h + block.alpha * n
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * block.w_pre
    q, k, v, z, a = (x.to(BF).float() @ block.inp.weight.float().T).split(block.sizes, -1)
    q, k, v, z = (t.unflatten(-1, (block.heads, -1)) for t in (q, k, v, z))
    k = torch.nn.functional.normalize(k, dim=-1)
    g = torch.nn.functional.logsigmoid(a + 4.0)
    S = torch.zeros(y.shape[0], block.heads, block.dk, block.dv, device=y.device)
    o = []
    for t in range(y.shape[1]):
        S = torch.exp(g[:, t])[..., None, None] * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        o.append(block.scale * torch.einsum("bhk,bhkv->bhv", q[:, t], S))
    o = torch.stack(o, 1)
    o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + 1e-6) * block.w_gate * torch.nn.functional.silu(z)
    return o.flatten(-2) @ block.out.weight.float().T


def test_block_gradients(example):
    torch.manual_seed(1)
    block = example.Block(64, 2, 64, 64).cuda()
    y, h = torch.randn(2, 40, 64, device="cuda").to(BF).requires_grad_(), torch.randn(2, 40, 64, device="cuda").requires_grad_()
    w = torch.randn(2, 40, 64, device="cuda")
    params = [y, h, *block.parameters()]
    out, _, _ = block(y, h)
    got = torch.autograd.grad((out.float() * w).sum(), params)
    plain = plain_block(block, y.float(), h)
    want = torch.autograd.grad((plain * w).sum(), params)
    # about ten bf16 roundings of independent sign lie between the input and a gradient: 10^0.5 x 2.3e-3 = 7e-3 in
    # the root mean square, and what they are multiplied by (norms, normalised keys) at most doubles it
    assert ref.rel(out, plain.detach()) <= 1.5e-2
    for a, b in zip(got, want):
        assert ref.rel(a, b) <= 1.5e-2


def test_example(example):
    losses, errors = example.main(steps=20, verbose=False)
    assert losses[-1] < 0.9 * losses[0]
    assert errors[None] <= 2e-2          # bf16 roundings of two orders of computation
    # 20 writes of E4M3 (relative step up to 2^-4) or INT8 (2^-8 of a block's largest) on a state of that precision
    assert errors["e4m3"] <= 0.15 and errors["int8"] <= 0.05
