"""A linear-attention block trained for a few steps, then used: a prompt in one chunked call and tokens one by
one, with the recurrent state kept in 8 bits.

    python examples/la_layer.py

The block: residual norm (the norm before it, and the one after the block before) -> q, k, v, gate z and log-decay
g by linear maps -> la_chunk_fwd / la_decode_step -> gated norm per head -> output map. The linear maps are torch's;
everything between them is this library's, with the gradients of la_chunk_bwd, gated_norm_bwd and
residual_norm_bwd.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_state_qat_gb300 as gdn  # noqa: E402

BF = torch.bfloat16


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, scale):
        o, hT = gdn.la_chunk_fwd(q, k, v, g, scale=scale)
        ctx.save_for_backward(q, k, v, g)
        ctx.scale = scale
        ctx.mark_non_differentiable(hT)
        return o, hT

    @staticmethod
    def backward(ctx, do, _):
        dq, dk, dv, dg, _ = gdn.la_chunk_bwd(*ctx.saved_tensors, dout=do.contiguous(), scale=ctx.scale, want_dh0=False)
        return dq, dk, dv, dg, None


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, w):
        ctx.save_for_backward(x, z, w)
        return gdn.gated_norm_fwd(x, z, w)

    @staticmethod
    def backward(ctx, dy):
        return gdn.gated_norm_bwd(dy.contiguous(), *ctx.saved_tensors)


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, h, w_pre, w_post, alpha):
        ctx.save_for_backward(y, h, w_pre, w_post)
        ctx.alpha = alpha
        return gdn.residual_norm_fwd(y, h, w_pre, w_post, alpha=alpha)

    @staticmethod
    def backward(ctx, dh_out, dx):
        y, h, w_pre, w_post = ctx.saved_tensors
        dy, dh, d1, d2 = gdn.residual_norm_bwd(dx.contiguous(), dh_out.contiguous(), y, h, w_pre, w_post, alpha=ctx.alpha)
        return dy, dh, d1, d2, None


class Block(torch.nn.Module):
    def __init__(self, width, heads, dk, dv, alpha=0.5):
        super().__init__()
        self.heads, self.dk, self.dv, self.alpha, self.scale = heads, dk, dv, alpha, dk ** -0.5
        self.sizes = [heads * dk, heads * dk, heads * dv, heads * dv, heads]
        self.inp = torch.nn.Linear(width, sum(self.sizes), bias=False, dtype=BF)
        self.out = torch.nn.Linear(heads * dv, width, bias=False, dtype=BF)
        self.w_pre, self.w_post = (torch.nn.Parameter(torch.ones(width)) for _ in range(2))
        self.w_gate = torch.nn.Parameter(torch.ones(dv))

    def maps(self, x):
        q, k, v, z, a = self.inp(x).split(self.sizes, -1)
        H = self.heads
        q, k, v, z = (t.unflatten(-1, (H, -1)).contiguous() for t in (q, k, v, z))
        k = torch.nn.functional.normalize(k.float(), dim=-1).to(BF)
        return q, k, v, z, torch.nn.functional.logsigmoid(a.float() + 4.0)

    def forward(self, y, h):
        """y: the output of the block before; h: the residual stream. Returns (output, stream, final state)."""
        h, x = ResidualNorm.apply(y, h, self.w_pre, self.w_post, self.alpha)
        q, k, v, z, g = self.maps(x)
        o, state = LinearAttention.apply(q, k, v, g, self.scale)
        return self.out(GatedNorm.apply(o, z, self.w_gate).flatten(-2)), h, state

    @torch.no_grad()
    def step(self, y, h, state, codec):
        """One token of every sequence; the state is updated in place, and held in 8 bits where a codec is given."""
        h, x = gdn.residual_norm_fwd(y, h, self.w_pre, self.w_post, alpha=self.alpha)
        q, k, v, z, g = self.maps(x)
        o = gdn.la_decode_step(q, k, v, g, state, state_qdq=codec is not None, codec=codec or "e4m3", scale=self.scale)
        return self.out(gdn.gated_norm_fwd(o, z, self.w_gate).flatten(-2)), h


def quantize(state, codec):
    """The handoff from the prompt to the decode steps: the state as the codec stores it."""
    if codec == "e4m3":
        return gdn.fp8_tile_qdq(state.flatten(0, 1), 64, scales=False)[0].view_as(state)
    return gdn.int8_block_qdq(state, 32, scales=False)[0] if codec == "int8" else state


def main(steps=30, B=4, T=300, width=256, heads=4, dk=64, dv=128, verbose=True):
    torch.manual_seed(0)
    block = Block(width, heads, dk, dv).cuda()
    y, h = torch.randn(B, T, width, device="cuda").to(BF), torch.randn(B, T, width, device="cuda")
    target = torch.roll(y.float(), 3, 1)              # to be found three tokens back
    opt = torch.optim.Adam(block.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        opt.zero_grad()
        out, _, _ = block(y, h)
        loss = (out.float() - target)[:, 3:].square().mean()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    if verbose:
        print(f"training loss {losses[0]:.3f} -> {losses[-1]:.3f} in {steps} steps")
    prompt = T - 20
    with torch.no_grad():
        whole, _, _ = block(y, h)
        errors = {}
        for codec in (None, "e4m3", "int8"):
            _, _, state = block(y[:, :prompt].contiguous(), h[:, :prompt].contiguous())
            state = quantize(state, codec)
            tokens = [block.step(y[:, t].contiguous(), h[:, t].contiguous(), state, codec)[0] for t in range(prompt, T)]
            got, want = torch.stack(tokens, 1).float(), whole[:, prompt:].float()
            errors[codec] = ((got - want).norm() / want.norm()).item()
            if verbose:
                print(f"20 tokens after a prompt of {prompt}, state in {codec or 'fp32'}: relative difference "
                      f"{errors[codec]:.1e} from the chunked call")
    return losses, errors


if __name__ == "__main__":
    main()
