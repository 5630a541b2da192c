"""A state space block on this library's operators: prompts, single tokens and
a training step.

    python examples/state_space_block.py [--channels 2048] [--tokens 4096]

The block is projection -> causal convolution -> selective scan -> projection,
with the norms, the gate and the residual sum around it.  The projections are
torch products; everything between them is one call each:

  prompts   ps_causal_conv and ps_selective_scan over packed sequences, whose
            final rows and states go into the pools of the sequences in flight
  decoding  ps_causal_conv_step and ps_selective_scan_step on those pools
  training  the same forward calls with checkpoints, then the *_bwd calls,
            joined to autograd by the functions below
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import device_wide_prefix_chained_amd as dw  # noqa: E402


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, offsets):
        ctx.save_for_backward(x, weight, bias, offsets)
        return dw.ps_causal_conv(x, weight, bias, offsets=offsets)

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias, offsets = ctx.saved_tensors
        g = dw.ps_causal_conv_bwd(x, weight, dout.contiguous(), bias, offsets=offsets)
        return g.dx, g.dweight, g.dbias, None


class Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, dt, A, B, C, D, z, dt_bias, offsets):
        rows = dw.ps_selective_scan_checkpoint_rows(x.shape[0], A.shape[1])
        kept = torch.empty(rows, *A.shape, dtype=torch.float32, device=x.device)
        ctx.save_for_backward(x, dt, A, B, C, D, z, dt_bias, offsets, kept)
        return dw.ps_selective_scan(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, offsets=offsets, checkpoints=kept)

    @staticmethod
    def backward(ctx, dout):
        x, dt, A, B, C, D, z, dt_bias, offsets, kept = ctx.saved_tensors
        g = dw.ps_selective_scan_bwd(x, dt, A, B, C, dout.contiguous(), kept, D=D, z=z, dt_bias=dt_bias, offsets=offsets)
        return g.dx, g.ddt, g.dA, g.dB, g.dC, g.dD, g.dz, g.ddt_bias, None


class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, residual, gate, scale, post, pre):
        r, out = dw.ps_block_norm(y, residual, gate=gate, scale=scale, post_weight=post, pre_weight=pre)
        ctx.save_for_backward(y, r, gate, scale, post, pre)
        return r, out

    @staticmethod
    def backward(ctx, dr, dout):
        y, r, gate, scale, post, pre = ctx.saved_tensors
        g = dw.ps_block_norm_bwd(y, r, dout.contiguous(), dr.contiguous(), gate=gate, scale=scale, post_weight=post,
                                 pre_weight=pre)
        return g.dy, g.dresidual, g.dgate, g.dscale, g.dpost_weight, g.dpre_weight


class Block:
    """One block of width `channels`; `inner` channels in the scan."""

    def __init__(self, channels, inner, states=16, width=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=device) * scale  # noqa: E731
        self.inner, self.states, self.width, self.dtype = inner, states, width, dtype
        # x | z | dt | B | C of the scan and the gate of the norm, in one projection
        self.cuts = [inner, inner, inner, states, states, channels]
        self.w_in = r(channels, sum(self.cuts), scale=channels ** -0.5).to(dtype)
        self.w_out = r(inner, channels, scale=inner ** -0.5).to(dtype)
        self.conv_w, self.conv_b = r(inner, width, scale=width ** -0.5), r(inner, scale=0.1)
        self.A = -torch.arange(1, states + 1, device=device, dtype=torch.float32).repeat(inner, 1)
        self.D, self.dt_bias = torch.ones(inner, device=device), r(inner, scale=0.1) - 4.0
        self.scale, self.post, self.pre = (torch.ones(channels, device=device) for _ in range(3))
        self.parameters = [self.w_in, self.w_out, self.conv_w, self.conv_b, self.A, self.D, self.dt_bias, self.scale,
                           self.post, self.pre]

    def _split(self, h):
        x, z, dt, B, C, gate = (h @ self.w_in).split(self.cuts, dim=1)  # strided slices: no copies
        return x, z, dt, B.unflatten(1, (1, self.states)), C.unflatten(1, (1, self.states)), gate

    def prompts(self, residual, h, offsets, conv_rows, scan_states):
        """Packed prompts; their last rows and states are written to the pools."""
        x, z, dt, B, C, gate = self._split(h)
        x = dw.ps_causal_conv(x, self.conv_w, self.conv_b, offsets=offsets, final=conv_rows)
        y = dw.ps_selective_scan(x, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias, offsets=offsets,
                                 final=scan_states)
        return dw.ps_block_norm(y @ self.w_out, residual, gate=gate, scale=self.scale, post_weight=self.post,
                                pre_weight=self.pre)

    def token(self, residual, h, slots, conv_rows, scan_states):
        """One token for each row; the pools are updated in place."""
        x, z, dt, B, C, gate = self._split(h)
        x = dw.ps_causal_conv_step(x, conv_rows, self.conv_w, self.conv_b, slots=slots)
        y = dw.ps_selective_scan_step(x, scan_states, dt, self.A, B, C, D=self.D, z=z, dt_bias=self.dt_bias, slots=slots)
        return dw.ps_block_norm(y @ self.w_out, residual, gate=gate, scale=self.scale, post_weight=self.post,
                                pre_weight=self.pre)

    def train(self, residual, h, offsets):
        x, z, dt, B, C, gate = self._split(h)
        x = Conv.apply(x, self.conv_w, self.conv_b, offsets)
        y = Scan.apply(x, dt, self.A, B, C, self.D, z, self.dt_bias, offsets)
        return Norm.apply(y @ self.w_out, residual, gate, self.scale, self.post, self.pre)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--channels", type=int, default=1024)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--decode", type=int, default=8)
    a = ap.parse_args()
    block = Block(a.channels, 2 * a.channels)
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(a.tokens, a.channels, generator=g, device="cuda").to(block.dtype)
    residual = torch.randn(a.tokens, a.channels, generator=g, device="cuda")
    offsets = torch.tensor([0, a.tokens // 3, a.tokens // 3, a.tokens], dtype=torch.int32, device="cuda")
    seqs = offsets.numel() - 1

    # prompts, then decoding from what they left
    rows = torch.empty(seqs, block.width - 1, block.inner, dtype=block.dtype, device="cuda")
    states = torch.empty(seqs, block.inner, block.states, device="cuda")
    r, out = block.prompts(residual, h, offsets, rows, states)
    slots = torch.arange(seqs, dtype=torch.int32, device="cuda")
    hr, hx = residual[:seqs], h[:seqs]
    for _ in range(a.decode):
        hr, hx = block.token(hr, hx, slots, rows, states)
    print("prompts: %d tokens in %d sequences, then %d steps of %d tokens; out rms %.3f, last token rms %.3f"
          % (a.tokens, seqs, a.decode, seqs, out.float().square().mean().sqrt(), hx.float().square().mean().sqrt()))

    # a training step
    for p in block.parameters:
        p.requires_grad_(True)
    r, out = block.train(residual, h, offsets)
    loss = out.float().square().mean() + 0.1 * r.square().mean()
    loss.backward()
    norms = [float(p.grad.float().norm()) for p in block.parameters]
    print("training: loss %.4f, gradient norms %s" % (float(loss.detach()), " ".join("%.3g" % n for n in norms)))
    assert all(n == n and n < float("inf") for n in norms)


if __name__ == "__main__":
    main()
