"""A block with the gated delta rule on this library's operators: prompts,
single tokens and a training step.

    python examples/delta_block.py [--channels 1024] [--tokens 4096]

The block is layer norm -> projection -> causal convolution over queries, keys
and values -> gated delta rule -> layer norm of every head -> projection, added
to its input.  The projections and the gates' functions are torch's; the rest is
one call each:

  prompts   ps_layer_norm, ps_causal_conv and ps_gated_delta over packed
            sequences, whose final rows and states go into the pools of the
            sequences in flight
  decoding  ps_causal_conv_step and ps_gated_delta_step on those pools
  training  the same forward calls with checkpoints, then the *_bwd calls,
            joined to autograd by the functions below
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import device_wide_prefix_chained_amd as dw  # noqa: E402
from state_space_block import Conv  # noqa: E402


class Delta(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, offsets):
        tokens, heads, value_dim = v.shape
        seqs = 1 if offsets is None else offsets.numel() - 1
        floats = dw.ps_gated_delta_checkpoint_floats(tokens, seqs, heads, q.shape[2], value_dim)
        kept = torch.empty(floats, dtype=torch.float32, device=q.device)
        ctx.save_for_backward(q, k, v, g, beta, offsets, kept)
        return dw.ps_gated_delta(q, k, v, g, beta, normalize=True, offsets=offsets, checkpoints=kept)

    @staticmethod
    def backward(ctx, dout):
        q, k, v, g, beta, offsets, kept = ctx.saved_tensors
        d = dw.ps_gated_delta_bwd(q, k, v, g, beta, dout.contiguous(), kept, normalize=True, offsets=offsets)
        return d.dq, d.dk, d.dv, d.dg, d.dbeta, None


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return dw.ps_layer_norm(x, weight, bias)

    @staticmethod
    def backward(ctx, dout):
        x, weight, bias = ctx.saved_tensors
        d = dw.ps_layer_norm_bwd(x, dout.contiguous(), weight, bias)
        return d.dx, d.dweight, d.dbias


class Block:
    """One block of width `channels`: `heads` heads of values, which share
    `kheads` heads of queries and keys."""

    def __init__(self, channels, heads, kheads, key_dim=64, value_dim=64, width=4, dtype=torch.bfloat16, device="cuda",
                 seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, scale=1.0: torch.randn(*s, generator=g, device=device) * scale  # noqa: E731
        self.heads, self.kheads, self.key_dim, self.value_dim = heads, kheads, key_dim, value_dim
        self.width, self.dtype = width, dtype
        # q | k | v together go through the convolution; then the two gates
        self.parts = [kheads * key_dim, kheads * key_dim, heads * value_dim]
        self.inner = sum(self.parts)
        self.cuts = [self.inner, heads, heads]
        self.w_in = r(channels, sum(self.cuts), scale=channels ** -0.5).to(dtype)
        self.w_out = r(heads * value_dim, channels, scale=(heads * value_dim) ** -0.5).to(dtype)
        self.conv_w, self.conv_b = r(self.inner, width, scale=width ** -0.5), r(self.inner, scale=0.1)
        self.rate, self.rate_bias = r(heads, scale=0.3), r(heads, scale=0.1) - 3.0
        self.in_w, self.in_b = 1.0 + r(channels, scale=0.1), r(channels, scale=0.1)
        self.head_w, self.head_b = 1.0 + r(value_dim, scale=0.1), r(value_dim, scale=0.1)
        self.parameters = [self.w_in, self.w_out, self.conv_w, self.conv_b, self.rate, self.rate_bias, self.in_w,
                           self.in_b, self.head_w, self.head_b]

    def _split(self, h):
        x, g, beta = (h @ self.w_in).split(self.cuts, dim=1)  # strided slices: no copies
        g = -torch.exp(self.rate) * torch.nn.functional.softplus(g.float() + self.rate_bias)
        return x, g, torch.sigmoid(beta.float())

    def _heads(self, x):
        q, k, v = x.split(self.parts, dim=1)
        return (q.unflatten(1, (self.kheads, self.key_dim)), k.unflatten(1, (self.kheads, self.key_dim)),
                v.unflatten(1, (self.heads, self.value_dim)))

    def _out(self, x, o, norm):
        o = norm(o.reshape(-1, self.value_dim), self.head_w, self.head_b).reshape(x.shape[0], -1)
        return x + o @ self.w_out

    def prompts(self, x, offsets, conv_rows, states):
        """Packed prompts; their last rows and states are written to the pools."""
        c, g, beta = self._split(dw.ps_layer_norm(x, self.in_w, self.in_b))
        c = dw.ps_causal_conv(c, self.conv_w, self.conv_b, offsets=offsets, final=conv_rows)
        o = dw.ps_gated_delta(*self._heads(c), g, beta, normalize=True, offsets=offsets, final=states)
        return self._out(x, o, dw.ps_layer_norm)

    def token(self, x, slots, conv_rows, states):
        """One token for each row; the pools are updated in place."""
        c, g, beta = self._split(dw.ps_layer_norm(x, self.in_w, self.in_b))
        c = dw.ps_causal_conv_step(c, conv_rows, self.conv_w, self.conv_b, slots=slots)
        o = dw.ps_gated_delta_step(*self._heads(c), states, g, beta, normalize=True, slots=slots)
        return self._out(x, o, dw.ps_layer_norm)

    def train(self, x, offsets):
        c, g, beta = self._split(LayerNorm.apply(x, self.in_w, self.in_b))
        c = Conv.apply(c, self.conv_w, self.conv_b, offsets)
        o = Delta.apply(*self._heads(c), g, beta, offsets)
        return self._out(x, o, LayerNorm.apply)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--channels", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kheads", type=int, default=16)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--decode", type=int, default=8)
    a = ap.parse_args(argv)
    block = Block(a.channels, a.heads, a.kheads)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, a.channels, generator=g, device="cuda").to(block.dtype)
    offsets = torch.tensor([0, a.tokens // 3, a.tokens // 3, a.tokens], dtype=torch.int32, device="cuda")
    seqs = offsets.numel() - 1

    # prompts, then decoding from what they left
    rows = torch.empty(seqs, block.width - 1, block.inner, dtype=block.dtype, device="cuda")
    states = torch.empty(seqs, a.heads, block.key_dim, block.value_dim, device="cuda")
    out = block.prompts(x, offsets, rows, states)
    slots = torch.arange(seqs, dtype=torch.int32, device="cuda")
    token = out[:seqs]
    for _ in range(a.decode):
        token = block.token(token, slots, rows, states)
    print("prompts: %d tokens in %d sequences, then %d steps of %d tokens; out rms %.3f, last token rms %.3f"
          % (a.tokens, seqs, a.decode, seqs, out.float().square().mean().sqrt(), token.float().square().mean().sqrt()))

    # a training step
    for p in block.parameters:
        p.requires_grad_(True)
    loss = block.train(x, offsets).float().square().mean()
    loss.backward()
    norms = [float(p.grad.float().norm()) for p in block.parameters]
    print("training: loss %.4f, gradient norms %s" % (float(loss.detach()), " ".join("%.3g" % n for n in norms)))
    assert all(n == n and n < float("inf") for n in norms)


if __name__ == "__main__":
    main()
