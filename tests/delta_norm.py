"""The gated delta rule's results against its formula in 64 bits (delta_ref) by the
norm over each head's rows: what the bounds of single elements in delta_ref, which
allow every rounding the worst direction, are too wide to see.

Errors of many elements have signs of their own, so in a norm errors add up by their
squares, and the lengths that a bound multiplies by do not meet.  What a value passes
in a chunk are the products that delta_ref counts, eight, each off by 2^-22 of its
terms: two fp16 planes hold a number to that, and a sum of up to 320 fp32 terms is off
by less (sqrt(320) 2^-24 / 2 = 2^-20.8 if all terms were as long as the sum).  Over up
to 32 chunks, through which a state may keep all that was added to it, that is
sqrt(8 * 32) 2^-22 = 2^-18 of the result's own norm.  Gradients go through the forward
chain and the one back, and join both in one more product of each: four times as much.

The last rounding is taken off each element by itself: a number w + d that is rounded
to its type is off from w by at most half a step and |d|, so what is left of |got - w|
over half a step of the larger of the two is at most |d|, and its norm that of d."""
from __future__ import annotations

import torch

from block_ref import f64

FORWARD, GRADIENT = 2.0 ** -18, 2.0 ** -16


def tolerance(name):
    return FORWARD if name in ("out", "final", "state") else GRADIENT


def half_step(kind, v):
    """Half the distance of the type's numbers at v (subnormal ones below its least)."""
    info = torch.finfo(kind)
    least = torch.full_like(v, info.tiny)
    return torch.ldexp(torch.full_like(v, info.eps / 4), torch.frexp(torch.maximum(v.abs(), least))[1])


def off_by(got, want):
    """For each head (dimension 1), the norm of what got is off by over its rounding,
    in wanted norms."""
    kind, got, want = got.dtype, f64(got), f64(want)
    over = ((got - want).abs() - half_step(kind, torch.maximum(got.abs(), want.abs()))).clamp(min=0.0)
    over = torch.where(torch.isnan(got), torch.full_like(over, float("inf")), over)
    heads = lambda t: t.transpose(0, 1).flatten(1).norm(dim=1)  # noqa: E731
    off = heads(over)
    return torch.where(off == 0, off, off / heads(want))


def close(name, got, want):
    off, tol = off_by(got, want), tolerance(name)
    assert bool((off <= tol).all()), "%s: heads are off by %s of their norms, tolerance %.2e" % (
        name, " ".join("%.2e" % float(v) for v in off[:8]), tol)


def decays(tokens, heads, generator):
    """Log decays by head: what is left after a chunk is 0.6 of a state for the first,
    the next three forget four times as fast as the one before."""
    rate = torch.tensor([2.0 ** -6 * 4.0 ** (h % 4) for h in range(heads)])
    return -rate * torch.rand(tokens, heads, generator=generator)
